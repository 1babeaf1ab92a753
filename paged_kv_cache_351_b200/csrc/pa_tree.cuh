// Speculative decoding over the paged cache (sm_100a): attention of a tree
// of drafted tokens, and the move of the accepted path's K/V.
//
// Tree attention.  Sequence i brings n_i drafted tokens, rows query_start[i]
// .. query_start[i+1] - 1, whose K/V already sit at cache positions c_i ..
// c_i + n_i - 1 (c_i = context_lens[i] - n_i).  Row j sees every committed
// key t < c_i and the drafted key c_i + u if bit u of its mask row is set:
//   out[r, h] = sum_{t visible} softmax_t(scale * <q[r,h], K_i[t, g]>) V_i[t, g],
//   g = h / G;  a row that sees nothing is zero.
//
// Work list (both kernels below).  A unit is (sequence, kv head, tile of R
// query rows), the rows being the unit's drafted tokens times the G query
// heads of the kv head, so that a K/V page is read once for all of them; it
// is a run of key tiles of KT tokens.  The workers (CTAs) of a persistent
// grid take equal contiguous ranges of the flattened list of units, whatever
// the mix of lengths; a unit counts as its tiles plus LEAD (what a unit costs
// beside its tiles, in tiles), which stand before its first tile and hold no
// work.  A unit cut by a range boundary leaves one share per worker (output
// before the division, running max, denominator), merged in worker order, so
// that the result does not depend on timing:
//  * in general whoever counts in a unit's last tiles merges them on the spot.
//    Nobody waits for anybody, and every counter is zero again when the launch
//    ends;
//  * with at most a unit for every four CTAs of the grid (the host knows no
//    lengths) a second launch merges them, spread over the GPU, since a long
//    unit may leave a share in each of a hundred CTAs, which one CTA would
//    read alone: 20,000 tokens of one kv head 27 us against 112 on the spot,
//    8,000 of eight 26 against 34, fp32 8,000 of one 36 against 150.  Short
//    contexts, of a few shares a unit, pay 1 to 4 us for that launch: 500
//    tokens of eight kv heads 16.0 against 15.0, of 32 units 20.0 against
//    16.3, of 72 units 24.2 against 20.0 (and 3,000 of 72 units 38.3 against
//    35.9).
#pragma once

#include "pa_common.cuh"
#include "pa_decode.cuh"

namespace pa {

struct TreeArgs {
  void* out;            // [T, H, D]
  const void* q;        // [T, H, D]
  const void* kc;
  const void* vc;
  const int32_t* bt;    // [B, max_nb]
  const int32_t* ctx;   // [B] tokens in the cache, the drafted ones included
  const int32_t* qs;    // [B + 1] first row of each sequence
  const uint32_t* mask; // [T, words]
  int64_t q_st, q_sh, o_st, o_sh, bt_stride, mask_stride;
  int32_t B, T, Hkv, lg, max_nb, num_blocks, words, max_q;  // lg: log2 of the query heads per kv head
  float scale_log2;  // scale * log2(e)
  int32_t min_len;   // least list length per worker
  int32_t split;     // 1: units may be cut between workers (shares below)
  float4* sh_o;      // shares: two slots per worker; see tree_share
  float2* sh_ml;     // [slot][R] (running max in log2 units, denominator)
  unsigned int* cnt; // shares merged on the spot: per worker and warp (or half), tiles of the unit that starts
                     // there counted in so far
  struct TreeCut* cut;  // shares merged by a second launch (else null): by the unit's number in the list
  int32_t* units;       // and the units in the list
  uint64_t timeout_ns;
};

// What the merge needs of a unit: its shares (0: it was not cut), the worker
// that holds its first tile, its rows.
struct TreeCut {
  int ns, wa, h, rt;
  int q0, n, c0, pad;
};

// Dims 4 d .. 4 d + 3 of row r of a share: rows side by side, in blocks of at
// most 128, so that the threads of a warp, one row each, write and read runs.
template <int D, int R>
__device__ __forceinline__ float4* tree_share(const TreeArgs& a, int slot, int r, int d) {
  constexpr int RB = R < 128 ? R : 128;
  return a.sh_o + ((int64_t(slot) * (R / RB) + r / RB) * (D / 4) + d) * RB + r % RB;
}

// The drafted rows of sequence i (n = 0: none, or a range that does not fit).
struct TreeSeq {
  int q0, n, c0;  // first row, rows, committed tokens
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int i) {
  const int64_t q0 = __ldg(a.qs + i), q1 = __ldg(a.qs + i + 1);
  const int ctx = __ldg(a.ctx + i);
  const int64_t n = q1 - q0;
  if (q0 < 0 || n < 0 || q1 > a.T || n > ctx || ctx > a.max_nb * kBS || n > a.max_q) {
    if (blockIdx.x == 0) flag(PA_DEV_BAD_CONTEXT);
    return TreeSeq{0, 0, 0};
  }
  return TreeSeq{int(q0), int(n), ctx - int(n)};
}

// Position in the flattened list: sequence, kv head, row tile, position in
// the unit (LEAD, then its key tiles).
struct TreePos {
  int i, h, rt, p;
  int number;   // of the unit in the list (if a.cut)
  int rts, nt;  // row tiles of each kv head of the sequence (0: no drafted rows), key tiles of each unit
  TreeSeq s;
};

// A worker's part of one unit: key tiles [b, e) (none if the part lies in the
// lead), and where the part ends in the unit's list.
struct TreeSeg {
  int b, e, pe;
};

template <int LEAD>
__device__ __forceinline__ TreeSeg tree_seg(const TreePos& x, int left) {
  TreeSeg g;
  g.pe = x.nt + LEAD - x.p < left ? x.nt + LEAD : x.p + left;
  g.b = max(0, x.p - LEAD);
  g.e = max(0, g.pe - LEAD);
  return g;
}

template <int R, int KT>
__device__ __forceinline__ void tree_shape(const TreeArgs& a, TreePos& x) {
  x.s = tree_seq(a, x.i);
  x.rts = ((x.s.n << a.lg) + R - 1) / R;
  x.nt = x.s.n > 0 ? (x.s.c0 + x.s.n + KT - 1) / KT : 0;
}

// Next unit of the list (x.p = 0), skipping sequences without drafted rows.
template <int R, int KT>
__device__ __forceinline__ void tree_next_unit(const TreeArgs& a, TreePos& x) {
  x.p = 0;
  ++x.number;
  if (++x.rt < x.rts) return;
  x.rt = 0;
  if (++x.h < a.Hkv) return;
  x.h = 0;
  do {
    ++x.i;
    if (x.i >= a.B) return;
    tree_shape<R, KT>(a, x);
  } while (x.rts == 0);
}

// Whole block: this worker's range [lo, hi) of the list, the list's length, and the position of lo.  smem: 41 ints.
//
// Workers past N = W / min_len (at least 1, at most the grid) get nothing: a
// short list is cut into fewer pieces, since a share costs a write and the
// merge a read, and no worker of the others is empty.
struct TreeRange {
  int W, N;    // length of the list, workers
  int per, rem;  // W / N, W % N
  int lo, hi;
  TreePos at;
  // first position of worker w: ceil(w W / N), in 32 bits (N is at most the
  // grid, below 2^15, so w rem + N does not overflow)
  __device__ __forceinline__ int first(int w) const { return w * per + (w * rem + N - 1) / N; }
  // the worker that holds position x: an estimate, then exact
  __device__ __forceinline__ int owner(int x) const {
    int w = min(N - 1, int(__fdividef(float(x), float(per) + __fdividef(float(rem), float(N)))));
    while (first(w) > x) --w;
    while (w + 1 < N && first(w + 1) <= x) ++w;
    return w;
  }
};

template <int R, int KT, int LEAD>
__device__ __forceinline__ TreeRange tree_range(const TreeArgs& a, int* smem) {
  const int nthr = blockDim.x;
  const int per = (a.B + nthr - 1) / nthr;
  const int i0 = min(a.B, int(threadIdx.x) * per), i1 = min(a.B, i0 + per);
  int local = 0;
  for (int i = i0; i < i1; ++i) {
    TreePos x;
    x.i = i;
    tree_shape<R, KT>(a, x);
    local += x.rts * a.Hkv * (x.nt + LEAD);
  }
  int total;
  const int first = block_exclusive_scan(local, smem, &total);
  int unit0 = 0;  // units before this thread's sequences
  if (a.cut != nullptr) {
    int units = 0;
    for (int i = i0; i < i1; ++i) {
      TreePos x;
      x.i = i;
      tree_shape<R, KT>(a, x);
      units += x.rts * a.Hkv;
    }
    int all;
    unit0 = block_exclusive_scan(units, smem, &all);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.units = all;
  }
  TreeRange r;
  r.W = total;
  r.N = max(1, min(int(gridDim.x), total / a.min_len));
  r.per = total / r.N;
  r.rem = total - r.per * r.N;
  const int w = min(int(blockIdx.x), r.N);
  r.lo = r.first(w);
  r.hi = w < r.N ? r.first(w + 1) : r.lo;
  // the thread that owns the tile finds its sequence; without a split both
  // ends move down to the start of their unit
  for (int e = 0; e < 2; ++e) {
    const int b = e == 0 ? r.lo : r.hi;
    if (b < r.W && b >= first && b < first + local) {
      int base = first, units = unit0;
      for (int i = i0; i < i1; ++i) {
        TreePos x;
        x.i = i;
        tree_shape<R, KT>(a, x);
        const int len = x.nt + LEAD, t = x.rts * a.Hkv * len;
        if (b < base + t) {
          const int off = b - base;
          smem[32 + 4 * e + 0] = i;
          smem[32 + 4 * e + 1] = off / len;
          smem[32 + 4 * e + 2] = a.split ? off % len : 0;
          smem[32 + 4 * e + 3] = a.split ? 0 : off % len;
          if (e == 0) smem[40] = units + off / len;
          break;
        }
        base += t;
        units += x.rts * a.Hkv;
      }
    }
  }
  __syncthreads();
  if (r.lo < r.W) {
    r.at.i = smem[32];
    r.at.p = smem[34];
    r.at.number = smem[40];
    tree_shape<R, KT>(a, r.at);
    r.at.h = smem[33] / r.at.rts;
    r.at.rt = smem[33] - r.at.h * r.at.rts;
    r.lo -= smem[35];
  }
  if (r.hi < r.W) r.hi -= smem[39];
  __syncthreads();
  return r;
}

// For the second launch, by one thread of a worker at each unit that starts in
// its range: whether it is cut.
__device__ __forceinline__ TreeCut tree_cut(const TreeRange& rg, const TreePos& x, const TreeSeg& g, int unit0) {
  const bool cut = g.e < x.nt;
  return TreeCut{cut ? rg.owner(unit0 + x.nt - 1) - int(blockIdx.x) + 1 : 0, int(blockIdx.x), x.h, x.rt,
                 x.s.q0, x.s.n, x.s.c0, 0};
}

// Bits of the 32 drafted keys u0 .. u0 + 31 that row `row` sees (u0 may be
// negative: committed keys are all seen, and so are no keys past the draft).
__device__ __forceinline__ uint32_t tree_word(const TreeArgs& a, int64_t row, int n, int w) {
  if (w < 0 || w >= a.words || w * 32 >= n) return 0u;
  const uint32_t x = __ldg(a.mask + row * a.mask_stride + w);
  const int left = n - w * 32;
  return left >= 32 ? x : x & ((1u << left) - 1u);
}

__device__ __forceinline__ uint32_t tree_seen32(const TreeArgs& a, int64_t row, int n, int u0) {
  if (u0 >= 0) {
    const int w = u0 >> 5, sh = u0 & 31;
    return __funnelshift_r(tree_word(a, row, n, w), sh ? tree_word(a, row, n, w + 1) : 0u, sh);
  }
  if (u0 <= -32) return 0xffffffffu;
  const int k = -u0;  // committed keys in the low k bits, 1 <= k <= 31
  return (tree_word(a, row, n, 0) << k) | ((1u << k) - 1u);
}

// 1 / (a row's denominator), which is 0 only where no logit is above
// -infinity: NaN then (0 / 0), but 0 for a row that sees nothing, whose output
// is zero.
__device__ __forceinline__ float tree_inverse(const TreeArgs& a, float l, int c0, int n, int64_t row) {
  if (l != 0.f) return 1.f / l;
  if (c0 > 0) return NAN;
  for (int w = 0; w * 32 < n; ++w)
    if (tree_word(a, row, n, w) != 0u) return NAN;
  return 0.f;
}

// ---- CUDA-core kernel ----------------------------------------------------
// fp32 caches: products and sums in fp32, no tensor-core rounding.  Eight warps
// of RW query rows each; tiles of 32 keys come into two stages of shared
// memory by asynchronous 16-byte copies, the next tile while this one is
// computed.  Scores: lane = key, the query rows broadcast from shared memory
// (K rows padded to D + 4 floats, so that 16-byte reads of 32 consecutive rows
// touch every bank once per phase).  Weighted sum: lane = D / 32 dims, the
// probabilities broadcast from shared memory.  Per 4 dims and key, a 16-byte
// read of K (or V) and one of each row's query (or probability) serve 4 RW
// products, which is why a warp takes up to 8 rows.  Nothing is at its limit
// (16 sequences of 2,000 tokens, trees of 20, 32 heads on 8: FMA pipe 33%,
// shared-memory pipe 46% on average and 74% in the busiest SM): the time goes
// to two block barriers per 32 keys and to waiting for shared memory with 16
// warps an SM (2.3 cycles each per issued instruction), and a sequence's last
// unit, of 16 of its 80 rows there, reads all keys for two of its eight warps
// at work.  (That batch: 1.03 ms with four warps of 4 rows and no copies
// ahead, 0.68 with 8 rows and copies ahead, 0.66 with eight such warps, 16
// TFLOP/s; 4 x 4,000 tokens, trees of 64, 8 heads on 1: 0.35, 0.23, 0.18 ms.)
constexpr int kTsKeys = 32;
constexpr int kTsWarps = 8;
constexpr int kTsLead = 1;

template <int D, int RW>
struct TreeSimt {
  static constexpr int R = kTsWarps * RW;
  static constexpr int KSTR = D + 4;                                // floats per row of K in shared memory
  static constexpr int STAGE = kTsKeys * KSTR + kTsKeys * D;        // floats: K, V
  static constexpr int Q0 = 2 * STAGE, P0 = Q0 + R * D, S0 = P0 + kTsWarps * kTsKeys * RW;
  static constexpr size_t SMEM = size_t(S0 + 64) * 4;
};

// 16 bytes into shared memory, asynchronously; zeros if !valid.
__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}

template <int D, int RW>
__global__ void __launch_bounds__(kTsWarps * 32) tree_simt_kernel(const TreeArgs a) {
  using C = TreeSimt<D, RW>;
  constexpr int VPR = D / 4, PER = D / 32, R = C::R;
  extern __shared__ __align__(128) unsigned char smem[];
  float* const stage0 = reinterpret_cast<float*>(smem);
  float* const Qs = stage0 + C::Q0;
  int* scratch = reinterpret_cast<int*>(stage0 + C::S0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* const Ps = stage0 + C::P0 + warp * kTsKeys * RW;  // [key][row]

  pdl_wait();
  pdl_launch_dependents();
  const TreeRange rg = tree_range<R, kTsKeys, kTsLead>(a, scratch);
  TreePos x = rg.at;
  const float* kc = static_cast<const float*>(a.kc);
  const float* vc = static_cast<const float*>(a.vc);

  for (int cx = rg.lo; cx < rg.hi;) {
    // ---- one segment: this worker's tiles of one unit ----
    const TreeSeg sg = tree_seg<kTsLead>(x, rg.hi - cx);
    if (sg.b == sg.e) {
      cx += sg.pe - x.p;
      if (cx < rg.hi) tree_next_unit<R, kTsKeys>(a, x);
      continue;
    }
    const int kvh = x.h, r0 = x.rt * R, gm = (1 << a.lg) - 1;
    const int rows = min(R, (x.s.n << a.lg) - r0);
    const int kv_len = x.s.c0 + x.s.n;
    const int32_t* bt = a.bt + int64_t(x.i) * a.bt_stride;
    auto load = [&](int p) {  // tile p into its stage; keys past the end are zeros
      float* const Ks = stage0 + (p & 1) * C::STAGE;
      float* const Vs = Ks + kTsKeys * C::KSTR;
#pragma unroll 4
      for (int e = threadIdx.x; e < kTsKeys * VPR; e += kTsWarps * 32) {
        const int t = e / VPR, c = e % VPR, key = p * kTsKeys + t;
        const bool valid = key < kv_len;
        int blk = valid ? __ldg(bt + key / kBS) : 0;
        if (unsigned(blk) >= unsigned(a.num_blocks)) {
          flag(PA_DEV_BAD_BLOCK);
          blk = 0;
        }
        const int64_t off = ((int64_t(blk) * a.Hkv + kvh) * kBS + key % kBS) * D + c * 4;
        cp_async16(Ks + t * C::KSTR + c * 4, kc + off, valid);
        cp_async16(Vs + t * D + c * 4, vc + off, valid);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(sg.b);
    for (int e = threadIdx.x; e < R * VPR; e += kTsWarps * 32) {
      const int r = e / VPR, c = e % VPR;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int tok = (r0 + r) >> a.lg, j = (r0 + r) & gm;
        f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (x.s.q0 + tok) * a.q_st +
                                             ((kvh << a.lg) + j) * a.q_sh + c * 4);
      }
      const float k = a.scale_log2;
      reinterpret_cast<float4*>(Qs + r * D)[c] = make_float4(f.x * k, f.y * k, f.z * k, f.w * k);
    }
    float o[RW][PER], m[RW], l[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[r][e] = 0.f;
    }
    for (int p = sg.b; p < sg.e; ++p) {
      const int key0 = p * kTsKeys;
      if (p + 1 < sg.e) {
        load(p + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();  // every thread's copies of this tile, and the query rows, are there
      if (warp * RW < rows) {
        const float* const Ks = stage0 + (p & 1) * C::STAGE;
        const float* const Vs = Ks + kTsKeys * C::KSTR;
        float s[RW];
#pragma unroll
        for (int r = 0; r < RW; ++r) s[r] = 0.f;
        const float4* kr = reinterpret_cast<const float4*>(Ks + lane * C::KSTR);
        const float4* qr = reinterpret_cast<const float4*>(Qs + warp * RW * D);
#pragma unroll 4
        for (int d = 0; d < VPR; ++d) {
          const float4 k4 = kr[d];
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float4 q4 = qr[r * VPR + d];
            s[r] = fmaf(q4.x, k4.x, s[r]);
            s[r] = fmaf(q4.y, k4.y, s[r]);
            s[r] = fmaf(q4.z, k4.z, s[r]);
            s[r] = fmaf(q4.w, k4.w, s[r]);
          }
        }
        const bool tree = key0 + kTsKeys > x.s.c0;  // some keys are drafted, or past the end
        uint32_t seen[RW];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const int row = r0 + warp * RW + r;
          seen[r] = 0xffffffffu;
          if (tree)
            seen[r] = row < (x.s.n << a.lg) ? tree_seen32(a, x.s.q0 + (row >> a.lg), x.s.n, key0 - x.s.c0) : 0u;
          const bool vis = (seen[r] >> lane) & 1u;
          if (!vis) s[r] = -INFINITY;
          float mx = s[r];
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
          const float mn = fmaxf(m[r], mx);
          // no key seen so far, or only logits of -infinity, which weigh nothing
          // beside the finite ones that may follow
          const float mu = mn == -INFINITY ? 0.f : mn;
          const float al = ex2(m[r] - mu);
          m[r] = mn;
          s[r] = vis ? ex2(s[r] - mu) : 0.f;
          l[r] = l[r] * al + s[r];
#pragma unroll
          for (int e = 0; e < PER; ++e) o[r][e] *= al;
        }
        if constexpr (RW == 2) {
          *reinterpret_cast<float2*>(Ps + lane * RW) = make_float2(s[0], s[1]);
        } else {
#pragma unroll
          for (int r = 0; r < RW; r += 4)
            *reinterpret_cast<float4*>(Ps + lane * RW + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
        }
        __syncwarp();
        auto weigh = [&](int t, bool masked) {
          float v[PER];
#pragma unroll
          for (int e = 0; e < PER; ++e) v[e] = Vs[t * D + lane * PER + e];
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float pt = Ps[t * RW + r];
            if (masked && !((seen[r] >> t) & 1u)) continue;  // a masked V may hold anything
#pragma unroll
            for (int e = 0; e < PER; ++e) o[r][e] = fmaf(pt, v[e], o[r][e]);
          }
        };
        if (!tree) {
#pragma unroll 4
          for (int t = 0; t < kTsKeys; ++t) weigh(t, false);
        } else {
          const int nk = min(kTsKeys, kv_len - key0);
#pragma unroll 1
          for (int t = 0; t < nk; ++t) weigh(t, true);
        }
      }
      __syncthreads();  // the stage may be filled again
    }
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], k);

    // ---- the segment's result: rows of the output, or a share of a cut unit ----
    const bool whole = sg.e - sg.b == x.nt;
    const int unit0 = cx - x.p + kTsLead;  // the unit's first tile in the list
    if (a.cut != nullptr && threadIdx.x == 0 && sg.b == 0) a.cut[x.number] = tree_cut(rg, x, sg, unit0);
    bool write = whole;
    if (!whole) {
      const int slot = 2 * int(blockIdx.x) + (sg.b == 0);
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const int row = warp * RW + r;
        if (row >= rows) continue;
        float* dst = reinterpret_cast<float*>(tree_share<D, R>(a, slot, row, lane * PER / 4)) + lane * PER % 4;
#pragma unroll
        for (int e = 0; e < PER; ++e) __stcg(dst + e, o[r][e]);
        if (lane == 0) __stcg(a.sh_ml + slot * R + row, make_float2(m[r], l[r]));
      }
      const int wa = a.cut == nullptr ? rg.owner(unit0) : 0;
      write = a.cut == nullptr && share_done(a.cnt + wa * kTsWarps + warp, sg.e - sg.b, x.nt);
      if (write) {
        // Lane t holds the (max, denominator) pair of share k0 + t and turns
        // it into a weight; the weights are broadcast while every lane adds
        // its dims, several shares' loads in flight.
        const int ns = rg.owner(unit0 + x.nt - 1) - wa + 1;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          if (warp * RW + r >= rows) continue;
          const int64_t row0 = warp * RW + r;
          auto pair = [&](int k) {
            return k < ns ? __ldcg(a.sh_ml + share_slot(wa + k, wa) * R + row0) : make_float2(-INFINITY, 0.f);
          };
          float mx = -INFINITY;
          for (int k0 = 0; k0 < ns; k0 += 32) mx = fmaxf(mx, pair(k0 + lane).x);
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
          const float mu = mx == -INFINITY ? 0.f : mx;
          l[r] = 0.f;
#pragma unroll
          for (int e = 0; e < PER; ++e) o[r][e] = 0.f;
          for (int k0 = 0; k0 < ns; k0 += 32) {
            const float2 ml = pair(k0 + lane);
            const float wl = ex2(ml.x - mu);
            l[r] += ml.y * wl;
            const int nk = min(32, ns - k0);
#pragma unroll 8
            for (int t = 0; t < nk; ++t) {
              const float w = __shfl_sync(0xffffffffu, wl, t);
              const float* src = reinterpret_cast<const float*>(tree_share<D, R>(
                                     a, int(share_slot(wa + k0 + t, wa)), int(row0), lane * PER / 4)) + lane * PER % 4;
#pragma unroll
              for (int e = 0; e < PER; ++e) o[r][e] = fmaf(w, __ldcg(src + e), o[r][e]);
            }
          }
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], k);
        }
      }
    }
    if (write) {
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        if (warp * RW + r >= rows) continue;
        const int row = r0 + warp * RW + r;
        const float inv = tree_inverse(a, l[r], x.s.c0, x.s.n, x.s.q0 + (row >> a.lg));
        float y[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) y[e] = o[r][e] * inv;
        store_out_small<float, PER>(static_cast<float*>(a.out) + (x.s.q0 + (row >> a.lg)) * a.o_st +
                                    ((kvh << a.lg) + (row & gm)) * a.o_sh + lane * PER,
                                y);
      }
    }
    cx += sg.pe - x.p;
    if (cx < rg.hi) tree_next_unit<R, kTsKeys>(a, x);
  }
}

// ---- merge by a second launch ---------------------------------------------------
// out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k over a unit's shares k.
// Block (x, y, z): unit x, RG of its rows, the z-th part of the dims; a thread
// holds one float4 of one row.  The 8 warps first reduce every row's maximum
// and denominator, each over every 8th share; then they split the block's
// dims and the shares, 8 of them in flight a thread.  Bound by latency (100
// shares of a unit are some 4 MB in L2).
constexpr int kTmThreads = 256;

template <typename T, int D, int R>
__global__ void __launch_bounds__(kTmThreads) tree_merge_kernel(const TreeArgs a) {
  constexpr int RG = R < 32 ? R : 32, DPL = 32 / RG, UN = 8;
  __shared__ float2 part[8][RG];
  __shared__ float4 sum[8][32];
  pdl_wait();
  pdl_launch_dependents();
  if (int(blockIdx.x) >= *a.units) return;
  const TreeCut c = a.cut[blockIdx.x];
  if (c.ns == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y * RG + lane % RG;
  if (c.rt * R + int(blockIdx.y) * RG >= (c.n << a.lg)) return;  // no such rows (the whole block)
  auto slot = [&](int k) { return 2 * (c.wa + k) + (k == 0); };
  auto pair = [&](int k) {
    return k < c.ns ? __ldcg(a.sh_ml + slot(k) * R + r) : make_float2(-INFINITY, 0.f);
  };
  float M = -INFINITY, L = 0.f;
  for (int k0 = warp; k0 < c.ns; k0 += 32) {
    float2 ml[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) ml[k] = pair(k0 + 8 * k);
    const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
    const float mu = mn == -INFINITY ? 0.f : mn;
    L *= ex2(M - mu);
    M = mn;
#pragma unroll
    for (int k = 0; k < 4; ++k) L += ml[k].y * ex2(ml[k].x - mu);
  }
  if (lane < RG) part[warp][lane] = make_float2(M, L);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, part[w][lane % RG].x);
  const float mu = M == -INFINITY ? 0.f : M;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) L += part[w][lane % RG].y * ex2(part[w][lane % RG].x - mu);

  // this warp's float4 of the dims, and its shares: k0 and every SPL
  const int count = D / 4 / gridDim.z;
  const int SPL = 8 * DPL / count, k0 = warp % SPL;
  const int d = blockIdx.z * count + warp / SPL * DPL + lane / RG;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = k0; k < c.ns; k += UN * SPL) {
    float4 v[UN];
    float w[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int ku = k + u * SPL;
      w[u] = ex2(pair(ku).x - mu);
      v[u] = ku < c.ns ? __ldcg(tree_share<D, R>(a, slot(ku), r, d)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      o.x = fmaf(w[u], v[u].x, o.x);
      o.y = fmaf(w[u], v[u].y, o.y);
      o.z = fmaf(w[u], v[u].z, o.z);
      o.w = fmaf(w[u], v[u].w, o.w);
    }
  }
  sum[warp][lane] = o;
  __syncthreads();
  if (k0 != 0) return;
  for (int w = 1; w < SPL; ++w) {
    const float4 y = sum[warp + w][lane];
    o = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
  }
  const int row = c.rt * R + r;
  if (row >= (c.n << a.lg)) return;
  const int tok = row >> a.lg;
  const float inv = tree_inverse(a, L, c.c0, c.n, c.q0 + tok);
  T* dst = static_cast<T*>(a.out) + int64_t(c.q0 + tok) * a.o_st + ((c.h << a.lg) + (row & ((1 << a.lg) - 1))) * a.o_sh;
  const float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  store_out_small<T, 4>(dst + 4 * d, y);
}

// ---- accepted path --------------------------------------------------------
// cache position c_i + k  <-  position c_i + accepted[i][k], k < count[i], for
// K and V of every head.  The accepted indices ascend strictly (children
// follow their parents in a draft), so accepted[k] >= k and a row is only
// ever overwritten after it was read, in the order k = 0, 1, ...  One thread
// owns one 16-byte column of a (sequence, head) and walks its path: no two
// threads touch the same bytes, so the walk needs no synchronisation.  Pure
// copy of a few rows a sequence, bound by the latency of its dependent steps
// (lengths, path, block ids, rows): lane k of each warp looks step k of the
// path up, 32 at a time, and kCommitBatch rows are loaded at once.
constexpr int kCommitBatch = 8;

struct CommitArgs {
  uint4* kc;
  uint4* vc;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qs;
  const int32_t* acc;
  const int32_t* count;
  int64_t bt_stride, acc_stride;
  int32_t B, Hkv, max_nb, num_blocks, P, vpr;
};

__global__ void __launch_bounds__(128) tree_commit_kernel(const CommitArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int per_seq = a.Hkv * 2 * a.vpr;
  const int i = blockIdx.y, lane = threadIdx.x & 31;
  const int id = blockIdx.x * blockDim.x + threadIdx.x;
  const int count = __ldg(a.count + i);
  const int64_t n = int64_t(__ldg(a.qs + i + 1)) - __ldg(a.qs + i);
  const int ctx = __ldg(a.ctx + i);
  if (count == 0) return;
  const int32_t* acc = a.acc + int64_t(i) * a.acc_stride;
  const int32_t* bt = a.bt + int64_t(i) * a.bt_stride;
  bool ok = count > 0 && count <= a.P && n >= count && n <= ctx && ctx <= a.max_nb * kBS;
  const int c0 = ctx - int(n);
  // The whole path first: strictly ascending in [0, n), every block in the
  // pool; else nothing of the sequence moves.  (Steps the next round reads
  // again; a path rarely has over 32.)
  int u = 0;
  bool blocks_ok = true;
  int64_t src = 0, dst = 0;  // this lane's step: row indices of head 0
  auto step = [&](int k0) {
    const int k = k0 + lane;
    bool good = true;
    u = k;
    if (k < count) {
      u = __ldg(acc + k);
      good = u >= k && u < n && (k == 0 || __ldg(acc + k - 1) < u);
      if (good) {
        const int sb = __ldg(bt + (c0 + u) / kBS), db = __ldg(bt + (c0 + k) / kBS);
        blocks_ok &= unsigned(sb) < unsigned(a.num_blocks) && unsigned(db) < unsigned(a.num_blocks);
        src = int64_t(sb) * a.Hkv * kBS + (c0 + u) % kBS;
        dst = int64_t(db) * a.Hkv * kBS + (c0 + k) % kBS;
      }
    }
    return __all_sync(0xffffffffu, good);
  };
  // the last round first, so that a path of one round is looked up once
  const int last = ok ? (count - 1) / 32 * 32 : 0;
  for (int k0 = last; ok && k0 >= 0; k0 -= 32) ok = step(k0);
  blocks_ok = __all_sync(0xffffffffu, blocks_ok);
  if (!ok || !blocks_ok) {
    if (id == 0) flag(ok ? PA_DEV_BAD_BLOCK : PA_DEV_BAD_CONTEXT);
    return;
  }
  const int c = id % a.vpr, kv = (id / a.vpr) & 1, h = id / (2 * a.vpr);
  uint4* const col = (kv ? a.vc : a.kc) + int64_t(h) * kBS * a.vpr + c;
  for (int k0 = 0; k0 < count; k0 += 32) {
    if (k0 > 0) step(k0);
    for (int k1 = 0; k1 < 32 && k0 + k1 < count; k1 += kCommitBatch) {
      uint4 row[kCommitBatch];
      int64_t to[kCommitBatch];
      bool move[kCommitBatch];
#pragma unroll
      for (int k = 0; k < kCommitBatch; ++k) {
        const int64_t from = __shfl_sync(0xffffffffu, src, k1 + k) * a.vpr;
        to[k] = __shfl_sync(0xffffffffu, dst, k1 + k) * a.vpr;
        const int at = __shfl_sync(0xffffffffu, u, k1 + k);  // (every lane, also those past the last column)
        move[k] = id < per_seq && at != k0 + k1 + k;
        if (move[k]) row[k] = __ldcg(col + from);
      }
#pragma unroll
      for (int k = 0; k < kCommitBatch; ++k)
        if (move[k]) col[to[k]] = row[k];
    }
  }
}

}  // namespace pa

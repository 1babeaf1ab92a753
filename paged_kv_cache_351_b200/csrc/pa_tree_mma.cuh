// Tree attention on the tensor cores (sm_100a), bf16 caches.  The operator,
// its work list and the shares of cut units are described in pa_tree.cuh.
//
// One CTA works on one unit at a time: HALVES x 128 query rows (drafted
// tokens times the G heads of a kv head) against key tiles of KT tokens.
//   S = Q K^T        tcgen05.mma, M = 128, N = KT, fp32 in TMEM;
//   P = exp(S - m)   one query row per thread, rounded to bf16 for the next
//                    product (the denominator sums the unrounded values);
//   O += P V         tcgen05.mma with P read from TMEM (bf16 pairs over S).
// P in bf16: the 16-bit products take both operands in one type, V's, at
// twice the rate and half the TMEM of 32-bit ones; a term is off by at most
// 2^-8 of itself, and the outputs' mean relative error against 64 bits goes
// from 0.0017 (their own rounding) to 0.0021-0.0023.
// A drafted step is bound by the K/V bytes while it has up to about 128 rows
// a unit: 64 KiB of K/V per 128 keys take 1.5 us of an SM's share of HBM, the
// padded M = 128 products 0.75 us.  Hence two variants:
//  * up to 128 rows: KT = 64, two S buffers (Q K^T of the next tile runs
//    while this one is in its softmax), 97 KiB of shared memory, 256 TMEM
//    columns: two CTAs per SM, so one streams while the other starts,
//    drains, merges or waits for its softmax;
//  * more rows: two halves that share every K/V tile in shared memory (the
//    K/V bytes an SM pulls would otherwise double), KT = 128, one CTA per
//    SM, the halves' products and softmaxes alternating; P V starts on the
//    first half of a tile's keys while the softmax is at the second.
// Roles: warp 0 loads K, warp 2 loads V, warp 3 loads Q (tiled TMA with
// 128-byte swizzle; a page is a [16 tokens][64 dims] box per half of the head
// dimension), warp 1 owns TMEM and issues the products, warps 4.. run the
// softmax and the epilogue.  The K and V rings run on across units.  Every
// wait is bounded by the caller's timeout, after which each role stops and
// waits (bounded) for its own copies or products in flight.
#pragma once

#include <cfloat>

#include "pa_prefill.cuh"
#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {

namespace tc {

// Whole warp: multiplies 8 consecutive fp32 columns of each lane's TMEM lane
// by f (one load, one store; few registers).  Complete with tmem_wait_st.
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f) {
  float v[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

}  // namespace tc

template <int D, int HALVES>
struct TreeMma {
  static constexpr int R = 128 * HALVES;
  static constexpr int KT = HALVES == 1 ? 64 : 128;
  static constexpr int NB = HALVES == 1 ? 2 : 1;  // S buffers per half
  // A unit's cost beside its tiles, in tiles (LLaMA batch of 16-token trees,
  // 12 tiles a unit: 0.197 ms with 0, 0.172 with 1, 0.154 with 2, 0.150 with
  // 3).
  static constexpr int LEAD = HALVES == 1 ? 3 : 1;
  static constexpr int NH = D / 64;               // 64-dim halves of the head dimension
  static constexpr int THREADS = 128 + HALVES * 128;
  static constexpr int CTAS = HALVES == 1 ? 2 : 1;  // per SM
  static constexpr uint32_t QHALF = 128 * 128;      // bytes of one 64-dim half of a 128-row Q tile
  static constexpr uint32_t QTILE = NH * QHALF;
  static constexpr uint32_t KHALF = KT * 128;
  static constexpr uint32_t STAGE = NH * KHALF;  // one K (or V) tile
  static constexpr int KST = D == 64 ? 4 : HALVES == 1 ? 2 : 3;
  static constexpr int VST = D == 64 ? 4 : 2;
  static constexpr int MAXT = PA_TREE_MAX_QUERY / KT + 1;  // key tiles that can hold drafted tokens
  static constexpr uint32_t K0 = HALVES * QTILE;
  static constexpr uint32_t V0 = K0 + KST * STAGE;
  static constexpr uint32_t BAR = V0 + VST * STAGE;
  static constexpr uint32_t SCAN = BAR + 256;            // 41 ints
  // [4][MAXT][4] words (see "Sanitise V"): warps of one half are at most two
  // segments apart, since a tile's products wait for all of them
  static constexpr uint32_t NONFIN = SCAN + 176;
  static constexpr uint32_t SMEM = NONFIN + 4 * MAXT * 4 * 4 + 1024;  // + alignment slack
  // TMEM columns: S buffers, then O of each half
  static constexpr uint32_t TO = HALVES * NB * KT;
  static constexpr uint32_t TCOLS = HALVES == 1 ? 256 : 512;
  static_assert(TO + HALVES * D <= TCOLS, "TMEM");
  static_assert(CTAS * (SMEM + 1024) <= 233472 && SMEM <= 232448, "shared memory");
};

// Barrier slots (8 bytes each).
enum TmBar : int {
  kTmKFull = 0,   // + stage (4)
  kTmKFree = 4,   // + stage (4)
  kTmVFull = 8,   // + stage (4)
  kTmVFree = 12,  // + stage (4)
  kTmQFull = 16,
  kTmQFree = 17,
  kTmSFull = 18,  // + half * NB + buffer (2)
  kTmPFull = 20,  // + half (2), 128 arrivals
  kTmODone = 22,  // + half (2)
  kTmDrain = 24,
  kTmBDone = 25,  // half B's warps have read a unit's results, 4 arrivals
  kTmSlot = 26,   // 4-byte TMEM base address
  kTmPPart = 27,  // + half (2), 128 arrivals: the first half of P's keys (two halves only)
  kTmLast = 29,   // + half * 4 bytes: this half completes a cut unit
};

// bf16 pair: a mask of the halves (low 0xffff, high 0xffff0000) that are infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// The largest of three; NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The four softmax warps of one half.
__device__ __forceinline__ void half_sync(int hx) { asm volatile("bar.sync %0, 128;" ::"r"(1 + hx) : "memory"); }

// The merge of a cut unit's shares, of ns workers from wa on, by the four warps
// of a half (all their lanes): 32 rows x D / parts dims a warp, the weights
// once, then 16 dims of up to four shares at a time.  Out of line, so that
// its registers do not burden the softmax.
template <int D, int HALVES>
__device__ __noinline__ void tree_merge(const TreeArgs& a, const TreePos x, int wa, int ns, int hx, int quad,
                                        int rows) {
  const int lane = threadIdx.x & 31;
  const int groups = (min(128, rows - hx * 128) + 31) / 32;
  const int parts = groups == 1 ? 4 : groups == 2 ? 2 : 1;
  const int r = quad % (4 / parts) * 32 + lane;
  const int dl = D / parts * (quad / (4 / parts)), dh = dl + D / parts;
  if (r / 32 >= groups) return;
  constexpr int R = TreeMma<D, HALVES>::R;
  auto slot_of = [&](int k) { return int(share_slot(wa + k, wa)); };
  auto pair = [&](int k) {
    return k < ns ? __ldcg(a.sh_ml + slot_of(k) * R + hx * 128 + r) : make_float2(-INFINITY, 0.f);
  };
  float M = -INFINITY, L = 0.f;
  for (int k0 = 0; k0 < ns; k0 += 4) {
    float2 ml[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) ml[k] = pair(k0 + k);
    const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
    const float mu = mn == -INFINITY ? 0.f : mn;
    L *= ex2(M - mu);
    M = mn;
#pragma unroll
    for (int k = 0; k < 4; ++k) L += ml[k].y * ex2(ml[k].x - mu);
  }
  const float mu = M == -INFINITY ? 0.f : M;
  const bool valid = hx * 128 + r < rows;
  const int row = x.rt * TreeMma<D, HALVES>::R + hx * 128 + r, tk = valid ? row >> a.lg : 0;
  const float inv = tree_inverse(a, L, x.s.c0, x.s.n, x.s.q0 + tk);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (x.s.q0 + tk) * a.o_st +
                       ((x.h << a.lg) + (row & ((1 << a.lg) - 1))) * a.o_sh;
#pragma unroll 1
  for (int d0 = dl; d0 < dh; d0 += 16) {
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < ns; k0 += 4) {
      float4 v[4][4];
      float w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool on = k0 + k < ns;
        w[k] = ex2(pair(k0 + k).x - mu);
        const float4* src = tree_share<D, R>(a, slot_of(k0 + k), hx * 128 + r, d0 / 4);
#pragma unroll
        for (int d = 0; d < 4; ++d) v[k][d] = on ? __ldcg(src + d * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          o[4 * d] = fmaf(w[k], v[k][d].x, o[4 * d]);
          o[4 * d + 1] = fmaf(w[k], v[k][d].y, o[4 * d + 1]);
          o[4 * d + 2] = fmaf(w[k], v[k][d].z, o[4 * d + 2]);
          o[4 * d + 3] = fmaf(w[k], v[k][d].w, o[4 * d + 3]);
        }
    }
    if (valid) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        reinterpret_cast<uint4*>(dst + d0)[e] = make_uint4(
            pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
            pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv), pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
    }
  }
}

template <int D, int HALVES>
__global__ void __launch_bounds__(TreeMma<D, HALVES>::THREADS, TreeMma<D, HALVES>::CTAS)
    tree_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeArgs a) {
  using C = TreeMma<D, HALVES>;
  constexpr int KT = C::KT, NB = C::NB, R = C::R;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + C::BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int st = 0; st < 16; ++st) mbar_init(bar(st), 1);
    mbar_init(bar(kTmQFull), 1);
    mbar_init(bar(kTmQFree), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kTmSFull + x), 1);
      mbar_init(bar(kTmPFull + x), 128);
      mbar_init(bar(kTmPPart + x), 128);
      mbar_init(bar(kTmODone + x), 1);
    }
    mbar_init(bar(kTmDrain), 1);
    mbar_init(bar(kTmBDone), 4);
    fence_barrier_init();
    tc::tma_prefetch_desc(&tm_q);
    tc::tma_prefetch_desc(&tm_k);
    tc::tma_prefetch_desc(&tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  const TreeRange rg = tree_range<R, KT, C::LEAD>(a, reinterpret_cast<int*>(gbase + C::SCAN));
  if (rg.lo >= rg.hi) return;  // the whole CTA: nothing allocated or in flight
  if (warp == 1) tc::tmem_alloc(bar(kTmSlot), C::TCOLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + C::BAR + 8 * kTmSlot);

  // Every role walks the same segments: this worker's key tiles [b, e) of one
  // unit after another.  t counts tiles, seg segments.
  TreePos x = rg.at;
  int cx = rg.lo;
  TreeSeg sg{0, 0, 0};
  auto unit_rows = [&](int& kvh, int& r0) {  // kv head, first row and rows of the unit
    kvh = x.h;
    r0 = x.rt * R;
    return min(R, (x.s.n << a.lg) - r0);
  };
  auto advance = [&]() {
    cx += sg.pe - x.p;
    if (cx < rg.hi) tree_next_unit<R, KT>(a, x);
  };
  // the segment at cx, past parts that hold no tile; false at the end
  auto next_seg = [&]() {
    while (cx < rg.hi) {
      sg = tree_seg<C::LEAD>(x, rg.hi - cx);
      if (sg.b < sg.e) return true;
      advance();
    }
    return false;
  };

  if (warp == 0 || warp == 2) {
    // ---------------- K and V producers ----------------
    const bool is_k = warp == 0;
    const int nst = is_k ? C::KST : C::VST;
    const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
    const uint32_t ring = base + (is_k ? C::K0 : C::V0);
    const int full0 = is_k ? kTmKFull : kTmVFull, free0 = is_k ? kTmKFree : kTmVFree;
    int t = 0;
    bool ok = true;
    while (ok && next_seg()) {
      int kvh, r0;
      unit_rows(kvh, r0);
      const int npages = (x.s.c0 + x.s.n + kBS - 1) / kBS;
      const int32_t* bt = a.bt + int64_t(x.i) * a.bt_stride;
      int win = -1, ids = 0;  // 32 block ids of the table from page `win` on, one per lane
      for (int p = sg.b; p < sg.e; ++p, ++t) {
        const int st = t % nst;
        const int p0 = p * (KT / kBS), np = min(KT / kBS, npages - p0);
        if (win < 0 || p0 + KT / kBS > win + 32) {
          win = p0;
          ids = p0 + lane < npages ? __ldg(bt + p0 + lane) : 0;
          if (unsigned(ids) >= unsigned(a.num_blocks)) {
            flag(PA_DEV_BAD_BLOCK);
            ids = 0;
          }
        }
        if (t >= nst && !(ok = warp_wait(bar(free0 + st), (t / nst - 1) & 1, a.timeout_ns))) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(full0 + st), uint32_t(np) * (C::NH * 2048u));
        for (int g = 0; g < np; ++g) {
          const int b = __shfl_sync(0xffffffffu, ids, p0 + g - win);
          if (lane == 0) {
            const uint32_t d = ring + uint32_t(st) * C::STAGE + uint32_t(g) * 2048u;
#pragma unroll
            for (int h = 0; h < C::NH; ++h)
              tc::tma_load_4d(d + uint32_t(h) * C::KHALF, tm, h * 64, 0, kvh, b, bar(full0 + st));
          }
        }
      }
      advance();
    }
    // before the CTA may exit, every copy it started must have landed
    for (int j = max(0, t - nst); j < t; ++j) mbar_wait_bounded(bar(full0 + j % nst), (j / nst) & 1, a.timeout_ns);
  } else if (warp == 3) {
    // ---------------- Q producer ----------------
    int seg = 0;
    bool ok = true;
    while (ok && next_seg()) {
      int kvh, r0;
      unit_rows(kvh, r0);
      if (seg > 0 && !(ok = warp_wait(bar(kTmQFree), (seg - 1) & 1, a.timeout_ns))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kTmQFull), HALVES * C::QTILE);
#pragma unroll
        for (int e = 0; e < HALVES * C::NH; ++e)
          tc::tma_load_3d(base + uint32_t(e) * C::QHALF, &tm_q, (e % C::NH) * 64, kvh << a.lg,
                          x.s.q0 + ((r0 + (e / C::NH) * 128) >> a.lg), bar(kTmQFull));
      }
      ++seg;
      advance();
    }
    if (seg > 0) mbar_wait_bounded(bar(kTmQFull), (seg - 1) & 1, a.timeout_ns);
  } else if (warp == 1) {
    // ---------------- product issuer ----------------
    constexpr uint32_t kIdQK = tc::idesc_bf16_f32(128, KT, false, false);
    constexpr uint32_t kIdPV = tc::idesc_bf16_f32(128, D, false, true);
    int cnt[2] = {0, 0};  // tiles of each half so far (Q K^T side)
    auto s_col = [&](int hx, int c) { return tmem + uint32_t((hx * NB + c % NB) * KT); };
    auto qk = [&](int t, int hx, int c) {  // S = Q K^T of tile t (lane 0); c = the half's tile count
      const uint32_t kb = base + C::K0 + uint32_t(t % C::KST) * C::STAGE;
      const uint32_t qb = base + uint32_t(hx) * C::QTILE;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc::mma_bf16_ss(s_col(hx, c), tc::desc_kmajor(qb + uint32_t(kk >> 2) * C::QHALF + uint32_t(kk & 3) * 32u),
                        tc::desc_kmajor(kb + uint32_t(kk >> 2) * C::KHALF + uint32_t(kk & 3) * 32u), kIdQK, kk > 0);
      tc::commit(bar(kTmSFull + hx * NB + c % NB));
    };
    auto pv = [&](int t, int hx, int c, bool first, int k0, int k1) {  // O (+)= P V of tile t, keys [16 k0, 16 k1) (lane 0)
      const uint32_t vb = base + C::V0 + uint32_t(t % C::VST) * C::STAGE;
#pragma unroll
      for (int kk = k0; kk < k1; ++kk)
        tc::mma_bf16_ts(tmem + C::TO + uint32_t(hx * D), s_col(hx, c) + uint32_t(kk) * 8u,
                        tc::desc_mnmajor(vb + uint32_t(kk) * 2048u, C::KHALF), kIdPV, !first || kk > 0);
      if (k1 == KT / 16) tc::commit(bar(kTmODone + hx));
    };
    int t = 0, seg = 0;
    bool ok = true;
    while (ok && next_seg()) {
      int kvh, r0;
      const bool has_b = HALVES == 2 && unit_rows(kvh, r0) > 128;
      const int nt = sg.e - sg.b;
      // Q K^T of the segment's tile j, both halves or one, then the stage is free
      auto issue_qk = [&](int j, int hx, bool last_half) {
        if (lane == 0) {
          qk(t + j, hx, cnt[hx]);
          if (last_half) {
            tc::commit(bar(kTmKFree + (t + j) % C::KST));
            if (j == nt - 1) tc::commit(bar(kTmQFree));
          }
        }
        __syncwarp();
        ++cnt[hx];
      };
      auto k_ready = [&](int j) {
        const bool r = warp_wait(bar(kTmKFull + (t + j) % C::KST), ((t + j) / C::KST) & 1, a.timeout_ns);
        tc::fence_after_sync();
        return r;
      };
      if (!(ok = warp_wait(bar(kTmQFull), seg & 1, a.timeout_ns) && k_ready(0))) break;
      issue_qk(0, 0, !has_b);
      if (has_b) issue_qk(0, 1, true);
      for (int j = 0; j < nt; ++j) {
        const int sv = (t + j) % C::VST;
        const bool more = j + 1 < nt;
        if constexpr (NB == 2) {
          // the other S buffer is free: P V of tile j - 1, which read it, was issued before
          if (more) {
            if (!(ok = k_ready(j + 1))) break;
            issue_qk(j + 1, 0, true);
          }
          const int c = cnt[0] - (more ? 2 : 1);
          if (!(ok = warp_wait(bar(kTmVFull + sv), ((t + j) / C::VST) & 1, a.timeout_ns))) break;
          if (!(ok = warp_wait(bar(kTmPFull), c & 1, a.timeout_ns))) break;
          tc::fence_after_sync();
          if (lane == 0) {
            pv(t + j, 0, c, j == 0, 0, KT / 16);
            tc::commit(bar(kTmVFree + sv));
          }
          __syncwarp();
        } else {
          const int ca = cnt[0] - 1, cb = cnt[1] - 1;
          if (!(ok = warp_wait(bar(kTmVFull + sv), ((t + j) / C::VST) & 1, a.timeout_ns))) break;
          // the first half of P's keys while the softmax is at the second
          if (!(ok = warp_wait(bar(kTmPPart), ca & 1, a.timeout_ns))) break;
          tc::fence_after_sync();
          if (lane == 0) pv(t + j, 0, ca, j == 0, 0, KT / 32);
          __syncwarp();
          if (!(ok = warp_wait(bar(kTmPFull), ca & 1, a.timeout_ns))) break;
          tc::fence_after_sync();
          if (lane == 0) {
            pv(t + j, 0, ca, j == 0, KT / 32, KT / 16);
            if (!has_b) tc::commit(bar(kTmVFree + sv));
          }
          __syncwarp();
          if (more) {
            if (!(ok = k_ready(j + 1))) break;
            issue_qk(j + 1, 0, !has_b);
          }
          if (has_b) {
            if (!(ok = warp_wait(bar(kTmPPart + 1), cb & 1, a.timeout_ns))) break;
            tc::fence_after_sync();
            if (lane == 0) pv(t + j, 1, cb, j == 0, 0, KT / 32);
            __syncwarp();
            if (!(ok = warp_wait(bar(kTmPFull + 1), cb & 1, a.timeout_ns))) break;
            tc::fence_after_sync();
            if (lane == 0) {
              pv(t + j, 1, cb, j == 0, KT / 32, KT / 16);
              tc::commit(bar(kTmVFree + sv));
            }
            __syncwarp();
            if (more) issue_qk(j + 1, 1, true);
          }
        }
      }
      t += nt;
      ++seg;
      advance();
    }
    // no product may still run when TMEM is released
    if (lane == 0) tc::commit(bar(kTmDrain));
    __syncwarp();
    mbar_wait_bounded(bar(kTmDrain), 0, a.timeout_ns);
  } else {
    // ---------------- softmax and epilogue: one query row per thread ----------------
    const int hx = (warp - 4) >> 2, quad = warp & 3;
    const int rr = quad * 32 + lane;  // row within the half = TMEM lane
    const uint32_t tl = tmem + (uint32_t(quad * 32) << 16);
    const uint32_t tO = tl + C::TO + uint32_t(hx * D);
    const float cl = a.scale_log2;
    // the exponent offset moves only when a row's max exceeds it by more than
    // 2^8, so that O is rarely rescaled (see prefill_kernel); finite for any
    // scale, since a row's first maximum is compared with -infinity + thr
    const float thr = fminf(8.f / cl, FLT_MAX);
    uint32_t* const nonfin = reinterpret_cast<uint32_t*>(gbase + C::NONFIN);
    int cnt = 0, t = 0, seg = 0;  // tiles of this half, tiles, segments
    int seg_b = 0;                // segments with a half B before this one
    bool ok = true, prev_b = false;
    for (; next_seg(); ++seg) {
      int kvh, r0;
      const int rows = unit_rows(kvh, r0);
      if (HALVES == 2) {
        // half A stays within a segment of half B, which reads what A noted
        // about V (units without a half B would let A run away)
        if (hx == 0 && prev_b && ok) ok = warp_wait(bar(kTmBDone), (seg_b - 1) & 1, a.timeout_ns);
        prev_b = rows > 128;
        seg_b += prev_b;
      }
      const int nt = sg.e - sg.b;
      const int c0 = x.s.c0, n = x.s.n, kv_len = c0 + n;
      const int urow = r0 + hx * 128 + rr;  // row of the sequence's (token, head) list
      const bool row_valid = hx * 128 + rr < rows;
      const bool live = hx * 128 + quad * 32 < rows;  // the warp has a row
      const int tok = urow >> a.lg, hg = urow - (tok << a.lg);
      const int64_t mrow = x.s.q0 + (row_valid ? tok : 0);
      float m_used = -INFINITY, l = 0.f;
      float cr = cl;  // the factor of this row's scores (log2 units)
      if (hx == 0 || rows > 128) {
        for (int j = 0; ok && j < nt; ++j, ++cnt) {
          const int key0 = (sg.b + j) * KT;
          const bool tree = key0 + KT > c0;  // drafted keys, or none, at the tile's end
          if (tree && hx == 0) {
            // Sanitise V: rows past the last key hold anything and drafted
            // tokens may, but P is zero in rows that do not see them, and 0
            // times infinity is NaN.  Clear the former, and infinite or NaN
            // elements of the latter; which drafted rows had any is kept for
            // the epilogue, which gives them to the rows that see them.  Each
            // warp takes KT / 4 keys.
            const int sv = (t + j) % C::VST;
            if (!(ok = warp_wait(bar(kTmVFull + sv), ((t + j) / C::VST) & 1, a.timeout_ns))) break;
            constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte chunks per row, rows per pass
            uint32_t bad = 0;
#pragma unroll 1
            for (int k = 0; k < KT / 4 / RPI; ++k) {
              const int kr = quad * (KT / 4) + k * RPI + lane / CPR, ch = lane % CPR;
              uint4* e = reinterpret_cast<uint4*>(gbase + C::V0 + uint32_t(sv) * C::STAGE +
                                                  uint32_t(ch >> 3) * C::KHALF + uint32_t(kr) * 128u +
                                                  uint32_t(ch & 7) * 16u);
              bool nf = false;
              if (key0 + kr >= kv_len) {
                *e = make_uint4(0u, 0u, 0u, 0u);
              } else if (key0 + kr >= c0) {
                const uint4 v = *e;
                const uint32_t w0 = nonfinite2(v.x), w1 = nonfinite2(v.y), w2 = nonfinite2(v.z), w3 = nonfinite2(v.w);
                nf = (w0 | w1 | w2 | w3) != 0u;
                if (nf) *e = make_uint4(v.x & ~w0, v.y & ~w1, v.z & ~w2, v.w & ~w3);
              }
              const uint32_t vote = __ballot_sync(0xffffffffu, nf);
#pragma unroll
              for (int q = 0; q < RPI; ++q)
                if ((vote >> (q * CPR)) & (CPR == 16 ? 0xFFFFu : 0xFFu)) bad |= 1u << (k * RPI + q);
            }
            if (lane == 0) nonfin[((seg & 3) * C::MAXT + (sg.b + j - c0 / KT)) * 4 + quad] = bad;
            tc::fence_proxy_async_smem();
            __syncwarp();
          }
          float mt = -INFINITY, alpha = 1.f, sum = 0.f;
          bool moved = false;
          // O may be rescaled, and P counted in, only after P V of the previous tile
          auto after_pv = [&]() {
            if (cnt == 0) return true;
            if (!warp_wait(bar(kTmODone + hx), (cnt - 1) & 1, a.timeout_ns)) return false;
            tc::fence_after_sync();
            if (live && moved && j > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) tc::tmem_scale8(tO + uint32_t(c) * 8u, alpha);
            }
            return true;
          };
          if (live) {
            uint32_t seen[KT / 32];
            if (tree) {
#pragma unroll
              for (int w = 0; w < KT / 32; ++w)
                seen[w] = row_valid ? tree_seen32(a, mrow, n, key0 + w * 32 - c0) : 0u;
            }
            if (!(ok = warp_wait(bar(kTmSFull + hx * NB + cnt % NB), (cnt / NB) & 1, a.timeout_ns))) break;
            tc::fence_after_sync();
            const uint32_t tS = tl + uint32_t((hx * NB + cnt % NB) * KT);
            float s[KT];
            __syncwarp();  // tcgen05.ld is warp-collective
            if constexpr (KT == 64)
              tc::tmem_ld64(tS, s);
            else
              tc::tmem_ld128(tS, s);
            if (tree) {
#pragma unroll
              for (int c = 0; c < KT; ++c) s[c] = (seen[c / 32] >> (c % 32)) & 1u ? s[c] : -INFINITY;
            }
            float m8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = s[k];
            if constexpr (HALVES == 1) {
#pragma unroll
              for (int c = 8; c < KT; ++c) m8[c & 7] = fmaxf(m8[c & 7], s[c]);
              mt = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                         fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
              moved = __any_sync(0xffffffffu, mt > m_used + thr);
            } else {
              // A NaN goes through the maximum, since the exponentials on the
              // FMA pipe (below) drop it.
#pragma unroll
              for (int c = 8; c < KT; c += 16)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  m8[k] = c + 8 + k < KT ? max3_nan(m8[k], s[c + k], s[c + 8 + k]) : max3_nan(m8[k], s[c + k], s[c + k]);
              mt = max3_nan(max3_nan(m8[0], m8[1], m8[2]), max3_nan(m8[3], m8[4], m8[5]), max3_nan(m8[6], m8[7], m8[7]));
              moved = __any_sync(0xffffffffu, !(mt <= m_used + thr));
            }
            if (moved) {
              float m_new = HALVES == 1 ? fmaxf(m_used, mt) : max3_nan(m_used, mt, mt);
              // +infinity: no exponential is finite, and the row is NaN
              if (HALVES == 2 && m_new == INFINITY) m_new = NAN;
              alpha = m_new == -INFINITY ? 1.f : ex2((m_used - m_new) * cl);  // 0 on a row's first visible tile
              m_used = m_new;
              // s * cl - mu (one rounding) brings out what mu was rounded by: up to
              // 2^-24 of it, within the error of the products in s, and a factor
              // common to the tiles of one mu; but it over- or underflows from 2^31
              // on.  From 2^30 on two scores that differ are at least 64 apart, so
              // that all but the largest weigh nothing, and they still do with a
              // smaller factor that keeps mu at 2^30.
              cr = fabsf(m_used * cl) > 1073741824.f && m_used != -INFINITY ? 1073741824.f / fabsf(m_used) : cl;
            }
            const float mu = m_used == -INFINITY ? 0.f : m_used * cr;
            if (HALVES == 2 && !(ok = after_pv())) break;
            float rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < KT / 32; ++ch) {
              if (HALVES == 2 && ch == KT / 64) {  // P's first half is complete
                tc::tmem_wait_st();
                tc::fence_before_sync();
                mbar_arrive(bar(kTmPPart + hx));
              }
              uint32_t pw[16];
#pragma unroll
              for (int c = ch * 32; c < ch * 32 + 32; c += 2) {
                float e0 = -mu, e1 = -mu;
                ffma2(e0, e1, s[c], s[c + 1], cr, cr);  // s * cl - mu
                // with two halves the special-function unit would be the
                // bottleneck: a quarter of the exponentials on the FMA pipe
                if (HALVES == 2 && !tree && ((c >> 3) & 3) == 3) {
                  ex2_poly2(e0, e1);
                } else {
                  e0 = ex2(e0);
                  e1 = ex2(e1);
                }
                pw[(c - ch * 32) >> 1] = pack_bf16x2(e0, e1);
                fadd2(rs[c & 7], rs[(c & 7) + 1], rs[c & 7], rs[(c & 7) + 1], e0, e1);
              }
              tc::tmem_st16(tS + uint32_t(ch) * 16u, pw);
            }
            sum = ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
          }
          if ((HALVES == 1 || !live) && !(ok = after_pv())) break;
          if (HALVES == 2 && !live) mbar_arrive(bar(kTmPPart + hx));
          if (live) tc::tmem_wait_st();
          l = l * alpha + sum;
          tc::fence_before_sync();
          mbar_arrive(bar(kTmPFull + hx));
        }
        if (ok) ok = warp_wait(bar(kTmODone + hx), (cnt - 1) & 1, a.timeout_ns);
        // the exponentials on the FMA pipe end at 2^-126, not at 0
        if (HALVES == 2 && m_used == -INFINITY) l = 0.f;
      }
      t += nt;
      const bool whole = nt == x.nt;
      const int unit0 = cx - x.p + C::LEAD;  // the unit's first tile in the list
      if (a.cut != nullptr && sg.b == 0 && threadIdx.x == 128) a.cut[x.number] = tree_cut(rg, x, sg, unit0);
      if (live) {
        // drafted tokens with infinite or NaN elements of V, in the segment's tiles
        const int tf = max(sg.b, c0 / KT);
        uint32_t any = 0;
        for (int p = tf; ok && p < sg.e; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            any |= reinterpret_cast<volatile uint32_t*>(nonfin)[((seg & 3) * C::MAXT + (p - c0 / KT)) * 4 + q];
        auto add_nonfinite = [&](float* o, int d0) {
          for (int p = tf; p < sg.e; ++p)
            for (int q = 0; q < 4; ++q) {
              uint32_t w = reinterpret_cast<volatile uint32_t*>(nonfin)[((seg & 3) * C::MAXT + (p - c0 / KT)) * 4 + q];
              for (; w != 0u; w &= w - 1u) {
                const int key = p * KT + q * (KT / 4) + __ffs(w) - 1, u = key - c0;
                if (!row_valid || !((tree_word(a, mrow, n, u >> 5) >> (u & 31)) & 1u)) continue;
                int blk = __ldg(a.bt + int64_t(x.i) * a.bt_stride + key / kBS);
                if (unsigned(blk) >= unsigned(a.num_blocks)) blk = 0;
                const uint32_t* v = reinterpret_cast<const uint32_t*>(
                    static_cast<const __nv_bfloat16*>(a.vc) + ((int64_t(blk) * a.Hkv + kvh) * kBS + key % kBS) * D + d0);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint32_t e = __ldg(v + i), nf = nonfinite2(e);
                  if (nf & 0xFFFFu) o[2 * i] += __uint_as_float(e << 16);
                  if (nf & 0xFFFF0000u) o[2 * i + 1] += __uint_as_float(e & 0xFFFF0000u);
                }
              }
            }
        };
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (x.s.q0 + tok) * a.o_st + ((kvh << a.lg) + hg) * a.o_sh;
        auto write_row = [&](int c, const float* o, float inv) {
          if (!row_valid) return;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 w;
            w.x = pack_bf16x2(o[8 * v + 0] * inv, o[8 * v + 1] * inv);
            w.y = pack_bf16x2(o[8 * v + 2] * inv, o[8 * v + 3] * inv);
            w.z = pack_bf16x2(o[8 * v + 4] * inv, o[8 * v + 5] * inv);
            w.w = pack_bf16x2(o[8 * v + 6] * inv, o[8 * v + 7] * inv);
            *reinterpret_cast<uint4*>(dst + c * 32 + v * 8) = w;
          }
        };
        if (ok) {
          tc::fence_after_sync();
          const int slot = 2 * int(blockIdx.x) + (sg.b == 0);
          const float inv = whole ? tree_inverse(a, l, c0, n, mrow) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            float o[64];
            __syncwarp();
            tc::tmem_ld64(tO + uint32_t(c) * 64u, o);
            if (any != 0u) {
              add_nonfinite(o, c * 64);
              add_nonfinite(o + 32, c * 64 + 32);
            }
            if (whole) {
              write_row(2 * c, o, inv);
              write_row(2 * c + 1, o + 32, inv);
            } else {
#pragma unroll
              for (int d = 0; d < 16; ++d)
                __stcg(tree_share<D, R>(a, slot, hx * 128 + rr, c * 16 + d),
                       make_float4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]));
            }
          }
          if (HALVES == 2 && hx == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kTmBDone));
          }
          if (!whole)
            __stcg(a.sh_ml + slot * R + hx * 128 + rr, make_float2(m_used == -INFINITY ? -INFINITY : m_used * cl, l));
        }
      } else if (HALVES == 2 && hx == 1 && rows > 128) {
        if (lane == 0) mbar_arrive(bar(kTmBDone));
      }
      if (!whole && rows > hx * 128 && a.cut == nullptr) {
        const int wa = rg.owner(unit0);
        // A cut unit: the half's tiles are counted in (after a timeout too,
        // so that the counters end at zero), and the half that completes the
        // unit merges the shares of its rows, its four warps together.  The
        // barriers are reached by all four warps whatever happened to them.
        half_sync(hx);
        int* const last = reinterpret_cast<int*>(gbase + C::BAR + 8 * kTmLast) + hx;
        if (quad == 0 && lane == 0)
          *reinterpret_cast<volatile int*>(last) = count_in(a.cnt + wa * HALVES + hx, unsigned(nt), unsigned(x.nt));
        half_sync(hx);
        if (*reinterpret_cast<volatile int*>(last) && ok) {
          const int ns = rg.owner(unit0 + x.nt - 1) - wa + 1;
          tree_merge<D, HALVES>(a, x, wa, ns, hx, quad, rows);
        }
      }
      advance();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TCOLS);
  }
}

}  // namespace pa

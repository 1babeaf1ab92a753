// Bounding a sequence's cache by accumulated attention weight (sm_100a): the
// accumulation behind a scored decode, the choice of the tokens that stay,
// and their move into fresh blocks.
#pragma once

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_decode.cuh"

namespace pa {

// ---- accumulation -----------------------------------------------------------
// After a scored decode left the logits (log2 units, [B][H_kv][cap][G]) and
// every row's log-sum-exp (log2 units, [B][H]) in the workspace:
//   scores[i, g, t] += sum_{j < G} 2^(logit[i, g, t, j] - lse[i, g G + j]),  t < ctx_i.
// The weights need the final denominator, which no page knows while it is
// read, hence the second pass over 4 G bytes a token (a second pass over K
// would read 64 times as much at head size 128 and G = 1).  Bound by those
// bytes plus 8 for the score; they are mostly still in L2 (320,000 tokens of 8
// kv heads, G = 4: 16 us with cold caches).  Each score has
// one writer and a fixed order of additions, so results do not vary.
struct AccumArgs {
  const float* logits;
  const float* lse;
  float* scores;
  const int32_t* ctx;
  int64_t s_sb, s_sh;  // strides of scores (elements)
  int32_t B, Hkv, cap, S;
};

constexpr int kAccTokens = 1024;  // per CTA and round

template <int G>
__global__ void __launch_bounds__(256) accumulate_scores_kernel(const AccumArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.y, i = blockIdx.z;
  int n = clamp_ctx(__ldg(a.ctx + i), a.cap);
  if (n > a.S) {
    if (blockIdx.x == 0 && g == 0 && threadIdx.x == 0) flag(PA_DEV_BAD_CONTEXT);
    n = a.S;
  }
  if (int(blockIdx.x) * kAccTokens >= n) return;
  float lse[G];
#pragma unroll
  for (int j = 0; j < G; ++j) lse[j] = a.lse[(int64_t(i) * a.Hkv + g) * G + j];
  const float* lg = a.logits + (int64_t(i) * a.Hkv + g) * a.cap * G;
  float* sc = a.scores + i * a.s_sb + g * a.s_sh;
  // four tokens a thread, their loads in flight together
  for (int t0 = blockIdx.x * kAccTokens + threadIdx.x; t0 < n; t0 += gridDim.x * kAccTokens) {
    float x[4][G], old[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = t0 + k * 256;
      if (t >= n) continue;
      old[k] = sc[t];
      const float* src = lg + int64_t(t) * G;
      if constexpr (G >= 4) {
#pragma unroll
        for (int j = 0; j < G; j += 4) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(src + j));
          x[k][j] = v.x, x[k][j + 1] = v.y, x[k][j + 2] = v.z, x[k][j + 3] = v.w;
        }
      } else if constexpr (G == 2) {
        const float2 v = __ldcs(reinterpret_cast<const float2*>(src));
        x[k][0] = v.x, x[k][1] = v.y;
      } else {
        x[k][0] = __ldcs(src);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t0 + k * 256 >= n) continue;
      float w = 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j) w += ex2(x[k][j] - lse[j]);
      sc[t0 + k * 256] = old[k] + w;
    }
  }
}

// ---- choice -------------------------------------------------------------------
// Sequence i keeps K = min(keep_lens[i], n) of its n tokens: the R =
// min(num_recent, K) newest, the S0 = min(num_sink, K - R) first, and of the
// others the K - R - S0 of largest score, ties to the lower position.
struct EvictArgs {
  const float* scores;
  float* scores_out;
  int32_t* kept;
  const int32_t* ctx;
  const int32_t* keep;
  const int32_t* bt;
  const int32_t* dt;
  uint4* kc;
  uint4* vc;
  int64_t s_sb, s_sh, o_sb, o_sh, k_sb, k_sh, bt_stride, dt_stride;
  int32_t B, Hkv, max_nb, dst_nb, num_blocks, S, So, P, sink, recent, vpr;
};

struct EvictSeq {
  int n, K, R, S0;  // tokens, kept, newest kept, first kept
  bool ok;
};

__device__ __forceinline__ EvictSeq evict_seq(const EvictArgs& a, int i) {
  EvictSeq s;
  s.n = __ldg(a.ctx + i);
  const int keep = __ldg(a.keep + i);
  s.K = min(keep, s.n);
  s.ok = s.n >= 0 && keep >= 0 && s.n <= a.max_nb * kBS && s.n <= a.S && s.K <= a.P && s.K <= a.So &&
         s.K <= a.dst_nb * kBS;
  s.R = min(a.recent, s.K);
  s.S0 = min(a.sink, s.K - s.R);
  return s;
}

// Order-preserving map of a score to an unsigned key: larger score, larger
// key; -0 equals +0, and NaN ranks with -infinity.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

// A cluster of C CTAs chooses for one (sequence, kv head), each warp over a run
// of its tokens: their keys stay in registers, KPT a lane (rows of up to
// 131072 tokens), or are read again in every pass (KPT = 0; a row stays in L2).
//  * The threshold, the need-th largest key of the competing tokens, comes
//    from a radix selection, 8 bits at a time below the keys' common prefix
//    (scores share their sign and most of their exponent): every CTA counts
//    its keys that match the digits found so far, the cluster's counts are
//    added up through distributed shared memory, and a suffix scan finds the
//    digit.  It ends early when a digit's keys stay all together, after two or
//    three passes for scores that differ.  Hot digits go to 8 neighbouring
//    copies of the count, by lane, so that a warp's lanes reach different
//    banks.
//  * Then every warp counts its tokens above the threshold and at it, and with
//    the sums before it (warps, then CTAs) writes those that stay: position =
//    above before + min(ties to keep, ties before).
// Integer sums only: the choice is exact and does not depend on timing.  Bound
// by the instructions and the latency of these steps; a row is 4 bytes a token against four K/V
// rows of 128 to 512 bytes for each token that stays.  (A search bit by bit
// instead, a count and an exchange a bit, measured 42 us for the LLaMA
// batch's 2048 rows and 146 us for 64 rows of 32 to 128 thousand tokens.)
constexpr int kSelCopies = 8;
static_assert(kSelCopies == 8, "read as two 16-byte vectors");

struct SelectSmem {
  uint4 hist[256][kSelCopies / 4];
  unsigned int tot[4][256];  // this CTA's counts of each pass
  unsigned int warp_sum[8];
  unsigned int all[16], any[16];  // per warp: and, or of its keys
  int gt[16], tie[16];            // per warp: tokens above the threshold, and at it
  unsigned int cta_all, cta_any;
  int cta_gt, cta_tie;
  unsigned int digit, need, exact;
};

template <int KPT, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) evict_select_kernel(const EvictArgs a, int warp_run) {
  namespace cg = cooperative_groups;
  __shared__ SelectSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  constexpr int NW = THREADS / 32;
  const int C = gridDim.x, rank = blockIdx.x;  // the cluster is the grid's x
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.y, i = blockIdx.z;
  const EvictSeq s = evict_seq(a, i);
  if (!s.ok) {  // the same in every CTA of the cluster
    if (g == 0 && rank == 0 && tid == 0) flag(PA_DEV_BAD_CONTEXT);
    return;
  }
  const float* sc = a.scores + i * a.s_sb + g * a.s_sh;
  float* so = a.scores_out + i * a.o_sb + g * a.o_sh;
  int32_t* kept = a.kept + i * a.k_sb + g * a.k_sh;
  const int lo = s.S0, hi = s.n - s.R;  // the tokens that compete
  // This warp's run: [w0, w0 + run).  A run is a multiple of 32 tokens
  // (warp_run with KPT = 0), so that no step of 32 reaches into the next
  // warp's: only tokens from n on lie past a run's end, and those neither
  // compete nor are protected.
  const int run = KPT > 0 ? 32 * KPT : warp_run;
  const int w0 = (rank * NW + warp) * run;
  const unsigned int mids = unsigned(hi - lo);
  auto load = [&](int t) { return unsigned(t - lo) < mids ? score_key(__ldg(sc + t)) : 0u; };  // 0: does not compete
  uint32_t key[KPT > 0 ? KPT : 1];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int k = 0; k < KPT; ++k) key[k] = load(w0 + 32 * k + lane);
  }
  auto each = [&](auto&& f) {  // f(token, key) for the run, the warp together
    if constexpr (KPT > 0) {
#pragma unroll
      for (int k = 0; k < KPT; ++k)
        if (w0 + 32 * k < s.n) f(w0 + 32 * k + lane, key[k]);  // (the warp together)
    } else {
      const int end = min(w0 + run, s.n);
      for (int t = w0; t < end; t += 32) f(t + lane, load(t + lane));
    }
  };
  for (int t = s.K + rank * THREADS + tid; t < a.So; t += C * THREADS) so[t] = 0.f;
  for (int t = s.K + rank * THREADS + tid; t < a.P; t += C * THREADS) kept[t] = -1;

  unsigned int need = unsigned(s.K - s.R - s.S0);
  uint32_t thr = need == 0 ? 0xffffffffu : 0u;  // keys above thr stay, and the first `ties` of those equal to it
  unsigned int ties = need == 0 ? 0u : 0xffffffffu;
  if (need > 0 && s.K < s.n) {
    // ---- the keys' common prefix ----
    uint32_t all = 0xffffffffu, any = 0u;
    each([&](int, uint32_t k) {
      if (k != 0u) all &= k;
      any |= k;
    });
    all = __reduce_and_sync(0xffffffffu, all);
    any = __reduce_or_sync(0xffffffffu, any);
    if (lane == 0) sm.all[warp] = all, sm.any[warp] = any;
    __syncthreads();
    all = __reduce_and_sync(0xffffffffu, lane < NW ? sm.all[lane] : 0xffffffffu);
    any = __reduce_or_sync(0xffffffffu, lane < NW ? sm.any[lane] : 0u);
    if (C > 1) {
      if (tid == 0) sm.cta_all = all, sm.cta_any = any;
      cl.sync();
      all = __reduce_and_sync(0xffffffffu, lane < C ? *cl.map_shared_rank(&sm.cta_all, lane) : 0xffffffffu);
      any = __reduce_or_sync(0xffffffffu, lane < C ? *cl.map_shared_rank(&sm.cta_any, lane) : 0u);
    }
    int left = 32 - __clz(all ^ any);  // bits below the prefix
    thr = left == 32 ? 0u : all & ~((1u << left) - 1u);
    // ---- digit by digit ----
    for (int p = 0; left > 0; ++p) {
      const int bits = min(8, left), shift = left - bits;
      for (int b = tid; b < 256 * kSelCopies / 4; b += THREADS) (&sm.hist[0][0])[b] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      unsigned int* const mine = reinterpret_cast<unsigned int*>(&sm.hist[0][0]) + (lane & (kSelCopies - 1));
      const uint32_t prefix = left == 32 ? 0u : thr >> left;
      each([&](int, uint32_t k) {
        if (k != 0u && (p == 0 || (k >> left) == prefix))
          atomicAdd(mine + ((k >> shift) & ((1u << bits) - 1u)) * kSelCopies, 1u);
      });
      __syncthreads();
      if (tid < 256) {
        const uint4 x = sm.hist[tid][0], y = sm.hist[tid][1];
        sm.tot[p][tid] = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
      }
      if (C > 1)
        cl.sync();
      else
        __syncthreads();
      // suffix sums over the digits, from the largest down
      unsigned int n = 0, suf = 0;
      if (tid < 256) {
        const int d = 255 - tid;
        if (C == 1) {
          n = sm.tot[p][d];
        } else {
#pragma unroll 8
          for (int r = 0; r < C; ++r) n += cl.map_shared_rank(&sm.tot[p][0], r)[d];
        }
        suf = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned int y = __shfl_up_sync(0xffffffffu, suf, o);
          if (lane >= o) suf += y;
        }
        if (lane == 31) sm.warp_sum[warp] = suf;
      }
      __syncthreads();
      if (tid < 256) {
        for (int w = 0; w < warp; ++w) suf += sm.warp_sum[w];
        if (suf >= need && suf - n < need) {
          sm.digit = 255 - tid;
          sm.need = need - (suf - n);
          sm.exact = suf == need;
        }
      }
      __syncthreads();
      thr |= sm.digit << shift;
      need = sm.need;
      left = shift;
      if (sm.exact) break;  // every key from thr on stays
      if (left == 0) ties = need;
    }
    if (all == any) ties = need;  // one key only
  }

  // ---- positions ----
  // Bit k of a lane's masks: its k-th token is above the threshold (or
  // protected), or at it.  (KPT = 0: 32 tokens a lane at a time.)
  const uint32_t below = (1u << lane) - 1u;
  auto is_tie = [&](int t, uint32_t k) { return k == thr && unsigned(t - lo) < mids; };
  auto is_gt = [&](int t, uint32_t k) { return k > thr || (t < s.n && unsigned(t - lo) >= mids); };
  int n_gt = 0, n_tie = 0;
  each([&](int t, uint32_t k) {
    n_gt += is_gt(t, k);
    n_tie += is_tie(t, k);
  });
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_tie = __reduce_add_sync(0xffffffffu, n_tie);
  if (lane == 0) {
    sm.gt[warp] = n_gt;
    sm.tie[warp] = n_tie;
  }
  __syncthreads();
  int b_gt = 0;
  unsigned int b_tie = 0;
  for (int w = 0; w < warp; ++w) {
    b_gt += sm.gt[w];
    b_tie += sm.tie[w];
  }
  if (C > 1) {
    if (tid == THREADS - 1) {
      sm.cta_gt = b_gt + n_gt;
      sm.cta_tie = int(b_tie) + n_tie;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      b_gt += *cl.map_shared_rank(&sm.cta_gt, r);
      b_tie += *cl.map_shared_rank(&sm.cta_tie, r);
    }
    cl.sync();  // no CTA leaves while another reads its counts
  }
  int done = b_gt + int(min(ties, b_tie));  // tokens that stay before this warp's
  // the ties of this warp all stay, or none does, or it holds the last that do
  const bool all_ties = b_tie + n_tie <= ties, no_ties = n_tie == 0 || b_tie >= ties;
  each([&](int t, uint32_t k) {
    bool stay = is_gt(t, k);
    if (!no_ties) {
      bool tie = is_tie(t, k);
      if (!all_ties) {
        const uint32_t m = __ballot_sync(0xffffffffu, tie);
        tie = tie && b_tie + __popc(m & below) < ties;
        b_tie += __popc(m);
      }
      stay |= tie;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, stay);
    const int pos = done + __popc(m & below);
    // (pos < K always, unless scores that are read again in every pass change
    // meanwhile)
    if (stay && (KPT > 0 || pos < s.K)) {
      kept[pos] = t;
      so[pos] = __ldg(sc + t);
    }
    done += __popc(m);
  });
}

// ---- move -----------------------------------------------------------------------
// K/V of kept token j of (sequence, kv head) -> position j of the destination
// table.  Pure copy.  A warp takes 32 kept tokens: lane l looks up token l's
// source and destination rows once, then the rows go 32 / VPR at a time as
// 16-byte vectors, four steps' K and V loads in flight.  Bound by the loads'
// latency: the LLaMA batch cut to half reads and writes 0.88 GB at 5.3 TB/s
// with three CTAs per SM; four (64 registers) took the whole call from 0.201
// to 0.194 ms.  (One kernel for the choice and the move, a CTA a row, measured
// slower, 0.193 against 0.164 + 0.025 ms: the longest rows are 40 times the
// shortest.)
template <int VPR>  // 16-byte vectors per row
__global__ void __launch_bounds__(256, 4) evict_move_kernel(const EvictArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.y, i = blockIdx.z;
  const EvictSeq s = evict_seq(a, i);
  if (!s.ok) return;
  const int lane = threadIdx.x & 31;
  const int32_t* kept = a.kept + i * a.k_sb + g * a.k_sh;
  const int32_t* bt = a.bt + int64_t(i) * a.bt_stride;
  const int32_t* dt = a.dt + int64_t(i) * a.dt_stride;
  constexpr int RPS = 32 / VPR;  // rows per step
  const int sub = lane / VPR, c = lane % VPR;
  const int step = gridDim.x * 8 * 32;
  for (int j0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 32; j0 < s.K; j0 += step) {
    int64_t src = -1, dst = 0;  // row indices, -1: nothing to move
    if (j0 + lane < s.K) {
      const int j = j0 + lane, t = kept[j];
      const int sb = __ldg(bt + t / kBS), db = __ldg(dt + j / kBS);
      if (unsigned(sb) >= unsigned(a.num_blocks) || unsigned(db) >= unsigned(a.num_blocks)) {
        flag(PA_DEV_BAD_BLOCK);
      } else {
        src = (int64_t(sb) * a.Hkv + g) * kBS + t % kBS;
        dst = (int64_t(db) * a.Hkv + g) * kBS + j % kBS;
      }
    }
    constexpr int U = VPR < 4 ? VPR : 4;
#pragma unroll 1
    for (int r0 = 0; r0 < VPR; r0 += U) {
      if (j0 + r0 * RPS >= s.K) break;
      uint4 k[U], v[U];
      int64_t d[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int who = (r0 + u) * RPS + sub;
        const int64_t sr = __shfl_sync(0xffffffffu, src, who);
        d[u] = __shfl_sync(0xffffffffu, dst, who) * VPR + c;
        on[u] = sr >= 0;
        if (on[u]) {
          k[u] = __ldcs(a.kc + sr * VPR + c);
          v[u] = __ldcs(a.vc + sr * VPR + c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on[u]) {
          __stcs(a.kc + d[u], k[u]);
          __stcs(a.vc + d[u], v[u]);
        }
    }
  }
}

}  // namespace pa

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
// bytes plus 8 for the score; they are mostly still in L2.  Each score has
// one writer and a fixed order of additions, so results do not vary.
struct AccumArgs {
  const float* logits;
  const float* lse;
  float* scores;
  const int32_t* ctx;
  int64_t s_sb, s_sh;  // strides of scores (elements)
  int32_t B, Hkv, cap, S;
};

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
  float lse[G];
#pragma unroll
  for (int j = 0; j < G; ++j) lse[j] = a.lse[(int64_t(i) * a.Hkv + g) * G + j];
  const float* lg = a.logits + (int64_t(i) * a.Hkv + g) * a.cap * G;
  float* sc = a.scores + i * a.s_sb + g * a.s_sh;
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x) {
    float x[G];
    if constexpr (G >= 4) {
#pragma unroll
      for (int j = 0; j < G; j += 4) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(lg + int64_t(t) * G + j));
        x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
      }
    } else if constexpr (G == 2) {
      const float2 v = __ldcs(reinterpret_cast<const float2*>(lg + int64_t(t) * G));
      x[0] = v.x, x[1] = v.y;
    } else {
      x[0] = __ldcs(lg + t);
    }
    float w = 0.f;
#pragma unroll
    for (int j = 0; j < G; ++j) w += ex2(x[j] - lse[j]);
    sc[t] += w;
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
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One cluster of C CTAs chooses for one (sequence, kv head): CTA r holds the
// scores of tokens [r chunk, (r + 1) chunk) in shared memory (IN_SMEM; rows too
// long for that are read again in every pass), so that a row is read once.
//  * The threshold, the need-th largest key of the competing tokens, comes
//    from a radix selection, 8 bits at a time: every CTA counts its keys that
//    match the digits found so far, adds up the cluster's counts through
//    distributed shared memory, and finds the digit by a suffix scan.  Hot
//    digits (scores share their exponents) go to 8 copies of the counts, by
//    lane.
//  * Then each warp takes a run of tokens, counts those above the threshold
//    and those at it, and with the sums before it (warps, then CTAs) writes
//    its tokens that stay: position = above before + min(need, ties before).
// Integer sums only: the choice is exact and does not depend on timing.
// Bound by latency: a row is 4 bytes a token against 4 K/V rows of 128 to
// 512 bytes for each that stays; the rule for C is in pa_evict.
constexpr int kSelCopies = 8;

struct SelectSmem {
  unsigned int hist[kSelCopies][256];
  unsigned int tot[4][256];  // this CTA's counts of each pass
  unsigned int warp_sum[32];
  int gt[32], tie[32];       // per warp: tokens above the threshold, and at it
  int cta_gt, cta_tie;
  unsigned int digit, need;
};

template <bool IN_SMEM>
__global__ void __launch_bounds__(512) evict_select_kernel(const EvictArgs a, int chunk) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(128) unsigned char smem[];
  SelectSmem& sm = *reinterpret_cast<SelectSmem*>(smem);
  float* const row = reinterpret_cast<float*>(smem + sizeof(SelectSmem));
  cg::cluster_group cl = cg::this_cluster();
  const int C = gridDim.x, rank = blockIdx.x;  // the cluster is the grid's x
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nthr >> 5;
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
  for (int t = s.K + rank * nthr + tid; t < a.So; t += C * nthr) so[t] = 0.f;
  for (int t = s.K + rank * nthr + tid; t < a.P; t += C * nthr) kept[t] = -1;
  if (s.K == s.n) {
    for (int t = rank * nthr + tid; t < s.n; t += C * nthr) {
      kept[t] = t;
      so[t] = __ldg(sc + t);
    }
    return;
  }
  const int lo = s.S0, hi = s.n - s.R;  // the tokens that compete
  const int t0 = min(s.n, rank * chunk), t1 = min(s.n, t0 + chunk);
  if constexpr (IN_SMEM) {
#pragma unroll 4
    for (int t = t0 + tid; t < t1; t += nthr) row[t - t0] = __ldg(sc + t);
  }
  auto score = [&](int t) { return IN_SMEM ? row[t - t0] : __ldg(sc + t); };

  unsigned int need = unsigned(s.K - s.R - s.S0);
  uint32_t thr = 0;  // the smallest key that stays; need: how many tokens of exactly that key do
  const bool none = need == 0;
  if (!none) {
    const int c0 = max(t0, lo), c1 = min(t1, hi);
    for (int p = 0; p < 4; ++p) {
      const int shift = 24 - 8 * p;
      for (int b = tid; b < kSelCopies * 256; b += nthr) (&sm.hist[0][0])[b] = 0;
      __syncthreads();
      for (int t = c0 + tid; t < c1; t += nthr) {
        const uint32_t k = score_key(score(t));
        if (p == 0 || (k >> (shift + 8)) == (thr >> (shift + 8)))
          atomicAdd(&sm.hist[lane & (kSelCopies - 1)][(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid < 256) {
        unsigned int n = 0;
#pragma unroll
        for (int c = 0; c < kSelCopies; ++c) n += sm.hist[c][tid];
        sm.tot[p][tid] = n;
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
        }
      }
      __syncthreads();
      thr |= sm.digit << shift;
      need = sm.need;
    }
  } else {
    __syncthreads();
  }

  // each warp's run of tokens, 32 at a time
  const int per = ((t1 - t0 + nw - 1) / nw + 31) / 32 * 32;
  const int w0 = min(t1, t0 + warp * per), w1 = min(t1, w0 + per);
  auto classify = [&](int t, float x, bool& gt, bool& tie) {
    const bool in = t < w1, mid = t >= lo && t < hi;
    const uint32_t k = score_key(x);
    gt = in && (!mid || (!none && k > thr));
    tie = in && mid && !none && k == thr;
  };
  int n_gt = 0, n_tie = 0;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    bool gt, tie;
    classify(t, t < w1 ? score(t) : 0.f, gt, tie);
    n_gt += __popc(__ballot_sync(0xffffffffu, gt));
    n_tie += __popc(__ballot_sync(0xffffffffu, tie));
  }
  if (lane == 0) {
    sm.gt[warp] = n_gt;
    sm.tie[warp] = n_tie;
  }
  __syncthreads();
  int b_gt = 0, b_tie = 0;
  for (int w = 0; w < warp; ++w) {
    b_gt += sm.gt[w];
    b_tie += sm.tie[w];
  }
  if (C > 1) {
    if (tid == nthr - 1) {
      sm.cta_gt = b_gt + n_gt;
      sm.cta_tie = b_tie + n_tie;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      b_gt += *cl.map_shared_rank(&sm.cta_gt, r);
      b_tie += *cl.map_shared_rank(&sm.cta_tie, r);
    }
    // no CTA leaves while another reads its counts
    cl.sync();
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    bool gt, tie;
    const float x = t < w1 ? score(t) : 0.f;
    classify(t, x, gt, tie);
    const uint32_t m_gt = __ballot_sync(0xffffffffu, gt), m_tie = __ballot_sync(0xffffffffu, tie);
    const int before = b_tie + __popc(m_tie & below);
    if (gt || (tie && before < int(need))) {
      const int pos = b_gt + __popc(m_gt & below) + min(int(need), before);
      kept[pos] = t;
      so[pos] = x;
    }
    b_gt += __popc(m_gt);
    b_tie += __popc(m_tie);
  }
}

// ---- move -----------------------------------------------------------------------
// K/V of kept token j of (sequence, kv head) -> position j of the destination
// table.  Pure copy.  A warp takes 32 kept tokens: lane l looks up token l's
// source and destination rows once, then the rows go 32 / VPR at a time as
// 16-byte vectors, four steps' K and V loads in flight.
template <int VPR>  // 16-byte vectors per row
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
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

// Bounding a sequence's cache by accumulated attention weight (sm_100a): the
// accumulation behind a scored decode, the choice of the tokens that stay,
// and their move into fresh blocks.
#pragma once

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

constexpr int kSelThreads = 512;

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ unsigned int hist[256];
  __shared__ int scratch[32];
  __shared__ unsigned int sh_digit, sh_need;
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.x, i = blockIdx.y;
  const EvictSeq s = evict_seq(a, i);
  if (!s.ok) {
    if (g == 0 && threadIdx.x == 0) flag(PA_DEV_BAD_CONTEXT);
    return;
  }
  const float* sc = a.scores + i * a.s_sb + g * a.s_sh;
  float* so = a.scores_out + i * a.o_sb + g * a.o_sh;
  int32_t* kept = a.kept + i * a.k_sb + g * a.k_sh;
  const int lo = s.S0, hi = s.n - s.R;  // the tokens that compete
  unsigned int need = unsigned(s.K - s.R - s.S0);
  // the need-th largest key of the competing tokens, digit by digit
  uint32_t prefix = 0;
  const bool all = s.K == s.n, none = need == 0;
  if (!all && !none) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int b = threadIdx.x; b < 256; b += kSelThreads) hist[b] = 0;
      __syncthreads();
      for (int t = lo + threadIdx.x; t < hi; t += kSelThreads) {
        const uint32_t k = score_key(__ldg(sc + t));
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        unsigned int left = need;
        int d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        sh_digit = unsigned(d);
        sh_need = left;
      }
      __syncthreads();
      prefix |= sh_digit << shift;
      need = sh_need;
    }
  }
  // prefix: the smallest key that stays; need: how many tokens of exactly that key do
  int done = 0, ties = 0;
  for (int t0 = 0; t0 < s.n; t0 += kSelThreads) {
    const int t = t0 + threadIdx.x;
    const float x = t < s.n ? __ldg(sc + t) : 0.f;
    const bool mid = t >= lo && t < hi;
    const uint32_t k = score_key(x);
    const int tie = !all && !none && mid && k == prefix;
    int n_tie, n_stay;
    const int rank = ties + block_exclusive_scan(tie, scratch, &n_tie);
    const int stay = t < s.n && (all || !mid || (!none && (k > prefix || (tie && rank < int(need)))));
    const int pos = done + block_exclusive_scan(stay, scratch, &n_stay);
    if (stay) {
      kept[pos] = t;
      so[pos] = x;
    }
    ties += n_tie;
    done += n_stay;
  }
  for (int t = s.K + threadIdx.x; t < a.So; t += kSelThreads) so[t] = 0.f;
  for (int t = s.K + threadIdx.x; t < a.P; t += kSelThreads) kept[t] = -1;
}

// ---- move -----------------------------------------------------------------------
// K/V of kept token j of (sequence, kv head) -> position j of the destination
// table.  Pure copy of 16-byte vectors.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.y, i = blockIdx.z;
  const EvictSeq s = evict_seq(a, i);
  if (!s.ok) return;
  const int32_t* kept = a.kept + i * a.k_sb + g * a.k_sh;
  const int32_t* bt = a.bt + int64_t(i) * a.bt_stride;
  const int32_t* dt = a.dt + int64_t(i) * a.dt_stride;
  const int64_t total = int64_t(s.K) * a.vpr;
  for (int64_t e = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += int64_t(gridDim.x) * blockDim.x) {
    const int j = int(e / a.vpr), c = int(e % a.vpr);
    const int t = kept[j];
    int sb = __ldg(bt + t / kBS);
    const int db = __ldg(dt + j / kBS);
    if (unsigned(sb) >= unsigned(a.num_blocks) || unsigned(db) >= unsigned(a.num_blocks)) {
      flag(PA_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t src = ((int64_t(sb) * a.Hkv + g) * kBS + t % kBS) * a.vpr + c;
    const int64_t dst = ((int64_t(db) * a.Hkv + g) * kBS + j % kBS) * a.vpr + c;
    const uint4 k = __ldcs(a.kc + src), v = __ldcs(a.vc + src);
    a.kc[dst] = k;
    a.vc[dst] = v;
  }
}

}  // namespace pa

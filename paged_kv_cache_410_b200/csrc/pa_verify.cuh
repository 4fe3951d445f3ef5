// Verification of drafted tokens against the target's probabilities (sm_100a).
//
// Speculative decoding keeps the target's distribution p when draft i, drawn
// from q, is accepted with probability min(1, p_i(x_i) / q_i(x_i)) and the
// first refused one is replaced by a draw from max(p - q, 0), normalised;
// when all are accepted one more token is drawn from the row after them.
// With the random numbers given,
//   accept i:  u_i q_i(x_i) < p_i(x_i)        (both sides exact in 64 bits)
//   draw:      the lowest token whose running sum of w passes u sum(w),
// w = max(p - q, 0) or p. The sums run in 64 bits: with 32 the token next to
// a border would depend on the order of the additions.
//
// Only the deciding row of p (and of q) is read whole: the accept test needs
// one value of each row before it. A cluster of kVerifyCtas CTAs takes one
// sequence; each warp sums a contiguous piece of the vocabulary, the pieces'
// sums are exchanged through distributed shared memory, and the one warp
// whose piece holds the border walks it again (from L2) to find the token.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kVerifyCtas = 8;      // CTAs per sequence (a portable cluster)
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyPieces = kVerifyCtas * kVerifyWarps;  // 128

struct VerifyParams {
  const int32_t* draft_tokens;  // [num_drafts]
  const int32_t* cu_drafts;     // [batch + 1]
  const void* target_probs;     // [num_drafts + batch][vocab]
  const void* draft_probs;      // [num_drafts][vocab], or null: q is 1 at the draft
  const float* accept_uniforms;  // [num_drafts]
  const float* sample_uniforms;  // [batch]
  int32_t* accepted;            // [batch]
  int32_t* tokens;              // [batch][max_drafts + 1]
  int64_t num_drafts;
  int vocab;
  int max_drafts;
};

template <>
__device__ __forceinline__ float to_f32<float>(float x) {
  return x;
}

// A probability; what is not a positive finite number counts as zero.
template <typename T>
__device__ __forceinline__ double prob(T x) {
  const float f = to_f32<T>(x);
  return f > 0.f && f < INFINITY ? static_cast<double>(f) : 0.0;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
}

// VEC: rows start on 16-byte boundaries (base pointers aligned, vocab * size
// a multiple of 16), so a lane takes 16 bytes at a time; else one value.
template <typename T, bool VEC>
__global__ void __cluster_dims__(kVerifyCtas, 1, 1) __launch_bounds__(kVerifyThreads)
    pa_verify_kernel(const VerifyParams p) {
  constexpr int VE = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  __shared__ double sums[2][kVerifyPieces];
  const int b = blockIdx.x / kVerifyCtas;
  const int rank = blockIdx.x % kVerifyCtas;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int start = __ldg(p.cu_drafts + b);
  const int end = __ldg(p.cu_drafts + b + 1);
  const int n = end - start;
  // (uniform over the cluster)
  if (start < 0 || n < 0 || end > p.num_drafts || n > p.max_drafts) {
    if (rank == 0 && threadIdx.x == 0) flag_error(PA_DEVERR_CHUNK);
    return;
  }
  const int64_t V = p.vocab;
  const T* target = reinterpret_cast<const T*>(p.target_probs) + (static_cast<int64_t>(start) + b) * V;
  const T* draft = p.draft_probs ? reinterpret_cast<const T*>(p.draft_probs) + start * V : nullptr;

  // every warp finds the first refused draft, 32 at a time
  int a = n;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool refused = false;
    if (i < n) {
      const int x = __ldg(p.draft_tokens + start + i);
      if (x < 0 || x >= p.vocab) {
        if (rank == 0 && warp == 0) flag_error(PA_DEVERR_TOKEN);
        refused = true;
      } else {
        const double pt = prob<T>(target[i * V + x]);
        const double qt = draft ? prob<T>(draft[i * V + x]) : 1.0;
        refused = !(static_cast<double>(__ldg(p.accept_uniforms + start + i)) * qt < pt);
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, refused);
    if (m) {
      a = i0 + __ffs(m) - 1;
      break;
    }
  }

  const T* prow = target + a * V;
  const T* qrow = draft && a < n ? draft + a * V : nullptr;
  // without draft probabilities the refused draft itself is what q removes
  const int gone = !draft && a < n ? __ldg(p.draft_tokens + start + a) : -1;
  const double u = fmax(static_cast<double>(__ldg(p.sample_uniforms + b)), 0.0);

  // this warp's piece of the vocabulary
  const int64_t piece = ((V + kVerifyPieces - 1) / kVerifyPieces + VE - 1) / VE * VE;
  const int g = rank * kVerifyWarps + warp;
  const int64_t lo = min(g * piece, V), hi = min(lo + piece, V);
  // weights of VE tokens from i (all below hi); `residual`: against q
  auto weights = [&](int64_t i, bool residual, double (&w)[VE]) {
    T pv[VE], qv[VE];
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(pv) = __ldg(reinterpret_cast<const uint4*>(prow + i));
      if (residual && qrow) *reinterpret_cast<uint4*>(qv) = __ldg(reinterpret_cast<const uint4*>(qrow + i));
    } else {
      pv[0] = prow[i];
      if (residual && qrow) qv[0] = qrow[i];
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      w[e] = prob<T>(pv[e]);
      if (residual) {
        if (qrow) w[e] = fmax(w[e] - prob<T>(qv[e]), 0.0);
        if (i + e == gone) w[e] = 0.0;
      }
    }
  };

  int pick = -1;       // (one lane of one warp of the cluster finds it)
  bool drawn = false;  // uniform over the cluster
  for (int attempt = 0; attempt < 2 && !drawn; ++attempt) {
    // where nothing is left of p - q (p <= q everywhere), the draw is from p
    const bool residual = attempt == 0;
    double s = 0.0;
#pragma unroll 4
    for (int64_t i = lo + lane * VE; i < hi; i += 32 * VE) {
      double w[VE];
      weights(i, residual, w);
#pragma unroll
      for (int e = 0; e < VE; ++e) s += w[e];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < kVerifyCtas) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n"
                   : "=r"(at)
                   : "r"(smem_addr(&sums[attempt][g])), "r"(lane));
      asm volatile("st.shared::cluster.f64 [%0], %1;\n" ::"r"(at), "d"(s) : "memory");
    }
    cluster_sync_all();
    // the pieces' running sums: lane holds four consecutive ones
    constexpr int PL = kVerifyPieces / 32;
    double c[PL], mine = 0.0;
#pragma unroll
    for (int e = 0; e < PL; ++e) mine += c[e] = sums[attempt][lane * PL + e];
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const double total = __shfl_sync(0xffffffffu, incl, 31);
    if (!(total > 0.0)) continue;
    drawn = true;
    const double t = u * total;
    // the first piece whose running sum passes t; behind it (u >= 1) the last
    // one with any weight
    double before = incl - mine, base = 0.0;
    int cross = -1, last = -1;
#pragma unroll
    for (int e = 0; e < PL; ++e) {
      if (c[e] > 0.0) last = lane * PL + e;
      if (cross < 0 && c[e] > 0.0 && before + c[e] > t) {
        cross = lane * PL + e;
        base = before;
      }
      before += c[e];
    }
    const unsigned found = __ballot_sync(0xffffffffu, cross >= 0);
    const unsigned some = __ballot_sync(0xffffffffu, last >= 0);
    const int src = found ? __ffs(found) - 1 : 31 - __clz(some);
    const int gs = __shfl_sync(0xffffffffu, found ? cross : last, src);
    base = __shfl_sync(0xffffffffu, base, src);
    if (gs != g) continue;  // (this warp is done; `drawn` ends the loop)
    const double lim = found ? t : INFINITY;
    int64_t tail = -1;  // the last token with weight so far
    for (int64_t i0 = lo; i0 < hi && pick < 0; i0 += 32 * VE) {
      const int64_t i = i0 + lane * VE;
      double w[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) w[e] = 0.0;
      if (i < hi) weights(i, residual, w);
      double own = 0.0;
#pragma unroll
      for (int e = 0; e < VE; ++e) own += w[e];
      double run = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      double at = base + (run - own);
      int64_t mine_pick = -1, mine_last = -1;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        at += w[e];
        if (w[e] > 0.0) {
          mine_last = i + e;
          if (mine_pick < 0 && at > lim) mine_pick = i + e;
        }
      }
      base += __shfl_sync(0xffffffffu, run, 31);
      const unsigned hit = __ballot_sync(0xffffffffu, mine_pick >= 0);
      const unsigned any = __ballot_sync(0xffffffffu, mine_last >= 0);
      if (any) tail = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(any));
      if (hit) pick = static_cast<int>(__shfl_sync(0xffffffffu, mine_pick, __ffs(hit) - 1));
    }
    // the piece's sum passed t by less than the additions' rounding
    if (pick < 0) pick = static_cast<int>(tail);
  }

  int32_t* row = p.tokens + static_cast<int64_t>(b) * (p.max_drafts + 1);
  if (pick >= 0 && lane == 0) row[a] = pick;
  if (rank == 0) {
    if (threadIdx.x == 0) {
      p.accepted[b] = a;
      if (!drawn) {
        row[a] = -1;
        flag_error(PA_DEVERR_PROBS);
      }
    }
    for (int i = threadIdx.x; i <= p.max_drafts; i += kVerifyThreads)
      if (i != a) row[i] = i < a ? p.draft_tokens[start + i] : -1;
  }
}

}  // namespace pa

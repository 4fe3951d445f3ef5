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
// one value of each row before it. A cluster of CL CTAs takes one sequence
// (CL = 8, 4, 2 or 1: as many as leave the batch one wave); each warp sums a
// contiguous piece of the vocabulary, the pieces' sums are exchanged through
// distributed shared memory, and the one warp
// whose piece holds the border reads it again (from L2) to find the token.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kVerifyMaxCtas = 8;   // CTAs per sequence at most (a portable cluster)
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

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
__device__ __forceinline__ float prob(T x) {
  const float f = to_f32<T>(x);
  return f > 0.f && f < INFINITY ? f : 0.f;
}
// a - b = hi + lo exactly (both 32 bits); its sign is hi's.
__device__ __forceinline__ float2 exact_difference(float a, float b) {
  const float s = __fsub_rn(a, b);
  const float t = __fsub_rn(s, a);
  return make_float2(s, __fsub_rn(__fsub_rn(a, __fsub_rn(s, t)), __fadd_rn(b, t)));
}

// The two halves of a barrier over the cluster's CTAs; each is executed by
// converged warps (.aligned).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
}

// Weights of VE tokens from i, each as the exact sum of two floats: of
// max(p - q, 0) (Q), or of p without the token `gone`.
template <typename T, int VE, bool Q>
__device__ __forceinline__ void verify_weights(const T* prow, const T* qrow, int i, int gone,
                                               float2 (&w)[VE]) {
  T pv[VE];
  [[maybe_unused]] T qv[VE];
  if constexpr (VE > 1) {
    *reinterpret_cast<uint4*>(pv) = __ldg(reinterpret_cast<const uint4*>(prow + i));
    if constexpr (Q) *reinterpret_cast<uint4*>(qv) = __ldg(reinterpret_cast<const uint4*>(qrow + i));
  } else {
    pv[0] = prow[i];
    if constexpr (Q) qv[0] = qrow[i];
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    if constexpr (Q) {
      w[e] = exact_difference(prob<T>(pv[e]), prob<T>(qv[e]));
      if (!(w[e].x > 0.f)) w[e] = make_float2(0.f, 0.f);
    } else {
      w[e] = make_float2(i + e == gone ? 0.f : prob<T>(pv[e]), 0.f);
    }
  }
}

// Their sum over tokens first, first + stride, ... < end (VE at a time); *last:
// the last token with weight. High and low parts are added up apart, each in 64
// bits (the low ones in 32 bits: 61.9 against 60.7 us at 256 rows of 131072).
template <typename T, int VE, bool Q>
__device__ __forceinline__ double verify_sum(const T* prow, const T* qrow, int gone, int first, int end,
                                             int stride, int* last) {
  double s = 0.0;
  [[maybe_unused]] double s_lo = 0.0;
#pragma unroll 4
  for (int i = first; i < end; i += stride) {
    float2 w[VE];
    verify_weights<T, VE, Q>(prow, qrow, i, gone, w);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      s += static_cast<double>(w[e].x);
      if constexpr (Q) s_lo += static_cast<double>(w[e].y);
      if (last && w[e].x > 0.f) *last = i + e;
    }
  }
  return s + s_lo;
}

// VEC: rows start on 16-byte boundaries (base pointers aligned, vocab * size
// a multiple of 16), so a lane takes 16 bytes at a time; else one value.
template <typename T, bool VEC, int CL>
__global__ void __launch_bounds__(kVerifyThreads, 2) pa_verify_kernel(const VerifyParams p) {
  constexpr int kPieces = CL * kVerifyWarps;
  constexpr int VE = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  __shared__ double sums[2][kPieces];
  __shared__ double part[kVerifyWarps];
  const int b = blockIdx.x / CL;
  const int rank = blockIdx.x % CL;
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
  // A CTA's shared memory may be written from the others only once it is known
  // to have started: every CTA says so here, and waits for all before its
  // first store (the reads of the row lie between).
  if constexpr (CL > 1) cluster_arrive();
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
        const double qt = draft ? prob<T>(draft[i * V + x]) : 1.f;
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
  const int64_t piece = ((V + kPieces - 1) / kPieces + VE - 1) / VE * VE;
  const int g = rank * kVerifyWarps + warp;
  const int lo = static_cast<int>(min(g * piece, V)), hi = static_cast<int>(min(lo + piece, V));
  int pick = -1;       // (one lane of one warp of the cluster finds it)
  bool drawn = false;  // uniform over the cluster
  for (int attempt = 0; attempt < 2 && !drawn; ++attempt) {
    // where nothing is left of p - q (p <= q everywhere), the draw is from p
    const bool against = attempt == 0 && qrow;
    const int gone_at = attempt == 0 ? gone : -1;
    double s = against ? verify_sum<T, VE, true>(prow, qrow, gone_at, lo + lane * VE, hi, 32 * VE, nullptr)
                       : verify_sum<T, VE, false>(prow, qrow, gone_at, lo + lane * VE, hi, 32 * VE, nullptr);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (CL == 1) {
      if (lane == 0) sums[attempt][g] = s;
      __syncthreads();
    } else {
      if (attempt == 0) cluster_wait();  // (every CTA of the cluster has started)
      if (lane < CL) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n"
                     : "=r"(at)
                     : "r"(smem_addr(&sums[attempt][g])), "r"(lane));
        asm volatile("st.shared::cluster.f64 [%0], %1;\n" ::"r"(at), "d"(s) : "memory");
      }
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
    // the pieces' running sums: lane holds PL consecutive ones
    constexpr int PL = (kPieces + 31) / 32;
    double c[PL], mine = 0.0;
#pragma unroll
    for (int e = 0; e < PL; ++e) mine += c[e] = lane * PL + e < kPieces ? sums[attempt][lane * PL + e] : 0.0;
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
    if (gs / kVerifyWarps != rank) continue;  // (another CTA's; `drawn` ends the loop)
    // this CTA's warps share the piece out again, and the warp whose share holds
    // the border gives each lane a contiguous run of it: the lane whose running
    // sum passes walks its run (a few tokens, from L1 and L2)
    const double lim = found ? t : INFINITY;
    const int p0 = static_cast<int>(min(gs * piece, V)), p1 = static_cast<int>(min(p0 + piece, V));
    const int share = static_cast<int>(((piece + kVerifyWarps - 1) / kVerifyWarps + VE - 1) / VE * VE);
    const int s0 = min(p0 + min(warp * share, p1 - p0), p1), s1 = min(s0 + min(share, p1 - s0), p1);
    double mine_sum = against ? verify_sum<T, VE, true>(prow, qrow, gone_at, s0 + lane * VE, s1, 32 * VE, nullptr)
                              : verify_sum<T, VE, false>(prow, qrow, gone_at, s0 + lane * VE, s1, 32 * VE, nullptr);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine_sum += __shfl_xor_sync(0xffffffffu, mine_sum, o);
    if (lane == 0) part[warp] = mine_sum;
    __syncthreads();
    int owner = -1, last_share = -1;
    double run_base = base;
#pragma unroll
    for (int k = 0; k < kVerifyWarps; ++k) {
      const double s_k = part[k];
      if (s_k > 0.0) last_share = k;
      if (owner < 0 && s_k > 0.0 && run_base + s_k > lim) {
        owner = k;
        base = run_base;
      }
      run_base += s_k;
    }
    // (none: u >= 1, or the piece's sum passed t by less than the additions'
    // rounding: the last token with weight)
    const bool crossed = owner >= 0;
    if ((crossed ? owner : last_share) != warp) continue;
    const int run = ((share + 31) / 32 + VE - 1) / VE * VE;
    const int r0 = min(s0 + min(lane * run, s1 - s0), s1), r1 = min(r0 + min(run, s1 - r0), s1);
    int mine_last = -1;  // the run's last token with weight
    const double own = against ? verify_sum<T, VE, true>(prow, qrow, gone_at, r0, r1, VE, &mine_last)
                               : verify_sum<T, VE, false>(prow, qrow, gone_at, r0, r1, VE, &mine_last);
    double upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, crossed && own > 0.0 && base + upto > lim);
    const unsigned any = __ballot_sync(0xffffffffu, mine_last >= 0);
    const int tail = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(any));
    if (hit) {
      const int src_lane = __ffs(hit) - 1;
      int found_at = -1;
      if (lane == src_lane) {
        double at = base + (upto - own);
        for (int i = r0; i < r1 && found_at < 0; i += VE) {
          float2 w[VE];
          if (against)
            verify_weights<T, VE, true>(prow, qrow, i, gone_at, w);
          else
            verify_weights<T, VE, false>(prow, qrow, i, gone_at, w);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            at += static_cast<double>(w[e].x) + static_cast<double>(w[e].y);
            if (found_at < 0 && w[e].x > 0.f && at > lim) found_at = i + e;
          }
        }
        // (the run's sum passed by less than the additions' rounding)
        if (found_at < 0) found_at = mine_last;
      }
      pick = __shfl_sync(0xffffffffu, found_at, src_lane);
    }
    // the piece's sum passed t by less than the additions' rounding
    if (pick < 0) pick = tail;
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

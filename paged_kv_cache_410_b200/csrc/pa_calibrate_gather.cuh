// An E4M3 cache's scales from the K/V it will hold, and cached tokens read
// back into contiguous rows (sm_100a).
//
// The KV cache article, section "再往后：压 KV 的三条路线", stores FP8 K/V
// with calibrated per-channel scaling factors: scale = max |x| / 448 (the
// largest E4M3 value), so that the largest value of a channel uses the whole
// range. pa_calibrate_kernel takes the maximum over tokens; both kernels are
// bound by HBM (every input byte is read once).
#pragma once

#include "pa_common.cuh"

namespace pa {

// ---- calibration --------------------------------------------------------------

struct CalibrateParams {
  const void* x[2];         // K, V: [num_tokens][columns] 16-bit
  float* amax[2];           // [columns], read and written
  float* scale[2];          // [columns]
  float* inv_scale[2];
  const int64_t* slots;     // [num_tokens] or null; tokens with slot < 0 do not count
  int64_t num_tokens;
  int64_t tokens_per_split;
  int columns;              // num_kv_heads * head_dim
};

constexpr float kE4m3Max = 448.f;
constexpr float kSmallestScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

__device__ __forceinline__ void write_scale(const CalibrateParams& p, int which, int c, float amax) {
  const float s = amax > 0.f ? fmaxf(amax / kE4m3Max, kSmallestScale) : 1.f;
  p.scale[which][c] = s;
  p.inv_scale[which][c] = 1.f / s;
}

// grid (token splits, column blocks, K / V); a thread owns 8 columns (16
// bytes) and every (256 / width)-th token of its split.
//
// |x| of 16-bit floats orders as its bits, two at a time: with the sign
// cleared, adding (0x8000 - bits of infinity) leaves finite values positive
// as 16-bit integers and makes infinities and NaN negative, so one packed
// signed maximum keeps the largest finite |x|.
template <bool BF16, bool ONE_SPLIT>
__global__ void __launch_bounds__(256) pa_calibrate_kernel(const CalibrateParams p) {
  constexpr uint32_t kBias = BF16 ? 0x00800080u : 0x04000400u;
  __shared__ uint4 part[256];
  const int which = blockIdx.z;
  const int groups = p.columns / 8;
  const int width = min(groups, 256);  // column groups of a block
  const int rows = 256 / width;        // tokens in parallel
  const int cg = blockIdx.y * width + threadIdx.x % width;
  const int r = threadIdx.x / width;
  const int64_t t0 = blockIdx.x * p.tokens_per_split;
  const int64_t t1 = min(t0 + p.tokens_per_split, p.num_tokens);
  uint4 m = make_uint4(kBias, kBias, kBias, kBias);  // |x| = 0
  if (r < rows && cg < groups) {
    const uint4* x = reinterpret_cast<const uint4*>(p.x[which]) + cg;
    auto take = [&](const uint4& v, uint32_t live) {
      m.x = __vmaxs2(m.x, (v.x & live) + kBias);
      m.y = __vmaxs2(m.y, (v.y & live) + kBias);
      m.z = __vmaxs2(m.z, (v.z & live) + kBias);
      m.w = __vmaxs2(m.w, (v.w & live) + kBias);
    };
    // kBatch tokens' loads in flight at a time (with the slots read in the same
    // loop the compiler waited for each)
    constexpr int kBatch = 8;
    const int64_t step = static_cast<int64_t>(rows) * kBatch;
    int64_t t = t0 + r;
    for (; t + step - rows < t1; t += step) {
      uint4 v[kBatch];
      int64_t s[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) v[k] = __ldg(x + (t + k * rows) * groups);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) s[k] = p.slots ? __ldg(p.slots + t + k * rows) : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) take(v[k], s[k] < 0 ? 0u : 0x7fff7fffu);
    }
    for (; t < t1; t += rows)
      take(__ldg(x + t * groups), p.slots && __ldg(p.slots + t) < 0 ? 0u : 0x7fff7fffu);
  }
  part[threadIdx.x] = m;
  __syncthreads();
  if (r != 0 || cg >= groups) return;
  for (int k = 1; k < rows; ++k) {
    const uint4 v = part[threadIdx.x + k * width];
    m.x = __vmaxs2(m.x, v.x);
    m.y = __vmaxs2(m.y, v.y);
    m.z = __vmaxs2(m.z, v.z);
    m.w = __vmaxs2(m.w, v.w);
  }
  const uint32_t w[4] = {m.x - kBias, m.y - kBias, m.z - kBias, m.w - kBias};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint16_t bits = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
    float f;
    if constexpr (BF16)
      f = __uint_as_float(static_cast<uint32_t>(bits) << 16);
    else
      f = __half2float(__ushort_as_half(bits));
    const int c = cg * 8 + e;
    if constexpr (ONE_SPLIT) {
      f = fmaxf(f, p.amax[which][c]);
      p.amax[which][c] = f;
      write_scale(p, which, c, f);
    } else {
      // non-negative floats order as their bits; the maximum does not depend
      // on the order of the atomics
      atomicMax(reinterpret_cast<int*>(p.amax[which] + c), __float_as_int(f));
    }
  }
}

__global__ void __launch_bounds__(256) pa_calibrate_scale_kernel(const CalibrateParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < p.columns) write_scale(p, blockIdx.y, c, p.amax[blockIdx.y][c]);
}

// ---- read-back ------------------------------------------------------------------

struct GatherParams {
  const void* cache[2];      // K, V
  void* out[2];              // [num_tokens][columns]
  const float* scale[2];     // E4M3: [columns]
  const int32_t* block_tables;
  const int32_t* first;      // [batch]: position of each sequence's first row
  const int32_t* cu;         // [batch + 1]
  int64_t num_blocks;
  int64_t num_tokens;
  int batch;
  int max_blocks_per_seq;
  int bs_log2;
  int columns;
};

constexpr int kGatherTokens = 32;  // most tokens of a CTA

// MODE 0: 16-bit copy; 1: E4M3 -> f16; 2: E4M3 -> bf16. A CTA takes `per`
// consecutive output rows: one thread per row finds its sequence and slot,
// then a thread keeps one 16-byte piece of the columns (with its scales in
// registers) for the rows it passes.
template <int MODE>
__global__ void __launch_bounds__(256) pa_gather_kernel(const GatherParams p, int per) {
  __shared__ int64_t slot[kGatherTokens];  // -1: zeros, -2: leave the row
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per;
  if (blockIdx.x == 0)
    for (int i = tid; i < p.batch; i += 256)
      if (p.cu[i] < 0 || p.cu[i + 1] < p.cu[i] || p.cu[i + 1] > p.num_tokens)
        flag_error(PA_DEVERR_CHUNK);
  if (tid < per) {
    const int64_t t = t0 + tid;
    int64_t s = -2;
    if (t < p.num_tokens) {
      // the last sequence that starts at or before t
      int lo = 0, hi = p.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid) <= t)
          lo = mid;
        else
          hi = mid;
      }
      const int start = __ldg(p.cu + lo), end = __ldg(p.cu + lo + 1);
      if (t >= start && t < end) {
        const int64_t pos = __ldg(p.first + lo) + (t - start);
        s = -1;
        if (pos < 0 || (pos >> p.bs_log2) >= p.max_blocks_per_seq) {
          flag_error(PA_DEVERR_CONTEXT_LEN);
        } else {
          const int id = __ldg(p.block_tables + static_cast<int64_t>(lo) * p.max_blocks_per_seq +
                               (pos >> p.bs_log2));
          if (id < 0 || id >= p.num_blocks)
            flag_error(PA_DEVERR_BLOCK_ID);
          else
            s = (static_cast<int64_t>(id) << p.bs_log2) + (pos & ((1 << p.bs_log2) - 1));
        }
      }
    }
    slot[tid] = s;
  }
  __syncthreads();
  constexpr int E = MODE == 0 ? 8 : 16;  // columns of a 16-byte piece
  const int pieces = p.columns / E;
  const int width = min(pieces, 256);
  const int rows = 256 / width;
  const int r0 = tid / width;
  if (r0 >= rows) return;
  for (int c = tid % width; c < pieces; c += width) {
    for (int which = 0; which < 2; ++which) {
      const uint4* src = reinterpret_cast<const uint4*>(p.cache[which]) + c;
      uint4* dst = reinterpret_cast<uint4*>(p.out[which]);
      [[maybe_unused]] float sc[E];
      if constexpr (MODE != 0) {
        const float4* f = reinterpret_cast<const float4*>(p.scale[which]) + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = __ldg(f + i);
          sc[4 * i] = v.x, sc[4 * i + 1] = v.y, sc[4 * i + 2] = v.z, sc[4 * i + 3] = v.w;
        }
      }
#pragma unroll 4
      for (int r = r0; r < per; r += rows) {
        const int64_t s = slot[r];
        if (s == -2) continue;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (s >= 0) v = __ldg(src + s * pieces);
        if constexpr (MODE == 0) {
          dst[(t0 + r) * pieces + c] = v;
        } else {
          // code -> f16 (exact) -> f32, times the scale, one rounding
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[2];
            e4m3x4_to_f16x2x2(w[i], h[0], h[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
              o[2 * i + k] = pack2<MODE == 2>(f.x * sc[4 * i + 2 * k], f.y * sc[4 * i + 2 * k + 1]);
            }
          }
          uint4* d = dst + (t0 + r) * (2 * pieces) + 2 * c;
          d[0] = make_uint4(o[0], o[1], o[2], o[3]);
          d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
  }
}

}  // namespace pa

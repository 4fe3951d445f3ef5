// Attention of chunks of new tokens over the paged cache (sm_100a).
//
// Sequence b brings n_b new tokens (rows cu[b] .. cu[b+1] of q), whose K/V
// the caller has already stored; the row of new token i sits at position
// p = L_b - n_b + i and attends the cached tokens max(0, p - w + 1) .. p
// (w = the window, unlimited without one):
//   out = sum_j 2^(s_j - m) V_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q.K_j.
//
// For one KV head the rows (token, query head of the group) of a run of new
// tokens against the cached tokens are a dense problem, so a CTA takes NT
// tiles of up to 128 such rows and walks the tokens in steps of 64:
//   S (128 x 64, f32, TMEM, two buffers) = Q (128 x D, smem) . K_step^T
//   P (128 x 64, 16-bit, TMEM)           = 2^(S - m), over S's own columns
//   O (128 x D, f32, TMEM)              += P (TMEM) . V_step (64 x D, smem)
// with the running maximum m and sum l of a row, in 32 bits, in the registers
// of the one thread that owns the row. P is rounded to the operands' 16 bits
// (2^-8 or 2^-11 of each weight: what the MMA takes); l sums the weights
// before that rounding. m moves only when a score passes it by 2^8, so that O
// is rarely rescaled. With f16 operands m is the maximum less kHeadroom, so that
// weights use the type's upper range: they lie below 2^15, keep 11 bits down to
// 2^-21 of the largest and are lost below 2^-32 (of a reference at the maximum
// itself 2^-14 and 2^-25: a long history behind one large score can weigh as much).
//
// K and V steps come through one ring of buffers (K0 V0 K1 V1 ...), filled by
// two TMA warps (16-bit caches with blocks of 8 tokens or more: whole
// 1024-byte swizzle atoms per box), or by four loader warps with cp.async
// (smaller blocks; E4M3 caches, which they widen to f16: exact; the K scale is
// folded into q, rounded once to f16, and the V scale into the result).
//
// What each row may not see is decided by selecting on S, so K of masked
// tokens never matters; V rows outside the CTA's token range (behind the
// last row's position, before the first row's window: recycled memory) are
// zeroed in shared memory, since 0 x NaN would reach the sum. Inside it a V that
// is not finite makes every row of the step NaN; rows that do not see it are
// found by their result and summed again (chunk_unseen_v).
//
// What bounds it, measured on B200s (perf/operators.py; a GPU's own clock and
// power make up to a tenth):
//  - drafts (64 requests, 2 to 8 new tokens, 512 to 4096 cached ones, 64 / 8
//    heads of 128, bf16): 120 to 133 us for 636 MB, 0.73 to 0.81 of the copy
//    bandwidth.
//    One-tile CTAs, two per SM; on a GPU that took up to 141, without the loads
//    the launch took 103 us, without the softmax 131: the loads and the tail are
//    what is left.
//  - prompts (2048 tokens over 16384, 64 / 8 heads, bf16): 1000 to 1045 us, 1.0
//    PFLOP/s, 0.58 to 0.61 of the cuBLAS burst (single launches of a cool GPU reach
//    915). A step of 64 tokens and 256 rows takes about
//    1850 clocks. Its MMAs alone take 1300 (a tcgen05.mma of N = 64 runs in 33
//    (A in TMEM) to 49 clocks, but one warp needs 60 to issue it), its
//    exponentials 1024; the rest is the chain S -> P -> P.V -> S of a tile
//    (about 110 clocks a wait, 60 a commit). Steps that were tried and lost: N = 128
//    with one S buffer per tile (the MMAs alone 1030 a step, but the two tiles
//    fall into step and wait together: 1277 us in all), two warps per row
//    (1526 us), one MMA warp per tile instead of two (1003 us), a quarter of the
//    exponentials as polynomials on the FMA pipe (976 against 937 us).
//  - E4M3 (a mixed batch of 32, 32 / 8 heads): 240 to 250 us; the same batch from
//    a f16 cache 134: the loader warps' copies in flight and widening set the pace
//    (twice the loader warps: 248 against 241).
#pragma once

#include "pa_prefix_umma.cuh"

namespace pa {

constexpr int kChunkStep = 64;  // cached tokens per step

struct ChunkParams {
  const void* q;              // [num_tokens][Hq][D]
  void* out;                  // [num_tokens][Hq][D]
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;       // E4M3 caches
  const float* v_scale;
  const int32_t* cu;          // [batch + 1]
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_o;                // [num_tokens * Hq][num_partitions][D] (split contexts)
  float2* ws_ml;              // [num_tokens * Hq][num_partitions]
  int64_t num_blocks;
  int64_t num_tokens;
  int batch;
  int num_q_heads;
  int num_kv_heads;
  int group;                  // query heads per KV head
  int head_rows;              // query heads of a group in one row tile: min(group, 128)
  int head_blocks;            // ceil(group / head_rows)
  int tile_tokens;            // new tokens in one row tile: 128 / head_rows
  int num_tiles;              // grid bound: CTA tiles over the batch
  int one_tile;               // every chunk fits one tile of a one-tile CTA
  int longest_first;          // (one_tile) visit the longest contexts first
  int min_new, max_new;       // the chunk lengths this launch takes (a mixed batch has two)
  int leading, trailing;      // the first, the second launch of a mixed batch
  int num_partitions;
  int partition_tokens;       // a multiple of the kernel's BN
  int max_blocks_per_seq;
  int bs_log2;
  int max_chunk;
  int max_context;
  int window;                 // 0: the whole history
  int num_slots;              // TMA: a slot past the map (loads zeros)
  int withhold_scores;        // test hook: row tiles (one bit each) whose S is not issued
  float scale_log2;           // |scale| * log2(e)
  float sign;                 // 1, -1 or 0: the sign of scale
};

// Which new tokens a CTA tile holds, and the cached tokens they attend.
struct ChunkTile {
  int b;        // sequence (-1: no rows, the CTA has nothing to do)
  int i0;       // first new token of the tile within the chunk
  int tokens;   // new tokens in the tile
  int64_t row;  // first row of q / out
  int pos0;     // position of token i0
  int lo, hi;   // cached tokens [lo, hi) any row of the tile attends
  int base;     // lo rounded down to the step: where the partitions start
};

// Tiles are laid over the batch without reading lengths on the host: sequence
// b owns tile indices from f(b) = cu[b] / t + b (t tokens per tile), which
// leaves it at least ceil(n_b / t) of them; surplus tiles have no rows. One
// warp finds b, the last sequence with f(b) <= x, 32 probes at a time. When
// every chunk fits one tile, x is the sequence itself.
__device__ __forceinline__ ChunkTile chunk_tile(const ChunkParams& p, int x, int t) {
  const int lane = threadIdx.x & 31;
  int lo = p.one_tile ? x : 0, hi = p.one_tile ? x + 1 : p.batch;
  while (hi - lo > 1) {
    const int stride = (hi - lo + 31) >> 5;
    const int at = lo + lane * stride;
    const bool below = at < hi && __ldg(p.cu + at) / t + at <= x;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * stride;
    hi = min(lo + stride, hi);
  }
  ChunkTile c;
  c.b = -1;
  c.i0 = c.tokens = c.pos0 = c.lo = c.hi = c.base = 0;
  c.row = 0;
  const int start = __ldg(p.cu + lo);
  const int end = __ldg(p.cu + lo + 1);
  const int L = __ldg(p.context_lens + lo);
  // a chunk outside [0, num_tokens) or longer than max_chunk is not touched
  if (start < 0 || end < start || end > p.num_tokens || end - start > p.max_chunk) {
    if (lane == 0) flag_error(PA_DEVERR_CHUNK);
    return c;
  }
  const int n = end - start;
  if (n < p.min_new || n > p.max_new) return c;
  const int64_t first = p.one_tile ? 0 : static_cast<int64_t>(x - (start / t + lo)) * t;
  if (first < 0 || first >= n) return c;
  c.b = lo;
  c.i0 = static_cast<int>(first);
  c.tokens = min(t, n - c.i0);
  c.row = static_cast<int64_t>(start) + c.i0;
  // a length the table or the launch cannot hold: the rows see no tokens
  if (L < n || L > p.max_context ||
      L > (static_cast<int64_t>(p.max_blocks_per_seq) << p.bs_log2)) {
    if (lane == 0) flag_error(PA_DEVERR_CONTEXT_LEN);
    return c;
  }
  c.pos0 = L - n + c.i0;
  c.hi = c.pos0 + c.tokens;
  c.lo = p.window > 0 ? max(0, c.pos0 - p.window + 1) : 0;
  c.base = c.lo / kChunkStep * kChunkStep;
  return c;
}

// The sequence with the x-th longest context (ties: the lower index first), by
// one warp: the key's bits are fixed from the top by counting the keys that
// are not below the candidate.
constexpr int kChunkOrderMax = 256;
__device__ __forceinline__ int chunk_longest(const ChunkParams& p, int x) {
  const int lane = threadIdx.x & 31;
  uint32_t key[kChunkOrderMax / 32];
#pragma unroll
  for (int k = 0; k < kChunkOrderMax / 32; ++k) {
    const int b = lane + 32 * k;
    key[k] = 0;
    if (b < p.batch) {
      int L = max(0, min(__ldg(p.context_lens + b), (1 << 22) - 1));
      if (p.window > 0) L = min(L, p.window);
      key[k] = (static_cast<uint32_t>(L + 1) << 8) | static_cast<uint32_t>(255 - b);
    }
  }
  uint32_t found = 0;
  for (int bit = 30; bit >= 0; --bit) {
    const uint32_t cand = found | (1u << bit);
    int n = 0;
#pragma unroll
    for (int k = 0; k < kChunkOrderMax / 32; ++k)
      if (32 * k < p.batch) n += __popc(__ballot_sync(0xffffffffu, key[k] >= cand));
    if (n > x) found = cand;
  }
  return min(255 - static_cast<int>(found & 255u), p.batch - 1);
}

// MODE: how K / V reach shared memory.
constexpr int kChunkTma = 0;     // TMA boxes (16-bit, blocks >= 8)
constexpr int kChunkCopy = 1;    // cp.async (16-bit, smaller blocks)
constexpr int kChunkE4m3 = 2;    // cp.async of codes, widened to f16

template <int D, int NT, int MODE>
struct ChunkCfg {
  static constexpr int BN = kChunkStep;
  // warps in groups of four (a register split is set per group): 4 NT softmax
  // warps; two TMA producers (K, V) or four loader warps; a warp per tile that
  // issues its S, and one per tile that issues its P.V; idle ones
  static constexpr int kSoftmaxWarps = 4 * NT;
  static constexpr int kLoadWarps = MODE == kChunkTma ? 2 : 4;
  static constexpr int kLoadThreads = 32 * kLoadWarps;
  static constexpr int kSWarp = kSoftmaxWarps + kLoadWarps;
  static constexpr int kPvWarp = kSWarp + NT;
  static constexpr int kWarps = (kPvWarp + NT + 3) / 4 * 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 1 ? 2 : 1;  // per SM
  // registers per thread: at launch (the register file over the CTAs' threads),
  // then moved from the other groups to the softmax warps, which hold a row of
  // BN scores each
  static constexpr int kLaunchRegs = 65536 / (kCtas * kThreads) / 8 * 8;
  static constexpr int kSoftmaxRegs =
      NT == 2 ? (MODE == kChunkTma ? 168 : 160) : (MODE == kChunkTma ? 152 : 128);
  static constexpr int kOtherRegs =
      (kWarps * kLaunchRegs - kSoftmaxWarps * kSoftmaxRegs) / (kWarps - kSoftmaxWarps) / 8 * 8;
  static_assert(kOtherRegs >= 56, "the split draws on the launch's registers");
  // TMEM columns: S (and P) of tile t, buffer i at (2 t + i) * BN, O of tile t
  // behind them
  static constexpr int kOCol = NT * 2 * BN;
  static constexpr int kColsUsed = kOCol + NT * D;
  static constexpr int kTmemCols = kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
  static_assert(kColsUsed <= 512, "TMEM holds 512 columns");
  static constexpr int kSlabs = D / 64;
  static constexpr int kQTile = kSlabs * kUmmaRows * 128;
  static constexpr int kBufSlab = BN * 128;
  static constexpr int kBuf = kSlabs * kBufSlab;  // one K or V step, 16-bit
  // E4M3: the codes of a K and a V step arrive in a raw stage first
  static constexpr int kRaw = MODE == kChunkE4m3 ? kBuf : 0;
  static constexpr int kRawStages = MODE == kChunkE4m3 ? (NT == 1 ? 2 : 4) : 0;
  // bytes for tiles: 224 KB for one CTA per SM, 112 KB for two
  static constexpr int kBudget = kCtas == 2 ? 112 * 1024 : 224 * 1024;
  static constexpr int kFit = (kBudget - NT * kQTile - kRawStages * kRaw) / kBuf;
  static constexpr int kBufs = kFit < 10 ? kFit : 10;
  static_assert(kBufs >= 3, "a K and a V step in use and one arriving");
  // Barriers of the ring: buffer n's use is phase n / kBars of barrier
  // n % kBars. kBars is even, so that a barrier serves K or V alone also where
  // an odd ring lets them share buffers: whoever waits for one has waited for
  // each of its earlier phases (a parity wait takes the phase before last for
  // its own otherwise: two producers that take turns on one barrier skip every
  // second phase).
  static constexpr int kBars = kBufs % 2 ? 2 * kBufs : kBufs;
  static_assert(kBars <= 10, "room for the barriers");
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + NT * kQTile;
  static constexpr int kRawOff = kRing + kBufs * kBuf;
  static constexpr int kBytes = kRawOff + kRawStages * kRaw;
  static constexpr int kSmall = 352;  // barriers, TMEM address, abort flag
  // (the base is 1024-byte aligned as it is: a block's dynamic shared memory
  // starts behind 1 KB of the system's; the kernel checks that the slack holds)
  static constexpr int kSlack = 512;
  static constexpr int kRequest = kSlack + kBytes + kSmall;
  static_assert(kRequest <= 227 * 1024, "shared memory of a block");
};

// mbar_wait_or_abort with little between the polls: the timer and the abort
// flag are looked at every 32nd time (reading %globaltimer at each poll made
// a step's hand-overs take longer than its MMAs).
__device__ __forceinline__ bool chunk_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) == 0) {
      uint32_t a;
      asm volatile("ld.volatile.shared.u32 %0, [%1];\n" : "=r"(a) : "r"(abort));
      if (a) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        asm volatile("st.volatile.shared.u32 [%0], %1;\n" ::"r"(abort), "r"(1u) : "memory");
        return false;
      }
    }
  }
}

// Whether the phase with parity `parity` is over, without waiting. A ready
// wait takes about 110 clocks from issue to branch; asking early hides them.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "  selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// mbar_arrive / mbar_arrive_expect_tx of one lane of a converged warp,
// predicated (a branch around them takes longer than they do).
__device__ __forceinline__ void mbar_arrive_by(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n"
      "  .reg .pred q;\n"
      "  setp.ne.b32 q, %1, 0;\n"
      "  @q mbarrier.arrive.shared::cta.b64 _, [%0];\n"
      "}\n" ::"r"(bar),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_by(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n"
      "  .reg .pred q;\n"
      "  setp.ne.b32 q, %2, 0;\n"
      "  @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
      "}\n" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}

__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// TMEM store of 16 consecutive 32-bit columns of this warp's lanes.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
template <int N>
__device__ __forceinline__ void set_more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Eight channels from 8 c of token j's K or V row of KV head hk, widened
// (zeros for a block outside the cache, as the loads give).
template <typename TQ, int D, int MODE>
__device__ __forceinline__ void chunk_row_piece(const ChunkParams& p, const void* cache,
                                                const int32_t* table, int hk, int j, int c,
                                                float (&x)[8]) {
  const int id = __ldg(table + (j >> p.bs_log2));
  const int64_t slot = (static_cast<int64_t>(id) << p.bs_log2) + (j & ((1 << p.bs_log2) - 1));
  const int64_t at = (slot * p.num_kv_heads + hk) * D + 8 * c;
  if (id < 0 || id >= p.num_blocks) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
  } else if constexpr (MODE == kChunkE4m3) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at));
    uint32_t h[4];
    e4m3x4_to_f16x2x2(w.x, h[0], h[1]);
    e4m3x4_to_f16x2x2(w.y, h[2], h[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
      x[2 * e] = f.x, x[2 * e + 1] = f.y;
    }
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const TQ*>(cache) + at));
    const TQ* e8 = reinterpret_cast<const TQ*>(&w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f32<TQ>(e8[e]);
  }
}

// P of a token that a row does not see is 0, and 0 x V is NaN where that V is
// not finite. A row whose result is not finite comes here (never in a run of
// finite V): the channels in which such a token of the CTA has a V that is not
// finite are summed again over the tokens the row sees, from its q in shared
// memory (sQ), and written over. Where the row is comes from what the CTA left in
// shared memory (`unit`) and the launch: kept in registers through the steps it
// cost prompts 2 to 4 %.
// A last token without a finite V costs 2048 rows over 16384 tokens (1.0 ms) 37 ms
// for one channel, 140 ms for all.
template <typename TQ, int D, int MODE>
__device__ __forceinline__ void chunk_unseen_v(const ChunkParams& p, uint32_t unit, uint32_t sQ,
                                               float scale_log2, float m, float l) {
  using TO = typename std::conditional<MODE == kChunkE4m3, __half, TQ>::type;
  uint32_t tid, cta;
  asm volatile("mov.u32 %0, %%tid.x;\n" : "=r"(tid));
  asm volatile("mov.u32 %0, %%ctaid.x;\n" : "=r"(cta));
  int b, row0, pos0, tokens;
  asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(b), "=r"(row0), "=r"(pos0), "=r"(tokens)
               : "r"(unit));
  const int part = cta % p.num_partitions;
  const int heads_at = cta / p.num_partitions % (p.head_blocks * p.num_kv_heads);
  const int hk = heads_at / p.head_blocks;
  const int tile = tid >> 7, my_row = tid & (kUmmaRows - 1), sw = my_row & 7;
  const int tok = tile * p.tile_tokens + my_row / p.head_rows;
  const int head = hk * p.group + heads_at % p.head_blocks * p.head_rows + my_row % p.head_rows;
  const int64_t row = (static_cast<int64_t>(row0) + tok) * p.num_q_heads + head;
  const int32_t* table = p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  // tokens of the CTA in this partition [t0, c1), and of the row [lo, hi]
  const int cta_lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
  const int c0 = cta_lo / kChunkStep * kChunkStep + part * p.partition_tokens;
  const int c1 = min(c0 + p.partition_tokens, pos0 + tokens);
  const int t0 = max(cta_lo, c0);
  const int lo = max(p.window > 0 ? max(0, pos0 + tok - p.window + 1) : 0, c0);
  const int hi = min(pos0 + tok, c1 - 1);
  const uint32_t qrow = sQ + tile * ((D / 64) * kUmmaRows * 128) + my_row * 128;
  auto put = [&](int d, float x) {
    if constexpr (MODE == kChunkE4m3) x *= __ldg(p.v_scale + static_cast<int64_t>(hk) * D + d);
    if (p.num_partitions > 1)
      p.ws_o[(row * p.num_partitions + part) * D + d] = x;
    else
      reinterpret_cast<TQ*>(p.out)[row * D + d] = from_f32<TQ>(x);
  };
  uint32_t bad[D / 32] = {};
  for (int j = t0; j < c1; ++j) {
    if (j >= lo && j <= hi) {
      j = hi;
      continue;
    }
#pragma unroll 1
    for (int c = 0; c < D / 8; ++c) {
      float x[8];
      chunk_row_piece<TQ, D, MODE>(p, p.v_cache, table, hk, j, c, x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(fabsf(x[e]) < INFINITY)) bad[c >> 2] |= 1u << ((c & 3) * 8 + e);
    }
  }
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) any |= bad[i];
  if (any == 0) return;  // the tokens it sees say so
  // 32 channels at a time: at most D / 32 passes over the row's K
#pragma unroll 1
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t mine = bad[i];
    if (mine == 0) continue;
    float acc[32] = {};
#pragma unroll 1
    for (int j = lo; j <= hi; ++j) {
      float s = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        float x[8];
        chunk_row_piece<TQ, D, MODE>(p, p.k_cache, table, hk, j, c, x);
        const uint4 w = lds128(qrow + (c >> 3) * (kUmmaRows * 128) + (((c & 7) ^ sw) << 4));
        const TO* q = reinterpret_cast<const TO*>(&w);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(to_f32<TO>(q[e]), x[e], s);
      }
      if (p.sign != 1.f) s *= p.sign;
      const float w = ex2(fmaf(s, scale_log2, -m));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[8];
        chunk_row_piece<TQ, D, MODE>(p, p.v_cache, table, hk, j, 4 * i + c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[8 * c + e] = fmaf(w, x[e], acc[8 * c + e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (mine >> e & 1) put(32 * i + e, l != 0.f ? acc[e] / l : 0.f);
  }
}

// Grid: tiles x KV heads x head blocks x partitions, partition fastest.
template <typename TQ, int D, int NT, int MODE>
__global__ void __launch_bounds__(ChunkCfg<D, NT, MODE>::kThreads,
                                  ChunkCfg<D, NT, MODE>::kCtas)
    pa_chunk_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
  using C = ChunkCfg<D, NT, MODE>;
  // the operands' type: an E4M3 cache is widened to f16, and q folded into it
  constexpr bool BF16 = MODE != kChunkE4m3 && std::is_same<TQ, __nv_bfloat16>::value;
  constexpr float kHeadroom = BF16 ? 0.f : 7.f;
  constexpr int BN = C::BN;
  constexpr int SLABS = C::kSlabs;
  constexpr int NBUF = C::kBufs;
  constexpr int NBAR = C::kBars;
  constexpr uint32_t kIdescS = umma_idesc<BF16, BN, false>();
  constexpr uint32_t kIdescPV = umma_idesc<BF16, D, true>();

  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t raw = smem_addr(smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t small = base + C::kBytes;
  if (base - raw > static_cast<uint32_t>(C::kSlack)) {  // (uniform; never so)
    if (threadIdx.x == 0) flag_error(PA_DEVERR_TIMEOUT);
    return;
  }
  const uint32_t bar_full = small;            // + 8 * (buffer's use % NBAR)
  const uint32_t bar_free = small + 80;       // + 8 * (buffer's use % NBAR)
  const uint32_t bar_s = small + 160;         // + 16 * tile + 8 * S buffer
  const uint32_t bar_p = small + 192;         // + 16 * tile + 8 * S buffer
  const uint32_t bar_pv = small + 272;        // + 16 * tile + 8 * S buffer
  const uint32_t s_live = small + 304;        // + 4 * softmax warp: whether it has rows
  const uint32_t bar_q = small + 240;
  const uint32_t bar_done = small + 248;
  const uint32_t unit = small + 336;          // where the CTA's rows are (chunk_unseen_v)
  const uint32_t tmem_slot = small + 264;
  const uint32_t abort = small + 268;
  const uint32_t sQ = base + C::kQ;
  const uint32_t sRing = base + C::kRing;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  // A mixed batch's second launch may start once every CTA of the first has
  // (they share nothing), and must not end before it, since work behind the
  // call waits for the second only: its last CTA waits for the first.
  if (p.leading) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.trailing && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");

  // one CTA looks at the whole of cu: chunks that overlap, run backwards or
  // leave [0, num_tokens) may own no tile that would notice
  if (blockIdx.x == 0)
    for (int i = tid; i < p.batch; i += C::kThreads)
      if (p.cu[i] < 0 || p.cu[i + 1] < p.cu[i] || p.cu[i + 1] > p.num_tokens)
        flag_error(PA_DEVERR_CHUNK);

  // this CTA's unit
  int u = blockIdx.x;
  const int part = u % p.num_partitions;
  u /= p.num_partitions;
  const int hb = u % p.head_blocks;
  u /= p.head_blocks;
  const int hk = u % p.num_kv_heads;
  // the batch's last tiles first (in a causal chunk they see the most tokens);
  // where every sequence is one tile, the longest contexts first (drafts of 64
  // requests with 512 to 4096 tokens: 138 -> 118 us)
  int x = p.num_tiles - 1 - u / p.num_kv_heads;
  if (NT == 1 && p.longest_first) {
    if (warp == 0) {
      const int b = chunk_longest(p, u / p.num_kv_heads);
      if (lane == 0) asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(tmem_slot), "r"(b) : "memory");
    }
    __syncthreads();
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(x) : "r"(tmem_slot));
    __syncthreads();  // (the slot receives the TMEM address next)
  }
  const ChunkTile ct = chunk_tile(p, x, NT * p.tile_tokens);
  if (ct.b < 0) return;
  const int h0 = hk * p.group + hb * p.head_rows;                 // first query head
  const int heads = min(p.head_rows, p.group - hb * p.head_rows);  // query heads here
  // this partition's tokens: steps of BN from c0
  const int c0 = ct.base + part * p.partition_tokens;
  const int c1 = min(c0 + p.partition_tokens, ct.hi);
  if (c0 >= c1 && part > 0) return;  // (partition 0 writes the zeros of rows without tokens)
  const int nsteps = c0 < c1 ? (c1 - c0 + BN - 1) / BN : 0;
  const int ntiles = (ct.tokens + p.tile_tokens - 1) / p.tile_tokens;
  // steps [tile_a, tile_b) that tile t's rows see any token of
  auto tile_b = [&](int t) {
    const int end = min(c1, ct.pos0 + min((t + 1) * p.tile_tokens, ct.tokens));
    return end > c0 ? (end - c0 + BN - 1) / BN : 0;
  };
  auto tile_a = [&](int t) {
    if (p.window <= 0) return 0;
    const int first = ct.pos0 + t * p.tile_tokens - p.window + 1;
    return min(first > c0 ? (first - c0) / BN : 0, tile_b(t));
  };

  if (warp == 0) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  // the row of a softmax thread: token (within the CTA tile) and query head
  const int tile = warp >> 2;
  const int my_row = tid & (kUmmaRows - 1);
  const int my_tok = tile * p.tile_tokens + my_row / p.head_rows;
  const int my_head = my_row % p.head_rows;
  const bool live = warp < C::kSoftmaxWarps && my_row < p.tile_tokens * p.head_rows &&
                    my_tok < ct.tokens && my_head < heads;
  const bool warp_live = __any_sync(0xffffffffu, live);
  if (NT == 2 && lane == 0 && warp < C::kSoftmaxWarps)
    asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(s_live + 4 * warp), "r"(warp_live ? 1u : 0u) : "memory");
  if (tid == C::kSWarp * 32) {
    for (int i = 0; i < NBAR; ++i) {
      mbar_init(bar_full + 8 * i, MODE == kChunkTma ? 1 : C::kLoadWarps);
      mbar_init(bar_free + 8 * i, NT);
    }
    for (int t = 0; t < NT; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar_s + 16 * t + 8 * i, 1);
        mbar_init(bar_p + 16 * t + 8 * i, 4);
        mbar_init(bar_pv + 16 * t + 8 * i, 1);
      }
    }
    mbar_init(bar_q, MODE == kChunkE4m3 ? 128 * NT : 1);
    mbar_init(bar_done, 2 * NT);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(unit), "r"(ct.b),
                 "r"(static_cast<int>(ct.row)), "r"(ct.pos0), "r"(ct.tokens)
                 : "memory");
    asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(abort), "r"(0u) : "memory");
    mbar_init_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(tmem) : "r"(tmem_slot));
  bool ok = true;
  // use n of the ring (K of step it: n = 2 it, V: 2 it + 1): its buffer, its
  // barriers, their phase, and the wait for the use before it to end
  auto buf = [&](int n) { return sRing + static_cast<uint32_t>(n % NBUF) * C::kBuf; };
  auto full_of = [&](int n) { return bar_full + 8 * (n % NBAR); };
  auto parity = [](int n) { return static_cast<uint32_t>((n / NBAR) & 1); };
  auto wait_free = [&](int n) {
    return n < NBUF || chunk_wait(bar_free + 8 * ((n - NBUF) % NBAR), parity(n - NBUF), abort);
  };
  const int32_t* table = p.block_tables + static_cast<int64_t>(ct.b) * p.max_blocks_per_seq;
  auto block_of = [&](int j) -> int {  // physical block of token j, -1 if out of range
    const int id = __ldg(table + (j >> p.bs_log2));
    if (id < 0 || id >= p.num_blocks) {
      flag_error(PA_DEVERR_BLOCK_ID);
      return -1;
    }
    return id;
  };

  // one warp loads the row tiles of q (16-bit operands: as they are; boxes of
  // the tile's tokens x its query heads; rows of other chunks come along) and
  // sees them land before the CTA exits
  auto load_q = [&]() {
    if (nsteps <= 0) return;
    if (lane == 0) mbar_arrive_expect_tx(bar_q, ntiles * SLABS * p.tile_tokens * p.head_rows * 128);
    __syncwarp();
    if (lane < ntiles * SLABS) {
      const int t = lane / SLABS;
      const int s = lane % SLABS;
      tma_load_3d(sQ + t * C::kQTile + s * (kUmmaRows * 128), &tm_q, bar_q, s * 64, h0,
                  static_cast<int>(ct.row) + t * p.tile_tokens);
    }
  };
  auto drain_q = [&]() {
    if (nsteps > 0 && lane == 0) mbar_wait(bar_q, 0);
  };

  // (one register change per group of four warps, at one place)
  if (warp < C::kSoftmaxWarps) {
    set_more_regs<C::kSoftmaxRegs>();
    // ---- softmax: thread = row --------------------------------------------------
    const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t_lane + tile * 2 * BN;
    const uint32_t tO = tmem + t_lane + C::kOCol + tile * D;
    const int64_t row = (ct.row + my_tok) * p.num_q_heads + h0 + my_head;
    const int pos = ct.pos0 + my_tok;
    const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float scale_log2 = p.scale_log2;
    if constexpr (MODE == kChunkE4m3) {
      // q' = q * k_scale in f16: each row is divided by the power of two of
      // its largest |q * k_scale| first (and its scale multiplied by it), so
      // that no product leaves f16's range whatever the scales
      if (nsteps > 0) {
        float mx = 0.f;
        const TQ* q = reinterpret_cast<const TQ*>(p.q) + row * D;
        const float4* ks = reinterpret_cast<const float4*>(p.k_scale + static_cast<int64_t>(hk) * D);
        auto piece = [&](int c, float (&y)[8]) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(q) + c);
          const TQ* e = reinterpret_cast<const TQ*>(&w);
          const float4 s0 = __ldg(ks + 2 * c), s1 = __ldg(ks + 2 * c + 1);
          const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = to_f32<TQ>(e[i]) * s[i];
        };
        if (live) {
#pragma unroll 2
          for (int c = 0; c < D / 8; ++c) {
            float y[8];
            piece(c, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(y[i]));
          }
        }
        int e2 = 0;
        if (mx > 0.f && mx < INFINITY) frexpf(mx, &e2);
        e2 = max(-120, min(e2, 120));
        const float down = ldexpf(1.f, -e2);
        scale_log2 *= ldexpf(1.f, e2);
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
          float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (live) piece(c, y);
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack2<false>(y[2 * i] * down, y[2 * i + 1] * down);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                           sQ + tile * C::kQTile + (c >> 3) * (kUmmaRows * 128) + my_row * 128 +
                           (((c & 7) ^ (my_row & 7)) << 4)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        fence_async_smem();
        mbar_arrive(bar_q);
      }
    }
    const int a = tile < ntiles ? tile_a(tile) : 0;
    const int b = tile < ntiles ? tile_b(tile) : 0;
    // the first and last position of this tile's rows: steps inside what all
    // of them see need no mask
    const int pos_first = ct.pos0 + tile * p.tile_tokens;
    const int pos_last = ct.pos0 + min((tile + 1) * p.tile_tokens, ct.tokens) - 1;
    float m_run = -INFINITY;
    float l_run = 0.f;
    // Turns of the exponential unit: warp w of tile 0 and warp w of tile 1 sit on
    // the same scheduler. In step they would use each pipe at the same time and
    // leave the others idle; in turn one computes its exponentials while the
    // other loads its scores, finds their maximum and stores P. Steps that both
    // tiles have, where both warps have rows; tile 0 starts. bar.sync has no limit
    // of its own: what bounds it is that both warps take all their turns, also one
    // whose other, bounded waits have failed (it takes the rest empty-handed,
    // below), so each is waited for by one that comes. (Turns on mbarriers or
    // polled flags, each wait with its limit: prompts 150 -> 160 us, 968 -> 1095 us.)
    int turn_a = 0, turn_b = 0;
    int next_turn = 0;  // the step of the next turn to take
    const int my_turn = 1 + tile * 4 + (warp & 3), other_turn = 1 + (tile ^ 1) * 4 + (warp & 3);
    if constexpr (NT == 2) {
      uint32_t other;
      asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(other) : "r"(s_live + 4 * (warp ^ 4)));
      if (ntiles == 2 && warp_live && other) {
        turn_a = max(tile_a(0), tile_a(1));
        turn_b = min(tile_b(0), tile_b(1));
        next_turn = turn_a;
        if (tile == 1 && turn_a < turn_b)
          asm volatile("bar.arrive %0, 64;\n" ::"r"(other_turn) : "memory");
      }
    }
    for (int it = a; it < b; ++it) {
      const int j0 = c0 + it * BN;
      const uint32_t tSi = tS + ((it - a) & 1) * BN;
      ok = __all_sync(0xffffffffu, chunk_wait(bar_s + 16 * tile + 8 * ((it - a) & 1),
                                              static_cast<uint32_t>(((it - a) >> 1) & 1), abort));
      if (!ok) break;
      tc_fence_after();
      // V rows that no row of the CTA attends: zeros (their blocks may hold
      // anything). Loader warps have put zeros there.
      auto zero_v = [&]() -> bool {
        if constexpr (MODE == kChunkTma) {
          const int z_hi = c1 - j0, z_lo = ct.lo - j0;
          if (z_hi < BN || z_lo > 0) {
            const int n = 2 * it + 1;
            ok = __all_sync(0xffffffffu,
                            chunk_wait(full_of(n), parity(n), abort));
            if (!ok) return false;
            for (int i = my_row; i < BN * SLABS * 8; i += 128) {
              const int r = i >> 3 & (BN - 1);
              if (r >= z_hi || r < z_lo)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(buf(n) + i * 16), "r"(0u)
                             : "memory");
            }
            fence_async_smem();
          }
        }
        return true;
      };
      if (warp_live) {
        // tokens this row does not attend
        const bool edge = j0 + BN - 1 > pos_first || (p.window > 0 && j0 <= pos_last - p.window) ||
                          j0 + BN > c1;
        const int see_hi = min(pos, c1 - 1) - j0;
        const int see_lo = first - j0;
        auto mask32 = [&](int c, float (&h)[32]) {
          if (p.sign != 1.f) {  // a negative or zero scale
#pragma unroll
            for (int j = 0; j < 32; ++j) h[j] *= p.sign;
          }
          if (edge) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j > see_hi || c + j < see_lo) h[j] = -INFINITY;
          }
        };
        // the row's maximum: four chains of three-input maxima (a NaN score is
        // passed over here and makes its weight, and so the row, NaN below)
        float m4[4];
        auto max32 = [&](const float (&h)[32], bool start) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const int i = (j >> 1) & 3;
            m4[i] = start && j < 8 ? max3(h[j], h[j + 1], h[j + 1]) : max3(m4[i], h[j], h[j + 1]);
          }
        };
        float s0[32], s1[32];
        tmem_ld32(tSi, s0);
        tmem_ld32(tSi + 32, s1);
        tmem_ld_wait();
        mask32(0, s0);
        max32(s0, true);
        mask32(32, s1);
        max32(s1, false);
        float mx = max3(max3(m4[0], m4[1], m4[2]), m4[3], m4[3]);
        mx *= scale_log2;
        // (the first finite maximum always moves it)
        const bool up = mx > m_run + (kHeadroom + kRescaleLog2);
        const float m_ref = up ? mx - kHeadroom : m_run;
        const float alpha = up ? ex2(m_run - m_ref) : 1.f;
        // a row that has seen no token yet keeps p = 2^(-inf) = 0
        const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t sc2 = pack_f32x2(scale_log2, scale_log2);
        const uint64_t nm2 = pack_f32x2(neg_m, neg_m);
        uint64_t sum2[2] = {0ull, 0ull};
        auto exp32 = [&](int c, const float (&h)[32]) {
          uint32_t pw[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint64_t y2 = fma_f32x2(pack_f32x2(h[j], h[j + 1]), sc2, nm2);
            const float2 y = unpack_f32x2(y2);
            const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
            sum2[(j >> 1) & 1] = add_f32x2(sum2[(j >> 1) & 1], pack_f32x2(e2.x, e2.y));
            pw[j / 2] = pack2<BF16>(e2.x, e2.y);
          }
          tmem_st16u(tSi + c / 2, pw);
        };
        // the exponentials of the two tiles' warps of one scheduler take turns
        const bool turn = it >= turn_a && it < turn_b;
        if (turn) asm volatile("bar.sync %0, 64;\n" ::"r"(my_turn) : "memory");
        exp32(0, s0);
        exp32(32, s1);
        if (turn && (tile == 0 || it + 1 < turn_b))
          asm volatile("bar.arrive %0, 64;\n" ::"r"(other_turn) : "memory");
        if (turn) next_turn = it + 1;
        const float2 t2 = unpack_f32x2(add_f32x2(sum2[0], sum2[1]));
        l_run = l_run * alpha + (t2.x + t2.y);
        m_run = m_ref;
        // rows whose reference maximum moved rescale their O row, once P.V(it - 1)
        // is done (a full S(it) says that P.V(it - 2) is)
        if (it > a && __any_sync(0xffffffffu, up)) {
          const int n = it - a - 1;
          ok = __all_sync(0xffffffffu, chunk_wait(bar_pv + 16 * tile + 8 * (n & 1),
                                                  static_cast<uint32_t>((n >> 1) & 1), abort));
          if (!ok) {
            tmem_st_wait();  // (P's store) before the CTA drains
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tO + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(tO + c, o);
          }
        }
        tmem_st_wait();
      }
      if (!zero_v()) break;
      tc_fence_before();
      __syncwarp();
      mbar_arrive_by(lane == 0, bar_p + 16 * tile + 8 * ((it - a) & 1));
    }
    if (!ok)
      for (; next_turn < turn_b; ++next_turn) {  // the turns of the steps given up
        asm volatile("bar.sync %0, 64;\n" ::"r"(my_turn) : "memory");
        if (tile == 0 || next_turn + 1 < turn_b)
          asm volatile("bar.arrive %0, 64;\n" ::"r"(other_turn) : "memory");
      }
    if (ok && b > a) {  // the last P.V
      const int n = b - a - 1;
      ok = __all_sync(0xffffffffu, chunk_wait(bar_pv + 16 * tile + 8 * (n & 1),
                                              static_cast<uint32_t>((n >> 1) & 1), abort));
      tc_fence_after();
    }
    // ---- the row's result (or its partial) -------------------------------------------
    if (ok && warp_live && tile < ntiles) {
      const bool any = b > a;
      const float inv = l_run != 0.f ? 1.f / l_run : 0.f;  // no token attended: zeros
      float finite = 0.f;  // 0 while every value of the row is
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (any) {
          tmem_ld32(tO + c, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          o[e] = any && l_run != 0.f ? o[e] * inv : 0.f;
          finite = fmaf(o[e], 0.f, finite);
        }
        if constexpr (MODE == kChunkE4m3) {
          const float4* vs = reinterpret_cast<const float4*>(p.v_scale + static_cast<int64_t>(hk) * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 s = __ldg(vs + e);
            o[4 * e] *= s.x;
            o[4 * e + 1] *= s.y;
            o[4 * e + 2] *= s.z;
            o[4 * e + 3] *= s.w;
          }
        }
        if (live) {
          if (p.num_partitions > 1) {
            float4* dst = reinterpret_cast<float4*>(p.ws_o + (row * p.num_partitions + part) * D + c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<TQ*>(p.out) + row * D + c);
            constexpr bool kOutBf16 = std::is_same<TQ, __nv_bfloat16>::value;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_uint4(pack2<kOutBf16>(o[8 * e], o[8 * e + 1]),
                                  pack2<kOutBf16>(o[8 * e + 2], o[8 * e + 3]),
                                  pack2<kOutBf16>(o[8 * e + 4], o[8 * e + 5]),
                                  pack2<kOutBf16>(o[8 * e + 6], o[8 * e + 7]));
          }
        }
      }
      if (live && finite != 0.f && mbar_wait(bar_q, 0))  // (Q's bytes have landed for this thread)
        chunk_unseen_v<TQ, D, MODE>(p, unit, sQ, scale_log2, m_run, l_run);
      if (live && p.num_partitions > 1)
        p.ws_ml[row * p.num_partitions + part] = make_float2(m_run, l_run);
    }
  } else if (MODE != kChunkTma && warp < C::kSWarp) {
    set_fewer_regs<C::kOtherRegs>();
    if constexpr (MODE != kChunkTma) {
      // ---- loader warps: 16-byte pieces with cp.async -------------------------
      const int lt = tid - C::kSoftmaxWarps * 32;
      constexpr int kElem = MODE == kChunkE4m3 ? 1 : 2;
      constexpr int kPieces = D * kElem / 16;            // per token row
      constexpr int kPer = BN * kPieces / C::kLoadThreads;  // per thread and step
      static_assert(kPer * C::kLoadThreads == BN * kPieces, "whole rounds");
      const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * D * kElem;
      const uint32_t sRaw = base + C::kRawOff;
      // block of each of this thread's rows of step `it`: -1 for tokens outside
      // [lo, c1) and bad blocks, which become zeros
      auto lookup = [&](int it, int (&id)[kPer]) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int j = c0 + it * BN + (lt + k * C::kLoadThreads) / kPieces;
          id[k] = j >= ct.lo && j < c1 ? block_of(j) : -1;
        }
      };
      // start the copies of a step's K and V (into the raw stage, or the ring
      // buffers themselves)
      auto start = [&](int it, const int (&id)[kPer]) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int piece = lt + k * C::kLoadThreads;
          const int r = piece / kPieces, c = piece % kPieces;
          const int j = c0 + it * BN + r;
          const int64_t at = ((static_cast<int64_t>(max(id[k], 0)) << p.bs_log2) + (j & ((1 << p.bs_log2) - 1))) *
                                 row_bytes + hk * (D * kElem) + c * 16;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const char* cache = reinterpret_cast<const char*>(kv ? p.v_cache : p.k_cache);
            uint32_t dst;
            if constexpr (MODE == kChunkE4m3)
              dst = sRaw + (it % C::kRawStages) * C::kRaw + kv * (C::kRaw / 2) + piece * 16;
            else
              dst = buf(2 * it + kv) + (c >> 3) * C::kBufSlab + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            cp_async_16(dst, id[k] < 0 ? cache : cache + at, id[k] < 0 ? 0u : 16u);
          }
        }
      };
      // finish a step whose copies (this thread's own) have landed
      auto finish = [&](int it) -> bool {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int n = 2 * it + kv;
          if constexpr (MODE == kChunkE4m3) {
            uint4 w[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k)
              w[k] = lds128(sRaw + (it % C::kRawStages) * C::kRaw + kv * (C::kRaw / 2) +
                            (lt + k * C::kLoadThreads) * 16);
            if (!wait_free(n)) return false;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              const int piece = lt + k * C::kLoadThreads;
              const int r = piece / kPieces, c = piece % kPieces;
              uint4 h[2];
              e4m3x4_to_f16x2x2(w[k].x, h[0].x, h[0].y);
              e4m3x4_to_f16x2x2(w[k].y, h[0].z, h[0].w);
              e4m3x4_to_f16x2x2(w[k].z, h[1].x, h[1].y);
              e4m3x4_to_f16x2x2(w[k].w, h[1].z, h[1].w);
              // the row's two slabs would meet in the same banks: the upper
              // slab's threads store their odd half first
              const bool odd = c >= 4;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int cc = 2 * c + (e ^ (odd ? 1 : 0));
                const uint4 v = (e ^ (odd ? 1 : 0)) ? h[1] : h[0];
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                                 buf(n) + (cc >> 3) * C::kBufSlab + r * 128 + (((cc & 7) ^ (r & 7)) << 4)),
                             "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
              }
            }
          }
          fence_async_smem();
          __syncwarp();
          mbar_arrive_by(lane == 0, full_of(n));
        }
        return true;
      };
      // copies run kAhead steps ahead of their use, table entries one more
      constexpr int kAhead = MODE == kChunkE4m3 ? C::kRawStages - 1 : NBUF / 2 - 1;
      if (MODE == kChunkCopy && warp == C::kSoftmaxWarps) load_q();
      int id[kPer];
      if (nsteps > 0) lookup(0, id);
      for (int n = 0; n < nsteps + kAhead; ++n) {
        if (n < nsteps) {
          if (MODE == kChunkCopy && !(wait_free(2 * n) && wait_free(2 * n + 1))) break;
          start(n, id);
          if (n + 1 < nsteps) lookup(n + 1, id);
        }
        cp_async_commit();
        if (n >= kAhead) {
          cp_async_wait<kAhead>();
          if (!finish(n - kAhead)) break;
        }
      }
      cp_async_wait<0>();
      if (MODE == kChunkCopy && warp == C::kSoftmaxWarps) drain_q();
    }
  } else {
    set_fewer_regs<C::kOtherRegs>();
    if (warp >= C::kSWarp && warp < C::kPvWarp + NT) {
      // ---- MMA issue: per tile one warp for S and one for P.V ------------------
      // S has two buffers per tile, so that S(it + 1) is there when the softmax
      // warps finish S(it). A warp needs about 60 clocks to issue an MMA (one of
      // N = 64 runs in 33 to 49), 110 for a wait and 60 for a commit, so a warp
      // for everything could not keep the tensor core busy; four can.
      if (nsteps > 0) {
        const bool is_s = warp < C::kPvWarp;
        const int t = (warp - C::kSWarp) % NT;
        const int a = t < ntiles ? tile_a(t) : 0;
        const int b = t < ntiles ? tile_b(t) : 0;
        const uint32_t tS = tmem + t * 2 * BN;
        const uint32_t tO = tmem + C::kOCol + t * D;
        // descriptors of Q's tile, and of the ring as K (both slabs K-major) and
        // as V (MN-major); offsets add in 16-byte units
        const uint64_t dq = sw128_desc(sQ + t * C::kQTile, 16, 1024);
        const uint64_t dkv = is_s ? sw128_desc(sRing, 16, 1024) : sw128_desc(sRing, C::kBufSlab, 1024);
        // this step's use of the ring, modulo NBAR
        int slot = is_s ? 0 : 1;
        uint32_t phase = 0;
        if (is_s) ok = chunk_wait(bar_q, 0, abort) && !(p.withhold_scores >> t & 1);
        // (a parity wait tells a phase from the one before or after only; so
        // every barrier here is waited for when its last phase but one is known
        // to be over and its next cannot end yet)
        bool ready = false;  // asked ahead whether the buffer is full
        for (int it = 0; ok && it < nsteps; ++it) {
          const bool mine = it >= a && it < b;
          const uint32_t i = (it - a) & 1, ph = ((it - a) >> 1) & 1;
          if (!ready) ready = mbar_test(bar_full + 8 * slot, phase);
          if (is_s && !(ok = ready || chunk_wait(bar_full + 8 * slot, phase, abort))) break;
          ready = ready || is_s;
          if (mine) {
            // S: the buffer's last P has been read; P.V: P is there
            if (is_s)
              ok = it - a < 2 || chunk_wait(bar_pv + 16 * t + 8 * i, ph ^ 1, abort);
            else
              ok = chunk_wait(bar_p + 16 * t + 8 * i, ph, abort);
          }
          if (!ok || !(ok = ready || chunk_wait(bar_full + 8 * slot, phase, abort))) break;
          const uint32_t free_bar = bar_free + 8 * slot;
          const int at = NBAR > NBUF && slot >= NBUF ? slot - NBUF : slot;
          const uint64_t dst = dkv + static_cast<uint32_t>(at * (C::kBuf >> 4));
          slot += 2;
          if (slot >= NBAR) {
            slot -= NBAR;
            phase ^= 1;
          }
          tc_fence_after();
          if (lane == 0) {
            if (mine && is_s) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_f16(tS + i * BN, dq + (((kk >> 2) * (kUmmaRows * 128) + (kk & 3) * 32) >> 4),
                         dst + (((kk >> 2) * C::kBufSlab + (kk & 3) * 32) >> 4), kIdescS, kk > 0);
              umma_commit(bar_s + 16 * t + 8 * i);
            } else if (mine) {
#pragma unroll
              for (int kk = 0; kk < BN / 16; ++kk)
                umma_f16_tmem_a(tO, tS + i * BN + kk * 8, dst + (kk * 16 * 128 >> 4), kIdescPV,
                                (it > a || kk > 0) ? 1u : 0u);
              umma_commit(bar_pv + 16 * t + 8 * i);
            }
            umma_commit(free_bar);
          }
          __syncwarp();
          ready = it + 1 < nsteps && mbar_test(bar_full + 8 * slot, phase);
        }
        // every issued MMA has completed before TMEM is released
        if (lane == 0) umma_commit(bar_done);
        __syncwarp();
        mbar_wait(bar_done, 0);
      }
    } else if (MODE == kChunkTma && warp < C::kSWarp) {
      // ---- TMA producers (K, and V): lane i issues box (unit i / SLABS, slab
      // i % SLABS) of each step
      const int kv = warp - C::kSoftmaxWarps;
      const CUtensorMap* map = kv ? &tm_v : &tm_k;
      if (lane == 0)
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
      const int bs_mask = (1 << p.bs_log2) - 1;
      const int unit = min(1 << p.bs_log2, BN);
      const int nbox = BN / unit * SLABS;  // <= 32
      const int u0 = lane / SLABS * unit;
      const int sl = lane % SLABS;
      // slot of this lane's unit in step `it`; units without a token of
      // [lo, hi), and bad blocks, read past the map: zeros. Their table
      // entries are not looked up.
      auto slot_of = [&](int it) -> int {
        const int j = c0 + it * BN + u0;
        if (lane >= nbox || j >= c1 || j + unit <= ct.lo) return p.num_slots;
        const int blk = block_of(j);
        return blk < 0 ? p.num_slots : (blk << p.bs_log2) + (j & bs_mask);
      };
      if (kv == 0) load_q();
      int issued = 0;  // steps
      int slot = nsteps > 0 ? slot_of(0) : 0;
      for (int it = 0; it < nsteps; ++it) {
        const int next = it + 1 < nsteps ? slot_of(it + 1) : 0;
        const int n = 2 * it + kv;
        if (!__all_sync(0xffffffffu, wait_free(n))) break;
        const uint32_t bar = full_of(n);
        mbar_arrive_expect_tx_by(lane == 0, bar, C::kBuf);
        __syncwarp();
        if (lane < nbox) tma_load_3d(buf(n) + sl * C::kBufSlab + u0 * 128, map, bar, sl * 64, hk, slot);
        issued = it + 1;
        slot = next;
      }
      // every issued copy has landed before the CTA can exit: the last one of
      // each barrier (the last copy's wait for its buffer says that those
      // before have)
      if (lane == 0)
        for (int it = max(issued - NBAR / 2, 0); it < issued; ++it)
          mbar_wait(full_of(2 * it + kv), parity(2 * it + kv));
      if (kv == 0) drain_q();
    }
  }

  tc_fence_before();
  __syncthreads();
  uint32_t aborted;
  asm volatile("ld.volatile.shared.u32 %0, [%1];\n" : "=r"(aborted) : "r"(abort));
  if (aborted && tid == 0) flag_error(PA_DEVERR_TIMEOUT);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Merge of a split context: one warp per row of a CTA tile, the row's
// partials that the attention kernel wrote (the tile's own token range says
// how many), weighted by l 2^(m - max m).
template <typename TQ, int D>
__global__ void __launch_bounds__(256) pa_chunk_merge_kernel(const ChunkParams p, int cta_tokens) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const ChunkTile ct = chunk_tile(p, blockIdx.x, cta_tokens);
  if (ct.b < 0) return;
  const int r = blockIdx.y * 8 + warp;  // row of the tile: (token, query head)
  if (r >= ct.tokens * p.num_q_heads) return;
  const int64_t row = ct.row * p.num_q_heads + r;
  const int parts = max(1, (ct.hi - ct.base + p.partition_tokens - 1) / p.partition_tokens);
  const float2* ml = p.ws_ml + row * p.num_partitions;
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 32) {
    const float2 v = ml[i];
    if (v.y != 0.f) m = fmaxf(m, v.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  constexpr int V = D / 32;  // channels per lane
  float acc[V] = {};
  float l = 0.f;
  const float* po = p.ws_o + row * p.num_partitions * D + lane * V;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 v = ml[i];
    const float w = v.y != 0.f ? v.y * ex2(v.x - m) : 0.f;
    l += w;
    float o[V];
    if constexpr (V == 4) {
      const float4 f = *reinterpret_cast<const float4*>(po + static_cast<int64_t>(i) * D);
      o[0] = f.x, o[1] = f.y, o[2] = f.z, o[3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(po + static_cast<int64_t>(i) * D);
      o[0] = f.x, o[1] = f.y;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] += w != 0.f ? w * o[e] : 0.f;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  TQ* out = reinterpret_cast<TQ*>(p.out) + row * D + lane * V;
  constexpr bool BF16 = std::is_same<TQ, __nv_bfloat16>::value;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv), pack2<BF16>(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(out) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
}

}  // namespace pa

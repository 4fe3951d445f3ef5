// The batched calls of the block manager (pa_bm_append_chunks, pa_bm_keep)
// when the host runs out of memory: every allocation of a call fails in turn.
// A call that reports PA_BM_ERR_CAPACITY must have changed nothing; one that
// returns PA_BM_OK must have done its work (at most some blocks stay out of
// the prefix cache); and the manager must go on and account for every block.
#include <cstdio>
#include <cstdlib>
#include <new>
#include <vector>

#include "pa_block_manager.h"

static long g_fail_at = -1;  // allocations until one fails (-1: none does)
static bool g_failed = false;

void* operator new(std::size_t n) {
  if (g_fail_at >= 0 && g_fail_at-- == 0) {
    g_failed = true;
    throw std::bad_alloc();
  }
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void* operator new(std::size_t n, const std::nothrow_t&) noexcept { return std::malloc(n ? n : 1); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

#define CHECK(x)                                                      \
  do {                                                                \
    if (!(x)) {                                                       \
      std::printf("line %d: %s (allocation %ld)\n", __LINE__, #x, at); \
      std::exit(1);                                                   \
    }                                                                 \
  } while (0)

constexpr int kBlocks = 24, kBs = 4, kMax = 16;
const int64_t kIds[4] = {1, 2, 3, 4};

struct State {
  std::vector<int32_t> all;
  bool operator==(const State& o) const { return all == o.all; }
};

static State state(pa_block_manager* bm, int n_seqs) {
  State s;
  s.all.push_back(static_cast<int32_t>(pa_bm_num_free_blocks(bm)));
  s.all.push_back(static_cast<int32_t>(pa_bm_num_cached_blocks(bm)));
  for (int b = 0; b < kBlocks; ++b) s.all.push_back(pa_bm_block_refcount(bm, b));
  std::vector<int32_t> tables(4 * kMax), lens(4);
  pa_bm_block_tables(bm, kIds, n_seqs, kMax, tables.data(), lens.data());
  s.all.insert(s.all.end(), tables.begin(), tables.end());
  s.all.insert(s.all.end(), lens.begin(), lens.end());
  return s;
}

// Sequences of which two share a partial block, one is cut inside a cached
// block, and cached blocks that only evictions give back.
static pa_block_manager* setup(long at) {
  pa_block_manager* bm = pa_bm_create(kBlocks, kBs, 1);
  std::vector<int32_t> t(64);
  for (int i = 0; i < 64; ++i) t[i] = i;
  CHECK(pa_bm_add_sequence(bm, 9, t.data() + 20, 16, nullptr) == PA_BM_OK);
  CHECK(pa_bm_free_sequence(bm, 9) == PA_BM_OK);
  CHECK(pa_bm_add_sequence(bm, 1, t.data(), 10, nullptr) == PA_BM_OK);
  CHECK(pa_bm_fork(bm, 1, 2) == PA_BM_OK);
  CHECK(pa_bm_add_sequence(bm, 3, t.data() + 40, 8, nullptr) == PA_BM_OK);
  const int64_t id = 3;
  const int32_t len = 7;
  CHECK(pa_bm_keep(bm, &id, &len, 1) == PA_BM_OK);
  CHECK(pa_bm_add_sequence(bm, 4, t.data() + 50, 1, nullptr) == PA_BM_OK);
  return bm;
}

static void finish(pa_block_manager* bm, long at) {
  // another chunk, cut again, then every block comes back
  const int32_t counts[4] = {1, 2, 1, 1}, tokens[5] = {7, 7, 7, 7, 7};
  int64_t slots[5];
  int32_t pairs[8], n = 0, lens[4], before[4];
  for (int i = 0; i < 4; ++i) before[i] = pa_bm_sequence_length(bm, kIds[i]);
  CHECK(pa_bm_append_chunks(bm, kIds, counts, 4, tokens, 1, slots, pairs, &n) == PA_BM_OK);
  for (int i = 0; i < 4; ++i) {
    CHECK(pa_bm_sequence_length(bm, kIds[i]) == before[i] + counts[i]);
    lens[i] = before[i];
  }
  CHECK(pa_bm_keep(bm, kIds, lens, 4) == PA_BM_OK);
  for (int i = 0; i < 4; ++i) CHECK(pa_bm_free_sequence(bm, kIds[i]) == PA_BM_OK);
  CHECK(pa_bm_num_free_blocks(bm) + pa_bm_num_cached_blocks(bm) == kBlocks);
  // and what is cached can be evicted: one sequence takes the whole pool
  std::vector<int32_t> t(kBlocks * kBs, 100);
  CHECK(pa_bm_add_sequence(bm, 50, t.data(), kBlocks * kBs, nullptr) == PA_BM_OK);
  CHECK(pa_bm_free_sequence(bm, 50) == PA_BM_OK);
  pa_bm_destroy(bm);
}

int main() {
  const int32_t counts[4] = {9, 5, 6, 15};
  std::vector<int32_t> tokens(35);
  for (int i = 0; i < 35; ++i) tokens[i] = 200 + i;
  int refused = 0, kept_going = 0;
  for (int offer = 0; offer < 2; ++offer)
    for (long at = 0;; ++at) {
      pa_block_manager* bm = setup(at);
      const State before = state(bm, 4);
      int64_t slots[35];
      int32_t pairs[8], n = 0;
      g_failed = false;
      g_fail_at = at;
      const int32_t rc =
          pa_bm_append_chunks(bm, kIds, counts, 4, tokens.data(), offer, slots, pairs, &n);
      g_fail_at = -1;
      const bool failed = g_failed;
      if (rc != PA_BM_OK) {
        CHECK(failed && rc == PA_BM_ERR_CAPACITY);
        CHECK(state(bm, 4) == before);
        ++refused;
      } else {
        kept_going += failed;
        const int32_t want[4] = {19, 15, 13, 16};
        for (int i = 0; i < 4; ++i) CHECK(pa_bm_sequence_length(bm, kIds[i]) == want[i]);
        CHECK(n == 2);  // (one of the sharers, and the sequence cut in a cached block)
        // the slots reported are the sequences' own
        int64_t own[35];
        int k = 0;
        for (int i = 0; i < 4; ++i) {
          CHECK(pa_bm_slots(bm, kIds[i], want[i] - counts[i], counts[i], own + k) == PA_BM_OK);
          k += counts[i];
        }
        for (int i = 0; i < 35; ++i) CHECK(own[i] == slots[i]);
      }
      finish(bm, at);
      if (!failed) break;
    }
  for (long at = 0;; ++at) {  // drafts, of which the batch keeps some
    pa_block_manager* bm = setup(at);
    int64_t slots[35];
    int32_t pairs[8], n = 0;
    CHECK(pa_bm_append_chunks(bm, kIds, counts, 4, tokens.data(), 0, slots, pairs, &n) == PA_BM_OK);
    const State before = state(bm, 4);
    const int32_t lens[4] = {17, 12, 8, 16};
    g_failed = false;
    g_fail_at = at;
    const int32_t rc = pa_bm_keep(bm, kIds, lens, 4);
    g_fail_at = -1;
    const bool failed = g_failed;
    if (rc != PA_BM_OK) {
      CHECK(failed && rc == PA_BM_ERR_CAPACITY);
      CHECK(state(bm, 4) == before);
      ++refused;
    } else {
      kept_going += failed;
      for (int i = 0; i < 4; ++i) CHECK(pa_bm_sequence_length(bm, kIds[i]) == lens[i]);
    }
    finish(bm, at);
    if (!failed) break;
  }
  long at = 0;
  CHECK(refused > 5 && kept_going > 5);
  std::printf("ok: %d refused, %d went on\n", refused, kept_going);
  return 0;
}

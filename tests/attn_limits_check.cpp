// CPU check of csrc/attn_plan.h at the largest sizes.
#include <cstdio>
#include <random>

#include "../w8a8_int8_quantized_amd/csrc/attn_plan.h"

using namespace w8;

#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      std::printf("failed: %s, line %d (round %d)\n", #c, __LINE__, round); \
      return 1;                                                           \
    }                                                                     \
  } while (0)

// The units that a call's sizes allow for are no fewer than its sequences have,
// and what sums to more than 32 bits hold never looks like less.
static int units() {
  std::mt19937 rng(2);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (uint32_t)(hi - lo + 1)); };
  for (int round = 0; round < 20000; ++round) {
    AttnShape a;
    a.B = pick(1, 40);
    a.Hkv = pick(1, 9);
    a.G = pick(1, 20);
    a.rows = 4 << pick(0, 4);
    a.page = 16 * pick(1, 6);
    a.max_pages = pick(0, round % 2 ? 3 : 200);
    a.causal = pick(0, 1);
    // (row tiles below 16 rows hold all rows of a sequence)
    const int longest = a.rows < 16 ? a.rows / a.G : pick(1, 300);
    if (longest < 1) continue;
    a.max_q = 0;
    a.T = 0;
    int n[40], len[40];
    for (int b = 0; b < a.B; ++b) {
      n[b] = pick(0, longest);
      len[b] = pick(0, 3) ? a.max_pages * a.page - pick(0, 40) : pick(0, a.max_pages * a.page);
      a.T += n[b];
      a.max_q = n[b] > a.max_q ? n[b] : a.max_q;
    }
    if (a.T == 0) continue;
    a.max_q += pick(0, 2);
    a.max_q = a.max_q < a.T ? a.max_q : a.T;
    if (a.rows < 16 && a.max_q * a.G > a.rows) continue;
    uint64_t total = 0;
    uint32_t sum = 0;
    for (int b = 0, at = 0; b < a.B; at += n[b++]) {
      const uint32_t u = attn_units(a, attn_seq(a, at, at + n[b], len[b]));
      total += u;
      sum = attn_add(sum, u);
    }
    CHECK(total <= attn_most_units(a));
    CHECK(sum == total);
  }
  const int round = 0;
  // 128 pieces of 2048 tokens, and 32 of 8192, beside a table for 131072
  AttnShape a = {128, 128 * 2048, 8, 4, 2048, 64, 2048, 1, 64};
  CHECK(attn_most_units(a) <= kAttnMostUnits);
  a.B = 32, a.max_q = 8192;
  CHECK(attn_most_units(a) <= kAttnMostUnits);
  // sizes whose product passes 64 bits
  a = {2147483647, 2147483647, 4096, 1, 2147483647, 16, 134217727, 1, 16};
  CHECK(attn_most_units(a) > kAttnMostUnits);
  CHECK(attn_add(0xffffffffu, 1) == 0xffffffffu && attn_add(0x80000000u, 0x80000000u) == 0xffffffffu);
  CHECK(attn_add(0xfffffffeu, 1) == 0xffffffffu && attn_add(3, 4) == 7);
  // 512 shares of the most units stay inside 32 bits
  CHECK((uint64_t)attn_share((uint32_t)kAttnMostUnits, 512) * 512 < 1ull << 32);
  return 0;
}

// Short segments have a workgroup each: few enough for one launch, whatever the table's width.
static int whole() {
  int round = 0;
  for (int pages = 0; pages < 300; pages += pages < 3 ? 1 : 33)
    for (int db = 32; db <= 256; db *= 2)
      for (int64_t segments = 1; segments < (int64_t)1 << 40; segments += 1 + segments / 7, ++round) {
        const AttnShape a = {1, 1, 1, 1, 1, 32, pages, 1, 4};
        if (attn_takes_whole(a, segments, db)) CHECK(segments * 64 * attn_whole_waves(db) < (int64_t)1 << 32);
        if (pages == 0 && segments <= 512) CHECK(attn_takes_whole(a, segments, db));
      }
  return 0;
}

// Sequences up to the longest: no sum leaves its type (built with checks for that).
static int longest() {
  const int round = 0;
  for (int page = 16; page <= 1 << 20; page *= 2) {
    const int pages = 2147483647 / page;
    for (int back = 0; back < 100; ++back) {
      for (int causal = 0; causal < 2; ++causal) {
        const AttnShape a = {1, 50, 1, 3, 50, page, pages, causal, 16};
        const AttnSeq s = attn_seq(a, 0, 50, pages * page - back);
        CHECK(s.L == pages * page - back && s.n == 50);
        const int last = attn_seen(a, s, 49);
        const uint32_t tiles = attn_tiles(a, s, 9);
        CHECK(last == s.L && tiles == ((uint64_t)last + 31) / 32);
        for (uint32_t t = tiles - 3; t < tiles; ++t) CHECK(attn_tile_full(t, last) == ((uint64_t)t * 32 + 32 <= (uint64_t)last));
        CHECK(attn_units(a, s) <= attn_most_units(a));
      }
    }
  }
  CHECK(!attn_tile_full(0, 0) && !attn_tile_full(0, 31) && attn_tile_full(0, 32));
  return 0;
}

int main() {
  if (units() || whole() || longest()) return 1;
  std::printf("ok\n");
  return 0;
}

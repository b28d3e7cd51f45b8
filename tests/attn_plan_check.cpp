// CPU check of csrc/attn_plan.h: the walk of the attention kernel's workgroups
// over units, and that of the joining kernel over pieces, on random sequences.
// Every tile of every segment is taken once, a segment's pieces are the ones
// that the joining kernel reads, in places that nothing else writes, and a
// workgroup begins one shared segment at most.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "../w8a8_int8_quantized_amd/csrc/attn_plan.h"

using namespace w8;

#define CHECK(c)                                             \
  do {                                                       \
    if (!(c)) {                                              \
      std::printf("failed: %s (round %d)\n", #c, round);     \
      return 1;                                              \
    }                                                        \
  } while (0)

typedef std::tuple<int, int, uint32_t> Segment;   // sequence, head, first row

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (uint32_t)(hi - lo + 1)); };
  for (int round = 0; round < 3000; ++round) {
    AttnShape a;
    a.B = pick(1, round % 3 ? 9 : 70);
    a.Hkv = pick(1, 5);
    a.G = pick(1, 9);
    a.rows = 4 << pick(0, 4);
    a.page = 16 * pick(1, 6);
    a.max_pages = pick(0, 30);
    a.causal = pick(0, 1);
    const uint32_t workgroups = (uint32_t)pick(1, round % 2 ? 1024 : 40);
    // starts and lengths, some of them nonsense
    std::vector<int> start(a.B + 1), len(a.B);
    int at = pick(0, 3);
    for (int b = 0; b <= a.B; ++b) {
      start[b] = at;
      at += pick(0, 4) == 0 ? 0 : pick(0, round % 5 ? 3 : 40);
    }
    a.T = pick(0, 9) ? at + pick(0, 2) : pick(0, at);
    a.max_q = pick(0, 3) ? a.T : pick(0, a.T);
    for (int b = 0; b < a.B; ++b) len[b] = pick(0, 5) == 0 ? 0 : pick(0, 30 * 96 + 50);
    if (pick(0, 3) == 0) {
      start[pick(0, a.B)] = pick(-2000000000, 2000000000);
      len[pick(0, a.B - 1)] = pick(-2000000000, 2000000000);
    }
    std::vector<AttnSeq> seq(a.B);
    std::vector<uint32_t> base(a.B + 1, 0);
    for (int b = 0; b < a.B; ++b) {
      seq[b] = attn_seq(a, start[b], start[b + 1], len[b]);
      CHECK(seq[b].row0 >= 0 && seq[b].n >= 0 && seq[b].row0 + seq[b].n <= a.T && seq[b].n <= a.max_q);
      CHECK(seq[b].L >= 0 && seq[b].L <= a.max_pages * a.page);
      for (int i = 0; i < seq[b].n; ++i) {
        const int s = attn_seen(a, seq[b], i);
        CHECK(s >= 0 && s <= seq[b].L && (!i || s >= attn_seen(a, seq[b], i - 1)));
      }
      base[b + 1] = base[b] + attn_units(a, seq[b]);
    }
    const uint32_t total = base[a.B], share = attn_share(total, workgroups);
    CHECK((uint64_t)share * workgroups >= total);
    std::map<Segment, std::vector<int>> taken;               // times each tile is taken
    std::map<Segment, std::vector<uint32_t>> pieces;         // places, in order of workgroups
    std::map<Segment, std::pair<uint32_t, uint32_t>> split;  // the workgroup that began it, followers
    std::set<uint32_t> used;
    for (uint32_t w = 0; w < workgroups; ++w) {
      const uint32_t lo = w * share, hi = lo + share < total ? lo + share : total;
      int splits = 0, b = 0;
      while (lo < hi && lo >= base[b + 1]) ++b;
      for (uint32_t u = lo; u < hi;) {
        if (u >= base[b + 1]) {
          ++b;
          continue;
        }
        const AttnSeg g = attn_segment(a, seq[b], attn_head(a, seq[b]), u - base[b], hi - base[b]);
        CHECK(g.units > 0 && u + g.units <= hi);
        u += g.units;
        CHECK(g.h >= 0 && g.h < a.Hkv && g.row_0 < g.rows && g.first <= g.last && g.last <= g.tiles);
        if (g.first == g.last) continue;
        // as many tiles as the last row sees
        const uint32_t last_row = g.row_0 + (uint32_t)a.rows < g.rows ? g.row_0 + (uint32_t)a.rows - 1 : g.rows - 1;
        const int most = attn_seen(a, seq[b], (int)(last_row / (uint32_t)a.G));
        CHECK((int)g.tiles == (most > 0 ? (most + 31) / 32 : 1));
        const Segment s(b, g.h, g.row_0);
        auto& t = taken[s];
        t.resize(g.tiles);
        for (uint32_t i = g.first; i < g.last; ++i) ++t[i];
        if (g.first == 0 && g.last == g.tiles) continue;
        const uint32_t x = attn_place(w, g.first == 0);
        CHECK(x < 2 * workgroups && used.insert(x).second);
        pieces[s].push_back(x);
        if (g.first == 0) {
          split[s] = {w, attn_followers(g.tiles, g.last, share)};
          CHECK(++splits == 1);          // one record to a workgroup
        }
      }
    }
    uint32_t segments = 0;
    for (int b = 0; b < a.B; ++b) segments += (uint32_t)a.Hkv * attn_head(a, seq[b]).row_tiles;
    CHECK(taken.size() == segments);
    for (auto& t : taken)
      for (int n : t.second) CHECK(n == 1);
    CHECK(split.size() == pieces.size());
    for (auto& s : split) {
      CHECK(s.second.second > 0 && s.second.first + s.second.second < workgroups);
      std::vector<uint32_t> reads;
      for (uint32_t v = 0; v <= s.second.second; ++v) reads.push_back(attn_place(s.second.first + v, v == 0));
      CHECK(reads == pieces[s.first]);
    }
  }
  std::printf("ok\n");
  return 0;
}

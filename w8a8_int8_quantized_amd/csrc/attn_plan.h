// How attention over a quantised cache (attn.hip) is shared out, in plain C++:
// the kernels and the host use the same rules, and tests/attn_plan_check.cpp
// checks them on the CPU.
//
// A segment is one row tile (rows are query token x query head of a key head's
// group) of one key head of one sequence; it holds the tiles of 32 cached
// tokens that its rows see.  Segments lie one behind the other (sequence, key
// head, row tile), each as attn_start units for its beginning and end (loads
// that wait for loads, the join of the waves) and a unit per tile.  Workgroup w
// takes units [w share, (w + 1) share): whole segments, and pieces of those
// that straddle its borders: the end of one that began before, and the
// beginning of one that goes on.
//
// With causal masks later row tiles see more.  A head's row tiles lie in pairs
// (the last with the first, the last but one with the second, ..), whose tiles
// add up to nearly the same for all: a pair has a fixed number of units, the
// few that its two segments leave are empty, and so the place of every segment
// follows by division.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define W8_HD __host__ __device__ __forceinline__
#else
#define W8_HD inline
#endif

namespace w8 {

constexpr int kAttnTile = 32;     // cached tokens to a unit
constexpr int kAttnWaves = 4;     // waves to a workgroup, each with a part of its tiles

struct AttnShape {
  int B, T, Hkv, G, max_q, page, max_pages, causal;
  int rows;   // rows to a row tile
};

// One sequence: its first query token, how many it has, its cached tokens.
struct AttnSeq {
  int row0, n, L;
};

// Units that a segment counts for beside its tiles.  Measured: decode batches
// of 64 sequences up to 16384 tokens 102, 98, 98 and 100 us with 8, 16, 24 and
// 40 (111 with 2), prompts' pieces beside single tokens 203, 176, 167 and 166.
W8_HD uint32_t attn_start(const AttnShape& a) { return a.rows > 16 ? 28u : 16u; }

// From the values in the arrays, which the host has not seen: clamped to what
// the call's shapes allow, so that nothing outside is read or written.
W8_HD AttnSeq attn_seq(const AttnShape& a, int q0, int q1, int len) {
  AttnSeq s;
  s.row0 = q0 < 0 ? 0 : (q0 > a.T ? a.T : q0);
  const int end = q1 < s.row0 ? s.row0 : (q1 > a.T ? a.T : q1);
  s.n = end - s.row0 < a.max_q ? end - s.row0 : a.max_q;
  const int64_t cap = (int64_t)a.max_pages * a.page;
  s.L = len < 0 ? 0 : (len > cap ? (int)cap : len);
  return s;
}

// Keys that query token i of the sequence sees.
W8_HD int attn_seen(const AttnShape& a, const AttnSeq& s, int i) {
  if (!a.causal) return s.L;
  const int64_t k = (int64_t)s.L - s.n + i + 1;
  return k < 0 ? 0 : (int)k;
}

// Tiles that row tile rt sees; one that sees nothing has a tile too, which
// gives its rows their zeros.
W8_HD uint32_t attn_tiles(const AttnShape& a, const AttnSeq& s, uint32_t rt) {
  const int64_t last = ((int64_t)(rt + 1) * a.rows - 1) / a.G;
  const int seen = attn_seen(a, s, last < s.n ? (int)last : s.n - 1);
  return seen > 0 ? ((uint32_t)seen + kAttnTile - 1) / kAttnTile : 1u;
}

// Whether `seen` tokens hold all of tile t.  (Lengths go to 2^31 - 16, so a
// tile's end may be 2^31.)
W8_HD bool attn_tile_full(uint32_t t, int seen) { return (t + 1) * (uint32_t)kAttnTile <= (uint32_t)seen; }

// A key head of a sequence: its row tiles, the units of a pair of them, and
// all its units.
struct AttnHead {
  uint32_t row_tiles, pair, units;
};
W8_HD AttnHead attn_head(const AttnShape& a, const AttnSeq& s) {
  AttnHead h;
  h.row_tiles = (uint32_t)(((int64_t)s.n * a.G + a.rows - 1) / a.rows);
  h.pair = 0;
  if (h.row_tiles > 1) {
    if (a.causal && s.L >= s.n) {
      // the last tokens of row tiles k and row_tiles - 1 - k add up to `most` at most
      const int64_t most = 2 * (int64_t)(s.L - s.n) + ((int64_t)(h.row_tiles + 1) * a.rows - 2) / a.G + 2;
      h.pair = (uint32_t)((most + 2 * kAttnTile - 2) / kAttnTile);
    } else {
      h.pair = 2 * attn_tiles(a, s, h.row_tiles - 1);
    }
    h.pair += 2 * attn_start(a);
  }
  h.units = h.row_tiles / 2 * h.pair;
  if (h.row_tiles & 1) h.units += attn_start(a) + attn_tiles(a, s, h.row_tiles / 2);
  return h;
}
W8_HD uint32_t attn_units(const AttnShape& a, const AttnSeq& s) { return (uint32_t)a.Hkv * attn_head(a, s).units; }

// Units of several sequences; more than 32 bits hold stay at the largest number,
// which is only reached where starts contradict the call's sizes.
W8_HD uint32_t attn_add(uint32_t a, uint32_t b) { return a + b < a ? ~0u : a + b; }

// The units of a call's sequences at most, whatever its arrays hold within its
// sizes: T query tokens in all fill T G / rows row tiles of a key head and
// begin one more for each sequence, and each counts its start and the tiles of
// the whole table (a pair's two up to 30 more than these, see attn_head).
inline uint64_t attn_most_units(const AttnShape& a) {
  const int64_t each = (int64_t)a.B * (((int64_t)a.max_q * a.G + a.rows - 1) / a.rows);
  const int64_t all = (int64_t)a.T * a.G / a.rows + a.B;
  const int64_t row_tiles = (each < all ? each : all) * a.Hkv;
  if (row_tiles >> 36) return ~0ull;
  return (uint64_t)row_tiles * (uint64_t)(((int64_t)a.max_pages * a.page + kAttnTile - 1) / kAttnTile + 33);
}
// What the kernels count up to (and a share more than that).
constexpr uint64_t kAttnMostUnits = 0xfffff000u;

// Units to a workgroup: an even share, but two tiles to a wave at least.
W8_HD uint32_t attn_share(uint32_t total, uint32_t workgroups) {
  const uint32_t even = (total + workgroups - 1) / workgroups;
  const uint32_t least = 2 * kAttnWaves;
  return even > least ? even : least;
}

// The segment that holds unit u of a sequence (u and hi from the sequence's
// first unit; units of the workgroup end before hi): the key head, the first
// row and the rows there are, the units from u to its end or the workgroup's,
// and the tiles among them, from `first` to before `last` of `tiles`.  Without
// tiles (only units of a beginning, or empty ones) there is nothing to do.
struct AttnSeg {
  int h;
  uint32_t row_0, rows, units, tiles, first, last;
};
W8_HD AttnSeg attn_segment(const AttnShape& a, const AttnSeq& s, const AttnHead& hd, uint32_t u, uint32_t hi) {
  AttnSeg g;
  const uint32_t h = u / hd.units, v = u - h * hd.units, left = hi - u;
  const uint32_t k = hd.pair ? v / hd.pair : 0;
  const uint32_t start = attn_start(a);
  uint32_t from = v, rt = hd.row_tiles / 2;
  g.h = (int)h;
  g.rows = (uint32_t)s.n * (uint32_t)a.G;
  bool second = false;
  if (k < hd.row_tiles / 2) {
    rt = hd.row_tiles - 1 - k;
    from = v - k * hd.pair;
    const uint32_t longer = start + attn_tiles(a, s, rt);
    if (from >= longer) {
      rt = k;
      from -= longer;
      second = true;
    }
  } else {
    from = v - hd.row_tiles / 2 * hd.pair;
  }
  g.tiles = attn_tiles(a, s, rt);
  g.row_0 = rt * (uint32_t)a.rows;
  const uint32_t each = start + g.tiles;
  if (second && from >= each) {   // the empty units of a pair
    const uint32_t rest = (k + 1) * hd.pair - v;
    g.units = rest < left ? rest : left;
    g.first = g.last = 0;
    return g;
  }
  const uint32_t to = left < each - from ? from + left : each;
  g.units = to - from;
  g.first = from > start ? from - start : 0;
  g.last = to > start ? to - start : 0;
  return g;
}

// Short segments are not shared: a workgroup of more waves to each, without a
// search and without a second kernel (which also saves its launch on the
// host).  The waves whose rings of two or four tiles fit in LDS, for rows of db
// bytes.
constexpr W8_HD int attn_whole_waves(int db) { return db <= 64 ? 16 : db == 128 ? 8 : 4; }

// Segments that many, of which none is longer than the block table is wide.  A
// few can be spread over the GPU, so their waves' runs have to be short; with
// more than a workgroup to a CU the wide workgroups wait for each other.
// Measured, us whole and shared, 128 channels of 4 bits: 8 segments of 1000
// tokens 10.8 and 12.1, of 1500 12.5 and 12.0, of 2000 14.4 and 12.4; 64 of 2200
// 17.1 and 17.2, of 3400 20.5 and 18.6; 128 of 1500 13.8 and 18.4, of 3500 20.9
// and 23.2; 256 of 1200 14.4 and 20.4, of 3400 25.1 and 30.8; 512 of 500 17.4 and
// 17.8, of 1500 29 and 24; nothing between 256 and 512.  The table's width stands
// for the lengths, which are on the device: one that is wider than its sequences
// need has them shared (32 of up to 1200 under a table for 131072 tokens 17 us,
// 12.5 with one for 1200).
W8_HD bool attn_takes_whole(const AttnShape& a, int64_t segments, int db) {
  const int64_t most = ((int64_t)a.max_pages * a.page + kAttnTile - 1) / kAttnTile;
  const int64_t run = segments <= 128 ? 3 + segments / 32 : segments <= 256 ? 7 : segments <= 512 ? 1 : 0;
  return segments <= 512 && most <= run * attn_whole_waves(db);   // (a table without pages has none)
}

// A segment of `tiles` tiles of which the workgroup that takes the first ends
// with `last`: the workgroups that take the others, one behind the other.
W8_HD uint32_t attn_followers(uint32_t tiles, uint32_t last, uint32_t share) {
  return (tiles - last + share - 1) / share;
}

// The place of a workgroup's piece of a segment that it shares with others:
// one for the segment that it begins, one for the segment that began before.
W8_HD uint32_t attn_place(uint32_t workgroup, bool begins) { return 2 * workgroup + (begins ? 1u : 0u); }

}  // namespace w8

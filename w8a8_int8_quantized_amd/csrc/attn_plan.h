// How attention over a quantised cache (attn.hip) is shared out, in plain C++:
// the kernels and the host use the same rules, and tests/attn_plan_check.cpp
// checks them on the CPU.
//
// A segment is one row tile (rows are query token x query head of a key head's
// group) of one key head of one sequence; it holds the sequence's tiles of 32
// cached tokens.  Segments lie one behind the other (sequence, key head, row
// tile), each as kAttnStart units for its beginning and end (loads that wait
// for loads, the join of the waves) and a unit per tile.  Workgroup w takes
// units [w share, (w + 1) share): whole segments, and pieces of those that
// straddle its borders: the end of one that began before, and the beginning of
// one that goes on.
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
constexpr uint32_t kAttnStart = 16;   // units that a segment counts for beside its tiles

struct AttnShape {
  int B, T, Hkv, G, max_q, page, max_pages, causal;
  int rows;   // rows to a row tile
};

// One sequence: its first query token, how many it has, its cached tokens.
struct AttnSeq {
  int row0, n, L;
};

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

// Tiles of a sequence; one without cached tokens has a tile too, which holds
// nothing and gives its rows their zeros.
W8_HD uint32_t attn_tiles(int L) {
  return L > 0 ? (uint32_t)(L + kAttnTile - 1) / kAttnTile : 1u;
}

W8_HD uint32_t attn_row_tiles(int n, int G, int rows) {
  return (uint32_t)(((int64_t)n * G + rows - 1) / rows);
}

W8_HD uint32_t attn_units(const AttnShape& a, const AttnSeq& s) {
  return (uint32_t)a.Hkv * attn_row_tiles(s.n, a.G, a.rows) * (attn_tiles(s.L) + kAttnStart);
}

// Keys that query token i of the sequence sees.
W8_HD int attn_seen(const AttnShape& a, const AttnSeq& s, int i) {
  if (!a.causal) return s.L;
  const int64_t k = (int64_t)s.L - s.n + i + 1;
  return k < 0 ? 0 : (int)k;
}

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
// tiles (only units of the beginning) there is nothing to do.
struct AttnSeg {
  int h;
  uint32_t row_0, rows, units, tiles, first, last;
};
W8_HD AttnSeg attn_segment(const AttnShape& a, const AttnSeq& s, uint32_t u, uint32_t hi) {
  AttnSeg g;
  g.tiles = attn_tiles(s.L);
  const uint32_t each = g.tiles + kAttnStart, nrt = attn_row_tiles(s.n, a.G, a.rows), seg = u / each;
  const uint32_t from = u - seg * each, to = hi - u < each - from ? from + (hi - u) : each;
  g.units = to - from;
  g.first = from > kAttnStart ? from - kAttnStart : 0;
  g.last = to > kAttnStart ? to - kAttnStart : 0;
  g.h = (int)(seg / nrt);
  g.row_0 = (seg - (uint32_t)g.h * nrt) * (uint32_t)a.rows;
  g.rows = (uint32_t)s.n * (uint32_t)a.G;
  return g;
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

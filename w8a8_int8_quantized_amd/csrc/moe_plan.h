// The launch rules of the few-token experts (moe.hip): which variant of each
// kernel a call takes, its grid and its LDS, from the sizes alone.  Plain C++,
// so that they are checked on the CPU over the sizes the call takes, and so
// that tests can tell which variant a case reaches.
#pragma once

#include <cstddef>
#include <cstdint>

namespace w8 {

constexpr int kMaxPairs = 1024;
constexpr int kGuWaves = 4, kDownWaves = 8;

// Pairs and codes whose h every down workgroup quantises for itself, at most:
// 0.8 us of each workgroup per 8192 codes, most of it while the first weights
// are under way, against a kernel of 4.7 us (K = 7168, I = 2048: 32768 codes
// 44.0 us against 41.8 + 4.7, 65536 codes 76.5 against 68.5 + 4.7).
constexpr int64_t kLdsPairs = 64, kLdsCodes = 32768;

// Up to this K the experts may be split over workgroups.
constexpr int64_t kSplitMaxK = 4096;

// Down sums' places in LDS, with all else there: at most this many bytes for
// more than one place per unit.
constexpr size_t kDownLds = 131072;

constexpr bool moe_quant_in_down(int64_t P, int64_t I) { return P <= kLdsPairs && P * I <= kLdsCodes; }

struct MoePlan {
  int most;                    // chosen experts, at most
  int gu_mf, gu_fc, gu_wk;     // k_moe_gate_up's template arguments
  bool in_down;                // h's codes from k_moe_down, else from k_moe_quant
  int down_mf, down_fn;        // k_moe_down's fragments of rows and columns
  int cw, z;                   // columns per workgroup, workgroups per columns
  int smax;                    // places per unit
  size_t gu_lds, down_lds;     // dynamic LDS, bytes
};

// The down kernel's columns per workgroup and workgroups per columns: those of
// the least time of the fullest CU, its workgroups' blocks times the 128-byte
// lines of a block (a weight row each, a row of h each, the scales) at about
// 4.5 ns a line, and 6 us for the combine kernel where the experts are split over
// workgroups (z > 1: few columns, many pairs; a workgroup of few columns loads
// more of h than of the weights).  K = 256, I = 2816, 24 experts, 84 pairs:
// 64 workgroups of 4 columns 24 us, 256 of 16 columns and a sixteenth of the
// experts 5 us and the combine.
inline void moe_down_grid(MoePlan* p, int64_t P, int64_t K, int64_t IB) {
  p->cw = 16;
  p->z = 1;
  double best = 1e30;
  for (int z = 1; z <= (p->in_down || K > kSplitMaxK ? 1 : 16); z *= 2)
    for (int cw = 32; cw >= 4; cw -= 4) {
      const int64_t wgs = (K + cw - 1) / cw * z, blocks = (p->most + z - 1) / z * IB;
      const double lines = cw + 2 + (p->in_down ? 0.0 : (double)P / p->most);
      const double t = (double)((wgs + 255) / 256) * blocks * lines * 4.5e-3 + (z > 1 ? 6.0 : 0.0);
      if (t < best) {
        best = t;
        p->cw = cw;
        p->z = z;
      }
    }
}

inline MoePlan moe_plan(int64_t T, int64_t topk, int64_t E, int64_t I, int64_t K) {
  MoePlan p;
  const int64_t P = T * topk, IB = I / 128, KB = K / 128;
  p.most = (int)(P < E ? P : E);

  // gate_up: experts of many rows four fragments of rows at a time, two
  // workgroups per CU (8 experts of 64 rows: 73 us, 94 with 16 columns and
  // three); others two fragments and four workgroups (16 to 23 rows: 52 us, 66
  // with four fragments and 16 columns).  Columns per workgroup: 32 load the activations half as often as
  // 16, which spread few columns more evenly (one token of 8 experts,
  // K = 7168, I = 2048: 43 us with 32, 45 with 16; 7 experts, I = 256: 21 and
  // 16); 64, with half the waves per column, for short K, where a workgroup's
  // start is most of its time (K = 256, 24 experts, I = 2816: 13 us, 17, 27)
  const int64_t w16 = I / 16 * p.most, w32 = w16 / 2;
  const bool narrow = 5 * ((w16 + 255) / 256) * 16 < 4 * ((w32 + 255) / 256) * 32;
  p.gu_mf = P > 24 * E ? 4 : 2;
  p.gu_wk = p.gu_mf == 2 && K <= 1024 && w16 / 4 >= 512 ? 2 : 4;
  p.gu_fc = p.gu_mf == 2 && p.gu_wk == 4 && narrow ? 1 : 2;
  const size_t sums = (size_t)(kGuWaves / p.gu_wk) * (p.gu_wk - 1) * 2 * p.gu_fc * p.gu_mf * 1024;
  const size_t owner = (size_t)E * 4, scales = (size_t)(2 * KB + 16 * p.gu_mf * (KB | 1)) * 4;
  p.gu_lds = sums > owner ? sums : owner;
  if (scales > p.gu_lds) p.gu_lds = scales;

  // down: rows per unit by the mean rows of an expert: a unit of more rows than its
  // expert has costs registers, one of fewer reads the weights again (32
  // experts of 16 rows: 105 us with 32, 134 with 64)
  p.in_down = moe_quant_in_down(P, I);
  moe_down_grid(&p, P, K, IB);
  p.down_mf = p.in_down || P <= 12 * E ? 1 : P <= 28 * E ? 2 : 4;
  p.down_fn = p.cw <= 16 ? 1 : 2;
  const size_t place = (size_t)P * p.down_fn * 64;
  const size_t rest = (size_t)(P * 14 + 15) / 16 * 16 +
                      (p.in_down ? (size_t)(P * IB + 3) / 4 * 16 + (size_t)P * (I + 16) : 0);
  // pieces of a unit, at most: where units are fewer than the waves, or no
  // multiple of them (K = 7168, I = 2048, uncut, two, four and eight pieces:
  // one pair 9.1, 8.5, 7.8 and 9.0 us; one expert of 64 rows 16.8, 14.5, 14.6
  // and 15.7; nine experts of 14 rows 39.7, 38.1, 37.4 and 37.5; I = 512,
  // K = 2048 the same within 0.5 us)
  constexpr int kMaxPieces = 4;
  p.smax = 1;
  while (p.smax * 2 <= IB && p.smax < kMaxPieces && p.smax * 2 * place + rest <= kDownLds) p.smax *= 2;
  p.down_lds = p.smax * place + rest;
  return p;
}

}  // namespace w8

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

// Up to this K the experts may be split over workgroups.  Down and combine
// together, split as moe_down_grid chooses against unsplit, us: I = 2816, 24
// experts, 84 pairs: K = 256 18.0 against 36.1, 512 19.6 and 36.5, 1024 25.0 and
// 37.8, 2048 36.9 and 46.3, 4096 61 and 58; I = 1024, 32 experts, 512 pairs: 256
// 16.9 and 34.2, 1024 21.1 and 34.7, 2048 29.4 and 38.6, 4096 46.4 and 46.6.  At
// K = 7168 two workgroups to the columns lose (104 against 89, 78 against 61).
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
// 64 workgroups of 4 columns 36 us, 256 of 16 columns and a sixteenth of the
// experts 12 us and the combine's 4.5.
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

  // Rows per pass and per unit go by the mean rows of an expert, T topk / E:
  // slots without an expert count as rows, since the ids are on the device.
  // (64 tokens, 8 of 256 experts of which 32 are here, 69 rows: down 87 us with
  // the two fragments of the mean, 79 with one.)  Figures at K = 7168,
  // I = 2048.
  //
  // gate_up: experts of many rows four fragments of rows at a time, two
  // workgroups per CU, others two fragments and four workgroups.  Rows spread
  // as ids drawn at random (more than 32 rows take two fragments twice), 32
  // experts of 24 rows in the mean 219 us with four and 191 with two, of 28
  // 227 and 242, of 32 231 and 295; 16 experts of 28 114 and 100, of 32 119 and
  // 149.
  //
  // Columns per workgroup: 32 load the activations half as often as 16, which
  // spread few columns more evenly (one token of 8 experts: 43 us with 32, 45
  // with 16; 7 experts, I = 256: 21 and 16); 64, with half the waves per column,
  // for short K, where a workgroup's start is most of its time (I = 2816, 24
  // experts, 84 pairs, with 64, 32 and 16: K = 256 17.8, 21.4 and 34 us; 512
  // 22.4, 26.8 and 41; 1024 33.9, 34.6 and 49; 1536 47.5, 49.5 and 58; 2048
  // 58, 55 and 64; I = 2048, 16 experts, 64 pairs: K = 256 10.8, 12.1 and 17.9;
  // 1024 18.5, 19.4 and 26.3; 2048 28.4, 29.6 and 34.2)
  const int64_t w16 = I / 16 * p.most, w32 = w16 / 2;
  const bool narrow = 5 * ((w16 + 255) / 256) * 16 < 4 * ((w32 + 255) / 256) * 32;
  p.gu_mf = P > 24 * E ? 4 : 2;
  p.gu_wk = p.gu_mf == 2 && K <= 1024 && w16 / 4 >= 512 ? 2 : 4;
  p.gu_fc = p.gu_mf == 2 && p.gu_wk == 4 && narrow ? 1 : 2;
  const size_t sums = (size_t)(kGuWaves / p.gu_wk) * (p.gu_wk - 1) * 2 * p.gu_fc * p.gu_mf * 1024;
  const size_t owner = (size_t)E * 4, scales = (size_t)(2 * KB + 16 * p.gu_mf * (KB | 1)) * 4;
  p.gu_lds = sums > owner ? sums : owner;
  if (scales > p.gu_lds) p.gu_lds = scales;

  // down: a unit of more rows than its expert has costs registers and blocks in
  // flight, one of fewer reads the weights again (32 experts, rows spread as
  // above, with 16, 32 and 64 rows to a unit: mean 12 99, 104 and 134 us; 16
  // 124, 110 and 136; 24 169, 123 and 143; 28 180, 135 and 147; 32 203, 157 and
  // 151)
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

// CPU check of csrc/moe_plan.h.  Without arguments: what the kernels take for
// granted holds over the sizes the call takes, and each distinct form is
// printed ("gate MF FC WK", "down LDSH MF FN split", "places LDSH smax").
// With an argument: a plan per line of "T topk E I K" from standard input.
#include <cstdio>
#include <set>
#include <string>

#include "../w8a8_int8_quantized_amd/csrc/moe_plan.h"

using namespace w8;

#define CHECK(c)                                                                               \
  do {                                                                                         \
    if (!(c)) {                                                                                \
      std::printf("failed: %s (T %d topk %d E %d I %d K %d)\n", #c, T, topk, E, I, K);        \
      return 1;                                                                                \
    }                                                                                          \
  } while (0)

static std::string gate(const MoePlan& p) {
  return "gate " + std::to_string(p.gu_mf) + " " + std::to_string(p.gu_fc) + " " + std::to_string(p.gu_wk);
}
static std::string down(const MoePlan& p) {
  return "down " + std::to_string(p.in_down) + " " + std::to_string(p.down_mf) + " " + std::to_string(p.down_fn) +
         " " + std::to_string(p.z > 1);
}
static std::string places(const MoePlan& p) {
  return "places " + std::to_string(p.in_down) + " " + std::to_string(p.smax);
}

int main(int argc, char**) {
  int T, topk, E, I, K;
  if (argc > 1) {
    while (std::scanf("%d %d %d %d %d", &T, &topk, &E, &I, &K) == 5) {
      const MoePlan p = moe_plan(T, topk, E, I, K);
      std::printf("%s,%s,%s\n", gate(p).c_str(), down(p).c_str(), places(p).c_str());
    }
    return 0;
  }
  std::set<std::string> forms;
  const int sides[] = {128, 256, 384, 640, 896, 1024, 1152, 2048, 2688, 2816, 4096, 4224, 7168, 16384, 32768};
  const int experts[] = {1, 2, 3, 5, 8, 16, 24, 32, 43, 64, 96, 128, 160, 256, 1000, 4096};
  const size_t kCu = 160 * 1024;   // LDS of a CU
  for (T = 1; T <= 64; ++T)
    for (topk = 1; topk <= 16; ++topk)
      for (int e : experts)
        for (int i : sides)
          for (int k : sides) {
            E = e, I = i, K = k;
            const MoePlan p = moe_plan(T, topk, E, I, K);
            const int P = T * topk;
            forms.insert(gate(p));
            forms.insert(down(p));
            forms.insert(places(p));
            CHECK(P <= kMaxPairs && p.most >= 1 && p.most <= P && p.most <= E);
            // the grid covers I exactly; a workgroup's columns lie in one 128-row block of the weights
            const int cols = 16 * p.gu_fc * (kGuWaves / p.gu_wk);
            CHECK(I % cols == 0 && 128 % (16 * p.gu_fc) == 0);
            // LDS: beside the static arrays (tokens of the pairs, counts; 4 KB hold them)
            CHECK(p.gu_lds + 4096 <= kCu && p.gu_lds >= (size_t)E * 4);
            CHECK(p.cw % 4 == 0 && p.cw >= 4 && p.cw <= 16 * p.down_fn);
            CHECK(p.z == 1 || (!p.in_down && K <= kSplitMaxK));
            CHECK(p.smax == 1 || p.smax == 2 || p.smax == 4);
            CHECK(p.smax <= I / 128 && p.down_lds + 256 <= kCu);
            // a lane per chosen expert and four passes of 64 groups where h is quantised in the kernel
            CHECK(!p.in_down || (P <= 64 && P * (I / 128) <= 256 && p.down_mf == 1));
          }
  for (const std::string& f : forms) std::printf("%s\n", f.c_str());
  return 0;
}

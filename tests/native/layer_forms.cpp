// Prints the kernel forms that the layer operators' plans choose
// (tests/test_layers_forms_cpu.py). Host only.
//
//   layer_forms scan     every form that a wide grid of sizes reaches, each
//                        with the smallest product that reaches it
//   layer_forms          for each line "operator m n k" of the input its forms
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "layer_plan.h"

namespace {

using namespace fp8bl::plan;

const char* const kTileName[] = {"256-row tiles", "128-row tiles", "64-row tiles"};

// Outputs of a split part go through the join in quads where rows are whole
// quads and there are enough of them.
std::string join_of(int64_t m, int64_t n, int64_t width) {
  return n % 4 == 0 && m * width >= (1 << 18) ? ", join of quads" : ", join";
}

std::vector<std::string> forms(const std::string& op, int64_t m, int64_t n, int64_t k) {
  std::vector<std::string> out;
  const bool back = op == "linear_act_backward" || op == "glu_backward", two = op == "glu_backward";
  const bool pair = op == "glu";
  const std::string name = back ? (two ? "gradient of two: " : "gradient: ") : pair ? "pair: " : "linear: ";
  const int products = two ? 2 : 1;
  if (streams(back ? kInputGradient : pair ? kPair : kLinear, m, n, (pair ? 2 : products) * n * k)) {
    if (back) {
      const GradientPlan p = plan_gradient_skinny(n, k, products);
      out.push_back(name + "stream, " + (m <= 16 ? "16" : "32") + " rows" +
                    (p.splits > 1 ? join_of(m, k, k) : ", unsplit"));
      return out;
    }
    const int cols = pair ? 16 : 32;
    const StreamPlan p = plan_layer((n + cols - 1) / cols, k);
    std::string path;
    with_path(m, (n + cols - 1) / cols * p.splits, pair, [&](auto v) {
      using P = decltype(v);
      path = std::to_string(16 * P::MT) + " rows, X in " + (P::kLds ? "LDS" : "registers") + ", steps of " +
             std::to_string(P::KW);
    });
    out.push_back(name + "stream, " + path + (p.splits > 1 ? join_of(m, n, n) : ", unsplit"));
    return out;
  }
  const int64_t width = back ? k : n;
  const int cols = pair ? kTileCols / 2 : kTileCols;
  const ProductPlan p = back ? plan_product(m, k, cols, n, products, 1) : plan_product(m, n, cols, k, 1, pair ? 2 : 1);
  for (int i = 0; i < p.parts; ++i) {
    const Part& part = p.part[i];
    const bool split = part.plan.splits > 1;
    out.push_back(name + kTileName[part.plan.tile] + (split ? ", split" : ", unsplit") +
                  (width % 4 ? ", odd rows" : "") + (m <= 32 ? ", few rows" : "") + (p.parts > 1 ? i ? ", columns left over" : ", whole rounds" : "") +
                  (split ? join_of(m, width, width - (int64_t)part.tile0 * cols) : ""));
  }
  return out;
}

}  // namespace

int main(int argc, char** argv) {
  const char* const ops[] = {"linear_act", "linear_act_backward", "glu", "glu_backward"};
  if (argc > 1 && !std::strcmp(argv[1], "scan")) {
    const int64_t ms[] = {1,   2,   4,   5,   8,   16,  17,  24,  32,   33,   48,   64,   65,   77,   96,   128,
                          129, 192, 200, 256, 257, 300, 333, 384, 512,  513,  700,  768,  1000, 1024, 1500, 2048,
                          2304, 3000, 4096, 6144, 8192};
    const int64_t ns[] = {1,    8,    16,   36,   100,  264,  513,  784,  1000, 1024,  1443,  2048,  2560,  2819,  4096,
                          4224, 5120, 5121, 6000, 7168, 8192, 8200, 8448, 9001, 10240, 12288, 12800, 13824, 16001, 25600};
    const int64_t ks[] = {16, 64, 128, 336, 512, 784, 1024, 1552, 2048, 2560, 4096, 5120, 7168, 8192, 8448, 12288, 16384, 25600};
    std::map<std::string, std::pair<int64_t, std::string>> seen;
    for (const char* op : ops)
      for (int64_t m : ms)
        for (int64_t n : ns)
          for (int64_t k : ks)
            for (const std::string& f : forms(op, m, n, k)) {
              const int64_t size = m * n * k + n * k;
              const auto at = seen.find(f);
              if (at == seen.end() || size < at->second.first)
                seen[f] = {size, std::string(op) + " " + std::to_string(m) + " " + std::to_string(n) + " " + std::to_string(k)};
            }
    for (const auto& s : seen) std::printf("%s\t%s\n", s.first.c_str(), s.second.second.c_str());
    return 0;
  }
  char op[64];
  long long m, n, k;
  while (std::scanf("%63s %lld %lld %lld", op, &m, &n, &k) == 4)
    for (const std::string& f : forms(op, m, n, k)) std::printf("%s\n", f.c_str());
  return 0;
}

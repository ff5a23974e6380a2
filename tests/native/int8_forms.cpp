// Prints the kernel forms that the 8-bit integer linear's plans (csrc/int8_plan.h)
// choose (tests/test_int8_forms_cpu.py). Host only.
//
//   int8_forms scan   every form that a wide grid of sizes reaches, each with the
//                     smallest product that reaches it
//   int8_forms        for each line "m n k bf16" of the input its form
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>

#include "int8_plan.h"

namespace {

std::string form(int64_t m, int64_t n, int64_t k, bool bf16) {
  using namespace fp8bl;
  const std::string from = bf16 ? "" : " from codes";
  if (m <= kInt8SkinnyRows) {
    const Int8SkinnyPlan p = plan_skinny8(m, n, k);
    const bool fused = bf16 && int8_skinny_quantizes(m, k);
    if (bf16 && !fused) return form(m, n, k, false);       // the quantizer, then the product on codes
    const int step = fused ? (p.few ? 128 : 256) : m > 16 ? (p.few ? 128 : 256) : p.few || m > 1 ? 128 : 256;
    return std::string("stream, ") + (m > 16 ? "two row tiles" : m > 1 ? "one row tile" : "one row") +
           (p.few ? ", few columns" : ", many columns") + (fused ? ", quantized on the way" : "") +
           (p.splits > 1 ? ", split" : "") + (k % step ? ", K tail" : "") + from;
  }
  if (bf16) return form(m, n, k, false);
  const Int8Plan p = plan_int8(m, n, k);
  const Int8Cut c = cut_int8(m, n, k, kInt8Edge[p.tile], p.splits);
  const bool split = c.splits > 1;
  return "tiles of " + std::to_string(kInt8Edge[p.tile]) + (split ? ", split" : "") +
         (c.units > (p.tile == 2 ? 512 : 256) ? ", several rounds" : "") +
         (split ? (n % 4 ? ", rows of parts" : "") : p.tile < 2 && n % 64 == 0 ? ", whole lines" : n % 8 ? ", odd rows" : "") +
         (k % kInt8StepK ? ", K tail" : "");
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1 && !std::strcmp(argv[1], "scan")) {
    const int64_t ms[] = {1, 2, 5, 16, 17, 32, 33, 48, 64, 65, 77, 128, 129, 200, 256, 257, 333, 512, 700, 1000, 1025, 2048, 4096, 8192};
    const int64_t ns[] = {1, 8, 36, 100, 264, 513, 1000, 1024, 2048, 2819, 4096, 4097, 4104, 5120, 5121, 8000, 8192, 12288, 16001, 25600};
    const int64_t ks[] = {16, 128, 144, 256, 512, 528, 1024, 1040, 2048, 4096, 5120, 8192, 8208, 16384, 16400, 25600, 32768, 65552};
    std::map<std::string, std::pair<int64_t, std::string>> seen;
    for (int64_t m : ms)
      for (int64_t n : ns)
        for (int64_t k : ks)
          for (int bf16 = 0; bf16 < 2; ++bf16) {
            const std::string f = form(m, n, k, bf16);
            const int64_t size = m * n * k + n * k;
            const auto at = seen.find(f);
            if (at == seen.end() || size < at->second.first)
              seen[f] = {size, std::to_string(m) + " " + std::to_string(n) + " " + std::to_string(k) + " " + std::to_string(bf16)};
          }
    for (const auto& s : seen) std::printf("%s\t%s\n", s.first.c_str(), s.second.second.c_str());
    return 0;
  }
  long long m, n, k;
  int bf16;
  while (std::scanf("%lld %lld %lld %d", &m, &n, &k, &bf16) == 4) std::printf("%s\n", form(m, n, k, bf16 != 0).c_str());
  return 0;
}

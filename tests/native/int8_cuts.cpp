// Checks how the 8-bit integer linear cuts its products (csrc/int8_plan.h) over
// every accepted size that is extreme in some way (tests/test_int8_cuts_cpu.py).
// Host only. Prints the number of sizes checked, or the first that is wrong.
#include <cstdint>
#include <cstdio>

#include "int8_plan.h"

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 35, kInt = ((int64_t)1 << 31) - 1, kThreads = (int64_t)1 << 32;

// What is wrong with the cut of an accepted size, or null.
const char* wrong(int64_t m, int64_t n, int64_t k) {
  using namespace fp8bl;
  if (m <= kInt8SkinnyRows) {
    const Int8SkinnyPlan p = plan_skinny8(m, n, k);
    if (p.splits < 1 || p.k_split < 1 || p.k_split % 256 != 0) return "few rows: empty splits";
    if ((int64_t)p.k_split * p.splits < k || (int64_t)p.k_split * (p.splits - 1) >= k) return "few rows: K is not covered";
    return nullptr;
  }
  const Int8Plan p = plan_int8(m, n, k);
  if (p.tile < 0 || p.tile > 2 || p.splits < 1 || p.splits > 8) return "plan";
  const int64_t edge = kInt8Edge[p.tile];
  const Int8Cut c = cut_int8(m, n, k, (int)edge, p.splits);
  if (c.tiles_m * edge < m || (c.tiles_m - 1) * edge >= m) return "rows are not covered";
  if (c.tiles_n * edge < n || (c.tiles_n - 1) * edge >= n) return "columns are not covered";
  if (c.steps * kInt8StepK < k || (c.steps - 1) * kInt8StepK >= k) return "K is not covered";
  if (c.splits < 1 || c.splits > p.splits) return "splits";
  if (c.steps_per_unit * c.splits < c.steps || c.steps_per_unit * (c.splits - 1) >= c.steps) return "a split is empty";
  // the kernel counts units, and a tile's rows and columns, in 32 bits
  if (c.units < 1 || c.units != c.tiles_m * c.tiles_n * c.splits || c.units + 8192 > kInt) return "units";
  if ((c.tiles_m - 1) * edge > kInt || c.tiles_m > kInt - 4 || 4 * c.tiles_n > kInt) return "tiles";
  if (c.splits > 1 && m * ((n + 3) / 4) + 255 >= kThreads) return "the join's launch";
  return nullptr;
}

}  // namespace

int main() {
  const int64_t rows[] = {1, 2, 16, 17, 32, 33, 64, 65, 255, 256, 257, 1000, 4096, 65535, 65537, 1 << 20, (1 << 25) - 1, 1 << 28,
                          (int64_t)1 << 30, kInt - 256, kInt - 255, kInt - 128, kInt - 127, kInt - 64, kInt - 63, kInt - 1, kInt};
  const int64_t cols[] = {1, 2, 3, 4, 7, 8, 15, 16, 63, 64, 65, 128, 257, 1003, 4096, 4097, 8192, 25600, 131072, (1 << 20) - 1, 1 << 20};
  const int64_t depths[] = {16, 32, 112, 128, 144, 512, 528, 1024, 4096, 8192, 8208, 16384, 16400, 25600, 65536, 131040, 131056};
  long long checked = 0;
  for (int64_t m : rows)
    for (int64_t n : cols)
      for (int64_t k : depths) {
        if (m * k >= kMaxElems || n * k >= kMaxElems || m * n >= kMaxElems) continue;
        ++checked;
        if (const char* what = wrong(m, n, k)) {
          std::printf("%lld x %lld x %lld: %s\n", (long long)m, (long long)n, (long long)k, what);
          return 1;
        }
      }
  std::printf("%lld\n", checked);
  return 0;
}

// How the root-mean-square norm deals rows out, walked over all widths: every
// column has a thread, no workgroup is empty or larger than its kernel's
// launch bound, every k is one that has a kernel, and a workgroup's groups fit
// its LDS and the words of the row's sum.  Prints the first mistake and fails.
#include <cstdio>
#include <cstdlib>

#include "norm_shape.h"

using namespace fp8sg;

static void need(bool ok, const char* what, long rows, long cols) {
  if (ok) return;
  std::printf("%s: rows %ld cols %ld\n", what, rows, cols);
  std::exit(1);
}

int main() {
  const long rows_of[] = {0, 1, 2, 7, 255, 256, 257, 511, 512, 513, 1000, 4096, 65536, 2147483647};
  for (long cols = 1; cols <= 32768; ++cols) {
    const long slots = (cols + 7) / 8;
    for (long rows : rows_of) {
      const RowShape f = rms_row_shape(rows, cols);
      need((long)f.k * f.nt >= slots, "forward: columns without a thread", rows, cols);
      need(f.wave ? f.nt == 64 && (f.k == 1 || f.k == 2) : f.k >= 1 && f.k <= 4,
           "forward: no such kernel", rows, cols);
      need(cols >= 8 || (f.wave && f.k == 1), "forward: short rows are a wave's", rows, cols);
      need(f.nt % 64 == 0 && f.nt <= (f.k == 2 || f.k == 4 ? 1024 : 512), "forward: launch bound",
           rows, cols);
      for (int f32 = 0; f32 < 2; ++f32)
        need(rms_fwd_waves(f.k, f32) * 64 / (f.wave ? 256 : f.nt) >= 1,
             "forward: no workgroup held", rows, cols);
      const BwdShape b = rms_bwd_shape(rows, cols);
      need((long)b.k * b.nt >= slots, "backward: columns without a thread", rows, cols);
      need(b.k == 1 || b.k == 2 || b.k == 4, "backward: no such kernel", rows, cols);
      need(cols >= 8 || b.k == 1, "backward: short rows have one slot", rows, cols);
      need(b.nt >= 64 && b.nt % 64 == 0 && b.groups >= 1 && b.nt * b.groups <= kRmsBwdThreads,
           "backward: launch bound", rows, cols);
      need(b.grid <= 256 && b.grid <= rows && (rows == 0) == (b.grid == 0),
           "backward: workgroups", rows, cols);
      need((b.groups - 1L) * 8 * b.nt * 4 <= 48 * 1024, "backward: LDS", rows, cols);
      need(b.groups * (b.nt >> 6) <= 16, "backward: words of the sum", rows, cols);
    }
  }
  std::puts("ok");
  return 0;
}

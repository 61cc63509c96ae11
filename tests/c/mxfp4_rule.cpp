// For each line "R E Nw KB x_rows gathered cus" of the input, the kernel that the products by expert
// of microscaled FP4 rows take: "rows waves per_cu wide direct".
#include <stdio.h>

#include "grouped_mxfp4_rule.h"

int main() {
  long long R, E, Nw, KB, x_rows, gathered, cus;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld", &R, &E, &Nw, &KB, &x_rows, &gathered, &cus) == 7) {
    const rmoe::MxSizes s{R, E, Nw, KB, x_rows, gathered != 0, static_cast<int>(cus)};
    const rmoe::MxTiles t = rmoe::mx_tiles(s);
    printf("%d %d %d %d %d\n", t.rows, t.waves, t.per_cu, t.wide,
           t.rows == rmoe::kMxBig.rows ? 0 : rmoe::mx_direct(s, t));
  }
  return 0;
}

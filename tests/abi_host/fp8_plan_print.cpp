// Prints the launch plans of csrc/fp8_layout.h. Each line of the input is
// "dense m n k fast" or "grouped rows experts n blocks exact"; the answers are
// "stream tile t_main r_tiles splits" and "tile".
#include <stdio.h>

#include "../../gguf_block_quantized_qmv_amd/csrc/fp8_layout.h"

int main() {
  char what[16];
  int a, b, c, d, e;
  while (scanf("%15s", what) == 1) {
    if (what[0] == 'd') {
      if (scanf("%d %d %d %d", &a, &b, &c, &d) != 4) return 1;
      const qmv::fp8::DensePlan p = qmv::fp8::dense_plan(a, b, c, d != 0);
      printf("%d %d %d %d %d\n", p.stream, p.tile, p.t_main, p.r_tiles, p.splits);
    } else {
      if (scanf("%d %d %d %d %d", &a, &b, &c, &d, &e) != 5) return 1;
      printf("%d\n", qmv::fp8::grouped_tile(a, b, c, d, e != 0));
    }
  }
  return 0;
}

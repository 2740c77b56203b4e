// Prints the kernel that plan_logits8 (fh_host.cpp) chooses for each line
// "rows v d ldo out_size" of the standard input: "tiles 64 128" or "rows 16 32".
#include <stdio.h>

#include "../../two_stage_retrieval_amd/csrc/fh_host.h"

int main() {
  long long rows, v, ldo;
  int d, size;
  while (scanf("%lld %lld %d %lld %d", &rows, &v, &d, &ldo, &size) == 5) {
    const fh::Logits8Plan p = fh::plan_logits8(rows, v, d, ldo, size);
    printf("%s %d %d\n", p.tiles ? "tiles" : "rows", p.bm, p.bn);
  }
  return 0;
}

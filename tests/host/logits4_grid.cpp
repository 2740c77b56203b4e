// For each line "rows v f32" of the standard input: the kernel that plan_logits4
// chooses, the threads of its launch, and what check_logits_int4 (fh_host.cpp)
// says of a call of that size.
#include <stdio.h>

#include "../../two_stage_retrieval_amd/csrc/fh_host.h"

int main() {
  static const char* const kNames[] = {"kRows16", "kRows32", "k16x128", "k32x256",
                                       "k48x256", "k64x128", "k64x256", "k64x512"};
  void* const P = (void*)0x10000;   // aligned, never read
  long long rows, v;
  int f32;
  while (scanf("%lld %lld %d", &rows, &v, &f32) == 3) {
    const fh::Logits4Plan plan = fh::plan_logits4(rows, v, f32 != 0);
    const int64_t ld = (v + 7) / 8 * 8;
    const int st = fh::check_logits_int4(P, 128, f32 ? FH_DTYPE_F32 : FH_DTYPE_BF16, (int32_t)rows,
                                         P, 64, P, nullptr, ld, 128, v, 128, P, FH_DTYPE_BF16, ld);
    printf("%s %lld %d\n", kNames[(int)plan], (long long)fh::logits4_threads(plan, rows, v), st);
  }
  return 0;
}

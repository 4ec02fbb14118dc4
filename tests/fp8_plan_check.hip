// Host-only: which kernel rq_gemm_fp8 runs (built and run by tests/test_fp8_plan.py;
// no GPU code is executed).  Reads calls from stdin, a line each:
//   M  out_type  with_workspace  count  N K  N K ...
// and prints a line for each: the kernel and its ranges of K.
#include <cstdio>

#include "rq_gemm_fp8.hip"

static const char* const NAMES[] = {"ROWS16", "ROWS64", "RING1X2", "RING2X2", "RING4X2", "RING4X3", "RING4X4",
                                    "RING8X1", "RING8X2", "WIDE64", "WIDE128", "FP128", "FP256", "FP64"};
static_assert(sizeof(NAMES) / sizeof(NAMES[0]) == rq::FP64 + 1 && rq::FP256 == 12 && rq::WIDE64 == 9 &&
                  rq::RING8X1 == 7 && rq::RING4X4 == 6,
              "names of the kernels");

int main() {
  int ws;
  rq::Fp8Args a{};
  while (scanf("%d %d %d %d", &a.M, &a.out, &ws, &a.count) == 4) {
    if (a.count < 1 || a.count > rq::FP8_BATCH) return 1;
    for (int i = 0; i < a.count; i++)
      if (scanf("%d %d", &a.p[i].N, &a.p[i].K) != 2) return 1;
    const rq::Plan c = rq::choose(a, ws != 0);
    printf("%s %d\n", NAMES[c.kind], c.splits);
  }
  return 0;
}

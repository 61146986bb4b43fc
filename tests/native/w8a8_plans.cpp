// Host driver: for every line "M N K may_split off ld" of the input, the kernel that the 8-bit product
// takes, as "tile splits tail shifted" (names as in w8a8_plan.hpp, the tail or "-").  off: the byte of a cache
// line that both operands start at, ld: their row pitch.
#include <stdio.h>

#include "../../mxfp4_microscaled_quantization_amd/csrc/w8a8_plan.hpp"

int main() {
  const char* names[mxq::TILES] = {"256x256", "128x256", "128x128", "64x128", "128x64", "64x64", "64x32", "32x64", "32x32", "128x128_SHORT"};
  long long M, N, K, ld;
  int may_split, off;
  while (scanf("%lld %lld %lld %d %d %lld", &M, &N, &K, &may_split, &off, &ld) == 6) {
    const mxq::Plan p = mxq::plan_w8a8(M, N, K, may_split != 0);
    printf("%s %d %s %d\n", names[p.tile], p.splits, p.tail < 0 ? "-" : names[p.tail], mxq::shifted(K, off, ld, off, ld) ? 1 : 0);
  }
  return 0;
}

// The row kernels' generator (drop_offset, philox4x32_10 in fl_rows.cuh, the functions the kernels call), on the CPU.
// Reads lines "big block seed offset", each a 64-bit number; prints the four words of that block, with the form for blocks
// below 2^32 (big 0) or for any (big 1).
#include <cinttypes>
#include <cstdio>
#include <cstring>

#include "../../gemm_bias_activation_tcgen05_b200/csrc/fl_rows.cuh"

int main() {
  uint64_t big, block, seed, offset;
  while (std::scanf("%" SCNu64 " %" SCNu64 " %" SCNu64 " %" SCNu64, &big, &block, &seed, &offset) == 4) {
    fl::DropParams d;
    std::memset(&d, 0, sizeof(d));
    fl::set_drop_keys(&d, seed);
    d.offset = offset;
    const fl::DropOffset o = fl::drop_offset(d);
    const uint4 w = big ? fl::philox4x32_10<true>(block, o, d) : fl::philox4x32_10<false>(block, o, d);
    std::printf("%u %u %u %u\n", w.x, w.y, w.z, w.w);
  }
  return 0;
}

// kv8_attend's kernels for heads of 128 and e4m3 codes (one translation unit each, built in parallel).
#include "kv8_attend.cuh"

namespace qmv {
namespace attend {
int launch_128_e4m3(const Args& a, int rows, bool mods, int blocks, cudaStream_t s) {
  return launch_rows<128, QMV_KV_E4M3>(a, rows, mods, blocks, s);
}
}  // namespace attend
}  // namespace qmv

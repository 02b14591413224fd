// kv8_attend's kernels for heads of 64 and e4m3 codes (one translation unit each, built in parallel).
#include "kv8_attend.cuh"

namespace qmv {
namespace attend {
int launch_64_e4m3(const Args& a, int rows, bool mods, int blocks, cudaStream_t s) {
  return launch_rows<64, QMV_KV_E4M3>(a, rows, mods, blocks, s);
}
}  // namespace attend
}  // namespace qmv

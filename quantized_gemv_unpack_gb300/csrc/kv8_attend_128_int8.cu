// kv8_attend's kernels for heads of 128 and int8 codes (one translation unit each, built in parallel).
#include "kv8_attend.cuh"

namespace qmv {
namespace attend {
int launch_128_int8(const Args& a, int rows, bool mods, int blocks, cudaStream_t s) {
  return launch_rows<128, QMV_KV_INT8>(a, rows, mods, blocks, s);
}
}  // namespace attend
}  // namespace qmv

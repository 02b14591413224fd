// kv8_attend's prompt kernels for heads of 128 and int8 codes.
#include "kv8_prompt.cuh"

namespace qmv {
namespace prompt {
int launch_128_int8(const Args& a, bool mods, bool split, int blocks, cudaStream_t s) {
  return launch_any<128, QMV_KV_INT8>(a, mods, split, blocks, s);
}
}  // namespace prompt
}  // namespace qmv

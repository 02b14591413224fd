// kv8_attend's prompt kernels for int8 codes.
#include "kv8_prompt.cuh"

namespace qmv {
namespace prompt {
int launch_int8(const Args& a, int head_dim, bool mods, int blocks, cudaStream_t s) {
  return launch_dim<QMV_KV_INT8>(a, head_dim, mods, blocks, s);
}
}  // namespace prompt
}  // namespace qmv

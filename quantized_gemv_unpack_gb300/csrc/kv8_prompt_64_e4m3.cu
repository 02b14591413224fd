// kv8_attend's prompt kernels for heads of 64 and e4m3 codes.
#include "kv8_prompt.cuh"

namespace qmv {
namespace prompt {
int launch_64_e4m3(const Args& a, bool mods, bool split, int blocks, cudaStream_t s) {
  return launch_any<64, QMV_KV_E4M3>(a, mods, split, blocks, s);
}
}  // namespace prompt
}  // namespace qmv

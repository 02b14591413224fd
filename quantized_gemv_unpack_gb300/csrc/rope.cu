// Rotary positions with several axes (rope_run) and the rotation's descriptor.
//
// out = x rotated pair by pair: 2 * bytes(x) of traffic and three products per
// pair, so the kernel is a copy with some arithmetic. A block takes some tokens,
// computes their angles once (sine and cosine cost about 40 instructions a pair)
// into shared memory and applies them to all its heads, sixteen values per thread
// in two 16-byte pieces (16-bit types). No table of angles is read and none has to
// be made for a longer context.
//
// Few tokens are split over the heads (16 of them per block), so that a decode
// token's 48 heads are three blocks rather than one long loop.
//
// Measured: 8192 tokens of 48 heads of 128, bf16, three axes: 34.9 us, 5.8 TB/s (0.85
// of the measured copy rate); 4095 tokens of 16 heads of 64 in fp32: 7.5 us; one token 1.9 us in a
// captured graph, 4.3 issued from the host. Two,
// three or eight tokens per block and three loads in flight per thread were no faster.
#include "kv8.cuh"

#include <cmath>
#include <cstring>

namespace qmv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTokensPerBlock = 4;

struct RopeArgs {
  qmv_rope r;
  const void* x;
  void* out;
  const int32_t* positions;
  int64_t ldx, ldo, ldp, n_tokens;
  int n_heads, out_type, tokens_per_block, heads_per_block;
  float sign;
};

template <typename TI>
__global__ void __launch_bounds__(kRopeThreads, sizeof(TI) == 4 ? 3 : 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 angles[kMaxTokensPerBlock * QMV_ROPE_MAX_PAIRS];   // read two pairs at a time
  kv8::follow_previous();
  const int h0 = blockIdx.y * a.heads_per_block;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_block;
  kv8::rope_tokens<TI>(a.r, static_cast<const TI*>(a.x), a.ldx, t0, (int)min((int64_t)a.tokens_per_block, a.n_tokens - t0),
                       h0, min(a.n_heads, h0 + a.heads_per_block), a.positions, a.ldp, a.out, a.out_type, a.ldo, a.sign,
                       angles, threadIdx.x, blockDim.x);
}

}  // namespace

namespace kv8 {
int check_rope(const qmv_rope* r) {
  if (!r) return fail(QMV_ERR_ARG, "rope is NULL");
  if (r->abi_version != QMV_ABI_VERSION) return fail(QMV_ERR_ARG, "rope abi_version %u, library %d", r->abi_version, QMV_ABI_VERSION);
  if (r->head_dim < 16 || r->head_dim > 2 * QMV_ROPE_MAX_PAIRS || r->head_dim % 16 || r->rot_dim < 16 ||
      r->rot_dim > r->head_dim || r->rot_dim % 16)
    return fail(QMV_ERR_ARG, "head_dim=%d rot_dim=%d: multiples of 16, rot_dim <= head_dim <= %d", r->head_dim, r->rot_dim,
                2 * QMV_ROPE_MAX_PAIRS);
  if (r->n_axes < 1 || r->n_axes > QMV_ROPE_MAX_AXES) return fail(QMV_ERR_ARG, "n_axes=%d outside 1..%d", r->n_axes, QMV_ROPE_MAX_AXES);
  for (int i = 0; i < r->rot_dim / 2; ++i)
    if (r->axis[i] >= r->n_axes) return fail(QMV_ERR_ARG, "pair %d: axis %d of %d", i, r->axis[i], r->n_axes);
  return QMV_OK;
}

int rope_launch(const qmv_rope* rope, const void* x, int x_type, int64_t n_tokens, int n_heads, int64_t ldx,
                const int32_t* positions, int64_t ldp, void* out, int out_type, int64_t ldo, int inverse, cudaStream_t s) {
  int rc = check_rope(rope);
  if (rc) return rc;
  const int xs = dtype_size(x_type), os = dtype_size(out_type);
  if (!xs || !os) return fail(QMV_ERR_ARG, "x_type=%d out_type=%d", x_type, out_type);
  if (n_tokens < 0 || n_heads < 1 || n_tokens > INT32_MAX || n_heads > 65536)
    return fail(QMV_ERR_ARG, "n_tokens=%lld n_heads=%d", (long long)n_tokens, n_heads);
  const int64_t row = (int64_t)n_heads * rope->head_dim;
  if (ldx < row || ldo < row || ldp < n_tokens) return fail(QMV_ERR_ARG, "ldx=%lld ldo=%lld ldp=%lld", (long long)ldx, (long long)ldo, (long long)ldp);
  if (ldx * xs % 16 || ldo * os % 16) return fail(QMV_ERR_ALIGN, "rows of x and out must be 16-byte aligned");
  if (n_tokens == 0) return QMV_OK;
  if (!x || !out || !positions) return fail(QMV_ERR_ARG, "NULL x, out or positions");
  if (!aligned16(x) || !aligned16(out) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(QMV_ERR_ALIGN, "x and out must be 16-byte aligned, positions 4-byte");
  if (x == out && (x_type != out_type || ldx != ldo)) return fail(QMV_ERR_ARG, "in place needs one type and one stride");

  RopeArgs a;
  a.r = *rope;
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.ldx = ldx;
  a.ldo = ldo;
  a.ldp = ldp;
  a.n_tokens = n_tokens;
  a.n_heads = n_heads;
  a.out_type = out_type;
  a.sign = inverse ? -1.f : 1.f;
  // Enough tokens for four blocks per SM: all heads in one block, four tokens at a time. Fewer: one token and 16 heads.
  const bool split = n_tokens < 4 * sm_count();
  a.tokens_per_block = split ? 1 : kMaxTokensPerBlock;
  a.heads_per_block = split && n_heads > 16 ? 16 : n_heads;
  const dim3 grid((unsigned)((n_tokens + a.tokens_per_block - 1) / a.tokens_per_block),
                  (unsigned)((n_heads + a.heads_per_block - 1) / a.heads_per_block));
  // a block of few heads has one chunk per thread
  const int chunks = a.heads_per_block * (rope->head_dim / 16);
  const int block = chunks >= kRopeThreads ? kRopeThreads : (chunks + 31) / 32 * 32;
  const void* f = x_type == QMV_F32 ? (const void*)rope_kernel<float>
                  : x_type == QMV_BF16 ? (const void*)rope_kernel<__nv_bfloat16> : (const void*)rope_kernel<__half>;
  void* args[] = {&a};
  cudaError_t e = launch_early(f, grid, block, args, 0, s);
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return QMV_OK;
}
}  // namespace kv8
}  // namespace qmv

using namespace qmv;

extern "C" {

int rope_desc(int32_t head_dim, int32_t rot_dim, int32_t n_axes, int32_t interleaved, const double* inv_freq,
              const int32_t* axis, qmv_rope* out) {
  if (!out || !inv_freq) return fail(QMV_ERR_ARG, "NULL inv_freq or out");
  qmv_rope r;
  memset(&r, 0, sizeof(r));
  r.abi_version = QMV_ABI_VERSION;
  r.head_dim = head_dim;
  r.rot_dim = rot_dim;
  r.n_axes = n_axes;
  r.interleaved = interleaved ? 1 : 0;
  int rc = kv8::check_rope(&r);
  if (rc) return rc;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (axis && (axis[i] < 0 || axis[i] >= n_axes)) return fail(QMV_ERR_ARG, "pair %d: axis %d of %d", i, axis[i], n_axes);
    r.axis[i] = axis ? (uint8_t)axis[i] : 0;
    double t = inv_freq[i] * 0.15915494309189535;  // 1 / 2 pi
    if (!(std::fabs(t) < 1e15)) return fail(QMV_ERR_ARG, "inv_freq[%d] is not a finite frequency", i);
    t -= std::floor(t);
    // t is below 1, so the product is below 2^64 (1 - 2^-53 at most)
    r.turn[i] = t >= 1.0 ? 0 : (uint64_t)(t * 18446744073709551616.0);
  }
  *out = r;
  return QMV_OK;
}

int rope_run(const qmv_rope* rope, const void* x, int x_type, int64_t n_tokens, int32_t n_heads, int64_t ldx,
             const int32_t* positions, int64_t ldp, void* out, int out_type, int64_t ldo, int inverse, void* stream) {
  return kv8::rope_launch(rope, x, x_type, n_tokens, n_heads, ldx, positions, ldp, out, out_type, ldo, inverse,
                          static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// Embedding rows out of a packed matrix (qmv_embed):
//   out[t][k] = scale * q[token t][k] * s[token t][k / 128].
//
// A copy with a decode: K bits / 8 + K / 64 bytes in and K values out per token, so
// the stores are its bound. A thread makes eight consecutive values of each of
// several tokens: one store of 16 bytes (32 for fp32), next to its neighbours', and
// one to four small loads of codes, all of them in flight before the first use.
// Codes lie per token in pieces of 16 to 512 bytes, whatever the layout, and a
// warp's loads share their sectors.
#include "kv8.cuh"

namespace qmv {
namespace {

using kv8::follow_previous;

constexpr int kEmbedThreads = 128;

struct Args {
  const unsigned char* codes;
  const uint16_t* scales;
  const int32_t* tokens;
  void* out;
  int* err;
  int64_t n_tokens, ldo;
  int32_t N, K, pieces;      // pieces: blocks of threads that a token takes
  float scale;
};

// The codes of columns 8 c .. 8 c + 7 of row n as one word, before their order in it is undone, and the place of their scale.
template <int FMT>
__device__ __forceinline__ uint32_t load_codes(const Args& a, int64_t n, int c) {
  const int b = c / 16;                                            // block of 128 columns
  const int KB = a.K / 128;
  if constexpr (FMT == QMV_TERNARY2 || FMT == QMV_INT4) {
    // row-group records: 16 rows x up to 8 blocks, row after row
    const int64_t block = (n / 16) * 16 * KB + (b / 8) * 128 + (n % 16) * min(8, KB - b / 8 * 8) + b % 8;
    if constexpr (FMT == QMV_TERNARY2) return *reinterpret_cast<const uint32_t*>(a.codes + block * 32 + (c % 16) / 2 * 4);
    return *reinterpret_cast<const uint32_t*>(a.codes + block * 64 + (c % 16) * 4);
  } else {
    // byte lookup: a row's bytes of a block in halves of 32, each turned by n % 32
    const int64_t NG = (a.N + 31) / 32, record = b * NG + n / 32;
    const int r = (int)(n % 32);
    uint32_t w = 0;
    if constexpr (FMT == QMV_TERNARY2_LUT) {
      const unsigned char* p = a.codes + record * 1024 + r * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = ((c % 16) * 2 + i - r) & 31;
        w |= (uint32_t)p[t / 16 * 512 + t % 16] << (8 * i);
      }
    } else {
      const unsigned char* p = a.codes + record * 2048 + r * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int byte = (c % 16) * 4 + i, t = (byte & 32) + ((byte - r) & 31);
        w |= (uint32_t)p[t / 16 * 512 + t % 16] << (8 * i);
      }
    }
    return w;
  }
}
template <int FMT>
__device__ __forceinline__ int64_t scale_at(const Args& a, int64_t n, int c) {
  if constexpr (FMT == QMV_TERNARY2 || FMT == QMV_INT4) return scale_index(n, c / 16, scale_steps(a.K));
  return (int64_t)(c / 16) * ((a.N + 31) / 32 * 32) + n;
}
// Whole numbers of the eight columns; true where a code is none of its format's.
template <int FMT>
__device__ __forceinline__ bool decode(uint32_t w, int c, int (&q)[8]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (FMT == QMV_TERNARY2) {
      const int r = (c & 1) * 8 + i;
      const uint32_t u = (w >> (r % 2 ? 15 + r : r)) & 3u;
      bad |= u == 3u;
      q[i] = u == 3u ? 0 : (int)(u & 1u) - (int)(u >> 1);
    } else if constexpr (FMT == QMV_TERNARY2_LUT) {
      const uint32_t u = (w >> (2 * i)) & 3u;
      bad |= u == 3u;
      q[i] = u == 3u ? 0 : (int)(u & 1u) - (int)(u >> 1);
    } else {
      const uint32_t u = (w >> (FMT == QMV_INT4 ? (i % 2 ? 14 + 2 * i : 2 * i) : 4 * i)) & 15u;
      q[i] = (int)(u ^ 8u) - 8;
    }
  }
  return bad;
}

// U tokens per block of threads.
template <int FMT, typename TO, int U>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const Args a) {
  follow_previous();
  const int c = (int)(blockIdx.x % a.pieces) * kEmbedThreads + threadIdx.x;
  const int64_t t0 = (int64_t)(blockIdx.x / a.pieces) * U;
  if (c * 8 >= a.K) return;
  int32_t n[U];
  uint32_t w[U];
  uint16_t s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) n[u] = t0 + u < a.n_tokens ? a.tokens[t0 + u] : -1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    w[u] = 0;
    s[u] = 0;
    if (n[u] >= 0 && n[u] < a.N) {
      w[u] = load_codes<FMT>(a, n[u], c);
      s[u] = a.scales[scale_at<FMT>(a, n[u], c)];
    }
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (t0 + u >= a.n_tokens) break;
    int q[8];
    float v[8];
    bad |= n[u] >= a.N;
    bad |= decode<FMT>(w[u], c, q);
    const float f = __half2float(__ushort_as_half(s[u]));
    // q * s is exact (4 and 11 bits): one rounding to fp32, one to the output's type
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn((float)q[i] * f, a.scale);
    kv8::store8(static_cast<TO*>(a.out) + (t0 + u) * a.ldo + c * 8, v);
  }
  if (bad) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
}

template <int FMT, int U>
const void* of_type(int type) {
  return type == QMV_F32 ? reinterpret_cast<const void*>(embed_kernel<FMT, float, U>)
         : type == QMV_BF16 ? reinterpret_cast<const void*>(embed_kernel<FMT, __nv_bfloat16, U>)
                            : reinterpret_cast<const void*>(embed_kernel<FMT, __half, U>);
}
template <int U>
const void* of_format(int format, int type) {
  return format == QMV_TERNARY2 ? of_type<QMV_TERNARY2, U>(type)
         : format == QMV_TERNARY2_LUT ? of_type<QMV_TERNARY2_LUT, U>(type)
         : format == QMV_INT4 ? of_type<QMV_INT4, U>(type) : of_type<QMV_INT4_LUT, U>(type);
}

constexpr int kMany = 8;   // 8190 tokens of 5120 columns, INT4 to bf16: 23.8, 20.0 and 19.3 us with 2, 4 and 8

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

int qmv_embed(const qmv_desc* desc, const void* packed, const int32_t* tokens, int64_t n_tokens, float scale, void* out, int out_type,
              int64_t ldo, void* stream) {
  if (!desc) return fail(QMV_ERR_ARG, "desc is NULL");
  const int format = (int)desc->format;
  if (format != QMV_TERNARY2 && format != QMV_TERNARY2_LUT && format != QMV_INT4 && format != QMV_INT4_LUT)
    return fail(format >= QMV_TERNARY2 && format <= QMV_INT4_LUT ? QMV_ERR_UNSUPPORTED : QMV_ERR_ARG,
                "format %d: embedding rows come out of ternary and INT4 matrices in either layout", format);
  int rc = check_desc(desc, format);
  if (rc) return rc;
  qmv_desc ref;
  rc = qmv_pack_desc(format, desc->N, desc->K, desc->group, &ref);
  if (rc) return rc;
  if (ref.off[0] != desc->off[0] || ref.off[1] != desc->off[1] || ref.bytes[0] != desc->bytes[0] || ref.bytes[1] != desc->bytes[1])
    return fail(QMV_ERR_ARG, "desc sections do not match the layout of a %lld x %lld matrix", (long long)desc->N, (long long)desc->K);
  if (desc->N > INT32_MAX / 2 || desc->K > (1 << 26)) return fail(QMV_ERR_UNSUPPORTED, "matrix too large");
  const int os = kv8::dtype_size(out_type);
  if (!os) return fail(QMV_ERR_ARG, "out_type=%d", out_type);
  if (n_tokens < 0 || n_tokens > INT32_MAX || ldo < desc->K) return fail(QMV_ERR_ARG, "n_tokens=%lld ldo=%lld", (long long)n_tokens, (long long)ldo);
  if (ldo * os % 16) return fail(QMV_ERR_ALIGN, "output rows must be 16-byte aligned");
  if (!(fabsf(scale) <= 3.4028235e38f)) return fail(QMV_ERR_ARG, "scale is not finite");
  if (n_tokens == 0) return QMV_OK;
  if (!packed || !tokens || !out) return fail(QMV_ERR_ARG, "NULL packed, tokens or out");
  if (!aligned16(packed) || !aligned16(out) || (reinterpret_cast<uintptr_t>(tokens) & 3u))
    return fail(QMV_ERR_ALIGN, "packed and out must be 16-byte aligned, tokens 4-byte");
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");
  Args a;
  a.codes = static_cast<const unsigned char*>(packed) + desc->off[0];
  a.scales = reinterpret_cast<const uint16_t*>(static_cast<const unsigned char*>(packed) + desc->off[1]);
  a.tokens = tokens;
  a.out = out;
  a.err = err;
  a.n_tokens = n_tokens;
  a.ldo = ldo;
  a.N = (int32_t)desc->N;
  a.K = (int32_t)desc->K;
  a.scale = scale;
  a.pieces = (int32_t)((desc->K / 8 + kEmbedThreads - 1) / kEmbedThreads);
  // several tokens per block where there are enough to fill the device all the same
  const bool many = n_tokens / kMany * a.pieces >= 16 * (int64_t)sm_count();
  const int64_t blocks = (n_tokens + (many ? kMany : 1) - 1) / (many ? kMany : 1) * a.pieces;
  if (blocks > INT32_MAX) return fail(QMV_ERR_UNSUPPORTED, "n_tokens=%lld of %lld columns", (long long)n_tokens, (long long)desc->K);
  const void* f = many ? of_format<kMany>(format, out_type) : of_format<1>(format, out_type);
  void* args[] = {&a};
  cudaError_t e = kv8::launch_early(f, dim3((unsigned)blocks), kEmbedThreads, args, 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "qmv_embed launch");
  return QMV_OK;
}

}  // extern "C"

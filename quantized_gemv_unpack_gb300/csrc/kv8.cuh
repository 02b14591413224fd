// Pieces shared by the paged 8-bit KV cache kernels (kv_plan.cu, rope.cu,
// kv8_append.cu, kv8_attend.cu): the cache's tile layout, code conversions,
// 8-value loads and stores of the activation types, and the rotation's angle.
#pragma once

#include <cuda_fp8.h>

#include "qmv_internal.cuh"

namespace qmv {
namespace kv8 {

// ----------------------------------------------------------------------------- launches

// Kernels of this family are set up while the stream's kernel before them still ends: launch_early lets a grid begin when
// every block of that kernel has ended or has called let_next_begin, and follow_previous, called by all threads before the
// first access to memory that another kernel may use, waits until that kernel has ended and its writes are seen. So the
// order of a stream stays, less the launch's own time. Calls in a row, in us: one-token attention 12.3 -> 9.7, a decode
// step's append and read back 14.4 -> 10.2, kv_plan 6.3 -> 5.1. Only kernels of one block per SM call let_next_begin: with it
// the many small blocks of a rotation or an append come to lie unevenly over the SMs while they wait (7.6 and 10.2 us
// without it become 11.2 and 15.1).
__device__ __forceinline__ void follow_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
inline cudaError_t launch_early(const void* kernel, dim3 grid, int threads, void** args, size_t smem, cudaStream_t s, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

constexpr int kPage = QMV_KV_PAGE;

int check_kv_desc(const qmv_kv_desc* d);
int check_rope(const qmv_rope* r);
int rope_launch(const qmv_rope* rope, const void* x, int x_type, int64_t n_tokens, int n_heads, int64_t ldx,
                const int32_t* positions, int64_t ldp, void* out, int out_type, int64_t ldo, int inverse, cudaStream_t s);
inline int dtype_size(int t) { return t == QMV_F32 ? 4 : (t == QMV_BF16 || t == QMV_F16 ? 2 : 0); }

// Byte of (token, d) in a K tile. Eight tokens (token / 16, token % 2) of one
// 64-value piece of d lie in 512 consecutive bytes: one 16-byte load per lane of
// a warp is the B fragments of four m16n8k16 steps (kv8_attend.cu).
__host__ __device__ __forceinline__ int k_byte(int token, int d, int D) {
  return ((((token & 15) >> 1) * (D >> 6) + (d >> 6)) * 8 + (token >> 4) * 2 + (token & 1)) * 64 + (d & 63);
}
// Byte of (token, d) in a V tile.
__host__ __device__ __forceinline__ int v_byte(int token, int d) { return d * kPage + token; }

// ---- codes

template <int TYPE>
__device__ __forceinline__ float code_top() {
  return TYPE == QMV_KV_INT8 ? 127.f : 448.f;
}
// A page's scale is 0 or at least the smallest normal number, so that its reciprocal is finite: of a smaller one it would be
// infinite, which makes a code of 0 a NaN when it is rounded again. Values below half of that are stored as 0.
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126
__device__ __forceinline__ float grown_scale(float was, float largest, float top) {
  const float s = fmaxf(was, __fdiv_rn(largest, top));
  return s > 0.f ? fmaxf(s, kLeastScale) : 0.f;
}
// x * inv as a code byte, rounded to nearest even and held to +-top; NaN gives 0.
template <int TYPE>
__device__ __forceinline__ uint32_t encode(float y) {
  if constexpr (TYPE == QMV_KV_INT8) {
    // fmaxf takes the number of a (number, NaN) pair, so a NaN is tested first
    const float c = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
    return (uint32_t)(__float2int_rn(c) + 128);
  } else {
    const float c = y == y ? fminf(fmaxf(y, -448.f), 448.f) : 0.f;
    return (uint32_t)__nv_cvt_float_to_fp8(c, __NV_SATFINITE, __NV_E4M3);
  }
}
template <int TYPE>
__device__ __forceinline__ float decode(uint32_t b) {
  if constexpr (TYPE == QMV_KV_INT8) {
    return (float)((int)b - 128);
  } else {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
    return __half2float(__half(h));
  }
}

// Eight finite values of magnitude at most top * (1 + 2^-22) as codes, in two words. int8: adding 1.5 * 2^23 leaves the
// nearest whole number (ties to even) in the low byte of the sum.
template <int TYPE>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(v[4 * i + j], inv);
    if constexpr (TYPE == QMV_KV_INT8) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(__fadd_rn(y[j], 12582912.f));
      w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410) ^ 0x80808080u;
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}
// The same for any values.
template <int TYPE>
__device__ __forceinline__ uint2 encode8_any(const float (&v)[8], float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= encode<TYPE>(v[i] * inv) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// The values of eight codes, without the scale: exact.
template <int TYPE>
__device__ __forceinline__ void decode8(uint2 w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = i ? w.y : w.x;
    if constexpr (TYPE == QMV_KV_INT8) {
      // 2^23 + byte in the bits of a float
      v[4 * i] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7440)) - 8388736.f;
      v[4 * i + 1] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7441)) - 8388736.f;
      v[4 * i + 2] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7442)) - 8388736.f;
      v[4 * i + 3] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7443)) - 8388736.f;
    } else {
      const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xFFFFu), __NV_E4M3);
      const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x >> 16), __NV_E4M3);
      const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
      v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = b.x, v[4 * i + 3] = b.y;
    }
  }
}

// ---- eight consecutive values of an activation row (16-byte aligned)

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// the same with the type known at run time
__device__ __forceinline__ void store8_as(int type, void* base, int64_t i, const float (&v)[8]) {
  if (type == QMV_F32) store8(static_cast<float*>(base) + i, v);
  else if (type == QMV_BF16) store8(static_cast<__nv_bfloat16*>(base) + i, v);
  else store8(static_cast<__half*>(base) + i, v);
}

// ---- rotation

// Sixteen values of a head: chunk c (of head_dim / 16) is eight pairs, or past
// rot_dim sixteen values that pass through. Its values are two pieces of eight,
// at d0 and d1.
struct RopeChunk {
  int d0, d1;
  bool turned;
};
__device__ __forceinline__ RopeChunk rope_chunk(const qmv_rope& r, int c) {
  const bool turned = c * 16 < r.rot_dim;
  if (turned && !r.interleaved) return {8 * c, 8 * c + r.rot_dim / 2, true};
  return {16 * c, 16 * c + 8, turned};
}
// A pair's angle at a position: position * turn is exact modulo one turn; its top 32 bits, as half turns in [-1, 1), go
// to sincospif (an angle error of at most 2^-25 half turns from the conversion to fp32).
// The angles of n tokens (positions at pos, pos + 1, ...) into shared memory, by the block's threads, each pair's once
// for all heads that the block serves. Pairs 8c + 2i and 8c + 2i + 1 of token k are at 2 ((k * 4 + i) * chunks + c), so
// that the threads of neighbouring chunks read neighbouring 16-byte words. A thread keeps its pair from token to token: reading the descriptor (a
// kernel argument) at 32 places takes a warp 32 turns.
__device__ __forceinline__ void rope_angles(const qmv_rope& r, int n, const int32_t* pos, int64_t ldp, float sign,
                                            float2* angles, int tid, int threads) {
  const int pairs = r.rot_dim / 2, chunks = r.head_dim / 16;
  const int rows = threads >= pairs ? threads / pairs : 1;   // tokens at a time
  const int k0 = threads >= pairs ? tid / pairs : 0;
  if (k0 >= rows) return;
  for (int pair = tid - k0 * pairs; pair < pairs; pair += threads) {
    const uint64_t turn = r.turn[pair];
    const int32_t* p = pos + (int64_t)r.axis[pair] * ldp;
    for (int k = k0; k < n; k += rows) {
      const uint64_t ph = (uint64_t)(int64_t)p[k] * turn;
      const float h = (float)(int32_t)(ph >> 32) * 4.656612873077393e-10f;  // 2^-31
      float s, c;
      sincospif(h, &s, &c);
      angles[2 * ((k * 4 + ((pair & 7) >> 1)) * chunks + (pair >> 3)) + (pair & 1)] = make_float2(c, s * sign);
    }
  }
}
__device__ __forceinline__ void chunk_angles(const float2* angles, int k, int c, int chunks, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(angles)[(k * 4 + i) * chunks + c];
    cs[2 * i] = v.x;
    sn[2 * i] = v.y;
    cs[2 * i + 1] = v.z;
    sn[2 * i + 1] = v.w;
  }
}
__device__ __forceinline__ void rope_pair(float c, float s, float& a, float& b) {
  const float x = a;
  a = fmaf(-b, s, x * c);
  b = fmaf(x, s, b * c);
}
__device__ __forceinline__ void rope_turn(bool interleaved, const float (&cs)[8], const float (&sn)[8], float (&a)[8],
                                          float (&b)[8]) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rope_pair(cs[i], sn[i], a[i], b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rope_pair(cs[i], sn[i], a[2 * i], a[2 * i + 1]);
      rope_pair(cs[i + 4], sn[i + 4], b[2 * i], b[2 * i + 1]);
    }
  }
}

// Sixteen values of a head as they lie in memory.
template <typename TI>
struct Raw16 {
  static constexpr int W = sizeof(TI) / 2;   // 16-byte words per eight values
  uint4 w[2 * W];
};
template <typename TI>
__device__ __forceinline__ Raw16<TI> load_raw(const TI* p, int d0, int d1) {
  Raw16<TI> r;
  constexpr int W = Raw16<TI>::W;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    r.w[i] = reinterpret_cast<const uint4*>(p + d0)[i];
    r.w[W + i] = reinterpret_cast<const uint4*>(p + d1)[i];
  }
  return r;
}
template <typename TI>
__device__ __forceinline__ void unpack(const Raw16<TI>& r, float (&a)[8], float (&b)[8]) {
  load8(reinterpret_cast<const TI*>(&r.w[0]), a);
  load8(reinterpret_cast<const TI*>(&r.w[Raw16<TI>::W]), b);
}

// Largest magnitude among sixteen values as the bits of their type without the sign (an order that puts infinity and
// NaN on top): at or above odd_bits() some value is not finite.
template <typename TI>
__device__ __forceinline__ uint32_t raw_top(const Raw16<TI>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2 * Raw16<TI>::W; ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = sizeof(TI) == 4 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
  }
  return sizeof(TI) == 4 ? m : max(m & 0xFFFFu, m >> 16);
}
template <typename TI>
__device__ __forceinline__ constexpr uint32_t odd_bits();
template <>
__device__ __forceinline__ constexpr uint32_t odd_bits<float>() { return 0x7F800000u; }
template <>
__device__ __forceinline__ constexpr uint32_t odd_bits<__nv_bfloat16>() { return 0x7F80u; }
template <>
__device__ __forceinline__ constexpr uint32_t odd_bits<__half>() { return 0x7C00u; }
// Finite bits of raw_top as a float.
template <typename TI>
__device__ __forceinline__ float top_value(uint32_t bits) {
  if constexpr (sizeof(TI) == 4) return __uint_as_float(bits);
  else if constexpr (odd_bits<TI>() == 0x7F80u) return __uint_as_float(bits << 16);
  else return __half2float(__ushort_as_half((unsigned short)bits));
}

// Rotate heads [h0, h1) of the n tokens from t0 on, by the block's threads: a thread keeps its chunk and takes a (token,
// head) at a time, neighbouring threads neighbouring chunks. Its first two loads are in flight while the block
// computes the angles. `angles` (shared, 16-byte aligned) holds n * head_dim / 2 pairs.
template <typename TI>
__device__ __forceinline__ void rope_tokens(const qmv_rope& r, const TI* x, int64_t ldx, int64_t t0, int n, int h0, int h1,
                                            const int32_t* positions, int64_t ldp, void* out, int out_type, int64_t ldo,
                                            float sign, float2* angles, int tid, int threads) {
  constexpr int kAhead = 2;
  const int chunks = r.head_dim / 16, heads = h1 - h0;
  const int step = threads / chunks, y = tid / chunks, c = tid - y * chunks;
  const RopeChunk ch = rope_chunk(r, c);
  const bool inter = r.interleaved != 0;
  // (token, head) of this thread's next load, and of its next store
  int k = y / heads, h = y - k * heads;
  int k2 = k, h2 = h;
  if (y >= step) k = k2 = n;
  const int dk = step / heads, dh = step - dk * heads;
  auto next = [&](int& tk, int& th) {
    tk += dk;
    th += dh;
    if (th >= heads) {
      th -= heads;
      ++tk;
    }
  };
  const TI* px = x + t0 * ldx + (int64_t)h0 * r.head_dim;
  const int64_t po = t0 * ldo + (int64_t)h0 * r.head_dim;
  Raw16<TI> raw[kAhead];
  bool first = true;
  do {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k < n) raw[j] = load_raw(px + k * ldx + h * r.head_dim, ch.d0, ch.d1);
      next(k, h);
    }
    if (first) {
      rope_angles(r, n, positions + t0, ldp, sign, angles, tid, threads);
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k2 >= n) break;
      float a[8], b[8];
      unpack(raw[j], a, b);
      if (ch.turned) {
        float cs[8], sn[8];
        chunk_angles(angles, k2, c, chunks, cs, sn);
        rope_turn(inter, cs, sn, a, b);
      }
      const int64_t o = po + k2 * ldo + h2 * r.head_dim;
      store8_as(out_type, out, o + ch.d0, a);
      store8_as(out_type, out, o + ch.d1, b);
      next(k2, h2);
    }
  } while (k2 < n);
}

}  // namespace kv8
}  // namespace qmv

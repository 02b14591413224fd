// Pieces shared by the paged 8-bit KV cache kernels (kv_plan.cu, rope.cu,
// kv8_append.cu, kv8_attend.cu): the cache's tile layout, code conversions,
// 8-value loads and stores of the activation types, and the rotation's angle.
#pragma once

#include <cuda_fp8.h>

#include "qmv_internal.cuh"

namespace qmv {
namespace kv8 {

constexpr int kPage = QMV_KV_PAGE;

int check_kv_desc(const qmv_kv_desc* d);
int check_rope(const qmv_rope* r);
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
// Cosine and sine of chunk c's eight pairs for the token whose positions are at
// pos[axis * ldp]. The product position * turn is exact modulo one turn; the
// top 32 bits, as half turns in [-1, 1), go to sincospif (an angle error of at
// most 2^-25 half turns from the conversion to fp32).
__device__ __forceinline__ void rope_angles(const qmv_rope& r, int c, const int32_t* pos, int64_t ldp, float sign,
                                            float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = 8 * c + i;
    const int64_t p = pos[(int64_t)r.axis[pair] * ldp];
    const uint64_t ph = (uint64_t)p * r.turn[pair];
    const float h = (float)(int32_t)(ph >> 32) * 4.656612873077393e-10f;  // 2^-31
    sincospif(h, &sn[i], &cs[i]);
    sn[i] *= sign;
  }
}
__device__ __forceinline__ void rope_turn(bool interleaved, const float (&cs)[8], const float (&sn)[8], float (&a)[8],
                                          float (&b)[8]) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, sn[i]));
      b[i] = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, sn[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, sn[i]));
      a[2 * i + 1] = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, sn[i]));
      x = b[2 * i], y = b[2 * i + 1];
      b[2 * i] = __fsub_rn(__fmul_rn(x, cs[i + 4]), __fmul_rn(y, sn[i + 4]));
      b[2 * i + 1] = __fadd_rn(__fmul_rn(y, cs[i + 4]), __fmul_rn(x, sn[i + 4]));
    }
  }
}

// Rotate the heads of tokens [t0, t1) that this block serves: thread (c, y) of
// head_dim / 16 x rows threads takes chunk c of heads y, y + rows, ... and
// computes the chunk's angles once per token.
template <typename TI>
__device__ __forceinline__ void rope_tokens(const qmv_rope& r, const TI* x, int64_t ldx, int64_t t0, int64_t t1, int h0,
                                            int h1, const int32_t* positions, int64_t ldp, void* out, int out_type,
                                            int64_t ldo, float sign, int c, int y, int rows) {
  const RopeChunk ch = rope_chunk(r, c);
  for (int64_t t = t0; t < t1; ++t) {
    float cs[8], sn[8];
    if (ch.turned) rope_angles(r, c, positions + t, ldp, sign, cs, sn);
    for (int h = h0 + y; h < h1; h += rows) {
      float a[8], b[8];
      const TI* px = x + t * ldx + (int64_t)h * r.head_dim;
      load8(px + ch.d0, a);
      load8(px + ch.d1, b);
      if (ch.turned) rope_turn(r.interleaved != 0, cs, sn, a, b);
      const int64_t o = t * ldo + (int64_t)h * r.head_dim;
      store8_as(out_type, out, o + ch.d0, a);
      store8_as(out_type, out, o + ch.d1, b);
    }
  }
}

}  // namespace kv8
}  // namespace qmv

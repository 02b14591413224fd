// Log probabilities of given tokens, entropy, rank and top alternatives of rows
// of logits (logprob_run).
//
// One pass over a row: a thread keeps the largest value M it has seen, and with
// d_i = (x_i - M) scale log2 e the sums S = sum 2^d_i and U = sum 2^d_i d_i, which
// give lse = scale M + ln S and the entropy ln S - ln 2 U / S. Partial results of
// threads, warps and blocks join by S = sum S_p 2^D_p, U = sum (U_p + D_p S_p) 2^D_p,
// D_p their M less the largest. d is one fused multiply-add from the rounded product
// M scale log2 e, and what the rounding took is put back into the results. That is a part of
// every d, the largest value's own among them, and up to half a step of the product: with
// products of 2^32 and more it would take powers past fp32's range. So from 2^31 on (a mask of
// -1e10, a row of its type's lowest value) the difference comes first, which is slower; up to
// there it is at most 2^6, and a mask of -1e9 keeps to the fast path (1000 rows of 131072
// values bf16, all but one in a thousand masked so: 58 us, 84 where the difference is taken
// from 2^20 on).
//
// The top k (k <= 32) come from the threads' largest values: at least k values of a block reach the k-th of its threads'
// maxima, and hardly more do. So the pass keeps maxima alone, of each thread and of up to 32 parts of what it reads, and
// after it the parts that reach the threshold are read again, a thread's by its whole warp: for 64 rows of 128257 values fp32,
// k = 5, 14.7 us (with lists that grow during the pass 16.8), for 4095 rows of 131072 values bf16, k = 20, 205 us (277). Up to
// 64 candidates are sorted at once. Where there are more, equal values or fewer than k that are not masked, each warp puts its own
// into a list, one by one where few lanes have some, else 32 at a time by a bitonic sort and merge: 64 rows with three values that are
// not masked 36 us. Lists are sorted, an entry per lane, of 64-bit keys: the value in an order-preserving 32-bit form, then the
// index's complement, so that no two keys are equal, ties go to the lowest index and the result does not depend on the order in
// which candidates arrive. They join two by two, each in an exchange and a bitonic merge.
//
// A token's rank is counted where a thread's values reach it: in 16 bits two values per
// instruction, against the token's value or, before its place, the one below it.
//
// Bound by memory: a row is read once, through a ring of asynchronous copies in
// which a thread finds what it has asked for itself; in 16 bits the exponentials (16 per
// clock and SM) take three quarters of the time that the loads do. Few rows are cut over
// a cluster of up to eight blocks that join in distributed shared memory.
#include "cluster.cuh"
#include "kv8.cuh"

#include <type_traits>

namespace qmv {
namespace {

using namespace cluster;
using kv8::follow_previous;

constexpr int kManyThreads = 256, kFewThreads = 512;
constexpr int kMaxCluster = 8;   // the largest cluster that every device of this kind schedules
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Args {
  const void* x;
  const int32_t* tokens;
  float* logprob;
  int32_t* rank;
  float* lse;
  float* entropy;
  int32_t* top_index;
  float* top_logprob;
  int* err;
  int64_t ldx;
  int32_t V, top, cluster, piece;   // piece: values of a block, a multiple of a vector
  float scale, scale2, most;        // scale2 = scale * log2 e; most: see Scale
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// m: the largest value; s = sum 2^d and u = sum 2^d d with d the distance of a value from m.
struct Sums {
  float m, s, u;
};

// Half of v - m: the whole may pass fp32's range where its product with a small scale does not.
__device__ __forceinline__ float half_difference(float v, float m) { return fmaf(v, 0.5f, -0.5f * m); }

// Sums are taken against the rounded product of a largest value with scale2 as long as its magnitude is at most `most` (-1: never),
// else against the value itself.
struct Scale {
  float scale2, most;
  __device__ __forceinline__ bool plain(float m) const { return fabsf(m) <= most; }
  // distance in powers of 2 between what the sums of v and of m were taken against; a product that was not rounded is not here either
  __device__ __forceinline__ float between(float v, float m) const {
    const float pv = __fmul_rn(v, scale2), pm = __fmul_rn(m, scale2);
    if (plain(fmaxf(fabsf(v), fabsf(m)))) return __fsub_rn(pv, pm);
    return plain(m) ? fmaf(v, scale2, -pm) : plain(v) ? -fmaf(m, scale2, -pv) : half_difference(v, m) * (2.f * scale2);
  }
};
constexpr float kPlainProduct = 2147483648.f;   // 2^31

// The sum of the lanes' parts, in every lane.
__device__ __forceinline__ Sums join(Sums t, const Scale& k) {
  float m = t.m;
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  if (t.s != 0.f) {
    const float d = k.between(t.m, m), f = exp2_fast(d);
    // a part whose factor is 0 leaves nothing (or its NaN): -inf * 0 would be NaN
    t.u = f == 0.f ? t.s * 0.f : (t.u + d * t.s) * f;
    t.s *= f;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, d);
    t.u += __shfl_xor_sync(0xFFFFFFFFu, t.u, d);
  }
  return {m, t.s, t.u};
}

// Pairs of fp32 in one instruction each.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ void parts(Pair p, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p)); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Values in an order-preserving form: NaN as -inf, -0 as 0. Never 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  x = fmaxf(x, -INFINITY) + 0.f;
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o); }

using Key = unsigned long long;   // order_of(value) << 32 | ~index; 0: none
__device__ __forceinline__ Key key_of(float x, int i) { return (Key)order_of(x) << 32 | (uint32_t)~i; }

// Lanes' keys, largest first.
__device__ __forceinline__ Key step(Key k, int j, bool larger) {
  const Key o = __shfl_xor_sync(0xFFFFFFFFu, k, j);
  return (k > o) == larger ? k : o;
}
__device__ __forceinline__ Key merge_down(Key k, int lane) {
#pragma unroll
  for (int j = 16; j; j >>= 1) k = step(k, j, (lane & j) == 0);
  return k;
}
__device__ __forceinline__ Key sort_down(Key k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int j = n / 2; j; j >>= 1) k = step(k, j, ((lane & j) == 0) == ((lane & n) == 0 || n == 32));
  return k;
}
// The 32 largest of two lists.
__device__ __forceinline__ Key join_lists(Key a, Key b, int lane) {
  const Key r = __shfl_sync(0xFFFFFFFFu, b, 31 - lane);
  return merge_down(a > r ? a : r, lane);
}

// Lanes' values, largest first.
__device__ __forceinline__ uint32_t sort_down32(uint32_t k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int j = n / 2; j; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, k, j);
      k = ((lane & j) == 0) == ((lane & n) == 0 || n == 32) ? max(k, o) : min(k, o);
    }
  return k;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// Sixteen bytes of a row. In 16 bits lift puts a value in the place of -inf (and of what is below it) that is so far below `-most` that
// its power is 0, so that no distance is infinite; kMost: what `most` is held to for that.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr float kMost = INFINITY;
  static __device__ __forceinline__ void values(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ float largest(const uint4& w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ void lift(uint4&) {}     // done on the distances
  using Bound = float;
  static __device__ __forceinline__ Bound bound(float x) { return x; }
  static __device__ __forceinline__ Bound below(float x) {    // the value before x, which is neither 0 nor -inf
    return __uint_as_float(__float_as_uint(x) + (x > 0.f ? -1 : 1));
  }
  static __device__ __forceinline__ int over(const uint4& w, Bound b) {
    return (__uint_as_float(w.x) > b) + (__uint_as_float(w.y) > b) + (__uint_as_float(w.z) > b) + (__uint_as_float(w.w) > b);
  }
  static __device__ __forceinline__ float value(const uint4& w, int i) {
    return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
  }
  static __device__ __forceinline__ void put(uint4& w, int i, float x) {
    const uint32_t b = __float_as_uint(x);
    if (i == 0) w.x = b; else if (i == 1) w.y = b; else if (i == 2) w.z = b; else w.w = b;
  }
};
template <typename T, typename T2>
struct Vec16 {
  static constexpr int kN = 8;
  static __device__ __forceinline__ T2 two(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
  static __device__ __forceinline__ float largest(const uint4& w) {
    const T2 m = __hmax2(__hmax2(two(w.x), two(w.y)), __hmax2(two(w.z), two(w.w)));
    return fmaxf(to_f(m.x), to_f(m.y));
  }
  using Bound = T2;
  static __device__ __forceinline__ Bound bound(float x) { return T2(T(x), T(x)); }
  static __device__ __forceinline__ Bound below(float x) {
    T h = T(x);
    *reinterpret_cast<uint16_t*>(&h) += x > 0.f ? -1 : 1;
    return T2(h, h);
  }
  static __device__ __forceinline__ int over(const uint4& w, Bound b) {
    const T2 n = __hadd2(__hadd2(__hgt2(two(w.x), b), __hgt2(two(w.y), b)), __hadd2(__hgt2(two(w.z), b), __hgt2(two(w.w), b)));
    return (int)(to_f(n.x) + to_f(n.y));
  }
  static __device__ __forceinline__ float value(const uint4& w, int i) {
    const T2 h = two(i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w);
    return to_f(i & 1 ? h.y : h.x);
  }
  static __device__ __forceinline__ void put(uint4& w, int i, float x) {
    const T h = T(x);
    const uint32_t b = (uint32_t)*reinterpret_cast<const uint16_t*>(&h) << (16 * (i & 1)), keep = (i & 1) ? 0xFFFFu : 0xFFFF0000u;
    if (i < 2) w.x = (w.x & keep) | b; else if (i < 4) w.y = (w.y & keep) | b; else if (i < 6) w.z = (w.z & keep) | b; else w.w = (w.w & keep) | b;
  }
};
template <>
struct Vec<__nv_bfloat16> : Vec16<__nv_bfloat16, __nv_bfloat162> {
  static constexpr float kMost = INFINITY;                  // 2^31 / 0.05 is far enough from -1e30
  static __device__ __forceinline__ void values(const uint4& w, float (&v)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(r[i] << 16), v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t lift1(uint32_t w) {   // to -1e30 at least
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w), "r"(0xF149F149u));
    return y;
  }
  static __device__ __forceinline__ void lift(uint4& w) { w = make_uint4(lift1(w.x), lift1(w.y), lift1(w.z), lift1(w.w)); }
};
template <>
struct Vec<__half> : Vec16<__half, __half2> {
  // 5504 below it is the least value, whose power is then 0 for a scale2 of 0.05 and more
  static constexpr float kMost = 60000.f;
  static __device__ __forceinline__ void values(const uint4& w, float (&v)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint32_t lift1(uint32_t w) {   // to -65504 at least
    uint32_t y;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(w), "r"(0xFBFFFBFFu));
    return y;
  }
  static __device__ __forceinline__ void lift(uint4& w) { w = make_uint4(lift1(w.x), lift1(w.y), lift1(w.z), lift1(w.w)); }
};

constexpr int kAhead = 4, kGroups = 2;   // vectors of a thread at a time, and such groups on their way

constexpr int kFound = 64;       // candidates that are sorted at once
template <int WARPS>
struct TopShared {
  Key list[WARPS][32];
  Key lists[kMaxCluster][32];     // of the cluster's blocks, in its first
  Key found[kFound];              // candidates, in no order
  uint32_t most[WARPS][32];       // threads' largest values (order_of), each warp's and then several warps' in order
  uint16_t parts[32][32 * WARPS]; // threads' largest values in each part of what they read: the upper half of order_of
  int count;                      // of candidates
};
// The 32 largest of two lists of values.
__device__ __forceinline__ uint32_t join_lists32(uint32_t a, uint32_t b, int lane) {
  uint32_t k = max(a, __shfl_sync(0xFFFFFFFFu, b, 31 - lane));
#pragma unroll
  for (int j = 16; j; j >>= 1) {
    const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, k, j);
    k = (lane & j) == 0 ? max(k, o) : min(k, o);
  }
  return k;
}

// A list takes one key, the same in all lanes.
__device__ __forceinline__ Key insert(Key list, Key k, int lane) {
  const Key up = __shfl_up_sync(0xFFFFFFFFu, list, 1);
  return list > k ? list : lane == 0 || up > k ? k : up;
}

__device__ __forceinline__ void st_remote32(uint32_t p, uint32_t v) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory"); }
__device__ __forceinline__ void st_remote64(uint32_t p, Key v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(p), "l"(v) : "memory"); }

template <typename T, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprob_kernel(const __grid_constant__ Args a) {
  using V = Vec<T>;
  constexpr int N = V::kN, WARPS = THREADS / 32, kStep = THREADS * N * kAhead;
  __shared__ Sums sums[WARPS];
  __shared__ int aheads[WARPS];
  __shared__ Sums all_sums[kMaxCluster];                    // of the cluster's blocks, in its first
  __shared__ int all_ahead[kMaxCluster];
  __shared__ Sums total;
  __shared__ int total_ahead;
  extern __shared__ __align__(16) unsigned char row_smem[];
  TopShared<WARPS>& ts = *reinterpret_cast<TopShared<WARPS>*>(row_smem + kGroups * kAhead * THREADS * 16);   // there where TOP
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.cluster, part = C > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x / C;
  if constexpr (TOP) {
    if (tid == 0) ts.count = 0;
  }
  if (C > 1) cluster_arrive();                              // waited for before the first access to another block's memory
  follow_previous();
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  // vectors lie on 16-byte boundaries: position 0 is at or before the row's first value
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const T* base = x - skew;
  const int end = a.V + skew;                               // positions skew .. end - 1 are the row
  const int lo = part * a.piece, hi = min(end, lo + a.piece);
  const uint4* ring = reinterpret_cast<const uint4*>(row_smem) + tid;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const auto ask = [&](int g0, int place) {                 // the block's group at position g0
    const T* p = base + g0 + tid * N;
    const uint32_t to = ring_at + place * (kAhead * THREADS * 16);
    if (g0 >= skew && g0 + kStep <= hi) {
#pragma unroll
      for (int v = 0; v < kAhead; ++v) copy16(to + v * (THREADS * 16), p + v * (THREADS * N));
    } else {
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        const int at = g0 + (v * THREADS + tid) * N;
        if (at >= skew && at + N <= hi) copy16(to + v * (THREADS * 16), p + v * (THREADS * N));
      }
    }
    copies_end();
  };
  int token = -1;
  if (a.tokens) token = a.tokens[row];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) ask(lo + i * kStep, i);
  if (token >= a.V) {
    if (part == 0 && tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    token = -1;
  }
  T own_value = T(0.f);                                     // on its way, with a list, while the first values are summed
  if (token >= 0) own_value = x[token];
  const int given_at = min(hi, token + skew);               // positions before it come first among equals
  float given = INFINITY;                                   // no token: nothing to count
  bool lowest = false, counted = false;
  typename V::Bound at_given = V::bound(0.f), under_given = at_given;
  const auto know_given = [&]() {
    if (token < 0) return;
    given = fmaxf(to_f(own_value), -INFINITY);              // NaN ranks as -inf
    // given is -inf, which all values before its place precede, or an ordinary value, with one below it that compares as such
    lowest = given == -INFINITY, counted = fabsf(given) > 1e-4f;
    at_given = V::bound(given), under_given = V::below(given);
  };
  if constexpr (!TOP) know_given();                         // its wait is hidden by other blocks, and the loop leaner without it
  const Scale scale{a.scale2, fminf(a.most, V::kMost)};
  Sums t{-INFINITY, 0.f, 0.f};
  int ahead = 0;
  Key list = 0;
  int place = 0;
  // a thread's groups in up to 32 parts
  const int groups = (hi - lo + kStep - 1) / kStep, per_part = (groups + 31) / 32;
  float part_most = -INFINITY;
  int part_at = 0, in_part = 0;
  for (int g0 = lo; g0 < hi; g0 += kStep) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory");
    const bool inside = g0 >= skew && g0 + kStep <= hi;
    uint4 w[kAhead];
    float vmax[kAhead];
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      w[v] = ring[(place * kAhead + v) * THREADS];
      const int p = g0 + (v * THREADS + tid) * N;
      if (!inside && (p < skew || p + N > hi)) {            // the row's ends, value by value; -inf where there is none
#pragma unroll
        for (int i = 0; i < N; ++i) V::put(w[v], i, p + i >= skew && p + i < hi ? to_f(base[p + i]) : -INFINITY);
      }
      vmax[v] = fmaxf(V::largest(w[v]), -INFINITY);
    }
    ask(g0 + kGroups * kStep, place);
    place = place + 1 == kGroups ? 0 : place + 1;
    const float m = fmaxf(fmaxf(vmax[0], vmax[1]), fmaxf(vmax[2], vmax[3]));
    if (m > t.m) {
      if (t.s != 0.f) {
        const float d = scale.between(t.m, m), f = exp2_fast(d);
        t.u = f == 0.f ? t.s * 0.f : (t.u + d * t.s) * f;
        t.s *= f;
      }
      t.m = m;
    }
    Pair s2 = 0, u2 = 0;
    if (scale.plain(t.m) || (scale.most > 0.f && t.m == -INFINITY)) {
      const float r = t.m == -INFINITY ? 0.f : -__fmul_rn(t.m, a.scale2);
      const Pair ref2 = pair(r, r), scale2 = pair(a.scale2, a.scale2);
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        uint4 y = w[v];
        V::lift(y);
        float z[N];
        V::values(y, z);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          Pair d2 = fma2(pair(z[i], z[i + 1]), scale2, ref2);
          float d0, d1;
          parts(d2, d0, d1);
          if constexpr (N == 4) {                           // -256: its power is 0, and so is the product
            d0 = max_nan(d0, -256.f);
            d1 = max_nan(d1, -256.f);
            d2 = pair(d0, d1);
          }
          const Pair e = pair(exp2_fast(d0), exp2_fast(d1));
          s2 = add2(s2, e);
          u2 = fma2(e, d2, u2);
        }
      }
    } else {
      const float m0 = t.m == -INFINITY ? 0.f : t.m;
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        float z[N];
        V::values(w[v], z);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float d0 = max_nan(half_difference(z[i], m0) * (2.f * a.scale2), -256.f);
          const float d1 = max_nan(half_difference(z[i + 1], m0) * (2.f * a.scale2), -256.f);
          const Pair e = pair(exp2_fast(d0), exp2_fast(d1));
          s2 = add2(s2, e);
          u2 = fma2(e, pair(d0, d1), u2);
        }
      }
    }
    float s0, s1, u0, u1;
    parts(s2, s0, s1);
    parts(u2, u0, u1);
    t.s += s0 + s1;
    t.u += u0 + u1;
    if (TOP && g0 == lo) know_given();
    if (m >= given) {
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        const int p = g0 + (v * THREADS + tid) * N;
        const bool before = p + N <= given_at;
        if (counted && p >= skew && (before || p >= given_at)) {
          ahead += before && lowest ? N : V::over(w[v], before ? under_given : at_given);
        } else if (vmax[v] >= given) {
          float z[N];
          V::values(w[v], z);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float y = fmaxf(z[i], -INFINITY);
            ahead += (y > given) || (y == given && p + i >= skew && p + i < given_at);
          }
        }
      }
    }
    if constexpr (TOP) {
      part_most = in_part == 0 ? m : fmaxf(part_most, m);
      ts.parts[part_at][tid] = (uint16_t)(order_of(part_most) >> 16);
      if (++in_part == per_part) in_part = 0, ++part_at;
    }
  }

  // the block's results
  const uint32_t my_most = order_of(t.m);
  t = join(t, scale);
  ahead = __reduce_add_sync(0xFFFFFFFFu, ahead);
  if (lane == 0) {
    sums[warp] = t;
    aheads[warp] = ahead;
  }
  // Joins n (a power of two) sums, counts and lists into the last warp's t and ahead, and warp 0's list.
  const auto join_all = [&](const Sums* s, const int* c, Key (*l)[32], int n) {
    if (warp == WARPS - 1) {
      t = join(lane < n ? s[lane] : Sums{-INFINITY, 0.f, 0.f}, scale);
      ahead = __reduce_add_sync(0xFFFFFFFFu, lane < n ? c[lane] : 0);
    }
    if constexpr (TOP) {
      if (l == nullptr) return;
      for (int d = n / 2; d; d >>= 1) {
        if (warp < d) {
          list = join_lists(l[warp][lane], l[warp + d][lane], lane);
          l[warp][lane] = list;
        }
        if (d > 1) __syncthreads();
      }
    }
  };
  Key (*own)[32] = nullptr, (*others)[32] = nullptr;
  if constexpr (TOP) {
    others = ts.lists;
    // as many threads have a value of at least the k-th of their largest ones: what is below it is in no list
    uint32_t most = sort_down32(my_most, lane);
    ts.most[warp][lane] = most;
    __syncthreads();
    for (int d = WARPS / 2; d; d >>= 1) {
      if (warp < d) {
        most = join_lists32(most, ts.most[warp + d][lane], lane);
        ts.most[warp][lane] = most;
      }
      __syncthreads();
    }
    const uint32_t least_most = ts.most[0][a.top - 1];
    const float floor = value_of(least_most);
    const int vectors = groups * kAhead;                      // of a thread
    // Vector i of thread `of` at its position p, which is `end` where there is none; and which of its values are candidates.
    const auto read = [&](int i, int of, uint4& y, int& p) {
      p = lo + i / kAhead * kStep + (i % kAhead * THREADS + of) * N;
      if (i >= vectors || p >= hi || p + N <= skew) {
        p = end;
      } else if (p >= skew && p + N <= hi) {
        y = *reinterpret_cast<const uint4*>(base + p);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) V::put(y, e, p + e >= skew && p + e < hi ? to_f(base[p + e]) : -INFINITY);
      }
    };
    const auto candidates = [&](const uint4& y, int p) {
      uint32_t passes = 0;
      if (p == end || V::largest(y) < floor) return passes;
      float z[N];
      V::values(y, z);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (fmaxf(z[e], -INFINITY) >= floor && p + e >= skew && p + e < hi) passes |= 1u << e;
      return passes;
    };
    // the parts of each thread that have one, read again by its warp
    unsigned have = __ballot_sync(0xFFFFFFFFu, my_most >= least_most);
    for (; have; have &= have - 1) {
      const int of = warp * 32 + __ffs(have) - 1;
      unsigned where = __ballot_sync(0xFFFFFFFFu, lane * per_part < groups && ts.parts[lane][of] >= least_most >> 16);
      for (; where; where &= where - 1) {
        const int first = (__ffs(where) - 1) * per_part * kAhead;
        for (int i = lane; i < per_part * kAhead; i += 32) {
          uint4 y;
          int p;
          read(first + i, of, y, p);
          for (uint32_t passes = candidates(y, p); passes; passes &= passes - 1) {
            const int e = __ffs(passes) - 1, at = atomicAdd(&ts.count, 1);
            if (at >= kFound) break;
            ts.found[at] = key_of(V::value(y, e), p + e - skew);
          }
        }
      }
      // the warp as one: its lanes meet again in the next vote
      if (__any_sync(0xFFFFFFFFu, *(volatile int*)&ts.count > kFound)) break;
    }
    __syncthreads();
    const int count = ts.count;
    if (count <= kFound) {
      if (warp < 2) {
        list = 32 * warp + lane < count ? ts.found[32 * warp + lane] : 0;
        if (warp == 0 || count > 32) ts.list[warp][lane] = list = sort_down(list, lane);
      }
      if (count > 32) {
        __syncthreads();
        if (warp == 0) list = join_lists(list, ts.list[1][lane], lane);
      }
    } else {
      // more of them (equal values, or fewer than k that are not masked): each warp keeps a list, its lanes' values one by one
      own = ts.list;
      list = 0;
      Key least = 0;                                        // its k-th key
      for (int i = 0; i < vectors; i += kAhead) {
        const bool mine = ts.parts[i / kAhead / per_part][tid] >= least_most >> 16;
        if (!__any_sync(0xFFFFFFFFu, mine)) continue;
        uint4 y[kAhead];
        int p[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          p[u] = end;
          if (mine) read(i + u, tid, y[u], p[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          uint32_t passes = candidates(y[u], p[u]);
          while (__any_sync(0xFFFFFFFFu, passes != 0)) {
            const int e = __ffs(passes) - 1;
            Key k = passes ? key_of(V::value(y[u], e), p[u] + e - skew) : 0;
            passes &= passes - 1;
            if (k <= least) k = 0;
            unsigned lanes = __ballot_sync(0xFFFFFFFFu, k != 0);
            if (!lanes) continue;
            if (__popc(lanes) <= 8) {
              for (; lanes; lanes &= lanes - 1) list = insert(list, __shfl_sync(0xFFFFFFFFu, k, __ffs(lanes) - 1), lane);
            } else {
              list = join_lists(list, sort_down(k, lane), lane);
            }
            least = __shfl_sync(0xFFFFFFFFu, list, a.top - 1);
          }
        }
      }
      ts.list[warp][lane] = list;
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  join_all(sums, aheads, own, WARPS);
  if (C > 1) {
    cluster_wait();
    if (warp == WARPS - 1 && lane == 0) {
      const uint32_t p = remote(&all_sums[part], 0);
      st_remote32(p, __float_as_uint(t.m));
      st_remote32(p + 4, __float_as_uint(t.s));
      st_remote32(p + 8, __float_as_uint(t.u));
      st_remote32(remote(&all_ahead[part], 0), (uint32_t)ahead);
    }
    if constexpr (TOP) {
      if (warp == 0) st_remote64(remote(&ts.lists[part][lane], 0), list);
    }
    cluster_arrive();
    if (part != 0) return;
    cluster_wait();
    join_all(all_sums, all_ahead, others, C);
  }
  if (warp == WARPS - 1 && lane == 0) {
    total = t;
    total_ahead = ahead;
  }
  __syncthreads();
  if (warp != 0) return;
  t = total;
  ahead = total_ahead;
  // the sums against the value itself: what the product's rounding took is put back, its whole part exactly
  const float rest = scale.plain(t.m) ? fmaf(t.m, a.scale2, -__fmul_rn(t.m, a.scale2)) : 0.f, whole = rintf(rest);
  const float ln_s = fmaf(-kLn2, rest - whole, logf(ldexpf(t.s, -(int)whole)));
  const bool none = t.s == 0.f;                             // every value is -inf
  const auto log_p = [&](float v) {
    if (none) return -INFINITY;
    return v == -INFINITY ? (ln_s == ln_s ? -INFINITY : ln_s) : fmaf(half_difference(v, t.m), 2.f * a.scale, -ln_s);
  };
  if (lane == 0) {
    if (a.lse) a.lse[row] = none ? -INFINITY : fmaf(t.m, a.scale, ln_s);
    if (a.entropy) a.entropy[row] = none ? 0.f : fmaf(-kLn2, t.u / t.s - rest, ln_s);
    if (a.logprob) a.logprob[row] = token < 0 ? 0.f : log_p(given);
    if (a.rank) a.rank[row] = token < 0 ? -1 : ahead;
  }
  if constexpr (TOP) {
    if (lane < a.top && list != 0) {                        // top <= V: every one of these lanes has a key
      a.top_index[row * a.top + lane] = (int)~(uint32_t)list;
      a.top_logprob[row * a.top + lane] = log_p(value_of((uint32_t)(list >> 32)));
    }
  }
}

struct Choice {
  const void* kernel;
  size_t smem;
};
template <typename T, int THREADS>
Choice choice_of(bool top) {
  return {top ? reinterpret_cast<const void*>(logprob_kernel<T, true, THREADS>) : reinterpret_cast<const void*>(logprob_kernel<T, false, THREADS>),
          kGroups * kAhead * THREADS * 16 + (top ? sizeof(TopShared<THREADS / 32>) : 0)};
}
template <typename T>
Choice choose(bool top, bool few) {
  return few ? choice_of<T, kFewThreads>(top) : choice_of<T, kManyThreads>(top);
}

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

int logprob_run(const logprob_args* g, void* stream) {
  if (!g) return fail(QMV_ERR_ARG, "args is NULL");
  const int xs = kv8::dtype_size(g->x_type);
  if (!xs) return fail(QMV_ERR_ARG, "x_type=%d", g->x_type);
  if (g->n_rows < 0 || g->V < 1 || g->V > QMV_LOGPROB_MAX_V || g->ldx < g->V)
    return fail(QMV_ERR_ARG, "n_rows=%d V=%d ldx=%lld", g->n_rows, g->V, (long long)g->ldx);
  if (g->top < 0 || g->top > QMV_LOGPROB_MAX_TOP || g->top > g->V) return fail(QMV_ERR_ARG, "top=%d outside 0..%d or over V=%d", g->top, QMV_LOGPROB_MAX_TOP, g->V);
  if (!(g->scale > 0.f && g->scale <= 1e30f)) return fail(QMV_ERR_ARG, "scale=%g must be positive and finite", (double)g->scale);
  if (g->n_rows > 0) {
    if (!g->x) return fail(QMV_ERR_ARG, "x is NULL");
    if (!aligned16(g->x)) return fail(QMV_ERR_ALIGN, "x must be 16-byte aligned");
    if ((g->logprob || g->rank) && !g->tokens) return fail(QMV_ERR_ARG, "logprob and rank need tokens");
    if (g->top > 0 && (!g->top_index || !g->top_logprob)) return fail(QMV_ERR_ARG, "top needs top_index and top_logprob");
    const void* four[] = {g->tokens, g->logprob, g->rank, g->lse, g->entropy, g->top_index, g->top_logprob};
    for (const void* p : four)
      if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(QMV_ERR_ALIGN, "tokens and outputs must be 4-byte aligned");
  }
  if (g->n_rows == 0) return QMV_OK;
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");
  Args a;
  a.x = g->x;
  a.tokens = g->logprob || g->rank ? g->tokens : nullptr;
  a.logprob = g->logprob;
  a.rank = g->rank;
  a.lse = g->lse;
  a.entropy = g->entropy;
  a.top_index = g->top_index;
  a.top_logprob = g->top_logprob;
  a.err = err;
  a.ldx = g->ldx;
  a.V = g->V;
  a.top = g->top;
  a.scale = g->scale;
  a.scale2 = g->scale * kLog2E;
  a.most = a.scale2 >= 0.05f && a.scale2 <= 1e6f ? kPlainProduct / a.scale2 : -1.f;
  const int N = 16 / xs;
  a.cluster = 1;
  // A row is cut while there are then at most 3.5 blocks per SM, so that all are resident at once: more of them only repeat the first
  // steps of the lists and the joins. 128257 values fp32, top 5, us with 8, 4 and 2 blocks per row: 38 rows 12.3, 13.7, 17.6; 64 rows
  // 15.3, 14.5, 17.8; 100 rows 21.8, 17.5, 20.9; 150 rows 30.1, 26.4, 21.2.
  while (a.cluster < kMaxCluster && 4 * (int64_t)g->n_rows * a.cluster <= 7 * (int64_t)sm_count() && g->V / (2 * a.cluster) >= kManyThreads * N) a.cluster *= 2;
  const bool few = (int64_t)g->n_rows * a.cluster <= sm_count();   // a block per SM: twice the threads, all of a row's loads at once
  // positions of a row and of the skew before it, in vectors
  const int64_t vectors = (g->V + 2 * (int64_t)N - 2) / N;
  a.piece = (int32_t)((vectors + a.cluster - 1) / a.cluster * N);
  if ((int64_t)g->n_rows * a.cluster > INT32_MAX) return fail(QMV_ERR_UNSUPPORTED, "n_rows=%d", g->n_rows);
  const bool top = g->top > 0;
  const Choice c = g->x_type == QMV_F32 ? choose<float>(top, few) : g->x_type == QMV_BF16 ? choose<__nv_bfloat16>(top, few) : choose<__half>(top, few);
  int per_sm = 0;
  int rc = kernel_fit(c.kernel, few ? kFewThreads : kManyThreads, c.smem, &per_sm);
  if (rc) return rc;
  void* args[] = {&a};
  cudaError_t e = kv8::launch_early(c.kernel, dim3((unsigned)(g->n_rows * a.cluster)), few ? kFewThreads : kManyThreads, args, c.smem,
                                    static_cast<cudaStream_t>(stream), a.cluster);
  if (e != cudaSuccess) return cuda_fail(e, "logprob_run launch");
  return QMV_OK;
}

}  // extern "C"

// Log probabilities of given tokens, entropy, rank and top alternatives of rows
// of logits (logprob_run).
//
// One pass over a row: a thread keeps the largest value M it has seen, and with
// d_i = (x_i - M) scale log2 e the sums S = sum 2^d_i and U = sum 2^d_i d_i, which
// give lse = scale M + ln S and the entropy ln S - ln 2 U / S. The difference comes
// before the product: it overflows only to a power of 0, and a row of the type's
// lowest value is an ordinary row. Partial results of threads, warps and blocks
// join by S = sum S_p 2^D_p, U = sum (U_p + D_p S_p) 2^D_p, D_p their M less the
// largest.
//
// The top k (k <= 32) are kept by each warp as a sorted list, an entry per lane,
// of 64-bit keys: the value in an order-preserving 32-bit form, then the index's
// complement, so that no two keys are equal, ties go to the lowest index and
// the result does not depend on the order in which candidates arrive. A vector of
// loaded values whose largest does not reach the warp's k-th value (or that of
// any warp of the block) costs one vote; others push what passes into a buffer in
// shared memory, which goes into the list 32 at a time by a bitonic sort and
// merge. The first loads' lane maxima give a first threshold (the k-th largest of
// 32 of them is below k values), so that few pass from the start.
//
// Bound by memory: a row is read once. Few rows are cut over a cluster of up to
// eight blocks that join in distributed shared memory.
#include "kv8.cuh"

#include <type_traits>

namespace qmv {
namespace {

using kv8::follow_previous;

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
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
  float scale, scale2;              // scale2 = scale * log2 e
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

// m: the largest value; s = sum 2^d and u = sum 2^d d with d = (value - m) * scale2.
struct Sums {
  float m, s, u;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float scale2) {
  if (b.s == 0.f) return a;
  if (a.s == 0.f) return b;
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = (a.m - r.m) * scale2, db = (b.m - r.m) * scale2, fa = exp2_fast(da), fb = exp2_fast(db);
  // a part whose factor is 0 leaves nothing (or its NaN): -inf * 0 would be NaN
  r.s = a.s * fa + b.s * fb;
  r.u = (fa == 0.f ? a.s * 0.f : (a.u + da * a.s) * fa) + (fb == 0.f ? b.s * 0.f : (b.u + db * b.s) * fb);
  return r;
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
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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

template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
};
template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ void unpack(uint4 w, float (&v)[Vec<T>::kN]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

constexpr int kAhead = 4;         // vectors in flight per thread
constexpr int kBuffer = 32 * 8;   // candidates of one vector of a warp, at most

struct TopShared {
  Key list[kRowWarps][32];
  Key buffer[kRowWarps][kBuffer + 32];
  int count[kRowWarps];
  unsigned least;                 // the largest k-th value (order_of) that a warp of the block has seen
};

template <bool TOP>
struct Shared {
  Sums sums[kRowWarps];
  int ahead[kRowWarps];
  Sums block_sums;
  int block_ahead;
};

// A warp's list takes the buffer's keys, the last 32 of `n`.
__device__ __forceinline__ Key take(Key list, const Key* buffer, int n, int lane) {
  const int i = n - 32 + lane;
  Key k = i >= 0 ? buffer[i] : 0;
  return join_lists(list, sort_down(k, lane), lane);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ Key ld_remote64(uint32_t p) {
  Key v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(p) : "memory");
  return v;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kRowThreads, 4) logprob_kernel(const __grid_constant__ Args a) {
  constexpr int N = Vec<T>::kN;
  __shared__ Shared<TOP> sh;
  extern __shared__ __align__(16) unsigned char top_smem[];
  TopShared& ts = *reinterpret_cast<TopShared*>(top_smem);   // there where TOP
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.cluster, part = C > 1 ? (int)cluster_rank() : 0;
  const int64_t row = blockIdx.x / C;
  if constexpr (TOP) {
    if (lane == 0) ts.count[warp] = 0;
    if (tid == 0) ts.least = 0;
  }
  follow_previous();
  if constexpr (TOP) __syncthreads();
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  // vectors lie on 16-byte boundaries: position 0 is at or before the row's first value
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const T* base = x - skew;
  const int end = a.V + skew;                               // positions skew .. end - 1 are the row
  const int lo = part * a.piece, hi = min(end, lo + a.piece);
  int token = -1;
  if (a.tokens) token = a.tokens[row];
  if (token >= a.V) {
    if (part == 0 && tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    token = -1;
  }
  float given = 0.f;
  if (token >= 0) given = fmaxf(to_f(x[token]), -INFINITY);  // NaN ranks as -inf
  const int given_at = token + skew;
  Sums t{-INFINITY, 0.f, 0.f};
  int ahead = 0;
  Key list = 0, least = 0;                                  // the warp's list and its k-th key
  float floor = -INFINITY;                                  // values below it are in no list
  bool first = true;
  for (int p0 = lo + tid * N; p0 - tid * N < hi; p0 += kRowThreads * N * kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      const int p = p0 + v * kRowThreads * N;
      raw[v] = make_uint4(0, 0, 0, 0);
      if (p >= skew && p + N <= hi) raw[v] = __ldcs(reinterpret_cast<const uint4*>(base + p));
    }
    float z[kAhead][N], vmax[kAhead];
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      const int p = p0 + v * kRowThreads * N;
      unpack<T>(raw[v], z[v]);
      if (p < skew || p + N > hi) {                         // the row's ends, value by value; -inf where there is none
#pragma unroll
        for (int i = 0; i < N; ++i) z[v][i] = p + i >= skew && p + i < hi ? to_f(base[p + i]) : -INFINITY;
      }
      vmax[v] = z[v][0];
#pragma unroll
      for (int i = 1; i < N; ++i) vmax[v] = fmaxf(vmax[v], z[v][i]);
      vmax[v] = fmaxf(vmax[v], -INFINITY);
    }
    float m = vmax[0];
#pragma unroll
    for (int v = 1; v < kAhead; ++v) m = fmaxf(m, vmax[v]);
    if (m > t.m) {
      if (t.s > 0.f) {
        const float d = (t.m - m) * a.scale2, f = exp2_fast(d);
        t.u = f == 0.f ? 0.f : (t.u + d * t.s) * f;
        t.s *= f;
      }
      t.m = m;
    }
    const float ref = t.m == -INFINITY ? 0.f : -t.m;
    const Pair ref2 = pair(ref, ref), scale2 = pair(a.scale2, a.scale2);
    Pair s2 = 0, u2 = 0;
#pragma unroll
    for (int v = 0; v < kAhead; ++v)
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float d0, d1;
        parts(mul2(add2(pair(z[v][i], z[v][i + 1]), ref2), scale2), d0, d1);
        // -256: its power is 0, and so is the product
        d0 = max_nan(d0, -256.f);
        d1 = max_nan(d1, -256.f);
        const Pair e = pair(exp2_fast(d0), exp2_fast(d1));
        s2 = add2(s2, e);
        u2 = fma2(e, pair(d0, d1), u2);
      }
    float s0, s1, u0, u1;
    parts(s2, s0, s1);
    parts(u2, u0, u1);
    t.s += s0 + s1;
    t.u += u0 + u1;
    if (token >= 0 && m >= given) {
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        const int p = p0 + v * kRowThreads * N;
        if (vmax[v] < given) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float y = fmaxf(z[v][i], -INFINITY);
          const bool before = p + i >= skew && p + i < min(given_at, hi);   // of this block's, and with a lower index
          ahead += (y > given) || (y == given && before);
        }
      }
    }
    if constexpr (TOP) {
      if (first) {
        // k lanes have seen a value of at least the k-th largest of the lanes' maxima
        const Key s = sort_down((Key)order_of(m) << 32, lane);
        const unsigned o = (unsigned)(__shfl_sync(0xFFFFFFFFu, s, a.top - 1) >> 32);
        if (lane == 0) atomicMax(&ts.least, o);
        floor = value_of(o);
        first = false;
      }
      floor = fmaxf(floor, value_of(max(order_of(-INFINITY), *(volatile unsigned*)&ts.least)));
#pragma unroll
      for (int v = 0; v < kAhead; ++v) {
        const int p = p0 + v * kRowThreads * N;
        if (!__any_sync(0xFFFFFFFFu, vmax[v] >= floor)) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (fmaxf(z[v][i], -INFINITY) >= floor && p + i >= skew && p + i < hi) {
            const Key k = key_of(z[v][i], p + i - skew);
            if (k > least) ts.buffer[warp][atomicAdd(&ts.count[warp], 1)] = k;
          }
        }
        __syncwarp();
        int n = *(volatile int*)&ts.count[warp];
        if (n >= 32) {
          for (; n >= 32; n -= 32) list = take(list, ts.buffer[warp], n, lane);
          __syncwarp();
          if (lane == 0) ts.count[warp] = n;
          least = __shfl_sync(0xFFFFFFFFu, list, a.top - 1);
          if (least) {
            floor = fmaxf(floor, value_of((unsigned)(least >> 32)));
            if (lane == 0) atomicMax(&ts.least, (unsigned)(least >> 32));
          }
          __syncwarp();
        }
      }
    }
  }

  // the block's results
  if constexpr (TOP) {
    __syncwarp();
    list = take(list, ts.buffer[warp], *(volatile int*)&ts.count[warp], lane);   // fewer than 32 are left
    ts.list[warp][lane] = list;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const Sums o{__shfl_xor_sync(0xFFFFFFFFu, t.m, d), __shfl_xor_sync(0xFFFFFFFFu, t.s, d), __shfl_xor_sync(0xFFFFFFFFu, t.u, d)};
    t = join(t, o, a.scale2);
    ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, d);
  }
  if (lane == 0) {
    sh.sums[warp] = t;
    sh.ahead[warp] = ahead;
  }
  __syncthreads();
  if constexpr (TOP) {
    for (int d = kRowWarps / 2; d; d >>= 1) {
      if (warp < d) ts.list[warp][lane] = join_lists(ts.list[warp][lane], ts.list[warp + d][lane], lane);
      __syncthreads();
    }
  }
  if (warp == 0) {
    t = sh.sums[0];
    ahead = sh.ahead[0];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) {
      t = join(t, sh.sums[w], a.scale2);
      ahead += sh.ahead[w];
    }
    if constexpr (TOP) list = ts.list[0][lane];
  }
  if (C > 1) {
    if (tid == 0) {
      sh.block_sums = t;
      sh.block_ahead = ahead;
    }
    cluster_sync();
    if (part == 0 && warp == 0) {
      for (int c = 1; c < C; ++c) {
        const uint32_t p = remote(&sh.block_sums, c);
        const Sums o{__uint_as_float(ld_remote32(p)), __uint_as_float(ld_remote32(p + 4)), __uint_as_float(ld_remote32(p + 8))};
        t = join(t, o, a.scale2);
        ahead += (int)ld_remote32(remote(&sh.block_ahead, c));
        if constexpr (TOP) list = join_lists(list, ld_remote64(remote(&ts.list[0][lane], c)), lane);
      }
    }
    cluster_sync();                                         // the other blocks' memory has been read
  }
  if (part != 0 || warp != 0) return;
  const float log2_s = log2f(t.s);
  const bool none = t.s == 0.f;                             // every value is -inf
  const auto log_p = [&](float v) {
    if (none) return -INFINITY;
    return v == -INFINITY ? (log2_s == log2_s ? -INFINITY : log2_s) : fmaf(v - t.m, a.scale, -log2_s * kLn2);
  };
  if (lane == 0) {
    if (a.lse) a.lse[row] = none ? -INFINITY : fmaf(t.m, a.scale, log2_s * kLn2);
    if (a.entropy) a.entropy[row] = none ? 0.f : (log2_s - t.u / t.s) * kLn2;
    if (a.logprob) a.logprob[row] = token < 0 ? 0.f : log_p(to_f(x[token]));
    if (a.rank) a.rank[row] = token < 0 ? -1 : ahead;
  }
  if constexpr (TOP) {
    if (lane < a.top && list != 0) {                        // top <= V: every one of these lanes has a key
      const int i = (int)~(uint32_t)list;
      a.top_index[row * a.top + lane] = i;
      a.top_logprob[row * a.top + lane] = log_p(to_f(x[i]));
    }
  }
}

template <typename T>
const void* kernel_of(bool top) {
  return top ? reinterpret_cast<const void*>(logprob_kernel<T, true>) : reinterpret_cast<const void*>(logprob_kernel<T, false>);
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
  const int N = 16 / xs;
  a.cluster = 1;
  while (a.cluster < kMaxCluster && (int64_t)g->n_rows * a.cluster < 2 * sm_count() && g->V / (2 * a.cluster) >= kRowThreads * N) a.cluster *= 2;
  // positions of a row and of the skew before it, in vectors
  const int64_t vectors = (g->V + 2 * (int64_t)N - 2) / N;
  a.piece = (int32_t)((vectors + a.cluster - 1) / a.cluster * N);
  if ((int64_t)g->n_rows * a.cluster > INT32_MAX) return fail(QMV_ERR_UNSUPPORTED, "n_rows=%d", g->n_rows);
  const bool top = g->top > 0;
  const void* f = g->x_type == QMV_F32 ? kernel_of<float>(top) : g->x_type == QMV_BF16 ? kernel_of<__nv_bfloat16>(top) : kernel_of<__half>(top);
  void* args[] = {&a};
  cudaError_t e = kv8::launch_early(f, dim3((unsigned)(g->n_rows * a.cluster)), kRowThreads, args, top ? sizeof(TopShared) : 0,
                                    static_cast<cudaStream_t>(stream), a.cluster);
  if (e != cudaSuccess) return cuda_fail(e, "logprob_run launch");
  return QMV_OK;
}

}  // extern "C"

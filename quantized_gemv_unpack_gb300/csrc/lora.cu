// Low-rank adapters of many requests beside a shared projection: the step's
// grouping of tokens by adapter (lora_plan) and
//   y[t] += s_a * B_a^T (A_a x[t]),  a the adapter of token t        (lora_run).
//
// What a call has to move: x once, y in and out, the rank rows of the adapters in use; 2 r (K + N) operations per token and
// projection beside it. With few tokens per adapter the rank rows are most of it, with many y is. Both products run on what
// lies in memory as it is:
// * few tokens (lora_short_kernel): one launch. A cluster of blocks takes a tile of up to 16 tokens of one adapter and one
//   projection, each block a share of K in the first product and of N in the second; the sums between them meet in
//   distributed shared memory and never leave the chip. mma.sync m16n8k16, bf16 with fp32 sums.
// * many tokens (lora_first_kernel, lora_second_kernel): two launches with the finished values between them in the caller's
//   workspace. The first product is one of the fifth-generation tensor cores, 128 tokens by the rank; the second, whose y in and
//   out is the call's bulk, is mma.sync with B in registers and y through rings of asynchronous copies.
// In the mma.sync products operands are whole pieces of rows:
// * first product: a lane's 16 bytes of a row of x and of a row of A are eight consecutive k. A contraction may take its
//   index in any order, so these are the lane's pairs of two k16 steps: no shuffle.
// * second product: a lane's 8 bytes of a row of B are four consecutive n of one rank row; two rows zipped by byte permutes
//   are the pairs of four n8 blocks, so that a lane's sums are two runs of four columns of y (fp32), or one of eight (16 bits).
// The r values between the products are fp32 sums, handed on as bf16 parts, each the rounding of what the ones before it have
// left: three for an fp32 y, which hold all 24 bits, two for a 16-bit y, which leave 2^-17 (what the first leaves is below 2^-8 of the
// value's power of two, and rounded by half a step of at most 2^-17), where y itself is rounded to 2^-8 or 2^-11. One part would put
// 2^-8 of the adapter's whole product on y.
//
// Measured, us per call in a stream of calls (bytes that have to be moved, at their rate): one token of rank 16, K = N = 4096 5.1;
// 64 tokens of 48 adapters of ranks up to 64, K 5120, q|k|v 26 (75 MB, 2.9 TB/s); 80 of 12, rank 16, gate|up 12.6 (33 MB, 2.6 TB/s);
// 1023 of 24, ranks up to 128, K 13824, N 5120 57 (137 MB, 2.4 TB/s); 8190 of 5, rank 64, gate|up, bf16 188 (918 MB, 4.9 TB/s).
#include <type_traits>

#include "cluster.cuh"
#include "kv8.cuh"
#include "tcgen05.cuh"

namespace qmv {
namespace {

using namespace cluster;
using kv8::follow_previous;

constexpr int kMaxAdapters = QMV_LORA_MAX_ADAPTERS;
constexpr int kMaxRank = QMV_LORA_MAX_RANK;
constexpr int kSmallTile = 16, kLargeTile = 64;

// ----------------------------------------------------------------------------- plan

// A stable counting sort by one block. Each warp takes a range of the tokens and
// counts them per adapter, 32 at a time (lanes of one adapter find each other by
// a match, the first of them adds); sums over the warps, then over the adapters,
// give each warp its place per adapter. What a token finds in its warp's counter is
// its place among the warp's, kept in a register where a lane has at most 16 tokens,
// else found again in a second pass.
// Measured: 64 tokens of 48 adapters 3.0 us, 16384 tokens of 512 adapters 7.9 us.
constexpr int kPlanAhead = 16;   // tokens of a lane whose loads are in flight at once

__device__ __forceinline__ int scan_add(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

struct PlanArgs {
  const int32_t* ids;
  int32_t* order;
  int4* tiles;
  int* err;
  int n_tokens, n_adapters, tile, max_tiles;
};

__global__ void __launch_bounds__(1024) lora_plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const int A = a.n_adapters, T = a.n_tokens;
  int32_t* first = plan_smem;         // [A + 1] first place of an adapter's tokens
  int32_t* tile0 = first + A + 1;     // [A + 1] its first tile
  int32_t* hist = tile0 + A + 1;      // [warps][A]
  __shared__ int2 sums[32];
  for (int i = tid; i < warps * A; i += threads) hist[i] = 0;
  follow_previous();
  __syncthreads();
  const int chunk = ((T + warps - 1) / warps + 31) / 32 * 32;
  const int lo = min(T, warp * chunk), hi = min(T, lo + chunk);
  int32_t* mine = hist + warp * A;
  bool bad = false;
  // The warp's tokens from t0 on, 16 to a lane: each one's adapter and its place among the warp's tokens of it, or -1.
  const auto count = [&](int t0, int (&id)[kPlanAhead], int (&at)[kPlanAhead]) {
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      const int t = t0 + 32 * u + lane;
      id[u] = t < hi ? a.ids[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      if (t0 + 32 * u >= hi) break;
      bad |= id[u] >= A;
      if (id[u] >= A) id[u] = -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, id[u]);
      if (id[u] >= 0) at[u] = mine[id[u]] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (id[u] >= 0 && lane == __ffs(same) - 1) mine[id[u]] += __popc(same);
      __syncwarp();
    }
  };
  int id[kPlanAhead], at[kPlanAhead];
  const bool once = chunk <= 32 * kPlanAhead;
  if (once) {
    count(lo, id, at);
  } else {
    for (int t0 = lo; t0 < hi; t0 += 32 * kPlanAhead) count(t0, id, at);
  }
  if (bad) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
  __syncthreads();
  // per adapter: its warps' counts to their exclusive sums; then sums over the adapters, `threads` of them at a time
  int2 base = make_int2(0, 0);
  for (int a0 = 0; a0 < A; a0 += threads) {
    const int k = a0 + tid;
    int n = 0;
    if (k < A)
      for (int w = 0; w < warps; w += 8) {                    // warps is a multiple of eight
        int c[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) c[u] = hist[(w + u) * A + k];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          hist[(w + u) * A + k] = n;
          n += c[u];
        }
      }
    const int tiles = (n + a.tile - 1) / a.tile;
    const int sn = scan_add(n, lane), st = scan_add(tiles, lane);
    if (lane == 31) sums[warp] = make_int2(sn, st);
    __syncthreads();
    const int2 of = lane < warps ? sums[lane] : make_int2(0, 0);
    const int before_x = scan_add(of.x, lane), before_y = scan_add(of.y, lane);   // up to and with each warp's
    const int2 before = make_int2(base.x + __shfl_sync(0xFFFFFFFFu, before_x - of.x, warp), base.y + __shfl_sync(0xFFFFFFFFu, before_y - of.y, warp));
    const int2 all = make_int2(base.x + __shfl_sync(0xFFFFFFFFu, before_x, 31), base.y + __shfl_sync(0xFFFFFFFFu, before_y, 31));
    if (k < A) {
      first[k] = before.x + sn - n;
      tile0[k] = before.y + st - tiles;
    }
    base = all;
    __syncthreads();
  }
  if (tid == 0) {
    first[A] = base.x;
    tile0[A] = base.y;
  }
  __syncthreads();
  for (int t0 = lo; t0 < hi; t0 += 32 * kPlanAhead) {
    if (!once) count(t0, id, at);                             // from the counters that the sums have left
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      if (t0 + 32 * u >= hi) break;
      if (id[u] >= 0) a.order[first[id[u]] + at[u] + (once ? mine[id[u]] : 0)] = t0 + 32 * u + lane;
    }
  }
  for (int t = base.x + tid; t < T; t += threads) a.order[t] = -1;
  for (int i = tid; i < a.max_tiles; i += threads) {
    int4 v = make_int4(0, 0, 0, 0);
    if (i < base.y) {
      int l = 0, h = A;   // the last adapter whose first tile is not past i: the one that has it
      while (h - l > 1) {
        const int m = (l + h) >> 1;
        if (tile0[m] <= i) l = m;
        else h = m;
      }
      const int at = (i - tile0[l]) * a.tile;
      v = make_int4(l, first[l] + at, min(a.tile, first[l + 1] - first[l] - at), 0);
    }
    a.tiles[i] = v;
  }
}

// ----------------------------------------------------------------------------- run

constexpr int kCluster = 8;    // blocks of a tile: the largest cluster that every device of this kind schedules
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;

struct Task {
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  void* y;
  int64_t lda, ldb, ldy;
  int32_t N;
  int32_t wide;                // rows of y are 16-byte aligned
};

struct RunArgs {
  const __nv_bfloat16* x;
  const int32_t* order;
  const int32_t* table;
  const int4* tiles;
  const float* scale;
  int* err;
  int64_t ldx;
  int32_t K, n_tokens, n_adapters, pool_rows, max_tiles, n_tasks, cluster, tile, window, window2, slices;
  uint4* values;               // many tokens: what lies between the products, as the second one takes it
  Task t[QMV_LORA_MAX_TASKS];
};

__device__ __forceinline__ bool tile_fits(const RunArgs& a, const int4& v) {
  return v.x >= 0 && v.x < a.n_adapters && v.y >= 0 && v.z > 0 && v.z <= a.tile && v.y <= a.n_tokens - v.z;
}
__device__ __forceinline__ float4 sum(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ void st_remote(uint32_t p, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t p, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float4 ld_remote(uint32_t p) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two fp32 values as three bf16 pairs: the values, and twice what is left. An infinite or NaN value leaves nothing.
__device__ __forceinline__ uint32_t split(float& x, float& y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float hx = __low2float(h), hy = __high2float(h);
  x = fabsf(hx) <= 3.3e38f ? x - hx : 0.f;
  y = fabsf(hy) <= 3.3e38f ? y - hy : 0.f;
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Words of the values between the products, whose columns are rank rows j, j + 1, j, j + 1: 0 past the rank. There the first product
// has multiplied zeros, which an infinite value of x makes NaN.
__device__ __forceinline__ void keep_rank(float4& v, int j, int r) {
  if (j >= r) v.x = v.z = 0.f;
  if (j + 1 >= r) v.y = v.w = 0.f;
}

template <int Y>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (Y == QMV_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int Y>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (Y == QMV_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's values of a row of y: one piece of 16 bytes, or two: 512 bytes apart in a ring, 64 in y.
template <int WORDS>
__device__ __forceinline__ void ld_pieces(const unsigned char* p, uint32_t (&w)[WORDS]) {
#pragma unroll
  for (int i = 0; i < WORDS; i += 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + 128 * i);
    w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
  }
}
template <int WORDS>
__device__ __forceinline__ void st_pieces(char* p, const uint32_t (&w)[WORDS]) {
#pragma unroll
  for (int i = 0; i < WORDS; i += 4) *reinterpret_cast<uint4*>(p + 16 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}
// Where a lane's columns of 32 lie: eight consecutive ones in 16 bits, else four and, 16 columns on, four more, so that each access
// of a warp has whole sectors; and, per column of an n8 block of the products, the first of its four.
template <int Y>
__device__ __forceinline__ int own_column(int t4) { return Y == QMV_F32 ? 4 * t4 : 8 * t4; }
template <int Y>
__device__ __forceinline__ int block_column(int g) { return Y == QMV_F32 ? 16 * (g & 1) + 4 * (g >> 1) : 4 * g; }
// The sum of column c of the 2 * BLOCKS that a lane has of row HI (g or g + 8): block c % BLOCKS, half c / BLOCKS.
template <int HI, int BLOCKS>
__device__ __forceinline__ float column(const float (&d)[BLOCKS][4], int c) {
  return d[c % BLOCKS][2 * HI + c / BLOCKS];
}
// y += s * d over a lane's columns, whose values are w.
template <int Y, int HI, int BLOCKS, int WORDS>
__device__ __forceinline__ void add_row(char* p, float s, const float (&d)[BLOCKS][4], uint32_t (&w)[WORDS]) {
  if constexpr (Y == QMV_F32) {
#pragma unroll
    for (int c = 0; c < WORDS; ++c) w[c] = __float_as_uint(fmaf(s, column<HI>(d, c), __uint_as_float(w[c])));
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      const float2 v = unpack2<Y>(w[i]);
      w[i] = pack2<Y>(fmaf(s, column<HI>(d, 2 * i), v.x), fmaf(s, column<HI>(d, 2 * i + 1), v.y));
    }
  }
  st_pieces(p, w);
}
// The same value by value, up to column n from the first of them on.
template <int Y, int HI, int BLOCKS>
__device__ __forceinline__ void add_row_part(void* p, int n, float s, const float (&d)[BLOCKS][4]) {
#pragma unroll
  for (int c = 0; c < 2 * BLOCKS; ++c) {
    const int at = Y == QMV_F32 ? c % 4 + c / 4 * 16 : c;
    if (at >= n) break;
    const float v = column<HI>(d, c);
    if constexpr (Y == QMV_F32) {
      float* q = static_cast<float*>(p) + at;
      *q = fmaf(s, v, *q);
    } else if constexpr (Y == QMV_BF16) {
      __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + c;
      *q = __float2bfloat16_rn(fmaf(s, v, __bfloat162float(*q)));
    } else {
      __half* q = static_cast<__half*>(p) + c;
      *q = __float2half_rn(fmaf(s, v, __half2float(*q)));
    }
  }
}

// Infinite values of B. A value between the products is a sum of bf16 parts, and the parts after the first may be 0 or of the other
// sign: each of them times an infinite value of B is NaN, where the value itself gives an infinity. Where there are any, the values
// of B that are not finite meet the values between the products as a whole, one by one.

// The largest of three, NaN if one is.
__device__ __forceinline__ float most(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Few tokens: a lane's sums of the second product that are NaN, once more, value by value: rank rows j < r of b, from the lane's first
// column on, with the parts of rows g and g + 8 as the fragments have them. One look at the sums per step of 32 columns costs a token
// of rank 16 (K = N = 4096) 0.1 of 5.1 us.
template <int Y, int P3>
__device__ __noinline__ void sums_again(float* d, const uint4* frag, const __nv_bfloat16* b, int64_t ldb, int r, int cols, int lane) {
  const uint32_t* parts = reinterpret_cast<const uint32_t*>(frag);
  for (int c = 0; c < 8; ++c) {
    const int at = Y == QMV_F32 ? c % 4 + c / 4 * 16 : c;
    if (at >= cols) break;
    for (int hi = 0; hi < 2; ++hi) {
      float* to = d + c % 4 * 4 + 2 * hi + c / 4;
      if (*to == *to) continue;
      float sum = 0.f;
      for (int j = 0; j < r; ++j) {
        const float w = __bfloat162float(b[j * ldb + at]);
        for (int k = P3 - 1; k >= 0; --k) {
          const uint32_t two = parts[((j / 16 * P3 + k) * 32 + lane / 4 * 4 + j % 8 / 2) * 4 + j % 16 / 8 * 2 + hi];
          const float h = __uint_as_float(j & 1 ? two & 0xFFFF0000u : two << 16);
          if (k == 0 || fabsf(w) < INFINITY) sum = fmaf(h, w, sum);
        }
      }
      *to = sum;
    }
  }
}

// Many tokens: in B's registers +-1 stands for a value that is not finite, so that an infinite value between keeps its sign, and what
// it stands for is added to y afterwards (B with 0 in its place beside B itself, for the later parts, took registers that the
// second kernel does not have: 4096 tokens, rank 128, fp32 169 -> 206 us).
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w = (w & 0xFFFF8000u) | 0x3F80u;
  if ((w & 0x7F800000u) == 0x7F800000u) w = (w & 0x8000FFFFu) | 0x3F800000u;
  return w;
}
// A lane's column, of `count` tokens whose rows of y are row_y bytes away; values: the finished values of the run, KS * P3 * 32 words for
// each 16 tokens.
template <int Y, int KS, int P3>
__device__ __noinline__ void add_infinite(char* y, const int64_t* row_y, int count, const uint4* values, const __nv_bfloat16* b, int64_t ldb,
                                          int r, float scale) {
  const uint32_t* parts = reinterpret_cast<const uint32_t*>(values);
  for (int j = 0; j < r; ++j) {
    const float w = __bfloat162float(b[j * ldb]);
    if (fabsf(w) < INFINITY) continue;
    for (int i = 0; i < count; ++i) {
      if (row_y[i] < 0) continue;
      float h = 0.f;
      for (int k = P3 - 1; k >= 0; --k) {
        const uint32_t two = parts[(((int64_t)(i / 16 * KS + j / 16) * P3 + k) * 32 + i % 8 * 4 + j % 8 / 2) * 4 + j % 16 / 8 * 2 + i % 16 / 8];
        h += __uint_as_float(j & 1 ? two & 0xFFFF0000u : two << 16);
      }
      char* q = y + row_y[i];
      if constexpr (Y == QMV_F32) {
        *reinterpret_cast<float*>(q) += scale * (h * w);
      } else if constexpr (Y == QMV_BF16) {
        *reinterpret_cast<__nv_bfloat16*>(q) = __float2bfloat16_rn(__bfloat162float(*reinterpret_cast<__nv_bfloat16*>(q)) + scale * (h * w));
      } else {
        *reinterpret_cast<__half*>(q) = __float2half_rn(__half2float(*reinterpret_cast<__half*>(q)) + scale * (h * w));
      }
    }
  }
}

// ---- few tokens of an adapter
//
// A cluster takes up to 16 tokens of a tile. Each warp streams through its own ring of asynchronous copies: k32 steps of x and
// A, then 32-column steps of B and y, of which the first are on their way while the sums of the first product meet. A warp
// copies just what its own fragments need, so a step needs no barrier of the block (B in pieces of 16 bytes, which a lane
// shares with others of its warp: 64 tokens of 48 adapters 26 us, with 8-byte pieces of its own 30).
// Bound by a unit's chain: its tile, table and tokens (1.1 us), the first loads, the meeting (2.5 us) and the steps, two or
// three of which a warp has in flight; beyond 16 tokens per adapter also by L2, from which every tile reads its rank rows again. NB blocks
// of eight rank rows (the call's largest rank).
template <int NB, int Y>
struct Short {
  static constexpr bool F32 = Y == QMV_F32;
  static constexpr int kParts3 = F32 ? 3 : 2;                 // bf16 parts of the values between the products
  static constexpr int kSteps = NB / 2;                       // k16 steps of the second product
  static constexpr int kHalves = NB > 8 ? 2 : 1;              // in the first product a warp has at most 64 rank rows
  static constexpr int kParts = kLoraWarps / kHalves;         // and a share of the columns of x
  static constexpr int kBlocks = NB / kHalves;
  static constexpr int kWords = kSteps * 64;                  // 16-byte words of the tile's r values, in the order of the fragments
  static constexpr int kPieces = NB > 8 ? 4 : 1;              // steps that 32 columns of B take, so that a slot is no larger than the first product needs
  static constexpr int kFirst = (kBlocks + 2) * 512, kB = kSteps / kPieces * 1024, kSecond = kB + (F32 ? 2048 : 1024);
  static constexpr int kSlot = kFirst > kSecond ? kFirst : kSecond;
  static constexpr int kDepth = NB == 2 ? 4 : NB == 4 ? 3 : 2;   // what two blocks of an SM have room for
  // Whether the blocks of a cluster share the work on its sums (two exchanges) or each reads all of them (one). us: 256 tokens of 4
  // adapters, rank 128, K = N = 4096 16.8 and 20.3; 1000 tokens of rank 64, K = N = 5120 27.7 and 29.8; 1023 tokens of 8 adapters, rank
  // 32, q|k|v 28.2 and 27.2; one token of rank 16, K = N = 4096 5.0 and 4.8.
  static constexpr bool kShared = NB > 4;
  static constexpr int kFixed = kWords * 16 + kSteps * kParts3 * 512 + kLoraWarps * (int)sizeof(int);
  static constexpr int kSmem = kFixed + kLoraWarps * kDepth * kSlot;
};

template <int NB, int Y>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_short_kernel(const __grid_constant__ RunArgs a) {
  using S = Short<NB, Y>;
  constexpr int KS = S::kSteps, W = S::kWords, RB = S::kBlocks, P3 = S::kParts3, size = Y == QMV_F32 ? 4 : 2, WORDS = 2 * size, D = S::kDepth, KH = KS / S::kPieces;
  constexpr bool F32 = S::F32;
  extern __shared__ __align__(16) unsigned char lora_smem[];
  float4* mine = reinterpret_cast<float4*>(lora_smem);        // kShared: [C][2][W / 2 / C], the blocks' sums of this block's items; else [W], its own sums
  uint4* frag = reinterpret_cast<uint4*>(mine + W);           // [KS][P3][32]: the parts of the finished values
  int* sums_in = reinterpret_cast<int*>(frag + KS * P3 * 32); // [kLoraWarps]: the slot in which a warp left its sums
  unsigned char* rings = lora_smem + S::kFixed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int half = warp % S::kHalves, part = warp / S::kHalves;
  const int rank = (int)cluster_rank(), C = a.cluster, clusters = gridDim.x / C;
  unsigned char* ring = rings + warp * (D * S::kSlot);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  // B: eight rank rows of 64 bytes, the even ones and then the odd ones, each piece where neither its copy nor the reads of
  // the lane's four columns of rows 2 t4 and 2 t4 + 1 meet another lane's bank
  constexpr int kTurn = F32 ? 1 : 2;
  const int b_col = block_column<Y>(g);
  const int b_to = (g & 1) * 256 + ((g >> 1) ^ (g & 1)) * 64 + ((t4 ^ (g >> 2) * kTurn) * 16);
  const int b_even = t4 * 64 + ((b_col >> 3) ^ (t4 >> 1) * kTurn) * 16 + (b_col & 4) * 2, b_odd = 256 + (b_even ^ 64);
  const int j0 = half * 8 * RB;                               // this warp's first rank row in the first product
  if constexpr (S::kShared) cluster_arrive();
  follow_previous();
  bool waiting = S::kShared;                                  // for the cluster: to have begun, or to have read `mine`
  const int sixteens = a.tile / 16, units = a.max_tiles * sixteens;   // of a projection: a unit takes 16 tokens of a tile
  for (int unit = blockIdx.x / C; unit < units * a.n_tasks; unit += clusters) {
    const Task& t = a.t[unit / units];
    int4 tile = a.tiles[unit % units / sixteens];              // units of a tile side by side: the first finds its rank rows for all
    if (tile.z == 0) continue;
    const bool fits = tile_fits(a, tile);
    const int skip = unit % sixteens * 16;
    if (skip > 0 && (!fits || skip >= tile.z)) continue;      // a bad tile is reported by the first of its units
    tile.y += skip;
    tile.z = min(16, tile.z - skip);
    int row0 = 0, r = 0, tok0 = -1, tok1 = -1;                // this lane's tokens: rows g and g + 8 of the tile
    float scale = 0.f;
    if (fits) {
      if (g < tile.z) tok0 = a.order[tile.y + g];
      if (g + 8 < tile.z) tok1 = a.order[tile.y + g + 8];
      row0 = a.table[2 * tile.x];
      r = a.table[2 * tile.x + 1];
      scale = a.scale[tile.x];
    }
    if (!fits || row0 < 0 || r < 0 || r > 8 * NB || row0 > a.pool_rows - r) {
      if (rank == 0 && tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
      continue;
    }
    if (r == 0) continue;
    if ((g < tile.z && (tok0 < 0 || tok0 >= a.n_tokens)) || (g + 8 < tile.z && (tok1 < 0 || tok1 >= a.n_tokens))) {
      atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
      if (tok0 >= a.n_tokens) tok0 = -1;
      if (tok1 >= a.n_tokens) tok1 = -1;
    }
    __syncthreads();                                          // the unit before this one is done with frag and the rings
    const __nv_bfloat16* x0 = a.x + (int64_t)(tok0 < 0 ? 0 : tok0) * a.ldx;
    const __nv_bfloat16* x1 = a.x + (int64_t)(tok1 < 0 ? 0 : tok1) * a.ldx;
    char* y0 = static_cast<char*>(t.y) + (int64_t)(tok0 < 0 ? 0 : tok0) * t.ldy * size;
    char* y1 = static_cast<char*>(t.y) + (int64_t)(tok1 < 0 ? 0 : tok1) * t.ldy * size;

    // this block's columns of both products, and this warp's steps of them
    const int k_share = (a.K + C * 32 - 1) / (C * 32) * 32, n_share = (t.N + C * 32 - 1) / (C * 32) * 32;
    const int k_lo = rank * k_share, k_hi = min(a.K, k_lo + k_share), n_lo = rank * n_share, n_hi = min(t.N, n_lo + n_share);
    int k_next = k_lo + part * 32, n_next = n_lo + warp * 32, piece_next = 0, slot_in = 0, slot = 0;
    const __nv_bfloat16* pa = t.a + (int64_t)(row0 + j0 + g) * t.lda + 8 * t4;
    const __nv_bfloat16* pb = t.b + (int64_t)(row0 + g) * t.ldb + 8 * t4;
    const int64_t step_b = 8 * t.ldb;
    const int64_t step_a = 8 * t.lda;
    const auto ask = [&]() {
      const uint32_t to = ring_at + slot_in * S::kSlot + lane * 16;
      if (k_next < k_hi) {
        const int k = k_next + 8 * t4;
        if (k < k_hi) {
          if (tok0 >= 0) copy16(to, x0 + k);
          if (tok1 >= 0) copy16(to + 512, x1 + k);
          const __nv_bfloat16* p = pa + k_next;
#pragma unroll
          for (int i = 0; i < RB; ++i, p += step_a)
            if (j0 + 8 * i + g < r) copy16(to + 1024 + i * 512, p);
        }
        k_next += S::kParts * 32;
      } else if (n_next < n_hi) {
        const int col = n_next + 8 * t4, n = n_next + own_column<Y>(t4);
        if (col < t.N) {
          const __nv_bfloat16* p = pb + n_next + (int64_t)(16 * KH * piece_next) * t.ldb;
          const uint32_t at = slot_in * S::kSlot + b_to;
#pragma unroll
          for (int i = 0; i < 2 * KH; ++i, p += step_b) {
            if (16 * KH * piece_next + 8 * i + g >= r) continue;
            if (col + 8 <= t.N) {
              copy16(ring_at + at + i * 512, p);
            } else {                                          // the row's last values, one by one
              const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
              uint16_t* d = reinterpret_cast<uint16_t*>(ring + at + i * 512);
              for (int c = 0; c < 8; ++c) d[c] = col + c < t.N ? e[c] : (uint16_t)0;
            }
          }
        }
        const bool last = ++piece_next == S::kPieces;         // y comes with the last rank rows
        if (last) piece_next = 0;
        if (last && t.wide && (F32 ? n_next + 32 : n + 8) <= t.N) {
          if (tok0 >= 0) {
            copy16(to + S::kB, y0 + (int64_t)n * size);
            if constexpr (F32) copy16(to + S::kB + 512, y0 + (int64_t)n * size + 64);
          }
          if (tok1 >= 0) {
            copy16(to + S::kB + 256 * size, y1 + (int64_t)n * size);
            if constexpr (F32) copy16(to + S::kB + 256 * size + 512, y1 + (int64_t)n * size + 64);
          }
        }
        if (last) n_next += kLoraWarps * 32;
      }
      copies_end();
      slot_in = slot_in + 1 == D ? 0 : slot_in + 1;
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) ask();

    // ---- first product, over this block's share of K
    float acc[RB][4];
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    for (int k0 = k_lo + part * 32; k0 < k_hi; k0 += S::kParts * 32) {
      ask();
      asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      const unsigned char* st = ring + slot * S::kSlot + lane * 16;
      slot = slot + 1 == D ? 0 : slot + 1;
      const bool in = k0 + 8 * t4 < k_hi;
      uint4 p = make_uint4(0, 0, 0, 0), o = p;
      if (in && tok0 >= 0) p = *reinterpret_cast<const uint4*>(st);
      if (in && tok1 >= 0) o = *reinterpret_cast<const uint4*>(st + 512);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (j0 + 8 * i >= r) break;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in && j0 + 8 * i + g < r) w = *reinterpret_cast<const uint4*>(st + 1024 + i * 512);
        mma(acc[i], p.x, o.x, p.y, o.y, w.x, w.y);
        mma(acc[i], p.z, o.z, p.w, o.w, w.z, w.w);
      }
    }
    // the sums of the block's warps, each by way of its ring's free slot
    {
      float4* to = reinterpret_cast<float4*>(ring + slot_in * S::kSlot) + lane;
#pragma unroll
      for (int i = 0; i < RB; ++i) to[i * 32] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      if (lane == 0) sums_in[warp] = slot_in * S::kSlot;
    }
    __syncthreads();
    if (waiting) cluster_wait();
    // The cluster's sums, of which every block needs all. An item is a lane's eight values of one k16 step, two words.
    const auto of_warps = [&](int i) {                        // this block's sum of word i
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < S::kParts; ++p) {
        const int w = p * S::kHalves + i / 32 / RB;
        v = sum(v, reinterpret_cast<const float4*>(rings + w * (D * S::kSlot) + sums_in[w])[i % (32 * RB)]);
      }
      return v;
    };
    const auto parts_of = [&](int item, float4 u, float4 v, uint4 (&f)[P3]) {
      const int j = item / 32 * 16 + 2 * (item % 4);
      keep_rank(u, j, r);
      keep_rank(v, j + 8, r);
#pragma unroll
      for (int k = 0; k < P3; ++k) {
        f[k].x = split(u.x, u.y);
        f[k].y = split(u.z, u.w);
        f[k].z = split(v.x, v.y);
        f[k].w = split(v.z, v.w);
      }
    };
    constexpr int ITEMS = W / 2;
    if constexpr (S::kShared) {
      // each block finishes a share of the items: it gets their words from every block, and sends the parts to every block
      const int per = ITEMS / C;
      for (int i = tid; i < W; i += kLoraThreads) {
        if (8 * (i / 32) >= r) break;
        const int item = i / 64 * 32 + i % 32;
        st_remote(remote(mine + (rank * 2 + (i / 32 & 1)) * per + item % per, item / per), of_warps(i));
      }
      cluster_arrive();
      cluster_wait();
      const int at = tid % per, item = rank * per + at, j = item / 32 * 16;
      if (tid < ITEMS && j < r) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
        for (int c = 0; c < C; ++c) u = sum(u, mine[2 * c * per + at]);
        if (j + 8 < r)
          for (int c = 0; c < C; ++c) v = sum(v, mine[(2 * c + 1) * per + at]);
        uint4 f[P3];
        parts_of(item, u, v, f);
#pragma unroll
        for (int k = 0; k < P3; ++k) st_remote(remote(frag + (item / 32 * P3 + k) * 32 + item % 32, tid / per), f[k]);
      }
      cluster_arrive();
      cluster_wait();
      waiting = false;
    } else {
      for (int i = tid; i < W; i += kLoraThreads) mine[i] = of_warps(i);
      cluster_arrive();
      cluster_wait();
      for (int i = tid; i < ITEMS; i += kLoraThreads) {
        const int at = i / 32 * 64 + i % 32;
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 8
        for (int c = 0; c < C; ++c) {
          const uint32_t p = remote(mine + at, c);
          u = sum(u, ld_remote(p));
          v = sum(v, ld_remote(p + 32 * 16));
        }
        uint4 f[P3];
        parts_of(i, u, v, f);
#pragma unroll
        for (int k = 0; k < P3; ++k) frag[(i / 32 * P3 + k) * 32 + i % 32] = f[k];
      }
      cluster_arrive();
      waiting = true;
      __syncthreads();
    }

    // ---- second product, over this block's share of N
    const uint4* h = frag + lane;
    for (int n0 = n_lo + warp * 32; n0 < n_hi; n0 += kLoraWarps * 32) {
      const int n = n0 + own_column<Y>(t4);                   // first column of this lane's sums
      float d[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
      const unsigned char* st = ring;
#pragma unroll
      for (int hf = 0; hf < S::kPieces; ++hf) {
        __syncwarp();                                         // the slot that is asked for was other lanes' too
        ask();
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
        __syncwarp();
        st = ring + slot * S::kSlot;
        slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
        for (int e = 0; e < KH; ++e) {
          const int s = hf * KH + e;
          if (16 * s >= r) break;
          uint32_t b[4][2];
          const bool full = 16 * s + 16 <= r;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = 16 * s + 8 * i + 2 * t4;
            uint2 u = make_uint2(0, 0), v = u;
            if (full || j < r) u = *reinterpret_cast<const uint2*>(st + b_even + (2 * e + i) * 512);
            if (full || j + 1 < r) v = *reinterpret_cast<const uint2*>(st + b_odd + (2 * e + i) * 512);
            b[0][i] = __byte_perm(u.x, v.x, 0x5410);
            b[1][i] = __byte_perm(u.x, v.x, 0x7632);
            b[2][i] = __byte_perm(u.y, v.y, 0x5410);
            b[3][i] = __byte_perm(u.y, v.y, 0x7632);
          }
#pragma unroll
          for (int k = P3 - 1; k >= 0; --k) {
            const uint4 f = h[(s * P3 + k) * 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(d[i], f.x, f.y, f.z, f.w, b[i][0], b[i][1]);
          }
        }
      }
      const float any = most(most(most(d[0][0], d[0][1], d[0][2]), most(d[0][3], d[1][0], d[1][1]), most(d[1][2], d[1][3], d[2][0])),
                             most(d[2][1], d[2][2], d[2][3]), most(most(d[3][0], d[3][1], d[3][2]), d[3][3], d[3][3]));
      if (any != any) {                                       // an infinite value of B, or what is NaN all the same
        float e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = d[i / 4][i % 4];
        sums_again<Y, P3>(e, frag, t.b + (int64_t)row0 * t.ldb + n, t.ldb, r, t.N - n, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i / 4][i % 4] = e[i];
      }
      if (t.wide && (F32 ? n0 + 32 : n + 8) <= t.N) {
        uint32_t v[WORDS];
        const unsigned char* sy = st + S::kB + lane * 16;
        if (tok0 >= 0) ld_pieces(sy, v), add_row<Y, 0>(y0 + (int64_t)n * size, scale, d, v);
        if (tok1 >= 0) ld_pieces(sy + 256 * size, v), add_row<Y, 1>(y1 + (int64_t)n * size, scale, d, v);
      } else {
        if (tok0 >= 0) add_row_part<Y, 0>(y0 + (int64_t)n * size, t.N - n, scale, d);
        if (tok1 >= 0) add_row_part<Y, 1>(y1 + (int64_t)n * size, t.N - n, scale, d);
      }
    }
    copies_wait();
  }
  if (waiting) cluster_wait();
}

// ---- many tokens of an adapter
//
// Two kernels, with the values between them in the caller's workspace as the fragments of the second: one cluster's meeting
// per run of tokens would leave the memory idle for a third of the time (in one kernel: 282 us for 8190 tokens).
//
// lora_first_kernel: a cluster takes a run of up to 128 tokens of one adapter and one projection, each block a share of K.
// The product is one of the fifth-generation tensor cores (the tokens' 128 rows of x by the rank rows of A, 64 columns at a
// time, sums in tensor memory), so that the warps only copy; the blocks' sums meet in distributed shared memory. They wait for one
// another with tensor memory in hand: beside a block of another kernel that wants all of it an SM never has room for two of
// them (attention over prompts has 98 KB of shared memory or more), so that none is behind it for the other's.
//
// lora_second_kernel: a block takes 256 columns and a window of tokens. A warp owns 32 columns: their values of B stay in its
// registers while the tokens pass by; y comes through a ring in which each lane finds what it has asked for itself (registers
// as the targets of loads that far ahead were slower: a wait for one of them waits for all). On the tensor cores of the first
// product it was slower (8190 tokens, gate|up: 252 us with a thread per token, 283 with the sums turned in shared memory, 189 so):
// two groups of 32 columns per warp halve the reads of the values, but leave two blocks per SM for three (237).
// Of those 189 us the first kernel takes 40 (L2: x for each projection, A for each run), the second the rest: L1's data path is 69 %
// busy (the values for each warp, y in and out), the tensor cores 52 %, memory 58 %.
constexpr int kRunBlocks = 8;                                 // 16-token blocks of a run of the first kernel: one per warp
constexpr int kMostBlocks = 64;                               // of a window of the second

template <int NB, int Y>
struct Many {
  static constexpr bool F32 = Y == QMV_F32;
  static constexpr int kSteps = NB / 2, kParts3 = F32 ? 3 : 2;
  static constexpr int kBlockWords = kSteps * kParts3 * 32;   // 16-byte words of a 16-token block's finished values
  // first kernel
  static constexpr int kColumns = NB <= 4 ? 32 : 8 * NB;      // of tensor memory: the run's sums
  static constexpr int kCols = 64, kX = 16 * kRunBlocks * kCols * 2, kStage = kX + 8 * NB * kCols * 2, kStages = NB <= 4 ? 4 : 3;
  static constexpr int kSmem1 = kStages * kStage + 1024;      // the stages on a boundary of 1024 bytes
  // second kernel
  static constexpr int kBlockY = 16 * 32 * (F32 ? 4 : 2), kRingY = F32 && NB <= 8 ? 8192 : 4096, kAheadY = kRingY / kBlockY;
  static constexpr int kChunkBlocks = kBlockWords * 16 * 8 > 36 * 1024 ? 2 : 4, kChunkH = kChunkBlocks * kBlockWords * 16;
  static constexpr int kSmem2 = kLoraWarps * kRingY + 2 * kChunkH + 16 * kMostBlocks * (int)sizeof(int64_t);
};

// Whether tile v continues the run of tile u before it.
__device__ __forceinline__ bool follows(const RunArgs& a, const int4& u, const int4& v) {
  return tile_fits(a, u) && tile_fits(a, v) && u.x == v.x && u.z == a.tile && u.y + u.z == v.y;
}

template <int NB, int Y>
__global__ void __launch_bounds__(kLoraThreads, NB > 8 ? 2 : 3) lora_first_kernel(const __grid_constant__ RunArgs a) {
  using S = Many<NB, Y>;
  constexpr int KS = S::kSteps, P3 = S::kParts3, G = S::kStages;
  extern __shared__ __align__(16) unsigned char lora_smem[];
  __shared__ __align__(8) uint64_t done[G];                   // a stage's products
  __shared__ uint32_t tmem_at;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int rank = (int)cluster_rank(), C = a.cluster, clusters = gridDim.x / C;
  unsigned char* stages = lora_smem + (1024 - ((uint32_t)__cvta_generic_to_shared(lora_smem) & 1023)) % 1024;
  const uint32_t stages_at = (uint32_t)__cvta_generic_to_shared(stages);
  float4* mine = reinterpret_cast<float4*>(stages);           // after the columns: this block's sums, which the cluster reads
  if (warp == 0) umma::tmem_alloc<S::kColumns>(&tmem_at);
  if (tid == 0) {
    for (int i = 0; i < G; ++i) core::mbar_init(&done[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = tmem_at;
  // this thread's 16-byte pieces of a stage: piece c of rows r1, r1 + 32, ..., in the order of the 128-byte swizzle
  constexpr int ROWS = kLoraThreads / 8, TURNS_X = 16 * kRunBlocks / ROWS, TURNS_A = (8 * NB + ROWS - 1) / ROWS;
  const int c1 = tid % 8, r1 = tid / 8;
  const uint32_t to1 = r1 * 128 + (c1 ^ (r1 & 7)) * 16;
  int begun = 0;                                              // stages of all units so far
  follow_previous();
  for (int unit = blockIdx.x / C; unit < a.max_tiles * a.n_tasks; unit += clusters) {
    const Task& t = a.t[unit / a.max_tiles];
    const int first = unit % a.max_tiles;
    const int4 tile = a.tiles[first];
    if (tile.z == 0) continue;
    if (first % a.window && follows(a, a.tiles[first - 1], tile)) continue;   // another unit's
    int row0 = 0, r = 0;
    float scale = 1.f;                                        // 16-bit y: part of these values; fp32: of the second product's sums
    const bool good = tile_fits(a, tile);
    if (good) {
      row0 = a.table[2 * tile.x];
      r = a.table[2 * tile.x + 1];
      if constexpr (!S::F32) scale = a.scale[tile.x];
    }
    if (!good || row0 < 0 || r < 0 || r > 8 * NB || row0 > a.pool_rows - r) {
      if (rank == 0 && tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
      continue;
    }
    if (r == 0) continue;
    int count = tile.z;
    for (int4 last = tile; (first + (count - 1) / a.tile + 1) % a.window && first + (count - 1) / a.tile + 1 < a.max_tiles;) {
      const int4 v = a.tiles[first + (count - 1) / a.tile + 1];
      if (!follows(a, last, v)) break;
      count += v.z;
      last = v;
    }
    const int k_share = (a.K + C * 32 - 1) / (C * 32) * 32, k_lo = rank * k_share, k_hi = min(a.K, k_lo + k_share);
    const int n_stages = k_hi > k_lo ? (k_hi - k_lo + S::kCols - 1) / S::kCols : 0, rows = (r + 15) / 16 * 16;
    const __nv_bfloat16* px[TURNS_X];                         // nullptr: no token; its row of the product is of no use
#pragma unroll
    for (int i = 0; i < TURNS_X; ++i) {
      const int at = r1 + i * ROWS, k = at < count ? a.order[tile.y + at] : -1;
      if (at < count && (k < 0 || k >= a.n_tokens)) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
      px[i] = k < 0 || k >= a.n_tokens ? nullptr : a.x + (int64_t)k * a.ldx + k_lo + 8 * c1;
    }
    const __nv_bfloat16* pa = t.a + (int64_t)(row0 + r1) * t.lda + k_lo + 8 * c1;
    const int64_t step_a = ROWS * t.lda;
    // rank rows past the rank are 0: no copy reaches them
#pragma unroll
    for (int i = 0; i < TURNS_A; ++i) {
      const int j = r1 + i * ROWS;
      if (j >= r && j < rows)
        for (int g = 0; g < G; ++g) *reinterpret_cast<uint4*>(stages + g * S::kStage + S::kX + to1 + i * (ROWS * 128)) = make_uint4(0, 0, 0, 0);
    }
    const auto ask = [&](int q) {
      if (q < n_stages) {
        const int use = begun + q, slot = use % G, off = q * S::kCols;
        if (q >= G) core::mbar_wait(&done[slot], (use / G - 1) & 1, a.err);   // the stage's products before these
        const uint32_t to = stages_at + slot * S::kStage + to1;
        if (k_lo + off + 8 * c1 < k_hi) {
#pragma unroll
          for (int i = 0; i < TURNS_X; ++i)
            if (px[i]) copy16(to + i * (ROWS * 128), px[i] + off);
          const __nv_bfloat16* p = pa + off;
#pragma unroll
          for (int i = 0; i < TURNS_A; ++i, p += step_a)
            if (r1 + i * ROWS < r) copy16(to + S::kX + i * (ROWS * 128), p);
        } else {                                              // past the last column: 0 by 0
          unsigned char* z = stages + slot * S::kStage + to1;
#pragma unroll
          for (int i = 0; i < TURNS_X; ++i) *reinterpret_cast<uint4*>(z + i * (ROWS * 128)) = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < TURNS_A; ++i)
            if (r1 + i * ROWS < rows) *reinterpret_cast<uint4*>(z + S::kX + i * (ROWS * 128)) = make_uint4(0, 0, 0, 0);
        }
      }
      copies_end();
    };
    for (int q = 0; q < G - 1; ++q) ask(q);
    const uint32_t shape = umma::mma_shape_bf16(rows);
    for (int q = 0; q < n_stages; ++q) {
      asm volatile("cp.async.wait_group %0;" ::"n"(G - 2) : "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();                                        // the stage is there
      if (warp == 0) {
        umma::fence_after();
        if (umma::elected()) {
          const uint32_t st = stages_at + (begun + q) % G * S::kStage;
          const uint64_t xa = umma::operand(st), ab = umma::operand(st + S::kX);
#pragma unroll
          for (int e = 0; e < 4; ++e) umma::mma_ss(tmem, xa + 2 * e, ab + 2 * e, shape, q + e > 0);
          umma::commit(&done[(begun + q) % G]);
        }
        __syncwarp();
      }
      ask(q + G - 1);
    }
    const int blocks = (count + 15) / 16;
    if (n_stages) {
      const int use = begun + n_stages - 1;
      core::mbar_wait(&done[use % G], (use / G) & 1, a.err);  // the last stage's products, and with them all
    }
    begun += n_stages;
    copies_wait();
    __syncwarp();                                             // a warp reads tensor memory as a whole
    umma::fence_after();
    // tensor memory has a token per lane; `mine` the order of the second product's fragments
    {
      const int row = warp % 4 * 32 + lane, b = row / 16, g = row % 8, high = row % 16 / 8;
      for (int nb = warp / 4; nb < rows / 8; nb += 2) {
        uint32_t v[8];
        if (n_stages) {
          umma::tmem_ld8(tmem + ((uint32_t)(warp % 4 * 32) << 16) + nb * 8, v);
          umma::wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0;
        }
        if (b < blocks) {
          float* to = reinterpret_cast<float*>(mine + (b * NB + nb) * 32 + g * 4) + 2 * high;
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2*>(to + 4 * i) = make_uint2(v[2 * i], v[2 * i + 1]);
        }
      }
    }
    umma::fence_before();
    cluster_arrive();
    cluster_wait();
    // the cluster's sums, a share in each block: an item is a lane's eight values of one k16 step
    const int steps = rows / 16, items = blocks * steps * 32, share = (items + C - 1) / C;
    uint4* to = a.values + ((int64_t)(unit / a.max_tiles) * a.max_tiles + first) * (a.tile / 16) * S::kBlockWords;
    for (int i = rank * share + tid; i < min(items, (rank + 1) * share); i += kLoraThreads) {
      const int b = i / 32 / steps, s = i / 32 % steps, at = (b * NB + 2 * s) * 32 + i % 32;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 8
      for (int c = 0; c < C; ++c) {
        const uint32_t m = remote(mine + at, c);
        const float4 e = ld_remote(m), f = ld_remote(m + 32 * 16);
        u.x += e.x, u.y += e.y, u.z += e.z, u.w += e.w;
        v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
      }
      keep_rank(u, 16 * s + 2 * (i % 4), r);
      keep_rank(v, 16 * s + 8 + 2 * (i % 4), r);
      if constexpr (!S::F32) {
        u.x *= scale, u.y *= scale, u.z *= scale, u.w *= scale;
        v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
      }
#pragma unroll
      for (int k = 0; k < P3; ++k) {
        uint4 f;
        f.x = split(u.x, u.y);
        f.y = split(u.z, u.w);
        f.z = split(v.x, v.y);
        f.w = split(v.z, v.w);
        to[((b * KS + s) * P3 + k) * 32 + i % 32] = f;
      }
    }
    cluster_arrive();
    cluster_wait();                                           // the blocks' sums have been read
  }
  __syncthreads();
  if (warp == 0) umma::tmem_free<S::kColumns>(tmem);
}

template <int NB, int Y>
__global__ void __launch_bounds__(kLoraThreads, NB > 8 || Y == QMV_F32 ? 2 : 3) lora_second_kernel(const __grid_constant__ RunArgs a) {
  using S = Many<NB, Y>;
  constexpr int KS = S::kSteps, P3 = S::kParts3, size = Y == QMV_F32 ? 4 : 2, WORDS = 2 * size, AY = S::kAheadY, CB = S::kChunkBlocks;
  constexpr bool F32 = S::F32;
  extern __shared__ __align__(16) unsigned char lora_smem[];
  unsigned char* chunks = lora_smem + kLoraWarps * S::kRingY;      // two of finished values, each of kChunkBlocks 16-token blocks
  int64_t* row_y = reinterpret_cast<int64_t*>(chunks + 2 * S::kChunkH);   // bytes to each token's row of y; negative: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  unsigned char* ring = lora_smem + warp * S::kRingY + lane * 16;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring), chunks_at = (uint32_t)__cvta_generic_to_shared(chunks);
  const int windows = (a.max_tiles + a.window2 - 1) / a.window2;
  follow_previous();
  for (int unit = blockIdx.x; unit < windows * a.slices; unit += gridDim.x) {
    int slice = unit % a.slices, task = 0;
    while (slice >= (a.t[task].N + 255) / 256) slice -= (a.t[task++].N + 255) / 256;
    const Task& t = a.t[task];
    const int base = unit / a.slices * a.window2, tiles = min(a.window2, a.max_tiles - base);
    // this warp's columns; the first of this lane's sums, and of its loads of B
    const int n0 = slice * 256 + warp * 32, n = n0 + own_column<Y>(t4), col = n0 + block_column<Y>(g);
    const bool whole = t.wide && (F32 ? n0 + 32 : n + 8) <= t.N;
    char* y = static_cast<char*>(t.y);
    for (int j = 0; j < tiles;) {
      const int first = base + j++;
      const int4 tile = a.tiles[first];
      if (!tile_fits(a, tile)) continue;                           // an empty entry, or reported by the first kernel, as is a bad adapter
      const int row0 = a.table[2 * tile.x], r = a.table[2 * tile.x + 1];
      float scale = 1.f;                                      // 16-bit y: the finished values have it
      if constexpr (F32) scale = a.scale[tile.x];
      if (row0 < 0 || r <= 0 || r > 8 * NB || row0 > a.pool_rows - r) continue;
      int count = tile.z;
      for (int4 last = tile; j < tiles; ++j) {                // the adapter's next tiles
        const int4 v = a.tiles[base + j];
        if (!follows(a, last, v)) break;
        count += v.z;
        last = v;
      }
      __syncthreads();                                        // the run before this one is done with row_y and the chunks
      const int blocks = (count + 15) / 16;
      bool odd = false;
      for (int i = tid; i < blocks * 16; i += kLoraThreads) {
        const int k = i < count ? a.order[tile.y + i] : -1;
        const bool there = k >= 0 && k < a.n_tokens;
        row_y[i] = there ? (int64_t)k * t.ldy * size : -1;
        odd |= i < count && !there;
      }
      const uint4* values = a.values + ((int64_t)task * a.max_tiles + first) * (a.tile / 16) * S::kBlockWords;
      const auto load = [&](int c) {                          // chunk c of the finished values
        const int words = min(CB, blocks - c * CB) * S::kBlockWords;
        for (int i = tid; i < words; i += kLoraThreads)
          copy16(chunks_at + (c & 1) * S::kChunkH + i * 16, values + (int64_t)c * CB * S::kBlockWords + i);
        copies_end();
      };
      load(0);
      // 16-token blocks of this warp that need no look at what is there: all their columns, rank rows and tokens
      odd = __syncthreads_or(odd);
      const int plain_blocks = t.wide && n0 + 32 <= t.N && r > 16 * (KS - 1) && !odd ? count / 16 : 0;
      int m_in = 0, slot_in = 0, slot = 0;                    // the next block of y to ask for
      const char* yq = y + (int64_t)n * size;
      const auto ask = [&]() {
        if (m_in < blocks) {
          const int64_t ta = row_y[m_in * 16 + g], tb = row_y[m_in * 16 + g + 8];
          const uint32_t to = ring_at + slot_in * S::kBlockY;
          const bool plain = m_in < plain_blocks;
#pragma unroll
          for (int i = 0; i < size / 2; ++i) {
            if (plain || (whole && ta >= 0)) copy16(to + i * 512, yq + ta + i * 64);
            if (plain || (whole && tb >= 0)) copy16(to + S::kBlockY / 2 + i * 512, yq + tb + i * 64);
          }
        }
        copies_end();
        ++m_in;
        slot_in = slot_in + 1 == AY ? 0 : slot_in + 1;
      };
      for (int i = 0; i < AY - 1; ++i) ask();
      uint32_t b[KS][4][2];
      __nv_bfloat162 seen = __floats2bfloat162_rn(0.f, 0.f);  // 0 times every value of b: NaN where one is not finite
      const __nv_bfloat16* pb = t.b + (int64_t)(row0 + 2 * t4) * t.ldb + col;
      const int cols = t.N - col;                             // from this lane's first on
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int off = 16 * s + (i & 1) + 8 * (i >> 1);
          w[i] = make_uint2(0, 0);
          if (off + 2 * t4 < r && cols > 0) {
            const __nv_bfloat16* q = pb + (int64_t)off * t.ldb;
            if (cols >= 4) {
              w[i] = __ldg(reinterpret_cast<const uint2*>(q));
            } else {
              const uint16_t* e = reinterpret_cast<const uint16_t*>(q);
              w[i].x = e[0] | (cols > 1 ? (uint32_t)e[1] << 16 : 0u);
              w[i].y = cols > 2 ? e[2] : 0u;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          seen = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[i].x), zero, seen);
          seen = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[i].y), zero, seen);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          b[s][0][i] = __byte_perm(w[2 * i].x, w[2 * i + 1].x, 0x5410);
          b[s][1][i] = __byte_perm(w[2 * i].x, w[2 * i + 1].x, 0x7632);
          b[s][2][i] = __byte_perm(w[2 * i].y, w[2 * i + 1].y, 0x5410);
          b[s][3][i] = __byte_perm(w[2 * i].y, w[2 * i + 1].y, 0x7632);
        }
      }
      const bool finite = !__any_sync(0xFFFFFFFFu, __hisnan(seen.x) || __hisnan(seen.y));
      if (!finite) {
#pragma unroll
        for (int i = 0; i < 8 * KS; ++i) b[i / 8][i / 2 % 4][i % 2] = finite2(b[i / 8][i / 2 % 4][i % 2]);
      }
      // Block m: fp32 values of y are added in the end (one rounding), 16-bit ones are what the products are added to.
      const auto block = [&](auto plain, int m, const uint4* h) {
        constexpr bool PLAIN = decltype(plain)::value;
        const int64_t ta = row_y[m * 16 + g], tb = row_y[m * 16 + g + 8];
        const unsigned char* sy = ring + slot * S::kBlockY;
        uint32_t v[2][WORDS];
        ld_pieces(sy, v[0]);
        ld_pieces(sy + S::kBlockY / 2, v[1]);
        float d[4][4];
        if (F32 || !(PLAIN || whole)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i / 4][i % 4] = 0.f;
        } else if constexpr (!F32) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = unpack2<Y>(v[i / 4][i % 4]);
            const int c = 2 * (i % 4), hi = 2 * (i / 4);
            d[c % 4][hi + c / 4] = f.x;
            d[(c + 1) % 4][hi + (c + 1) / 4] = f.y;
          }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (!PLAIN && 16 * s >= r) break;
#pragma unroll
          for (int k = P3 - 1; k >= 0; --k) {
            const uint4 f = h[(s * P3 + k) * 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(d[i], f.x, f.y, f.z, f.w, b[s][i][0], b[s][i][1]);
          }
        }
        char* q = const_cast<char*>(yq);
        if (PLAIN || whole) {
          if constexpr (F32) {
            if (PLAIN || ta >= 0) add_row<Y, 0>(q + ta, scale, d, v[0]);
            if (PLAIN || tb >= 0) add_row<Y, 1>(q + tb, scale, d, v[1]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int c = 2 * (i % 4), hi = 2 * (i / 4);
              v[i / 4][i % 4] = pack2<Y>(d[c % 4][hi + c / 4], d[(c + 1) % 4][hi + (c + 1) / 4]);
            }
            if (PLAIN || ta >= 0) st_pieces(q + ta, v[0]);
            if (PLAIN || tb >= 0) st_pieces(q + tb, v[1]);
          }
        } else {
          if (ta >= 0) add_row_part<Y, 0>(q + ta, t.N - n, scale, d);
          if (tb >= 0) add_row_part<Y, 1>(q + tb, t.N - n, scale, d);
        }
      };
      for (int c = 0; c * CB < blocks; ++c) {
        // since chunk c: the prologue's AY - 1 groups of y, or the CB of the chunk before this one
        if (c == 0) asm volatile("cp.async.wait_group %0;" ::"n"(AY - 1) : "memory");
        else asm volatile("cp.async.wait_group %0;" ::"n"(CB) : "memory");
        __syncthreads();                                      // chunk c is there, and c - 1 has been read
        if ((c + 1) * CB < blocks) load(c + 1);
        else copies_end();
#pragma unroll 1
        for (int m = c * CB; m < min(blocks, (c + 1) * CB); ++m) {
          ask();
          // since this block's copies: AY - 1 groups of y, and of the finished values one or more
          asm volatile("cp.async.wait_group %0;" ::"n"(AY - 1) : "memory");
          const uint4* h = reinterpret_cast<const uint4*>(chunks + (c & 1) * S::kChunkH) + (m - c * CB) * S::kBlockWords + lane;
          if (m < plain_blocks) block(std::true_type{}, m, h);
          else block(std::false_type{}, m, h);
          slot = slot + 1 == AY ? 0 : slot + 1;
        }
      }
      copies_wait();
      if (!finite) {
        __syncwarp();                                         // the warp's rows of y are written
        if (n0 + lane < t.N)
          add_infinite<Y, KS, P3>(y + (int64_t)(n0 + lane) * size, row_y, count, values, t.b + (int64_t)row0 * t.ldb + n0 + lane, t.ldb, r, scale);
      }
    }
  }
}

// The kernels of a call and their shared memory.
struct Choice {
  const void* few;
  const void* first;
  const void* second;
  int few_smem, first_smem, second_smem, block_words;
};
template <int NB, int Y>
Choice choice_of() {
  return {reinterpret_cast<const void*>(lora_short_kernel<NB, Y>), reinterpret_cast<const void*>(lora_first_kernel<NB, Y>),
          reinterpret_cast<const void*>(lora_second_kernel<NB, Y>), Short<NB, Y>::kSmem, Many<NB, Y>::kSmem1, Many<NB, Y>::kSmem2, Many<NB, Y>::kBlockWords};
}
template <int Y>
Choice choose(int max_rank) {
  return max_rank <= 16 ? choice_of<2, Y>() : max_rank <= 32 ? choice_of<4, Y>() : max_rank <= 64 ? choice_of<8, Y>() : choice_of<16, Y>();
}

// Whether a call is one of many tokens per adapter, which takes the two kernels. us with the one kernel and with these, K 5120: 1024
// tokens of 5 adapters, rank 64, gate|up 80 and 88, q|k|v 42 and 35; 1536 of 5, gate|up 139 and 102; 4096 of 5, gate|up 278 and 199;
// 4096 of 60, rank 16, N 5120 50 and 56; 3000 of 200, rank 64, N 5120, bf16 77 and 115.
bool many_tokens(int64_t n_tokens, int64_t n_adapters) { return n_tokens >= 1280 && n_tokens >= 64 * n_adapters; }

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

int32_t lora_tile(int64_t n_tokens) { return n_tokens < 1024 ? kSmallTile : kLargeTile; }

int64_t lora_max_tiles(int64_t n_tokens, int64_t n_adapters) {
  if (n_tokens <= 0 || n_adapters <= 0) return 0;
  return n_tokens / lora_tile(n_tokens) + (n_tokens < n_adapters ? n_tokens : n_adapters);
}

size_t lora_workspace_size(int64_t n_tokens, int64_t n_adapters, int32_t max_rank, int32_t n_tasks) {
  if (n_tokens <= 0 || n_adapters <= 0 || max_rank <= 0 || max_rank > kMaxRank || n_tasks <= 0 || !many_tokens(n_tokens, n_adapters)) return 0;
  const int64_t steps = max_rank <= 16 ? 1 : max_rank <= 32 ? 2 : max_rank <= 64 ? 4 : 8;   // of 16 rank rows, as the kernels are made
  return (size_t)(lora_max_tiles(n_tokens, n_adapters) * (kLargeTile / 16) * n_tasks * steps * 3 * 512);
}

int lora_plan(const lora_plan_args* g, void* stream) {
  if (!g) return fail(QMV_ERR_ARG, "args is NULL");
  if (g->n_tokens < 0 || g->n_tokens > QMV_LORA_MAX_TOKENS) return fail(QMV_ERR_ARG, "n_tokens=%d outside 0..%d", g->n_tokens, QMV_LORA_MAX_TOKENS);
  if (g->n_adapters < 1 || g->n_adapters > kMaxAdapters) return fail(QMV_ERR_ARG, "n_adapters=%d outside 1..%d", g->n_adapters, kMaxAdapters);
  if (g->max_tiles < lora_max_tiles(g->n_tokens, g->n_adapters))
    return fail(QMV_ERR_ARG, "max_tiles=%d below lora_max_tiles=%lld", g->max_tiles, (long long)lora_max_tiles(g->n_tokens, g->n_adapters));
  if ((g->n_tokens > 0 && (!g->ids || !g->order)) || (g->max_tiles > 0 && !g->tiles)) return fail(QMV_ERR_ARG, "NULL ids, order or tiles");
  if ((reinterpret_cast<uintptr_t>(g->ids) | reinterpret_cast<uintptr_t>(g->order)) & 3u) return fail(QMV_ERR_ALIGN, "int32 arrays must be 4-byte aligned");
  if (!aligned16(g->tiles)) return fail(QMV_ERR_ALIGN, "tiles must be 16-byte aligned");
  if (g->max_tiles == 0) return QMV_OK;
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");
  PlanArgs a{g->ids, g->order, reinterpret_cast<int4*>(g->tiles), err, g->n_tokens, g->n_adapters, lora_tile(g->n_tokens), g->max_tiles};
  const void* f = reinterpret_cast<const void*>(lora_plan_kernel);
  // a warp for every 128 tokens, up to 32: fewer counters to clear and to sum where there are few
  const int warps = g->n_tokens >= 4096 ? 32 : g->n_tokens >= 512 ? 16 : 8;
  const auto bytes = [](int w, int adapters) { return (size_t)(2 * (adapters + 1) + w * adapters) * sizeof(int32_t); };
  int per_sm = 0;
  // asked for the most adapters: the library keeps an answer per size asked for
  int rc = kernel_fit(f, 1024, bytes(32, kMaxAdapters), &per_sm);
  if (rc) return rc;
  void* args[] = {&a};
  cudaError_t e = kv8::launch_early(f, dim3(1), 32 * warps, args, bytes(warps, g->n_adapters), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lora_plan launch");
  return QMV_OK;
}

int lora_run(const lora_args* g, const lora_task* tasks, int n_tasks, void* stream) {
  if (!g || !tasks) return fail(QMV_ERR_ARG, "args or tasks is NULL");
  if (n_tasks < 1 || n_tasks > QMV_LORA_MAX_TASKS) return fail(QMV_ERR_ARG, "n_tasks=%d outside 1..%d", n_tasks, QMV_LORA_MAX_TASKS);
  if (g->n_tokens < 0 || g->n_tokens > QMV_LORA_MAX_TOKENS) return fail(QMV_ERR_ARG, "n_tokens=%d outside 0..%d", g->n_tokens, QMV_LORA_MAX_TOKENS);
  if (g->n_adapters < 1 || g->n_adapters > kMaxAdapters) return fail(QMV_ERR_ARG, "n_adapters=%d outside 1..%d", g->n_adapters, kMaxAdapters);
  if (g->max_rank < 1 || g->max_rank > kMaxRank) return fail(QMV_ERR_ARG, "max_rank=%d outside 1..%d", g->max_rank, kMaxRank);
  if (g->pool_rows < 1) return fail(QMV_ERR_ARG, "pool_rows=%d", g->pool_rows);
  if (g->K < 8 || g->K % 8 || g->K > (1 << 26) || g->ldx < g->K) return fail(QMV_ERR_ARG, "K=%d ldx=%lld: K a multiple of 8, ldx >= K", g->K, (long long)g->ldx);
  if (g->max_tiles < lora_max_tiles(g->n_tokens, g->n_adapters))
    return fail(QMV_ERR_ARG, "max_tiles=%d below lora_max_tiles=%lld", g->max_tiles, (long long)lora_max_tiles(g->n_tokens, g->n_adapters));
  if (g->ldx % 8) return fail(QMV_ERR_ALIGN, "ldx=%lld must be a multiple of 8 (16-byte rows)", (long long)g->ldx);
  if (g->n_tokens > 0) {
    if (!g->x || !g->order || !g->tiles || !g->table || !g->scale) return fail(QMV_ERR_ARG, "NULL x, order, tiles, table or scale");
    if (!aligned16(g->x) || !aligned16(g->tiles)) return fail(QMV_ERR_ALIGN, "x and tiles must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(g->order) | reinterpret_cast<uintptr_t>(g->table) | reinterpret_cast<uintptr_t>(g->scale)) & 3u)
      return fail(QMV_ERR_ALIGN, "order, table and scale must be 4-byte aligned");
  }
  RunArgs a;
  a.x = static_cast<const __nv_bfloat16*>(g->x);
  a.order = g->order;
  a.table = g->table;
  a.tiles = reinterpret_cast<const int4*>(g->tiles);
  a.scale = g->scale;
  a.ldx = g->ldx;
  a.K = g->K;
  a.n_tokens = g->n_tokens;
  a.n_adapters = g->n_adapters;
  a.pool_rows = g->pool_rows;
  a.max_tiles = (int32_t)lora_max_tiles(g->n_tokens, g->n_adapters);   // what the workspace has room for: a longer list is empty from there on
  a.n_tasks = n_tasks;
  for (int i = 0; i < n_tasks; ++i) {
    const lora_task& k = tasks[i];
    const int ys = kv8::dtype_size(k.y_type);
    if (!ys) return fail(QMV_ERR_ARG, "task %d: y_type=%d", i, k.y_type);
    if (k.y_type != tasks[0].y_type) return fail(QMV_ERR_ARG, "task %d: y_type=%d beside %d: one type for a call", i, k.y_type, tasks[0].y_type);
    if (k.N < 1 || k.lda < g->K || k.ldb < k.N || k.ldy < k.N)
      return fail(QMV_ERR_ARG, "task %d: N=%d lda=%lld ldb=%lld ldy=%lld", i, k.N, (long long)k.lda, (long long)k.ldb, (long long)k.ldy);
    if (k.N > (1 << 26)) return fail(QMV_ERR_UNSUPPORTED, "task %d: N=%d over 2^26", i, k.N);
    if (k.lda % 8 || k.ldb % 8) return fail(QMV_ERR_ALIGN, "task %d: rows of a and b must be 16-byte aligned", i);
    if (g->n_tokens > 0) {
      if (!k.a || !k.b || !k.y) return fail(QMV_ERR_ARG, "task %d: NULL a, b or y", i);
      if (!aligned16(k.a) || !aligned16(k.b) || !aligned16(k.y)) return fail(QMV_ERR_ALIGN, "task %d: a, b and y must be 16-byte aligned", i);
    }
    a.t[i] = {static_cast<const __nv_bfloat16*>(k.a), static_cast<const __nv_bfloat16*>(k.b), k.y, k.lda, k.ldb, k.ldy, k.N, (int32_t)(k.ldy * ys % 16 == 0)};
  }
  if (g->n_tokens == 0) return QMV_OK;
  const size_t need = lora_workspace_size(g->n_tokens, g->n_adapters, g->max_rank, n_tasks);
  if (need && (!g->workspace || g->ws_bytes < need)) return fail(QMV_ERR_ARG, "workspace of %zu bytes, lora_workspace_size is %zu", g->ws_bytes, need);
  if (need && !aligned16(g->workspace)) return fail(QMV_ERR_ALIGN, "workspace must be 16-byte aligned");
  a.err = device_error_word();
  if (!a.err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");
  a.tile = lora_tile(g->n_tokens);
  const int type = tasks[0].y_type;
  const Choice c = type == QMV_F32 ? choose<QMV_F32>(g->max_rank) : type == QMV_BF16 ? choose<QMV_BF16>(g->max_rank) : choose<QMV_F16>(g->max_rank);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* args[] = {&a};
  const int64_t units = (int64_t)a.max_tiles * n_tasks;
  int per_sm = 0;
  // Clusters and blocks are one for every unit, up to eight rounds of them: the device hands them out as others end (units differ
  // by rank and N). Past that they take several each, so that a list with many empty tiles costs few launches of blocks.
  if (!many_tokens(g->n_tokens, g->n_adapters)) {
    int rc = kernel_fit(c.few, kLoraThreads, c.few_smem, &per_sm);
    if (rc) return rc;
    // A unit is 16 tokens of a tile and a projection. Few units are cut into eight blocks each, as long as all are resident at once;
    // more of them into four, up to two rounds, or two, since a unit has two meetings of its cluster whatever its size. us with 8, 4
    // and 2: 80 tokens of 12 adapters, rank 16, gate|up 11.9, 12.7, 20.1; 512 of 8, rank 64, gate|up 57, 41, 48; 64 of 48, rank 64,
    // q|k|v 33.0, 24.4, 27.7; 1000 of one, rank 64, gate|up 89, 79, 73; 1023 of 8, rank 32, q|k|v 51, 33, 27.
    const int64_t blocks = (int64_t)sm_count() * per_sm;
    // Counted without the units that are empty because a tile of 64 tokens has fewer.
    const int64_t full = (g->n_tokens / 16 + (int64_t)(g->n_tokens < g->n_adapters ? g->n_tokens : g->n_adapters)) * n_tasks;
    a.cluster = full * kCluster <= blocks + blocks / 4 ? kCluster : full * 4 <= 2 * blocks + blocks / 8 ? 4 : 2;
    const int64_t all = units * (a.tile / 16), most = 8 * blocks / a.cluster, clusters = all < most ? all : most;
    cudaError_t e = kv8::launch_early(c.few, dim3((unsigned)(clusters * a.cluster)), kLoraThreads, args, c.few_smem, s, a.cluster);
    if (e != cudaSuccess) return cuda_fail(e, "lora_run launch");
    return QMV_OK;
  }
  a.values = static_cast<uint4*>(g->workspace);
  int rc = kernel_fit(c.first, kLoraThreads, c.first_smem, &per_sm);
  if (rc) return rc;
  // four blocks per run where that fills the device twice, else eight: 8190 tokens, gate|up: 189 us with 4, 199 with 8
  a.cluster = units * kCluster > 2 * (int64_t)sm_count() * per_sm ? kCluster / 2 : kCluster;
  a.window = kRunBlocks * 16 / a.tile;
  a.slices = 0;
  for (int i = 0; i < n_tasks; ++i) a.slices += (tasks[i].N + 255) / 256;
  const int64_t most = 8 * (int64_t)sm_count() * per_sm / a.cluster, clusters = units < most ? units : most;
  rc = kernel_fit(c.second, kLoraThreads, c.second_smem, &per_sm);
  if (rc) return rc;
  // the second kernel's windows: up to 1024 tokens, as long as there are four blocks of them for each that is resident
  a.window2 = kMostBlocks * 16 / a.tile;
  while (a.window2 > 1 && (int64_t)((a.max_tiles + a.window2 - 1) / a.window2) * a.slices < 4 * (int64_t)sm_count() * per_sm) a.window2 /= 2;
  const int64_t pieces = (int64_t)((a.max_tiles + a.window2 - 1) / a.window2) * a.slices, most2 = 64 * (int64_t)sm_count() * per_sm;
  if (pieces > INT32_MAX) return fail(QMV_ERR_UNSUPPORTED, "max_tiles=%d of %d slices of columns", a.max_tiles, a.slices);
  cudaError_t e = kv8::launch_early(c.first, dim3((unsigned)(clusters * a.cluster)), kLoraThreads, args, c.first_smem, s, a.cluster);
  if (e != cudaSuccess) return cuda_fail(e, "lora_run launch (first product)");
  e = kv8::launch_early(c.second, dim3((unsigned)(pieces < most2 ? pieces : most2)), kLoraThreads, args, c.second_smem, s);
  if (e != cudaSuccess) return cuda_fail(e, "lora_run launch (second product)");
  return QMV_OK;
}

}  // extern "C"

// Low-rank adapters of many requests beside a shared projection: the step's
// grouping of tokens by adapter (lora_plan) and
//   y[t] += s_a * B_a^T (A_a x[t]),  a the adapter of token t        (lora_run).
//
// lora_run is bound by memory: a token's products cost 2 r (K + N) operations
// for K + 2 N moved values, and a single token's adapter is read once. One launch
// does both products, so that their r values in between never leave the chip: a
// cluster of eight blocks takes a tile of tokens of one adapter and one
// projection; each block forms the first product over an eighth of K, the
// partial sums meet through distributed shared memory, and each block takes an
// eighth of N in the second. Warp-level products (mma.sync m16n8k16, bf16 with
// fp32 sums) are far from their limit here (11 GFLOP against 0.9 GB for the
// largest measured call), and they take both operands as they lie in memory:
// * first product: a lane's 16 bytes of a row of x and of a row of A are eight
//   consecutive k. A contraction may take its index in any order, so these are
//   the lane's pairs of two k16 steps: no shuffle and no shared memory.
// * second product: a lane's 16 bytes of a row of B are eight consecutive n of
//   one rank row; two rows zipped by byte permutes are the pairs of eight n8
//   blocks, whose column m is n0 + 8 m + block. So a lane's sums are sixteen
//   consecutive columns of y: whole 32-byte sectors in and out.
// The r values in between are fp32 sums, handed to the second product as two
// bf16 parts (value and remainder: 2^-18 of each), so that an fp32 y keeps its
// precision.
#include "kv8.cuh"

namespace qmv {
namespace {

using kv8::follow_previous;

constexpr int kMaxAdapters = QMV_LORA_MAX_ADAPTERS;
constexpr int kMaxRank = QMV_LORA_MAX_RANK;
constexpr int kSmallTile = 16, kLargeTile = 64;

// ----------------------------------------------------------------------------- plan

// A stable counting sort by one block. Each warp takes a range of the tokens and
// counts them per adapter, 32 at a time (lanes of one adapter find each other by
// a match, the first of them adds); sums over the warps, then over the adapters,
// give each warp its place per adapter, and a second pass hands the places out.
constexpr int kPlanAhead = 8;   // loads in flight per lane

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
  for (int t0 = lo; t0 < hi; t0 += 32 * kPlanAhead) {
    int id[kPlanAhead];
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      const int t = t0 + 32 * u + lane;
      id[u] = t < hi ? a.ids[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      if (t0 + 32 * u >= hi) break;
      bad |= id[u] >= A;
      const int k = id[u] < A ? id[u] : -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, k);
      if (k >= 0 && lane == __ffs(same) - 1) mine[k] += __popc(same);
      __syncwarp();
    }
  }
  if (bad) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
  __syncthreads();
  // per adapter: its warps' counts to their exclusive sums; then sums over the adapters, `threads` of them at a time
  int2 base = make_int2(0, 0);
  for (int a0 = 0; a0 < A; a0 += threads) {
    const int k = a0 + tid;
    int n = 0;
    if (k < A)
      for (int w = 0; w < warps; ++w) {
        const int c = hist[w * A + k];
        hist[w * A + k] = n;
        n += c;
      }
    const int tiles = (n + a.tile - 1) / a.tile;
    const int sn = scan_add(n, lane), st = scan_add(tiles, lane);
    if (lane == 31) sums[warp] = make_int2(sn, st);
    __syncthreads();
    int2 before = base, all = base;
    for (int w = 0; w < warps; ++w) {
      const int2 s = sums[w];
      if (w < warp) before.x += s.x, before.y += s.y;
      all.x += s.x, all.y += s.y;
    }
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
    int id[kPlanAhead];
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      const int t = t0 + 32 * u + lane;
      id[u] = t < hi ? a.ids[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      if (t0 + 32 * u >= hi) break;
      const int k = id[u] < A ? id[u] : -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, k);
      if (k >= 0) a.order[first[k] + mine[k] + __popc(same & ((1u << lane) - 1))] = t0 + 32 * u + lane;
      __syncwarp();
      if (k >= 0 && lane == __ffs(same) - 1) mine[k] += __popc(same);
      __syncwarp();
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
  int32_t N, y_type;
  int32_t wide;                // rows of y are 32-byte aligned
};

struct RunArgs {
  const __nv_bfloat16* x;
  const int32_t* order;
  const int32_t* table;
  const int4* tiles;
  const float* scale;
  int* err;
  int64_t ldx;
  int32_t K, n_tokens, n_adapters, pool_rows, max_tiles, n_tasks;
  Task t[QMV_LORA_MAX_TASKS];
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_remote(uint32_t p) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_remote(uint32_t p, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_once(const void* p) { return __ldg(static_cast<const uint4*>(p)); }
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

__device__ __forceinline__ float2 unpack2(int type, uint32_t w) {
  if (type == QMV_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(int type, float x, float y) {
  if (type == QMV_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight consecutive values of a row of y, as they lie in memory: 32 bytes (fp32, one 256-bit access) or 16.
__device__ __forceinline__ void ld_row(int type, const void* p, uint32_t (&w)[8]) {
  if (type == QMV_F32) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}
// w += s * v, to memory. v: the sums of the eight columns, block by block (column c is block c % 4, half c / 4).
template <int HI>
__device__ __forceinline__ void add_row(int type, void* p, float s, const float (&acc)[4][4], uint32_t (&w)[8]) {
  if (type == QMV_F32) {
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = __float_as_uint(fmaf(s, acc[c & 3][2 * HI + (c >> 2)], __uint_as_float(w[c])));
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 2 * i;
      const float2 v = unpack2(type, w[i]);
      o[i] = pack2(type, fmaf(s, acc[c & 3][2 * HI + (c >> 2)], v.x), fmaf(s, acc[(c + 1) & 3][2 * HI + ((c + 1) >> 2)], v.y));
    }
    *static_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}
// The same value by value, up to column n of the row.
template <int HI>
__device__ __forceinline__ void add_row_part(int type, void* p, int n, float s, const float (&acc)[4][4]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (c >= n) break;
    const float v = acc[c & 3][2 * HI + (c >> 2)];
    if (type == QMV_F32) {
      float* q = static_cast<float*>(p) + c;
      *q = fmaf(s, v, *q);
    } else if (type == QMV_BF16) {
      __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + c;
      *q = __float2bfloat16_rn(fmaf(s, v, __bfloat162float(*q)));
    } else {
      __half* q = static_cast<__half*>(p) + c;
      *q = __float2half_rn(fmaf(s, v, __half2float(*q)));
    }
  }
}

// MT 16-token blocks per tile, NB blocks of eight rank rows (the call's largest rank).
template <int MT, int NB>
struct Shape {
  static constexpr int kSteps = NB / 2;                       // k16 steps of the second product
  static constexpr int kShare = kLoraWarps / MT;              // warps that share a 16-token block
  static constexpr int kHalves = NB > 8 ? 2 : 1;              // in the first product a warp has at most 64 rank rows
  static constexpr int kParts = kShare / kHalves;             // and a share of the columns of x
  static constexpr int kWords = MT * kSteps * 2 * 32;         // 16-byte words of the tile's r values, in the order of the fragments
  static constexpr int kSums = kParts > 2 ? kParts : 2;       // room for the warps' sums, then for the three parts of their total
  static constexpr size_t kSmem = (size_t)(kSums + 1) * kWords * 16 + 16 * MT * sizeof(int);
};
constexpr int kAhead = 2;                                     // k16 steps of B in flight

template <int MT, int NB>
__global__ void __launch_bounds__(kLoraThreads, NB <= 4 ? 3 : 2) lora_kernel(const __grid_constant__ RunArgs a) {
  using S = Shape<MT, NB>;
  constexpr int KS = S::kSteps, W = S::kWords, RB = NB / S::kHalves;
  extern __shared__ uint4 lora_smem[];
  float4* sums = reinterpret_cast<float4*>(lora_smem);        // [kParts][W]: the warps' sums
  uint4* frag = lora_smem;                                    // [MT][KS][3][32], after them: the three parts of the finished values
  float4* mine = sums + S::kSums * W;                        // [W]: this block's sums, which the cluster reads
  int* token = reinterpret_cast<int*>(mine + W);              // [16 * MT]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int mb = warp % MT, share = warp / MT;                // this warp's 16-token block, its share of columns
  const int half = share % S::kHalves, part = share / S::kHalves;
  const int rank = (int)cluster_rank();
  const int clusters = gridDim.x / kCluster;
  follow_previous();
  bool reading = false;                                       // other blocks may still read `mine`
  for (int unit = blockIdx.x / kCluster; unit < a.max_tiles * a.n_tasks; unit += clusters) {
    const Task& t = a.t[unit / a.max_tiles];
    const int4 tile = a.tiles[unit % a.max_tiles];
    if (tile.z == 0) continue;
    const bool fits = tile.x >= 0 && tile.x < a.n_adapters && tile.y >= 0 && tile.z > 0 && tile.z <= 16 * MT && tile.y <= a.n_tokens - tile.z;
    int row0 = 0, r = 0;
    float scale = 0.f;
    if (fits) {
      row0 = a.table[2 * tile.x];
      r = a.table[2 * tile.x + 1];
      scale = a.scale[tile.x];
    }
    if (!fits || row0 < 0 || r < 0 || r > 8 * NB || row0 > a.pool_rows - r) {
      if (rank == 0 && tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
      continue;
    }
    if (r == 0) continue;
    const int count = tile.z;
    __syncthreads();                                          // the unit before this one is done with token and frag
    if (tid < 16 * MT) {
      int k = -1;
      if (tid < count) {
        k = a.order[tile.y + tid];
        if (k < 0 || k >= a.n_tokens) {
          k = -1;
          atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
        }
      }
      token[tid] = k;
    }
    __syncthreads();
    const bool mine_used = mb * 16 < count;                   // false: this warp's tokens are none
    const int tok0 = token[mb * 16 + g], tok1 = token[mb * 16 + g + 8];

    // ---- first product, over this block's share of K
    float acc[RB][4];
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    const int j0 = half * 8 * RB;                             // this warp's first rank row
    if (mine_used && j0 < r) {
      const __nv_bfloat16* x0 = a.x + (int64_t)(tok0 < 0 ? 0 : tok0) * a.ldx;
      const __nv_bfloat16* x1 = a.x + (int64_t)(tok1 < 0 ? 0 : tok1) * a.ldx;
      const __nv_bfloat16* pa = t.a + (int64_t)(row0 + j0 + g) * t.lda;
      const int64_t step = 8 * t.lda;
      for (int k0 = (rank * S::kParts + part) * 32; k0 < a.K; k0 += kCluster * S::kParts * 32) {
        const int k = k0 + 8 * t4;
        const bool in = k < a.K;
        uint4 p = make_uint4(0, 0, 0, 0), q = p, w[RB];
        if (in && tok0 >= 0) p = ld_once(x0 + k);
        if (in && tok1 >= 0) q = ld_once(x1 + k);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          w[i] = make_uint4(0, 0, 0, 0);
          if (in && j0 + 8 * i + g < r) w[i] = ld_once(pa + i * step + k);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          if (j0 + 8 * i >= r) break;
          mma(acc[i], p.x, q.x, p.y, q.y, w[i].x, w[i].y);
          mma(acc[i], p.z, q.z, p.w, q.w, w[i].z, w[i].w);
        }
      }
    }
    float4* to = sums + ((part * MT + mb) * S::kHalves + half) * RB * 32 + lane;
#pragma unroll
    for (int i = 0; i < RB; ++i) to[i * 32] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
    if (reading) cluster_wait();
    for (int i = tid; i < W; i += kLoraThreads) {
      float4 v = sums[i];
#pragma unroll
      for (int p = 1; p < S::kParts; ++p) {
        const float4 o = sums[p * W + i];
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      mine[i] = v;
    }
    cluster_arrive();
    cluster_wait();

    // ---- the cluster's sums: item i is a lane's eight values of one k16 step
    const auto finish = [&](int i, uint4 (&f)[3]) {
      const int at = (i / 32) * 64 + i % 32;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        const uint32_t p = remote(mine + at, c);
        const float4 o = ld_remote(p), q = ld_remote(p + 32 * 16);
        u.x += o.x, u.y += o.y, u.z += o.z, u.w += o.w;
        v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        f[k].x = split(u.x, u.y);
        f[k].y = split(u.z, u.w);
        f[k].z = split(v.x, v.y);
        f[k].w = split(v.z, v.w);
      }
    };
    if constexpr (MT == 1) {
      // few values: every block takes all of them
      for (int i = tid; i < W / 2; i += kLoraThreads) {
        uint4 f[3];
        finish(i, f);
#pragma unroll
        for (int k = 0; k < 3; ++k) frag[((i / 32) * 3 + k) * 32 + i % 32] = f[k];
      }
      cluster_arrive();
      reading = true;
      __syncthreads();
    } else {
      // each block finishes an eighth and hands it to all
      for (int i = rank * (W / 16) + tid; i < (rank + 1) * (W / 16); i += kLoraThreads) {
        uint4 f[3];
        finish(i, f);
#pragma unroll
        for (int c = 0; c < kCluster; ++c)
#pragma unroll
          for (int k = 0; k < 3; ++k) st_remote(remote(frag + ((i / 32) * 3 + k) * 32 + i % 32, c), f[k]);
      }
      cluster_arrive();
      cluster_wait();
    }
    if (!mine_used) continue;

    // ---- second product, over this block's share of N: 32 columns at a time
    const int type = t.y_type, size = type == QMV_F32 ? 4 : 2;
    const bool third = type == QMV_F32;
    char* y0 = static_cast<char*>(t.y) + (int64_t)(tok0 < 0 ? 0 : tok0) * t.ldy * size;
    char* y1 = static_cast<char*>(t.y) + (int64_t)(tok1 < 0 ? 0 : tok1) * t.ldy * size;
    const uint4* h = frag + mb * KS * 96 + lane;
    for (int n0 = (rank * S::kShare + share) * 32; n0 < t.N; n0 += kCluster * S::kShare * 32) {
      const int n = n0 + 8 * t4, col = n0 + 4 * g;            // first column of this lane's sums, and of its loads of B
      const bool whole = t.wide && n + 8 <= t.N;
      uint32_t v0[8], v1[8];
      if (whole && tok0 >= 0) ld_row(type, y0 + (int64_t)n * size, v0);
      if (whole && tok1 >= 0) ld_row(type, y1 + (int64_t)n * size, v1);
      float d[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
      const __nv_bfloat16* pb = t.b + (int64_t)(row0 + 2 * t4) * t.ldb + col;
#pragma unroll
      for (int s0 = 0; s0 < KS; s0 += kAhead) {
        if (16 * s0 >= r) break;
        uint2 w[kAhead][4];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int off = 16 * (s0 + e) + (i & 1) + 8 * (i >> 1);
            w[e][i] = make_uint2(0, 0);
            if (s0 + e < KS && off + 2 * t4 < r && col < t.N) {
              const __nv_bfloat16* p = pb + (int64_t)off * t.ldb;
              if (col + 4 <= t.N) {
                w[e][i] = __ldg(reinterpret_cast<const uint2*>(p));
              } else {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
                w[e][i].x = q[0] | (col + 1 < t.N ? (uint32_t)q[1] << 16 : 0u);
                w[e][i].y = col + 2 < t.N ? q[2] : 0u;
              }
            }
          }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          if (s0 + e >= KS || 16 * (s0 + e) >= r) break;
          uint32_t b[4][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            b[0][i] = __byte_perm(w[e][2 * i].x, w[e][2 * i + 1].x, 0x5410);
            b[1][i] = __byte_perm(w[e][2 * i].x, w[e][2 * i + 1].x, 0x7632);
            b[2][i] = __byte_perm(w[e][2 * i].y, w[e][2 * i + 1].y, 0x5410);
            b[3][i] = __byte_perm(w[e][2 * i].y, w[e][2 * i + 1].y, 0x7632);
          }
          if (third) {
            const uint4 f = h[(s0 + e) * 96 + 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(d[i], f.x, f.y, f.z, f.w, b[i][0], b[i][1]);
          }
#pragma unroll
          for (int k = 1; k >= 0; --k) {
            const uint4 f = h[(s0 + e) * 96 + 32 * k];
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(d[i], f.x, f.y, f.z, f.w, b[i][0], b[i][1]);
          }
        }
      }
      if (whole) {
        if (tok0 >= 0) add_row<0>(type, y0 + (int64_t)n * size, scale, d, v0);
        if (tok1 >= 0) add_row<1>(type, y1 + (int64_t)n * size, scale, d, v1);
      } else {
        if (tok0 >= 0) add_row_part<0>(type, y0 + (int64_t)n * size, t.N - n, scale, d);
        if (tok1 >= 0) add_row_part<1>(type, y1 + (int64_t)n * size, t.N - n, scale, d);
      }
    }
  }
  if (reading) cluster_wait();
}

template <int MT>
const void* run_kernel(int max_rank, size_t* smem) {
  if (max_rank <= 16) return *smem = Shape<MT, 2>::kSmem, reinterpret_cast<const void*>(lora_kernel<MT, 2>);
  if (max_rank <= 32) return *smem = Shape<MT, 4>::kSmem, reinterpret_cast<const void*>(lora_kernel<MT, 4>);
  if (max_rank <= 64) return *smem = Shape<MT, 8>::kSmem, reinterpret_cast<const void*>(lora_kernel<MT, 8>);
  return *smem = Shape<MT, 16>::kSmem, reinterpret_cast<const void*>(lora_kernel<MT, 16>);
}

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

int32_t lora_tile(int64_t n_tokens) { return n_tokens < 1024 ? kSmallTile : kLargeTile; }

int64_t lora_max_tiles(int64_t n_tokens, int64_t n_adapters) {
  if (n_tokens <= 0 || n_adapters <= 0) return 0;
  return n_tokens / lora_tile(n_tokens) + (n_tokens < n_adapters ? n_tokens : n_adapters);
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
  a.max_tiles = g->max_tiles;
  a.n_tasks = n_tasks;
  for (int i = 0; i < n_tasks; ++i) {
    const lora_task& k = tasks[i];
    const int ys = kv8::dtype_size(k.y_type);
    if (!ys) return fail(QMV_ERR_ARG, "task %d: y_type=%d", i, k.y_type);
    if (k.N < 1 || k.lda < g->K || k.ldb < k.N || k.ldy < k.N)
      return fail(QMV_ERR_ARG, "task %d: N=%d lda=%lld ldb=%lld ldy=%lld", i, k.N, (long long)k.lda, (long long)k.ldb, (long long)k.ldy);
    if (k.lda % 8 || k.ldb % 8) return fail(QMV_ERR_ALIGN, "task %d: rows of a and b must be 16-byte aligned", i);
    if (g->n_tokens > 0) {
      if (!k.a || !k.b || !k.y) return fail(QMV_ERR_ARG, "task %d: NULL a, b or y", i);
      if (!aligned16(k.a) || !aligned16(k.b) || !aligned16(k.y)) return fail(QMV_ERR_ALIGN, "task %d: a, b and y must be 16-byte aligned", i);
    }
    a.t[i] = {static_cast<const __nv_bfloat16*>(k.a), static_cast<const __nv_bfloat16*>(k.b), k.y, k.lda, k.ldb, k.ldy, k.N, k.y_type,
              (int32_t)(k.ldy * ys % 32 == 0 && (reinterpret_cast<uintptr_t>(k.y) & 31u) == 0)};
  }
  if (g->n_tokens == 0) return QMV_OK;
  if ((int64_t)g->max_tiles * n_tasks > INT32_MAX / 2) return fail(QMV_ERR_UNSUPPORTED, "max_tiles=%d of %d tasks", g->max_tiles, n_tasks);
  a.err = device_error_word();
  if (!a.err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");
  size_t smem = 0;
  const void* f = lora_tile(g->n_tokens) == kSmallTile ? run_kernel<kSmallTile / 16>(g->max_rank, &smem) : run_kernel<kLargeTile / 16>(g->max_rank, &smem);
  int per_sm = 0;
  int rc = kernel_fit(f, kLoraThreads, smem, &per_sm);
  if (rc) return rc;
  const int64_t units = (int64_t)g->max_tiles * n_tasks, resident = (int64_t)sm_count() * per_sm / kCluster;
  const int clusters = (int)(units < resident ? units : resident);
  void* args[] = {&a};
  cudaError_t e = kv8::launch_early(f, dim3((unsigned)(clusters * kCluster)), kLoraThreads, args, smem, static_cast<cudaStream_t>(stream), kCluster);
  if (e != cudaSuccess) return cuda_fail(e, "lora_run launch");
  return QMV_OK;
}

}  // extern "C"

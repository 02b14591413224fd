// Attention of a prompt's many query rows over the paged 8-bit cache
// (kv8_attend), on the fifth-generation tensor cores (tcgen05, accumulators in
// tensor memory).
//
// A block takes two tiles of 128 query rows (new tokens times the query heads of
// one KV head) of one request and walks the keys they see, 128 at a time (two
// pages). Both products are K-major in shared memory with the 128-byte swizzle:
// S = Q K^T with Q and K as fp16, and O += P V with P read from tensor memory and
// V as it is stored, transposed. Work is split by warps:
//   warps 0-3, 4-7   softmax of tile 0 and tile 1: a thread owns a row
//   warps 8-14       load the query rows and the pages' codes and turn them into fp16 tiles
//   warp 15          one thread issues the products (issued by one lane)
// with the registers moved from the last eight warps to the softmax (setmaxnreg).
// The order PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1) keeps the tensor cores on one tile
// while the other's softmax runs, and the commit behind QK_t(j+1) also covers
// PV_t(j): when a tile's softmax sees its next scores, its O may be rescaled.
//
// A page's V scale s_v enters in the exponent: with s a score and u = s + log2(s_v), P = 2^(u - M + 9) against a
// reference M of the row's own largest u, so that each key's weight in P V is held to 2^-11 of itself or 2^-33 of the
// largest weight that the row has, whatever other rows see. The softmax's sum has a reference m of its own among the
// scores. Rescaling is put off: a reference moves, to a whole number, only when its maximum has grown by more than 6.5; so
// P stays below 2^16 in fp16 and the accumulator in tensor memory is read back a few times per row and not once per step.
//
// What bounds it: per step and tile 2 * 128 * 128 * D multiply-adds, 1024 tensor
// clocks for D = 128, against 128 exponentials per row thread (the exponential
// unit) and 16 codes per conversion lane and register. Three chunks of up to 1500
// tokens over up to 4096 keys (40 and 8 heads of 128): 204 us, 0.97 PFLOP/s, half of
// the measured peak. A step takes about 3300 clocks for 2048 of products, because
// each tile's chain of scores, maximum, exponentials and P is as long as that, and a
// tile's next scores go where its scores and then P were, so they wait for PV. (P
// leaves half of those columns free, room for the scores of half a step ahead.) With cap and slopes 420 us
// (scores below half the cap; 550 where both sides of it meet: three special-function results per score in place of one).
#pragma once

#include <type_traits>

#include "kv8_attend.cuh"
#include "tcgen05.cuh"

namespace qmv {
namespace prompt {

using attend::Args;
using attend::ex2;
using attend::kLn2;
using attend::kLog2e;
using attend::Req;
using kv8::kPage;
using namespace umma;

constexpr int kWarps = 16, kThreads = kWarps * 32, kKeyThreads = 128, kValueThreads = 96;
// 512 threads are launched with 128 registers each; 256 * 176 + 256 * 80 = 512 * 128
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
constexpr int kRows = 128, kStep = 128;  // rows of a tile, keys of a step
constexpr int kHeld = 512;               // parts times rows that a join holds in shared memory: what L1 keeps counts (below)
// Steps of a part at least, and steps up to which an item stays whole: 100 tokens of 24 and 4 heads over 600 take 22 us whole
// and 33 in two parts; 20 tokens of 8 heads over 2048 32 us with parts of 4 steps and 35 with 6.
constexpr int kChunk = 4, kWhole = 6;
// Items the roles may be apart. The converters and the products are three steps apart at most, and an item has a step; but a
// softmax group sits out items of one row tile, and nothing of such an item waits for it: it gives back what it is past.
constexpr int kItems = 8;
constexpr float kSlack = 6.5f, kLift = 9.f;   // what a maximum may pass its reference by; P is 2^9 at the reference: 2^15.5 at most
// A page whose V scale is so far below the row's others that its P is 0 in fp16 anyway counts as 2^-60 of the reference, so that
// its sum does not leave the range of fp32.
constexpr float kLeast = -60.f;

// ---- two fp32 operations in one instruction
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// attend::capped_near of two scores
__device__ __forceinline__ uint64_t capped_near2(uint64_t s, uint64_t factor, uint64_t unit) {
  using namespace attend;
  const uint64_t X = mul2(s, factor), x = mul2(s, unit), y = mul2(X, X);
  const uint64_t r = fma2(fma2(fma2(two(kCap3, kCap3), y, two(kCap2, kCap2)), y, two(kCap1, kCap1)), y, two(kCap0, kCap0));
  return fma2(x, mul2(y, r), x);
}

template <int D>
struct Smem {
  // fp16 tiles in pieces of 64 columns: rows of 128 bytes
  alignas(1024) unsigned char q[2][D / 64][kRows * 128];
  alignas(1024) unsigned char k[2][D / 64][kStep * 128];
  alignas(1024) unsigned char v[2][kStep / 64][D * 128];
  alignas(8) uint64_t item_full[kItems], item_done[kItems], q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2][2], o_full[2];
  float2 scale[4][2];   // of the step's two pages: K scale (negative: no such page), log2 of the V scale
  int item[kItems];
  uint32_t tmem;
  int tiles_max[kWarps];
};

template <int D, bool SPLIT>
struct Shared : Smem<D> {};
template <int D>
struct Shared<D, true> : Smem<D> {
  float2 parts[2][kHeld];   // (maximum, sum) of a row tile's parts and rows, then their factors
  int last[2];
};

// A barrier of softmax group `tile` alone.
__device__ __forceinline__ void group_sync(int tile) { asm volatile("bar.sync %0, 128;" ::"r"(1 + tile) : "memory"); }

// Join `entries` parts of a row tile (rows at first + e * stride of the workspace) into rows row1 .. row1 + rows - 1 of a
// request's KV head h, by the 128 threads of a softmax group; written by other blocks too: read past L1. As many rows at a
// time as their parts' maxima and sums fit `held`. A function of its own, so that its registers are not the step loop's.
template <int D>
__device__ __noinline__ void join_parts(const Args& a, int64_t first, int stride, int entries, int row1, int rows, int qs, int h,
                                        float2* held, int group, int t) {
  const int at_once = max(1, min(rows, kHeld / entries));
  for (int r0 = 0; r0 < rows; r0 += at_once) {
    const int nr = min(at_once, rows - r0);
    const float2* ml = a.part_ml + first + r0;
#pragma unroll 4
    for (int i = t; i < entries * nr; i += kRows) {
      const int e = i / nr;
      held[i] = __ldcg(ml + (int64_t)e * stride + i - e * nr);
    }
    group_sync(group);
    if (t < nr) {
      float top = -INFINITY, sum = 0.f;
      for (int e = 0; e < entries; ++e) top = fmaxf(top, held[e * nr + t].x);
      const float use = top == -INFINITY ? 0.f : top;
      for (int e = 0; e < entries; ++e) {
        const float2 v = held[e * nr + t];
        const float w = ex2(v.x - use);
        held[e * nr + t].x = w;
        sum += w * v.y;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      for (int e = 0; e < entries; ++e) held[e * nr + t].x *= inv;
      if (a.lse) {
        const int rx = row1 + r0 + t, tx = a.by_g(rx);
        a.lse[(int64_t)(qs + tx) * a.Hq + h * a.G + rx - tx * a.G] = sum == 0.f ? -INFINITY : (use + log2f(sum)) * kLn2;
      }
    }
    group_sync(group);
    // Eight pieces of four values per thread at a time, part after part. A row's pieces and the rows of a part follow one
    // another, so that piece u + 128 i lies 128 i pieces further on. (Fewer pieces and several parts in flight, unrolled, took
    // 21 us in place of 10 for 128 rows of three parts.)
    constexpr int Q = D / 4, AT = 8;
    for (int u0 = t; u0 < nr * Q; u0 += AT * kRows) {
      const float4* from = reinterpret_cast<const float4*>(a.part_o + (first + r0) * D) + u0;
      float4 sum[AT];
#pragma unroll
      for (int i = 0; i < AT; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int e = 0; e < entries; ++e, from += (int64_t)stride * Q) {
        float4 v[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) v[i] = u0 + i * kRows < nr * Q ? __ldcg(from + i * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < AT; ++i) {
          if (u0 + i * kRows >= nr * Q) continue;
          const float w = held[e * nr + u0 / Q + i * (kRows / Q)].x;
          sum[i].x += w * v[i].x;
          sum[i].y += w * v[i].y;
          sum[i].z += w * v[i].z;
          sum[i].w += w * v[i].w;
        }
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const int u = u0 + i * kRows;
        if (u >= nr * Q) continue;
        const int rx = row1 + r0 + u / Q, tx = a.by_g(rx);
        attend::store4_as(a.out_type, a.out, (int64_t)(qs + tx) * a.ldo + (int64_t)(h * a.G + rx - tx * a.G) * D + (u % Q) * 4, sum[i]);
      }
    }
    group_sync(group);
  }
}

// One block's piece of work: up to two row tiles of one (request, KV head).
struct Item {
  Req r;
  int h, row0, tiles;   // first row; row tiles of 128
  int p0, pages, steps; // pages of it that any of its rows sees (p0 < 0: none), in steps of two
  int base, part, parts;  // number without its part, and the part of its keys
};

// SPLIT: an item's keys may be cut into parts (a kernel of its own, because the step loop of one that also joins parts is
// slower: 229 us in place of 212 on prompt chunks of 1500 tokens over up to 4096 keys, when it also held 24 KB more
// shared memory, which L1 then lacks).
template <int D, int TYPE, bool MODS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Args a) {
  constexpr int KH = D / 64;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Shared<D, SPLIT>& sm = *reinterpret_cast<Shared<D, SPLIT>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

  if (warp == kWarps - 1) tmem_alloc<512>(&sm.tmem);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      core::mbar_init(&sm.q_full[i], 128);
      core::mbar_init(&sm.k_full[i], kKeyThreads);
      core::mbar_init(&sm.k_empty[i], 1);
      core::mbar_init(&sm.v_full[i], kValueThreads);
      core::mbar_init(&sm.v_empty[i], 1);
      core::mbar_init(&sm.s_full[i], 1);
      core::mbar_init(&sm.p_full[i][0], 128);
      core::mbar_init(&sm.p_full[i][1], 128);
      core::mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      core::mbar_init(&sm.item_full[i], 1);
      core::mbar_init(&sm.item_done[i], 8);   // the warps of the softmax
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  kv8::let_next_begin();
  kv8::follow_previous();
  // the largest number of row-tile pairs of a request
  int most = 0;
  for (int b = tid; b < a.B; b += kThreads) most = max(most, (attend::load_req4(a, b).y * a.G + 2 * kRows - 1) / (2 * kRows));
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) sm.tiles_max[warp] = most;
  fence_before();
  __syncthreads();
  fence_after();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) most = max(most, sm.tiles_max[i]);
  const uint32_t tmem = sm.tmem;
  // Items in the order of their tiles from the last (which sees the most keys) to the first, then request and head.
  // Blocks take them one after another from a counter: an item's cost varies by its request's context, and which block
  // computes it does not change its result.
  // Where there are fewer items than blocks, an item's keys are cut into up to n_split parts, each an item of its own; what
  // they leave is joined by the last of them to arrive.
  const int per = a.B * a.H, n_base = most * per;   // at most (rows + 255 B) / 256 * H: below 2^31 for any call the host lets through
  const int n_split = SPLIT && n_base > 0 && n_base <= (int)gridDim.x ? (int)gridDim.x / n_base : 1, n_items = n_base * n_split;
  auto item_of = [&](int i, Item& it) {
    it.base = SPLIT ? i / n_split : i;
    it.part = SPLIT ? i - it.base * n_split : 0;
    const int pair = most - 1 - it.base / per, rest = it.base % per;
    it.r = attend::make_req(a, rest / a.H, attend::load_req4(a, rest / a.H), kRows);
    it.h = rest % a.H;
    it.row0 = pair * 2 * kRows;
    if (it.row0 >= it.r.rows) return false;
    it.tiles = it.r.rows - it.row0 > kRows ? 2 : 1;
    attend::tile_pages(a, it.r, pair, 2 * kRows, it.p0, it.pages);
    it.steps = (it.pages + 1) / 2;
    it.parts = 1;
    if (SPLIT && n_split > 1) {
      const int chunk = it.steps <= kWhole ? it.steps : max((it.steps + n_split - 1) / n_split, kChunk), first = it.part * chunk;
      it.parts = (it.steps + chunk - 1) / chunk;
      if (it.part >= it.parts) return false;
      it.steps = min(chunk, it.steps - first);
      if (it.p0 >= 0) it.p0 += 2 * first;
      it.pages = min(it.pages - 2 * first, 2 * it.steps);
    }
    return true;
  };

  // the k-th item of this block, as the converters' first lane publishes it
  auto next_item = [&](uint32_t k, Item& it) {
    if (!core::mbar_wait(&sm.item_full[k % kItems], (k / kItems) & 1, a.err)) return false;
    const int i = sm.item[k % kItems];
    return i >= 0 && item_of(i, it);
  };

  uint32_t n = 0;   // steps taken so far, over all items: stage n & 1, parity (n >> 1) & 1

  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp < 8) {
    // ------------------------------------------------------------------ softmax of tile `tile`: a thread owns a row
    const int tile = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + tile * 128, o_at = tmem + lanes + 256 + tile * 128;
    uint32_t n_mine = 0;   // steps this tile has taken
    uint32_t n_out = 0;
    // The thread's query row at `at` (negative: zeros) as fp16 with its largest magnitude in [2^13, 2^14); returns the
    // factor from product to score. 16-bit rows are read in one flight, fp32 rows twice.
    auto query_row = [&](int64_t at) {
      const bool wide = a.x_type == QMV_F32;
      uint4 raw[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        raw[c] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && !wide) raw[c] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at)[c];
      }
      auto put = [&](int c, const float (&v)[8], float f) {
        *reinterpret_cast<uint4*>(&sm.q[tile][c >> 3][row * 128 + (((c & 7) ^ (row & 7)) << 4)]) =
            make_uint4(attend::pack_h2(v[0] * f, v[1] * f), attend::pack_h2(v[2] * f, v[3] * f),
                       attend::pack_h2(v[4] * f, v[5] * f), attend::pack_h2(v[6] * f, v[7] * f));
      };
      float top = 0.f;
      if (wide) {
        const float* x = static_cast<const float*>(a.q) + max(at, (int64_t)0);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          float v[8];
          kv8::load8(x + 8 * c, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) top = fmaxf(top, fabsf(v[q]));
        }
        if (at < 0) top = 0.f;
      } else {
        uint32_t most16 = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) most16 = __vmaxu2(most16, x[q] & 0x7FFF7FFFu);
        }
        most16 = max(most16 & 0xFFFFu, most16 >> 16);
        top = a.x_type == QMV_BF16 ? __uint_as_float(most16 << 16) : __half2float(__ushort_as_half((unsigned short)most16));
      }
      const int e = min(max(13 + 127 - (int)(__float_as_uint(top) >> 23), -126), 126);
      const float f = core::exp2i(e);
      if (wide) {
        const float* x = static_cast<const float*>(a.q) + max(at, (int64_t)0);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          float v[8];
          kv8::load8(x + 8 * c, v);
          put(c, v, at < 0 ? 0.f : f);
        }
      } else if (a.x_type == QMV_BF16) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          float v[8];
          kv8::load8(reinterpret_cast<const __nv_bfloat16*>(&raw[c]), v);
          put(c, v, f);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          float v[8];
          kv8::load8(reinterpret_cast<const __half*>(&raw[c]), v);
          put(c, v, f);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      attend::mbar_arrive(&sm.q_full[tile]);
      return core::exp2i(-e) * a.scale * (MODS ? 1.f : kLog2e);
    };
    Item it;
    for (uint32_t k = 0; next_item(k, it); ++k) {
      const bool in_use = tile < it.tiles;
      const int rr = it.row0 + tile * kRows + row;
      const bool real = rr < it.r.rows;
      const int last = min(rr, it.r.rows - 1), tok = a.by_g(last), hq = it.h * a.G + last - tok * a.G;
      float mult = 0.f;
      if (in_use) mult = query_row(real ? (int64_t)(it.r.qs + tok) * a.ldq + (int64_t)hq * D : (int64_t)-1);
      const int pos = it.r.ctx - it.r.qlen + tok;
      const int hi = min(max(pos + 1, it.r.pfx), it.r.ctx);
      const int lo = attend::first_key(a, pos);
      const int hi_all = __reduce_min_sync(0xFFFFFFFFu, hi), lo_all = __reduce_max_sync(0xFFFFFFFFu, lo);
      const float slope = MODS && a.slopes ? a.slopes[hq] * kLog2e : 0.f;
      float m = -INFINITY, l = 0.f, M = -INFINITY;   // references of scores and of scores with the V scale; sum in units of 2^m
      if (in_use) {
        for (int j = 0; j < it.steps; ++j) {
          core::mbar_wait(&sm.s_full[tile], n_mine & 1, a.err);
          fence_after();
          const float2 sc0 = sm.scale[(n + j) & 3][0], sc1 = sm.scale[(n + j) & 3][1];
          const int key0 = (it.p0 + 2 * j) * kPage;
          float f0 = fmaxf(mult * sc0.x, 1e-37f), f1 = fmaxf(mult * sc1.x, 1e-37f);
          const bool cut = sc0.x < 0.f || sc1.x < 0.f || key0 < lo_all || key0 + kStep > hi_all;
          uint32_t x[128];   // the row's scores, until their p goes back to the same columns
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, x + 32 * c);
          wait_ld();
          if (MODS) {
            // cap and distance bias: the scores as they are wanted, in units of log2
            if (a.softcap > 0.f) {
              const float c0 = attend::cap_factor(a.softcap, f0), c1 = attend::cap_factor(a.softcap, f1), cap = a.softcap * kLog2e;
              const float u0 = f0 * kLog2e, u1 = f1 * kLog2e;
              float big[2] = {0.f, 0.f};
#pragma unroll
              for (int q = 0; q < 128; q += 2)
                big[q >> 6] = fmaxf(big[q >> 6], fmaxf(fabsf(__uint_as_float(x[q])), fabsf(__uint_as_float(x[q + 1]))));
              // one branch for the warp: scores far below the cap, as they mostly are, need no special function
              if (__all_sync(0xFFFFFFFFu, fmaxf(big[0] * c0, big[1] * c1) <= attend::kNear)) {
#pragma unroll
                for (int q = 0; q < 128; q += 2) {
                  const float c = q < 64 ? c0 : c1, u = q < 64 ? u0 : u1;
                  float lo, hi;
                  split(capped_near2(two(__uint_as_float(x[q]), __uint_as_float(x[q + 1])), two(c, c), two(u, u)), lo, hi);
                  x[q] = __float_as_uint(lo);
                  x[q + 1] = __float_as_uint(hi);
                }
              } else {
#pragma unroll
                for (int q = 0; q < 128; ++q) x[q] = __float_as_uint(attend::capped(__uint_as_float(x[q]), q < 64 ? c0 : c1, q < 64 ? u0 : u1, cap));
              }
            } else {
#pragma unroll
              for (int q = 0; q < 128; ++q) x[q] = __float_as_uint(__uint_as_float(x[q]) * ((q < 64 ? f0 : f1) * kLog2e));
            }
            if (a.slopes) {
              const float gap = (float)(pos - key0);
#pragma unroll
              for (int q = 0; q < 128; ++q) x[q] = __float_as_uint(fmaf(-slope, fabsf(gap - q), __uint_as_float(x[q])));
            }
            f0 = f1 = 1.f;
          }
          if (cut) {
            const int from = max(lo, 0) - key0, to = hi - key0;
            const int from0 = sc0.x < 0.f ? kStep : from, from1 = sc1.x < 0.f ? kStep : from;
#pragma unroll
            for (int q = 0; q < 128; ++q)
              if (q < (q < 64 ? from0 : from1) || q >= to) x[q] = __float_as_uint(-INFINITY);
          }
          float top[4];   // of halves of the pages
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            top[c] = __uint_as_float(x[32 * c]);
#pragma unroll
            for (int q = 1; q < 31; q += 2)
              top[c] = fmaxf(top[c], fmaxf(__uint_as_float(x[32 * c + q]), __uint_as_float(x[32 * c + q + 1])));
            top[c] = fmaxf(top[c], __uint_as_float(x[32 * c + 31]));
          }
          const float top0 = fmaxf(top[0], top[1]) * f0, top1 = fmaxf(top[2], top[3]) * f1;

          // the references, and O after moving its own (a row that has seen no key yet has none: -infinity)
          const float mx = fmaxf(top0, top1), mu = fmaxf(top0 + sc0.y, top1 + sc1.y);
          if (__any_sync(0xFFFFFFFFu, mx > m + kSlack || mu > M + kSlack)) {
            const float m_to = mx > m + kSlack ? ceilf(mx) : m, M_to = mu > M + kSlack ? ceilf(mu) : M;
            if (m_to != m) l *= ex2(m - m_to);   // l is 0 until there is a reference
            const float fix = M_to != M && M != -INFINITY ? ex2(M - M_to) : 1.f;
            m = m_to;
            M = M_to;
            if (j > 0 && __any_sync(0xFFFFFFFFu, fix != 1.f)) {
              // eight columns at a time: the scores fill the registers
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) {
                uint32_t y[8];
                tmem_ld8(o_at + 8 * c, y);
                wait_ld();
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] = __float_as_uint(__uint_as_float(y[q]) * fix);
                tmem_st8(o_at + 8 * c, y);
              }
            }
          }
          const float use = m == -INFINITY ? 0.f : m, use_u = M == -INFINITY ? 0.f : M;
          // P = 2^(score + shift): sixteen-bit pairs to tensor memory, their sum to l
#pragma unroll
          for (int page = 0; page < 2; ++page) {
            const float f = page ? f1 : f0, shift = fmaxf((page ? sc1.y : sc0.y) - use_u + kLift, kLeast - use);
            const uint64_t f2 = two(f, f), off = two(shift, shift);
            uint64_t sum0 = two(0.f, 0.f), sum1 = sum0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t p[16];
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                const int at = 64 * page + 32 * c + 2 * q;
                float p0, p1;
                split(fma2(two(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), f2, off), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                if (q & 1) sum1 = add2(sum1, two(p0, p1));
                else sum0 = add2(sum0, two(p0, p1));
                p[q] = attend::pack_h2(p0, p1);
              }
              tmem_st16(s_at + 32 * page + 16 * c, p);
            }
            wait_st();
            fence_before();
            attend::mbar_arrive(&sm.p_full[tile][page]);   // the product with this page may begin
            float a0, a1;
            split(add2(sum0, sum1), a0, a1);
            l = fmaf(a0 + a1, ex2(-shift - use), l);
          }
          ++n_mine;
        }
        // ---- output
        core::mbar_wait(&sm.o_full[tile], n_out & 1, a.err);
        ++n_out;
        fence_after();
        const int64_t at = (int64_t)(it.r.qs + tok) * a.ldo + (int64_t)hq * D;
        const bool part = SPLIT && it.parts > 1;
        const int64_t mine = (int64_t)(it.base * n_split + it.part) * 2 * kRows + tile * kRows + row;   // of a part's rows
        // from units of 2^(M - 9) to those of 2^m, in two factors that stay in range
        const float half = l == 0.f ? 0.f : ex2(0.5f * (M - kLift - m)), rest = part || l == 0.f ? half : half / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t y[32];
          tmem_ld32(o_at + 32 * c, y);
          wait_ld();
          if (real) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float v[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) v[x] = l == 0.f ? 0.f : __uint_as_float(y[8 * q + x]) * half * rest;
              if (part) kv8::store8(a.part_o + mine * D + 32 * c + 8 * q, v);
              else kv8::store8_as(a.out_type, a.out, at + 32 * c + 8 * q, v);
            }
          }
        }
        if (!part && real && a.lse) a.lse[(int64_t)(it.r.qs + tok) * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        if constexpr (SPLIT) {
          if (part) {
            // the last of the row tile's parts to arrive joins them in their order
            if (real) a.part_ml[mine] = make_float2(m, l);
            __threadfence();
            group_sync(tile);
            if (row == 0) {
              int* counter = a.counters + 2 + it.base * 2 + tile;
              const int old = atomicAdd(counter, 1);
              sm.last[tile] = old == it.parts - 1;
              if (old == it.parts - 1) *counter = 0;
              __threadfence();
            }
            group_sync(tile);
            if (sm.last[tile]) {
              const int row1 = it.row0 + tile * kRows;
              join_parts<D>(a, (int64_t)it.base * n_split * 2 * kRows + tile * kRows, 2 * kRows, it.parts, row1,
                            min(kRows, it.r.rows - row1), it.r.qs, it.h, sm.parts[tile], tile, row);
            }
          }
        }
        fence_before();
      }
      n += it.steps;
      __syncwarp();
      if (lane == 0) attend::mbar_arrive(&sm.item_done[k % kItems]);
    }
  } else if (warp < kWarps - 1) {
    // ------------------------------------------------------------------ codes to fp16 tiles
    constexpr int P = kPage * D / 16;   // 16-byte pieces of a page's K or V tile
    int win = -1;                       // this lane's page of a window of 32
    // Pages 2 j and 2 j + 1 of the item: their pieces w, w + T, ... of the tile at byte `part` of a page's codes.
    auto fetch = [&](const Item& it, int j, int part, int w, auto& to, auto threads, float2* sc) {
      constexpr int T = decltype(threads)::value, U = (P + T - 1) / T;
      constexpr uint32_t zero = TYPE == QMV_KV_INT8 ? 0x80808080u : 0u;
      if ((j & 15) == 0) {
        win = -1;
        const int p = 2 * j + lane;
        if (it.p0 >= 0 && p < it.pages) {
          win = a.table[(int64_t)it.r.b * a.ld_table + it.p0 + p];
          if (win < 0 || win >= a.n_pages) {
            atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
            win = -1;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int page = __shfl_sync(0xFFFFFFFFu, win, (2 * j + e) & 31);
        const int64_t at = (int64_t)max(page, 0) * a.H + it.h;
        const uint4* src = reinterpret_cast<const uint4*>(a.cache + at * (2 * kPage * D) + part) + w;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          to[e * U + u] = make_uint4(zero, zero, zero, zero);
          if (page >= 0 && w + T * u < P) to[e * U + u] = src[T * u];
        }
        if (sc) {
          sc[e] = make_float2(-1.f, 0.f);
          if (page >= 0) sc[e] = reinterpret_cast<const float2*>(a.cache + a.scale_off)[at];
        }
      }
    };
    // sixteen codes to two 16-byte pieces of a row of 128 bytes (`at`: the first piece's place, swizzled)
    auto put = [&](unsigned char* tile, int at, uint4 x) {
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) attend::codes_to_half<TYPE>(attend::word4(x, k), o[2 * k], o[2 * k + 1]);
      *reinterpret_cast<uint4*>(tile + at) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(tile + (at ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
    };
    Item it;
    if (warp < 12) {
      // ---------------------------------------------------------------- K, the scales, the items
      constexpr int T = kKeyThreads, U = (P + T - 1) / T;
      const int w = tid - 256;
      int k_at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // piece ((g3 * KH + half) * 8 + g) * 4 + t: token 16 (g / 2) + 2 g3 + g % 2, values 64 half + 16 t ..
        const int q = w + T * u, t = q & 3, g = (q >> 2) & 7, half = KH == 2 ? (q >> 5) & 1 : 0, g3 = q >> (KH == 2 ? 6 : 5);
        const int row = 16 * (g >> 1) + 2 * g3 + (g & 1);
        k_at[u] = half * (kStep * 128) + row * 128 + (((2 * t) ^ (row & 7)) << 4);
      }
      // the first lane takes the block's next item
      auto take = [&](uint32_t k) {
        if (w != 0) return;
        if (k >= kItems) core::mbar_wait(&sm.item_done[k % kItems], (k / kItems - 1) & 1, a.err);   // its last use is over
        Item next;
        int i;
        do i = atomicAdd(a.counters, 1);
        while (i < n_items && !item_of(i, next));
        sm.item[k % kItems] = i < n_items ? i : -1;
        attend::mbar_arrive(&sm.item_full[k % kItems]);
      };
      take(0);
      for (uint32_t k = 0; next_item(k, it); ++k) {
        uint4 raw[2 * U];
        float2 sc[2];
        fetch(it, 0, 0, w, raw, std::integral_constant<int, T>(), sc);
        for (int j = 0; j < it.steps; ++j, ++n) {
          const int stage = n & 1;
          core::mbar_wait(&sm.k_empty[stage], ((n >> 1) & 1) ^ 1, a.err);
          // a page of zeros has no scale: it counts as less than any
          if (w < 2) {
            const float2 s = w ? sc[1] : sc[0];
            sm.scale[n & 3][w] = make_float2(s.x, s.y > 0.f ? log2f(s.y) : -150.f);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (w + T * u < P) put(sm.k[stage][0] + e * 64 * 128, k_at[u], raw[e * U + u]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          attend::mbar_arrive(&sm.k_full[stage]);
          if (j + 1 < it.steps) fetch(it, j + 1, 0, w, raw, std::integral_constant<int, T>(), sc);
        }
        take(k + 1);
      }
    } else {
      // ---------------------------------------------------------------- V
      constexpr int T = kValueThreads, U = (P + T - 1) / T;
      const int w = tid - 384;
      int v_at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = w + T * u;   // piece: value q / 4, tokens 16 (q % 4) ..
        v_at[u] = (q >> 2) * 128 + (((2 * (q & 3)) ^ ((q >> 2) & 7)) << 4);
      }
      for (uint32_t k = 0; next_item(k, it); ++k) {
        uint4 raw[2 * U];
        fetch(it, 0, kPage * D, w, raw, std::integral_constant<int, T>(), nullptr);
        for (int j = 0; j < it.steps; ++j, ++n) {
          const int stage = n & 1;
          const bool tail = (it.p0 + 2 * j + 2) * kPage > it.r.ctx;   // slots past the request's end may hold any byte
          core::mbar_wait(&sm.v_empty[stage], ((n >> 1) & 1) ^ 1, a.err);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              uint4 x = raw[e * U + u];
              if (TYPE == QMV_KV_E4M3 && tail)
                x = make_uint4(attend::drop_nan(x.x), attend::drop_nan(x.y), attend::drop_nan(x.z), attend::drop_nan(x.w));
              if (w + T * u < P) put(sm.v[stage][e], v_at[u], x);
            }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          attend::mbar_arrive(&sm.v_full[stage]);
          if (j + 1 < it.steps) fetch(it, j + 1, kPage * D, w, raw, std::integral_constant<int, T>(), nullptr);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ the products
    constexpr uint32_t qk = mma_shape(kStep), pv = mma_shape(D);
    uint32_t n_p[2] = {0, 0}, n_q[2] = {0, 0};   // steps and items each tile has taken
    Item it;
    for (uint32_t k = 0; next_item(k, it); ++k) {
      auto scores = [&](int tile, int stage) {
        if (attend::elected()) {
#pragma unroll
          for (int hh = 0; hh < KH; ++hh) {
            const uint64_t qa = operand(core::smem_addr(sm.q[tile][hh])), kb = operand(core::smem_addr(sm.k[stage][hh]));
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_ss(tmem + tile * 128, qa + 2 * s, kb + 2 * s, qk, hh + s > 0);
          }
          commit(&sm.s_full[tile]);
        }
        __syncwarp();
      };
      core::mbar_wait(&sm.k_full[n & 1], (n >> 1) & 1, a.err);
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        if (tile >= it.tiles) continue;
        core::mbar_wait(&sm.q_full[tile], n_q[tile] & 1, a.err);
        ++n_q[tile];
        fence_after();
        scores(tile, n & 1);
      }
      if (attend::elected()) commit(&sm.k_empty[n & 1]);
      __syncwarp();
      for (int j = 0; j < it.steps; ++j, ++n) {
        const int stage = n & 1, next = (n + 1) & 1;
        const bool more = j + 1 < it.steps;
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          if (tile >= it.tiles) continue;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            core::mbar_wait(&sm.p_full[tile][e], n_p[tile] & 1, a.err);
            if (tile == 0 && e == 0) core::mbar_wait(&sm.v_full[stage], (n >> 1) & 1, a.err);
            fence_after();
            if (attend::elected()) {
              const uint64_t vb = operand(core::smem_addr(sm.v[stage][e]));
#pragma unroll
              for (int s = 0; s < 4; ++s)
                mma_ts(tmem + 256 + tile * 128, tmem + tile * 128 + (e * 4 + s) * 8, vb + 2 * s, pv, j > 0 || e + s > 0);
              if (!more && e == 1) commit(&sm.o_full[tile]);
            }
            __syncwarp();
          }
          ++n_p[tile];
          if (more) {
            if (tile == 0) {
              core::mbar_wait(&sm.k_full[next], ((n + 1) >> 1) & 1, a.err);
              fence_after();
            }
            scores(tile, next);
          }
        }
        if (attend::elected()) {
          commit(&sm.v_empty[stage]);
          if (more) commit(&sm.k_empty[next]);
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kWarps - 1) tmem_free<512>(tmem);
  // the last block leaves the counters as it found them
  if (tid == 0 && atomicAdd(a.counters + 1, 1) == (int)gridDim.x - 1) a.counters[0] = a.counters[1] = 0;
}

template <int D, int TYPE, bool MODS, bool SPLIT>
int launch(const Args& a, int blocks, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(prompt_kernel<D, TYPE, MODS, SPLIT>);
  int per_sm = 0;
  int rc = kernel_fit(f, kThreads, sizeof(Shared<D, SPLIT>), &per_sm);
  if (rc) return rc;
  Args copy = a;
  void* args[] = {&copy};
  cudaError_t e = kv8::launch_early(f, dim3(blocks), kThreads, args, sizeof(Shared<D, SPLIT>), s);
  if (e != cudaSuccess) return cuda_fail(e, "kv8_attend launch");
  return QMV_OK;
}

// One translation unit per type of codes and head size.
int launch_64_int8(const Args& a, bool mods, bool split, int blocks, cudaStream_t s);
int launch_64_e4m3(const Args& a, bool mods, bool split, int blocks, cudaStream_t s);
int launch_128_int8(const Args& a, bool mods, bool split, int blocks, cudaStream_t s);
int launch_128_e4m3(const Args& a, bool mods, bool split, int blocks, cudaStream_t s);

template <int D, int TYPE>
int launch_any(const Args& a, bool mods, bool split, int blocks, cudaStream_t s) {
  if (split) return mods ? launch<D, TYPE, true, true>(a, blocks, s) : launch<D, TYPE, false, true>(a, blocks, s);
  return mods ? launch<D, TYPE, true, false>(a, blocks, s) : launch<D, TYPE, false, false>(a, blocks, s);
}

}  // namespace prompt
}  // namespace qmv

// Attention over the paged 8-bit KV cache for decode and verification steps
// (kv8_attend), on the warp-level tensor cores.
//
// Work. The query rows of a (request, KV head) are its new tokens times the G
// query heads that share the KV head; they are cut into tiles of 8 * N * R rows.
// A unit is one page of one (request, row tile, KV head); all units of a call, in
// that order with the pages innermost, form one line that is cut into equal
// pieces, one per stream. A block has kWarps / R streams of R warps each; every
// warp of a stream holds 8 * N rows and all of them read the stream's pages. So
// the streams' loads differ by one page at most, whatever the mix of lengths, and
// no schedule has to be made on the host: a block sums the units of all requests
// (one load per request, a block scan) and finds its streams' starts.
//
// A stream walks its piece of the line with the running maximum and sum of a
// softmax per row. Where it covers all pages of a tile it writes the result;
// else it leaves (sum p v, maximum, sum p) in shared memory (its last tile) or in
// the workspace (its first, while the ring is still in use). The block joins its
// streams' partial tiles, and the last block to arrive at a tile that is cut
// between blocks joins the blocks' in their order: the result does not depend
// on timing.
//
// What bounds it: the cache's bytes where there are many (64 requests of up to
// 16384 tokens, 1.16 GB: 184 us, 6.3 TB/s, 0.92 of the measured copy rate); for few
// requests the launch and a chain of dependent loads (one token over 300 tokens 7.5 us, over
// 1000 9.5), then the products of one page per stream at a time; with 25 rows the
// latency of mma.sync at two warps per scheduler (5 tokens over 32771: 42 us).
//
// Data. A page's K or V tile is one contiguous piece of 64 * D bytes, fetched by
// one bulk copy into the stream's ring, its two scales by an asynchronous 8-byte
// copy that completes on the same barrier. The products are taken transposed, S^T
// = K Q^T and O^T = V^T P^T, with the tokens (then the values of a head) as the 16
// rows of m16n8k16 and the query rows as its 8 columns: the rows of a decode step
// are few (5 for 40 query and 8 KV heads), so a tile of 8 wastes less than one of
// 16, and a code is turned into fp16 once for all N column tiles. The cache's
// tiles are stored in the order of the A fragments: a lane's 16 bytes of K are
// four k-steps of one token, its 16 bytes of V four k-steps (sixteen tokens) of
// one d, so both are read with conflict-free 16-byte loads, and P^T goes from
// accumulator to B fragment by one 8 x 8 transpose per eight tokens. Codes become
// fp16 exactly: int8 as 1024 + byte by a byte permute and a subtraction, e4m3 by
// the conversion instruction. q is scaled per row by a power of two into fp16, so
// q . k is exact up to its fp32 sum for fp16 and, down to 2^-27 of a row's largest
// value, bf16 queries (their 8 bits fit in 11); fp32 queries are rounded to 11 bits,
// since a second product with what is left of them would double the scores' work. The page's K scale multiplies the scores, its
// V scale the page's product with V: in fp32 both, after the sum over the page.
#pragma once

#include "gemv_core.cuh"
#include "kv8.cuh"
#include "tcgen05.cuh"

namespace qmv {
namespace attend {

using kv8::kPage;

struct Args {
  const unsigned char* cache;
  int64_t scale_off, n_pages;
  const void* q;
  void* out;
  float* lse;
  int64_t ldq, ldo, ld_table;
  int x_type, out_type;
  int B, T, Hq, H, G;
  const int32_t *q_start, *ctx, *table, *prefix;
  const float* slopes;
  int max_pages, window;
  float scale, softcap;
  float* part_o;         // [blocks][kPartRows][D]: the streams' first tiles, then two tiles of the block
  float2* part_ml;       // the same with one (maximum, sum) per row
  int* counters;         // [blocks], zero between calls
  uint32_t g_mul, g_shift;
  // n / G for n below 2^31: G's rounded-up reciprocal, exact in this range
  __device__ __forceinline__ int by_g(int n) const { return (int)(((uint64_t)(uint32_t)n * g_mul) >> g_shift); }
  int* err;
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A row's reference lies 2^15 below its maximum, so that p reaches 2^15 in fp16 and is held down to 2^-40 of the largest: against
// the maximum itself, keys below 2^-25 of it would leave the product with V but not the sum, however many they are.
constexpr float kLift = 15.f;
constexpr int kStreamRows = 128, kPartRows = 256;   // rows per block of the workspace: of its streams, in all

template <int D, int N, int R>
struct Shape {
  static constexpr int kWarps = D == 64 && N == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStreams = kWarps / R;
  static constexpr int kTile = kPage * D;   // bytes of a K or V tile
  // A ring of 128 KB: a tile of K and one of V for each warp (D = 128). With 64 requests up to 16384 tokens (1.16 GB): 188 us;
  // 195 with 192 KB, and 199 with twelve warps and 192 KB, because more bytes in flight are shared out less evenly between
  // near and far SMs and the slowest block ends the call; 194 with six warps.
  static constexpr int kStages = 128 * 1024 / kStreams / kTile;
  static_assert(kStages % 2 == 0, "K in even stages, V in odd ones");
  static constexpr int kRows = 8 * N * R;
  static constexpr int kReqs = 256;   // requests kept in shared memory
  // How tiles are cut between blocks. Up to kAlone pages in a call's longest tile each has a block of its own; else a block
  // takes kCut pages or more of one tile, or the line of all is cut evenly where that saves a block more than kUneven pages.
  static constexpr int kAlone = kStreams * 6, kCut = kStreams * 2, kUneven = kStreams * 4;
};

struct Req {
  int b, qs, qlen, ctx, pfx, rows, tiles;
};
__device__ __forceinline__ Req make_req(const Args& a, int b, int4 v, int tile_rows) {
  Req r;
  r.b = b;
  r.qs = v.x;
  r.qlen = v.y;
  r.ctx = v.z;
  r.pfx = v.w;
  r.rows = r.qlen * a.G;
  r.tiles = (r.rows + tile_rows - 1) / tile_rows;
  return r;
}
__device__ __forceinline__ int4 load_req4(const Args& a, int b) {
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], ctx = a.ctx[b], pfx = a.prefix ? a.prefix[b] : 0;
  const int s = min(max(q0, 0), a.T), e = min(max(q1, 0), a.T);
  return make_int4(s, max(e - s, 0), (int)min((int64_t)max(ctx, 0), (int64_t)a.max_pages * kPage), pfx);
}
// First key that a row at `pos` sees (0 or less: from the first on). A row before the first key sees the prefix alone, from its
// beginning; its position is left out of the subtraction, which then stays in range for every window.
__device__ __forceinline__ int first_key(const Args& a, int pos) { return a.window > 0 ? max(pos, 0) - a.window + 1 : 0; }
// Pages [p0, p0 + n) that hold the keys seen by a row tile; p0 = -1, n = 1 where it sees none.
__device__ __forceinline__ void tile_pages(const Args& a, const Req& r, int tile, int tile_rows, int& p0, int& n) {
  const int first = a.by_g(tile * tile_rows), last = a.by_g(min(r.rows, (tile + 1) * tile_rows) - 1);
  const int base = r.ctx - r.qlen;
  const int hi = min(max(base + last + 1, r.pfx), r.ctx);
  const int lo = max(0, first_key(a, base + first));
  if (hi <= lo) {
    p0 = -1;
    n = 1;
    return;
  }
  p0 = lo / kPage;
  n = (hi + kPage - 1) / kPage - p0;
}
// Units of a request; `longest`: the most pages that a tile of it has, or what it was.
__device__ __forceinline__ long long req_units(const Args& a, const Req& r, int tile_rows, int& longest) {
  long long u = 0;
  for (int k = 0; k < r.tiles; ++k) {
    int p0, n;
    tile_pages(a, r, k, tile_rows, p0, n);
    u += n;
    longest = max(longest, n);
  }
  return u * a.H;
}
// Blocks of a request whose tiles are cut into parts of up to `most` pages.
__device__ __forceinline__ int req_parts(const Args& a, const Req& r, int tile_rows, int most) {
  int c = 0;
  for (int k = 0; k < r.tiles; ++k) {
    int p0, n;
    tile_pages(a, r, k, tile_rows, p0, n);
    c += (n + most - 1) / most;
  }
  return c * a.H;
}

// A place on the line of units: a tile of a request, a KV head, and its pages.
struct Walk {
  Req r;
  int tile, h, p0, n;
  long long start;  // first unit of this (request, tile, head) on the line
};

// n units over k parts: part i begins at i * (n / k) + min(i, n % k).
struct Cut {
  long long q;
  int r;
  __device__ __forceinline__ long long at(int i) const { return i * q + min(i, r); }
  __device__ __forceinline__ int part_of(long long x) const {
    const long long big = r * (q + 1);
    return x < big ? (int)(x / (q + 1)) : r + (int)((x - big) / q);
  }
};
__device__ __forceinline__ Cut cut(long long n, int k) {
  if (n < (1ll << 31)) return {(long long)((unsigned)n / (unsigned)k), (int)((unsigned)n % (unsigned)k)};
  return {n / k, (int)(n % k)};
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap * tanh(x / cap) of the score x = s f in units of log2, from the product s. Far from zero it is cap - 2 cap /
// (exp(2 x / cap) + 1): the sum is 1 or more, so that the reciprocal of infinity is 0. Near zero that difference would keep an
// error of 2^-23 of the cap, however small the score; up to |x / cap| = 1/2 it is x + x y r(y), y = X^2 with X the argument of the
// base-2 exponential (2 log2(e) x / cap) and r of degree 3 through the Chebyshev nodes: within 2^-23 of the score. Prompts with a
// cap 345 us with the difference alone, 361 with the polynomial for a warp whose scores are all near, 508 with both for all.
// `factor` is X / s, held finite so that a product of 0 stays 0 under the smallest caps, `unit` x / s, `cap` in units of log2.
__device__ __forceinline__ float cap_factor(float softcap, float f) { return fminf(f * (2.f * kLog2e / softcap), 1e37f); }
constexpr float kCap3 = 3.744247806e-6f, kCap2 = -9.251437586e-5f, kCap1 = 1.923213713e-3f, kCap0 = -4.003772512e-2f;   // of r, from the highest
constexpr float kNear = kLog2e;   // |X| up to which the polynomial serves
__device__ __forceinline__ float capped_near(float s, float factor, float unit) {
  const float X = s * factor, x = s * unit, y = X * X;
  return fmaf(x, y * fmaf(fmaf(fmaf(kCap3, y, kCap2), y, kCap1), y, kCap0), x);
}
__device__ __forceinline__ float capped(float s, float factor, float unit, float cap) {
  const float X = s * factor;
  float q;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(ex2(X) + 1.f));
  return fabsf(X) <= kNear ? capped_near(s, factor, unit) : fmaf(-2.f * cap, q, cap);
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit values: row g, columns 2t and 2t + 1 in, row and column exchanged out
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return h2_bits(__floats2half2_rn(lo, hi)); }

// Four codes to two fp16 pairs, exactly.
template <int TYPE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (TYPE == QMV_KV_INT8) {
    const __half2 bias = __floats2half2_rn(1152.f, 1152.f);  // 1024 + 128
    const uint32_t l = __byte_perm(w, 0x64646464u, 0x4140), h = __byte_perm(w, 0x64646464u, 0x4342);
    lo = h2_bits(__hsub2(core::as_h2(l), bias));
    hi = h2_bits(__hsub2(core::as_h2(h), bias));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}
__device__ __forceinline__ uint32_t word4(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// Bytes that are an e4m3 NaN become 0.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w) { return w & ~__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

__device__ __forceinline__ void store_as(int type, void* base, int64_t i, float x, float y) {
  if (type == QMV_F32) *reinterpret_cast<float2*>(static_cast<float*>(base) + i) = make_float2(x, y);
  else if (type == QMV_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(base) + i) = h;
  } else {
    *reinterpret_cast<__half2*>(static_cast<__half*>(base) + i) = __floats2half2_rn(x, y);
  }
}
// Four values in one store; i is a multiple of four.
__device__ __forceinline__ void store4_as(int type, void* base, int64_t i, float4 v) {
  if (type == QMV_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = v;
  } else if (type == QMV_BF16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<uint2*>(static_cast<__half*>(base) + i) = make_uint2(pack_h2(v.x, v.y), pack_h2(v.z, v.w));
  }
}
// N pieces of eight query values at the offsets at[0..N) of q, of the type known at run time (a negative offset: zeros).
// The type is chosen once around all of them, so that their loads are in flight together.
template <typename T, int N>
__device__ __forceinline__ void load_pieces(const void* base, const int64_t (&at)[N], float (&v)[N][8]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (at[i] >= 0) {
      kv8::load8(static_cast<const T*>(base) + at[i], v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
}
template <int N>
__device__ __forceinline__ void load_pieces_as(int type, const void* base, const int64_t (&at)[N], float (&v)[N][8]) {
  if (type == QMV_BF16) load_pieces<__nv_bfloat16>(base, at, v);
  else if (type == QMV_F16) load_pieces<__half>(base, at, v);
  else load_pieces<float>(base, at, v);
}
// True in one lane of a warp, the same one each time.
using umma::elected;
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(core::smem_addr(bar)) : "memory");
}

// A stream's partial tile, as its block joins it.
struct Piece {
  long long start;  // of its tile on the line
  int n, len;       // pages of the tile, pages covered here (0: no piece)
  int b, tile, h;
  const float* o;   // its rows (shared or global memory)
  const float2* ml;
};

template <int D, int N, int R>
struct Smem {
  using S = Shape<D, N, R>;
  alignas(128) unsigned char ring[S::kStreams][S::kStages][S::kTile];
  alignas(8) uint64_t full[S::kStreams][S::kStages];
  alignas(8) uint64_t empty[S::kStreams][S::kStages];
  float2 scale[S::kStreams][S::kStages];
  float2 ml[S::kStreams][S::kRows];
  int4 req[S::kReqs];
  long long start_base[S::kStreams];
  long long start_off[S::kStreams];
  int start_b[S::kStreams];
  Piece piece[S::kStreams][2];
  const float* entry_o[S::kStreams * 2];
  const float2* entry_ml[S::kStreams * 2];
  long long warp_sum[S::kWarps];
  int warp_segs[S::kWarps];
  int last[2];
};

// Join E partial tiles of `rows` rows (ml(e, row): maximum and sum, o(e, row, d): four values) into the output or into
// (dst_o, dst_ml): a warp of W takes row `first` and every W-th after it, with no step of the whole block. Lane e holds
// the factor of part e (of 32 at a time); BATCH parts are in flight, which is what a join out of L2 waits for: 19 parts of 25
// rows cost 11 us with six. With D = 64 the two halves of a warp take turns with the parts.
template <int D, int W, int BATCH, typename MlFn, typename OFn>
__device__ __forceinline__ void join(const Args& a, int E, int rows, int first, MlFn ml, OFn o, bool to_out, int h, int qs, int row0,
                                     float* dst_o, float2* dst_ml) {
  constexpr int HALVES = 128 / D, LANES = 32 / HALVES;
  const int lane = threadIdx.x & 31, half = lane / LANES, d = (lane % LANES) * 4;
  float2 next = make_float2(-INFINITY, 0.f);
  if (lane < E && first < rows) next = ml(lane, first);
  for (int row = first; row < rows; row += W) {
    const float2 mine = next;
    if (lane < E && row + W < rows) next = ml(lane, row + W);
    float m = mine.x;
    for (int e = lane + 32; e < E; e += 32) m = fmaxf(m, ml(e, row).x);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    const float use = m == -INFINITY ? 0.f : m;
    float w = ex2(mine.x - use);
    float l = w * mine.y;
    for (int e = lane + 32; e < E; e += 32) {
      const float2 v = ml(e, row);
      l += ex2(v.x - use) * v.y;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < E; c += 32) {
      const int n = min(32, E - c);
      if (c > 0) w = lane < n ? ex2(ml(c + lane, row).x - use) : 0.f;
      for (int i0 = 0; i0 < n; i0 += BATCH * HALVES) {
        float4 v[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int i = i0 + j * HALVES + half;
          v[j] = i < n ? o(c + i, row, d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int i = i0 + j * HALVES + half;   // past the end: v is 0, and lanes from E on hold the factor of -inf, 0
          const float f = __shfl_sync(0xFFFFFFFFu, w, i & 31);
          s.x += f * v[j].x;
          s.y += f * v[j].y;
          s.z += f * v[j].z;
          s.w += f * v[j].w;
        }
      }
    }
    if (HALVES == 2) {
      s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, 16);
      s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, 16);
      s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, 16);
      s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, 16);
    }
    if (to_out) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int rr = row0 + row, tok = a.by_g(rr), hq = h * a.G + rr - tok * a.G;
      if (half == 0) {
        const int64_t at = (int64_t)(qs + tok) * a.ldo + (int64_t)hq * D + d;
        store4_as(a.out_type, a.out, at, make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv));
      }
      if (lane == 0 && a.lse) a.lse[(int64_t)(qs + tok) * a.Hq + hq] = l == 0.f ? -INFINITY : (use + log2f(l)) * kLn2;
    } else {
      if (half == 0) *reinterpret_cast<float4*>(dst_o + (int64_t)row * D + d) = s;
      if (lane == 0) dst_ml[row] = make_float2(m, l);
    }
  }
}

template <int D, int TYPE, int N, int R, bool MODS>
__global__ void __launch_bounds__(Shape<D, N, R>::kThreads, 1) attend_kernel(const __grid_constant__ Args a) {
  using S = Shape<D, N, R>;
  constexpr int MT = D / 16;    // 16-row tiles of V^T
  constexpr int KH = D / 64;    // 64-wide pieces of d
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem<D, N, R>& sm = *reinterpret_cast<Smem<D, N, R>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stream = warp / R, wr = warp % R;
  const int g = lane >> 2, t = lane & 3;

  // ---- the line of units, and where this block's streams begin
  if (tid < S::kStreams * S::kStages) {
    core::mbar_init(&sm.full[0][0] + tid, tid % 2 ? 1 : 2);   // K tiles (even stages) come with their page's scales
    core::mbar_init(&sm.empty[0][0] + tid, R);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < S::kStreams * 2) (&sm.piece[0][0] + tid)->len = 0;
  kv8::let_next_begin();
  kv8::follow_previous();
  // Up to 32 requests: lane b of every warp holds request b, and each warp sums for itself.
  const bool few = a.B <= 32;
  int4 held = make_int4(0, 0, 0, 0);
  long long mine = 0, before = 0, W = 0;   // units of this thread's requests, of those before them, of all
  int segs = 0, longest = 0;
  const int per = few ? 1 : (a.B + S::kThreads - 1) / S::kThreads;
  const int b0 = few ? lane : min(a.B, tid * per), b1 = min(a.B, b0 + per);
  for (int b = b0; b < b1; ++b) {
    held = load_req4(a, b);
    if (!few && b < S::kReqs) sm.req[b] = held;
    const Req r = make_req(a, b, held, S::kRows);
    mine += req_units(a, r, S::kRows, longest);
    segs += r.tiles * a.H;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  segs = __reduce_add_sync(0xFFFFFFFFu, segs);
  if (few) {
    W = __shfl_sync(0xFFFFFFFFu, incl, 31);
  } else {
    if (lane == 31) {
      sm.warp_sum[warp] = incl;
      sm.warp_segs[warp] = segs;
    }
    __syncthreads();
    segs = 0;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) {
      if (w < warp) before += sm.warp_sum[w];
      W += sm.warp_sum[w];
      segs += sm.warp_segs[w];
    }
  }
  before += incl - mine;
  if (W == 0) return;
  auto get_req = [&](int b) {
    int4 v;
    if (few)
      v = make_int4(__shfl_sync(0xFFFFFFFFu, held.x, b), __shfl_sync(0xFFFFFFFFu, held.y, b), __shfl_sync(0xFFFFFFFFu, held.z, b),
                    __shfl_sync(0xFFFFFFFFu, held.w, b));
    else
      v = b < S::kReqs ? sm.req[b] : load_req4(a, b);
    return make_req(a, b, v, S::kRows);
  };
  const int cta = blockIdx.x;
  Cut blocks = {0, 0};
  int units;                                 // of this block
  int start_b = 0;
  long long start_off = 0, start_base = 0;   // this stream's first unit: its request, its place there, where that begins
  int whose0 = 0, whose1 = -1;               // the blocks of this block's tile, where each block has pages of one tile only
  // Cuts at the tiles' ends: `most` pages or fewer in each part, the fewest (in steps of a page per stream) with which
  // there are no more parts than blocks.
  int most = 0, parts = 0;
  if (few && segs <= (int)gridDim.x && W < (1ll << 30)) {
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    const Req r = make_req(a, lane, held, S::kRows);
    if (longest <= S::kAlone) {
      most = longest;
      parts = r.tiles * a.H;
    } else {
      const int one = r.tiles == 1 ? (int)mine / a.H : 0;   // pages of a request that has one row tile
      const int even = ((int)W + gridDim.x - 1) / (int)gridDim.x;
      const int least = (max(even, S::kCut) + S::kStreams - 1) / S::kStreams * S::kStreams;
      for (int p = least; p <= max(least, even + S::kUneven); p += S::kStreams) {
        parts = r.tiles == 1 ? (one + p - 1) / p * a.H : req_parts(a, r, S::kRows, p);
        if (__reduce_add_sync(0xFFFFFFFFu, parts) <= (int)gridDim.x) {
          most = p;
          break;
        }
      }
    }
  }
  if (most > 0) {
    int incl_parts = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, incl_parts, o);
      if (lane >= o) incl_parts += u;
    }
    if (cta >= __shfl_sync(0xFFFFFFFFu, incl_parts, 31)) return;
    start_b = __popc(__ballot_sync(0xFFFFFFFFu, incl_parts <= cta));
    start_base = __shfl_sync(0xFFFFFFFFu, before, start_b);
    const Req r = get_req(start_b);
    int part = cta - __shfl_sync(0xFFFFFFFFu, incl_parts - parts, start_b), n = 0, each = 1;   // of the request, then of a tile
    for (int k = 0;; ++k) {
      int p0;
      tile_pages(a, r, k, S::kRows, p0, n);
      each = n <= most ? 1 : (n + most - 1) / most;
      if (part < each * a.H || k + 1 >= r.tiles) break;
      part -= each * a.H;
      start_off += (long long)n * a.H;
    }
    int h = part, first = 0;   // its first page
    units = n;
    if (each > 1) {
      h = part / each;
      part -= h * each;
      const Cut cuts = cut(n, each);
      first = (int)cuts.at(part);
      units = (int)cuts.at(part + 1) - first;
      whose0 = cta - part;
      whose1 = whose0 + each - 1;
    }
    start_off += (long long)h * n + first + cut(units, S::kStreams).at(stream);
  } else {
    // the line in equal pieces for as many blocks as the tiles have kCut pages on average, all of them at most
    int A = gridDim.x;
    if (segs < A) {
      const int span = segs * S::kCut;   // below 2^13
      const int want = W < (1ll << 30) ? segs * (int)(((unsigned)W + span - 1) / (unsigned)span) : A;
      if (want < A) A = want;
    }
    if (cta >= A) return;
    blocks = cut(W, A);
    const long long u0 = blocks.at(cta);
    units = (int)(blocks.at(cta + 1) - u0);
    const Cut streams = cut(units, S::kStreams);
    if (few) {
      const long long x = u0 + streams.at(stream);
      start_b = __popc(__ballot_sync(0xFFFFFFFFu, before + mine <= x));
      start_base = __shfl_sync(0xFFFFFFFFu, before, start_b & 31);
      start_off = x - start_base;
    } else if (before < u0 + units && before + mine > u0) {
      long long P = before;
      for (int b = b0; b < b1; ++b) {
        const long long ub =
            per == 1 ? mine : req_units(a, make_req(a, b, load_req4(a, b), S::kRows), S::kRows, longest);
        for (int i = 0; i < S::kStreams; ++i) {
          const long long x = u0 + streams.at(i);
          if (P <= x && x < P + ub) {
            sm.start_b[i] = b;
            sm.start_off[i] = x - P;
            sm.start_base[i] = P;
          }
        }
        P += ub;
      }
    }
  }
  const Cut streams = cut(units, S::kStreams);
  __syncthreads();
  if (!few) {
    start_b = sm.start_b[stream];
    start_off = sm.start_off[stream];
    start_base = sm.start_base[stream];
  }
  int left = (int)(streams.at(stream + 1) - streams.at(stream));

  auto walk_next = [&](Walk& w) {
    w.start += w.n;
    if (++w.h < a.H) return;
    w.h = 0;
    if (++w.tile >= w.r.tiles) {
      w.tile = 0;
      int b = w.r.b;
      do {
        if (++b >= a.B) {  // past the last unit
          w.r.b = b;
          return;
        }
        w.r = get_req(b);
      } while (w.r.tiles == 0);
    }
    tile_pages(a, w.r, w.tile, S::kRows, w.p0, w.n);
  };

  if (left > 0) {
    Walk cw;   // the tile being computed
    int cp;    // page within it
    {
      long long off = start_off, base = start_base;
      cw.r = get_req(start_b);
      cw.tile = 0;
      for (;;) {
        tile_pages(a, cw.r, cw.tile, S::kRows, cw.p0, cw.n);
        const long long n = (long long)cw.n * a.H;
        if (off < n || cw.tile + 1 >= cw.r.tiles) break;
        off -= n;
        base += n;
        ++cw.tile;
      }
      cw.h = (int)((unsigned)off / (unsigned)cw.n);   // below H * n < 2^31
      cp = (int)off - cw.h * cw.n;
      cw.start = base + (long long)cw.h * cw.n;
    }
    Walk iw = cw;   // the tile being fetched
    int ip = cp, ileft = left;
    int win_at = 0, win_n = 0;
    long long win_off = -1;   // this lane's page of a window of up to 32 units: where its codes of this head begin
    bool fetch_v = false;
    int istage = 0;
    uint32_t iphase = 1;   // parity of the empty barrier's phase that a first use passes at once

    auto fetch = [&]() {
      if (ileft == 0) return;
      if (!fetch_v && win_at == win_n) {
        win_at = 0;
        win_n = min(32, min(iw.n - ip, ileft));
        win_off = -1;
        if (lane < win_n && iw.p0 >= 0) {
          const int id = a.table[(int64_t)iw.r.b * a.ld_table + iw.p0 + ip + lane];
          if (id >= 0 && id < a.n_pages) win_off = ((int64_t)id * a.H + iw.h) * (2 * S::kTile);
          else atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
        }
      }
      const long long off = __shfl_sync(0xFFFFFFFFu, win_off, win_at);
      if (elected()) {
        if (R > 1) core::mbar_wait(&sm.empty[stream][istage], iphase, a.err);
        uint64_t* bar = &sm.full[stream][istage];
        if (off >= 0) {
          core::mbar_arrive_expect_tx(bar, S::kTile);
          core::bulk_g2s(sm.ring[stream][istage], a.cache + off + (fetch_v ? S::kTile : 0), S::kTile, bar);
          if (!fetch_v) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(core::smem_addr(&sm.scale[stream][istage])),
                         "l"(a.cache + a.scale_off + off / (2 * S::kTile) * 8)
                         : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(core::smem_addr(bar)) : "memory");
          }
        } else {
          if (!fetch_v) {
            sm.scale[stream][istage] = make_float2(-1.f, -1.f);
            mbar_arrive(bar);
          }
          mbar_arrive(bar);
        }
      }
      if (++istage == S::kStages) {
        istage = 0;
        iphase ^= 1;
      }
      if (fetch_v) {
        ++win_at;
        --ileft;
        if (++ip == iw.n) {
          ip = 0;
          walk_next(iw);
        }
      }
      fetch_v = !fetch_v;
    };
    const bool leader = wr == 0;
    // with several warps per stream a slot is refilled one item late, so that the leader seldom waits for the others
    if (leader)
#pragma unroll 1
      for (int i = 0; i < S::kStages - (R > 1 ? 1 : 0); ++i) fetch();

    int cstage = 0;
    uint32_t cphase = 0;
    auto release = [&]() {
      __syncwarp();
      if (R > 1 && lane == 0) mbar_arrive(&sm.empty[stream][cstage]);
      if (++cstage == S::kStages) {
        cstage = 0;
        cphase ^= 1;
      }
      if (leader) fetch();
    };

    bool first_piece = true;
#pragma unroll 1
    while (left > 0) {
      const int len = min(cw.n - cp, left);
      // ---- the query rows of this warp: lane (g, t) loads row g of each tile of eight, and holds the scores of rows
      // 2t and 2t + 1
      const int row0 = cw.tile * S::kRows + wr * 8 * N;
      const int nr = min(max(cw.r.rows - row0, 0), 8 * N);
      uint32_t qf[N][KH * 4][2];
      float mult[N][2], slope[N][2];      // product to score, without the page's scale; distance bias
      int lo[N][2], hi[N][2], pos[N][2];  // keys seen
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int row = min(row0 + 8 * n + g, cw.r.rows - 1), row_tok = a.by_g(row);
        const bool real = 8 * n + g < nr;
        const int64_t at = (int64_t)(cw.r.qs + row_tok) * a.ldq + (int64_t)(cw.h * a.G + row - row_tok * a.G) * D;
        float v[KH * 2][8];
        int64_t piece[KH * 2];
#pragma unroll
        for (int p = 0; p < KH * 2; ++p) piece[p] = real ? at + (p >> 1) * 64 + t * 16 + (p & 1) * 8 : -1;
        load_pieces_as(a.x_type, a.q, piece, v);
        float m = 0.f;
#pragma unroll
        for (int p = 0; p < KH * 2; ++p)
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[p][i]));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        // the row's largest magnitude goes to [2^13, 2^14)
        const int e = min(max(13 + 127 - (int)(__float_as_uint(m) >> 23), -126), 126);
        const float f = core::exp2i(e);
        const float back = core::exp2i(-e) * a.scale;
#pragma unroll
        for (int p = 0; p < KH * 2; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            qf[n][(p >> 1) * 4 + (p & 1) * 2 + (i >> 1)][i & 1] = pack_h2(v[p][2 * i] * f, v[p][2 * i + 1] * f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mult[n][c] = __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4 * c);
          const int rr = min(row0 + 8 * n + 2 * t + c, cw.r.rows - 1), tok = a.by_g(rr);
          pos[n][c] = cw.r.ctx - cw.r.qlen + tok;
          hi[n][c] = min(max(pos[n][c] + 1, cw.r.pfx), cw.r.ctx);
          lo[n][c] = first_key(a, pos[n][c]);
          slope[n][c] = 0.f;
          if (MODS) {
            if (a.slopes) slope[n][c] = a.slopes[cw.h * a.G + rr - tok * a.G] * kLog2e;
          } else {
            mult[n][c] *= kLog2e;
          }
        }
      }
      int lo_all = lo[0][0], hi_all = hi[0][0];   // keys that every row of the warp sees
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          lo_all = max(lo_all, lo[n][c]);
          hi_all = min(hi_all, hi[n][c]);
        }
      lo_all = max(lo_all, __shfl_xor_sync(0xFFFFFFFFu, lo_all, 1));
      hi_all = min(hi_all, __shfl_xor_sync(0xFFFFFFFFu, hi_all, 1));
      lo_all = max(lo_all, __shfl_xor_sync(0xFFFFFFFFu, lo_all, 2));
      hi_all = min(hi_all, __shfl_xor_sync(0xFFFFFFFFu, hi_all, 2));

      float o[N][MT][4];
      float m[N][2], l[N][2];
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }

#pragma unroll 1
      for (int u = 0; u < len; ++u) {
        const int key0 = (cw.p0 + cp + u) * kPage;
        core::mbar_wait(&sm.full[stream][cstage], cphase, a.err);
        const float2 scale = sm.scale[stream][cstage];
        const bool there = scale.x >= 0.f && nr > 0;
        uint32_t pf[N][8];
        float corr[N][2];
        const bool cut_page = key0 < lo_all || key0 + kPage > hi_all;
        if (there) {
          float s[N][4][4];   // tokens of column groups 2i and 2i + 1
          const uint4* kt = reinterpret_cast<const uint4*>(sm.ring[stream][cstage]) + lane;
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i][0] = s[n][i][1] = s[n][i][2] = s[n][i][3] = 0.f;
          // the four row tiles' chains of products side by side
#pragma unroll
          for (int hh = 0; hh < KH; ++hh) {
            uint4 w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = kt[(j * KH + hh) * 32];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t a0, a1, a2, a3;
                codes_to_half<TYPE>(word4(w[2 * i], k), a0, a2);
                codes_to_half<TYPE>(word4(w[2 * i + 1], k), a1, a3);
#pragma unroll
                for (int n = 0; n < N; ++n) mma16816(s[n][i], a0, a1, a2, a3, qf[n][hh * 4 + k][0], qf[n][hh * 4 + k][1]);
              }
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            // scores in units of log2; value c of group 2i + e is token 16 (g / 2) + 2 (2i + e) + g % 2, row 2t + c
            float f[2] = {fmaxf(mult[n][0] * scale.x, 1e-37f), fmaxf(mult[n][1] * scale.x, 1e-37f)};
            const int tok0 = key0 + 16 * (g >> 1) + (g & 1);
            if (MODS) {
              if (a.softcap > 0.f) {
                const float c2[2] = {cap_factor(a.softcap, f[0]), cap_factor(a.softcap, f[1])}, cap = a.softcap * kLog2e;
                const float unit[2] = {f[0] * kLog2e, f[1] * kLog2e};
                float big[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int c = 0; c < 2; ++c) big[c] = fmaxf(big[c], fmaxf(fabsf(s[n][i][c]), fabsf(s[n][i][c + 2])));
                // one branch for the warp: scores far below the cap, as they mostly are, need no special function
                if (__all_sync(0xFFFFFFFFu, fmaxf(big[0] * c2[0], big[1] * c2[1]) <= kNear)) {
#pragma unroll
                  for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[n][i][c] = capped_near(s[n][i][c], c2[c & 1], unit[c & 1]);
                } else {
#pragma unroll
                  for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[n][i][c] = capped(s[n][i][c], c2[c & 1], unit[c & 1], cap);
                }
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int c = 0; c < 4; ++c) s[n][i][c] *= f[c & 1] * kLog2e;
              }
              if (a.slopes) {
                const float gap[2] = {(float)(pos[n][0] - tok0), (float)(pos[n][1] - tok0)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int c = 0; c < 4; ++c)
                    s[n][i][c] = fmaf(-slope[n][c & 1], fabsf(gap[c & 1] - (4 * i + 2 * (c >> 1))), s[n][i][c]);
              }
              f[0] = f[1] = 1.f;
            }
            if (cut_page) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const int key = tok0 + 4 * i + 2 * (c >> 1);
                  if (key < lo[n][c & 1] || key >= hi[n][c & 1]) s[n][i][c] = -INFINITY;
                }
            }
            float mx[2], use[2], sum[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              mx[c] = fmaxf(s[n][0][c], s[n][0][c + 2]);
#pragma unroll
              for (int i = 1; i < 4; ++i) mx[c] = fmaxf(mx[c], fmaxf(s[n][i][c], s[n][i][c + 2]));
            }
#pragma unroll
            for (int o2 = 4; o2 < 32; o2 <<= 1) {
              mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], o2));
              mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], o2));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float mn = fmaxf(m[n][c], fmaf(mx[c], f[c], -kLift));
              use[c] = mn == -INFINITY ? 0.f : mn;
              corr[n][c] = ex2(m[n][c] - use[c]);
              m[n][c] = mn;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float p0 = ex2(fmaf(s[n][i][2 * e], f[0], -use[0])), p1 = ex2(fmaf(s[n][i][2 * e + 1], f[1], -use[1]));
                sum[0] += p0;
                sum[1] += p1;
                pf[n][2 * i + e] = transpose8(pack_h2(p0, p1));
              }
            l[n][0] = l[n][0] * corr[n][0] + sum[0];
            l[n][1] = l[n][1] * corr[n][1] + sum[1];
          }
        }
        release();
        core::mbar_wait(&sm.full[stream][cstage], cphase, a.err);
        if (there) {
          const uint4* vt = reinterpret_cast<const uint4*>(sm.ring[stream][cstage]) + lane;
          constexpr int S4 = MT < 4 ? MT : 4;   // row tiles side by side
#pragma unroll
          for (int i0 = 0; i0 < MT; i0 += S4) {
            uint4 w[2 * S4];
#pragma unroll
            for (int j = 0; j < 2 * S4; ++j) {
              w[j] = vt[(2 * i0 + j) * 32];
              // slots past the request's end may hold any byte: a NaN code there would not be hidden by p = 0
              if (TYPE == QMV_KV_E4M3 && cut_page) w[j] = make_uint4(drop_nan(w[j].x), drop_nan(w[j].y), drop_nan(w[j].z), drop_nan(w[j].w));
            }
            float c[N][S4][4];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
              for (int i = 0; i < S4; ++i) c[n][i][0] = c[n][i][1] = c[n][i][2] = c[n][i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int i = 0; i < S4; ++i) {
                uint32_t a0, a1, a2, a3;
                codes_to_half<TYPE>(word4(w[2 * i], k), a0, a2);
                codes_to_half<TYPE>(word4(w[2 * i + 1], k), a1, a3);
#pragma unroll
                for (int n = 0; n < N; ++n) mma16816(c[n][i], a0, a1, a2, a3, pf[n][2 * k], pf[n][2 * k + 1]);
              }
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
              for (int i = 0; i < S4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i0 + i][j] = fmaf(c[n][i][j], scale.y, o[n][i0 + i][j] * corr[n][j & 1]);
          }
        }
        release();
      }

      // ---- end of the piece: the row sums, then the output or a partial tile
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], o2);
      const bool whole = len == cw.n, final_piece = left == len;
      // the last partial tile of the stream lies in its ring (when every warp of the stream has read it), an earlier
      // one in the workspace
      float* po = nullptr;
      float2* pml = nullptr;
      if (!whole) {
        if (final_piece) {
          if (R > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + stream), "r"(R * 32) : "memory");
          po = reinterpret_cast<float*>(sm.ring[stream]);
          pml = sm.ml[stream];
        } else {
          const int64_t at = (int64_t)cta * kPartRows + stream * S::kRows;
          po = a.part_o + at * D;
          pml = a.part_ml + at;
        }
        if (leader && lane == 0) sm.piece[stream][first_piece ? 0 : 1] = Piece{cw.start, cw.n, len, cw.r.b, cw.tile, cw.h, po, pml};
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        // lanes g and g ^ 1 exchange, so that an even lane holds two neighbouring values of row 2t, an odd one of 2t + 1
        const int c = g & 1, r8 = 8 * n + 2 * t + c;
        const bool real = r8 < nr;
        const float lc = c ? l[n][1] : l[n][0], mc = c ? m[n][1] : m[n][0];
        const float f = whole ? (lc == 0.f ? 0.f : 1.f / lc) : 1.f;
        const int row = row0 + r8, tok = a.by_g(row);
        const int64_t at = (int64_t)(cw.r.qs + tok) * a.ldo + (int64_t)(cw.h * a.G + row - tok * a.G) * D;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float got = __shfl_xor_sync(0xFFFFFFFFu, c ? o[n][i][2 * e] : o[n][i][2 * e + 1], 4);
            const float keep = c ? o[n][i][2 * e + 1] : o[n][i][2 * e];
            const float x = (c ? got : keep) * f, y = (c ? keep : got) * f;
            const int d = 16 * i + 8 * e + (g & 6);
            if (real) {
              if (whole) store_as(a.out_type, a.out, at + d, x, y);
              else *reinterpret_cast<float2*>(po + (wr * 8 * N + r8) * D + d) = make_float2(x, y);
            }
          }
        if (real && g < 2) {
          if (!whole) pml[wr * 8 * N + r8] = make_float2(mc, lc);
          else if (a.lse) a.lse[(int64_t)(cw.r.qs + tok) * a.Hq + cw.h * a.G + row - tok * a.G] = lc == 0.f ? -INFINITY : (mc + log2f(lc)) * kLn2;
        }
      }
      first_piece = false;
      left -= len;
      cp = 0;
      if (left > 0) walk_next(cw);
    }
  }
  __syncthreads();

  // ---- join the partial tiles of this block's streams, tile by tile (in the order of the line)
  // Lane e of every warp holds entry e's place.
  long long p_start = -1;
  int p_len = 0;
  if (lane < S::kStreams * 2) {
    p_start = (&sm.piece[0][0])[lane].start;
    p_len = (&sm.piece[0][0])[lane].len;
  }
  const unsigned all = __ballot_sync(0xFFFFFFFFu, p_len > 0);
  unsigned todo = all;
  if (warp == 0 && p_len > 0) {
    const int at = __popc(all & ((1u << lane) - 1));
    sm.entry_o[at] = (&sm.piece[0][0])[lane].o;
    sm.entry_ml[at] = (&sm.piece[0][0])[lane].ml;
  }
  __syncthreads();
  int turn = 0;   // rows given out so far: the next tile's begin with the next warp
  int shared_tiles[2] = {-1, -1};   // entries of the (at most two) tiles that other blocks hold a part of
  auto slot_of = [&](const Piece& pc, int c) {   // the rows where block c leaves its part of the tile
    return (int64_t)c * kPartRows + kStreamRows + (whose1 >= 0 || pc.start < blocks.at(c) ? 0 : S::kRows);
  };
  auto blocks_of = [&](const Piece& pc, int& c0, int& c1) {   // the blocks that hold parts of the tile
    c0 = whose1 >= 0 ? whose0 : blocks.part_of(pc.start);
    c1 = whose1 >= 0 ? whose1 : blocks.part_of(pc.start + pc.n - 1);
  };
  while (todo) {
    const int e0 = __ffs(todo) - 1;
    const long long start = __shfl_sync(0xFFFFFFFFu, p_start, e0);
    const unsigned same = __ballot_sync(0xFFFFFFFFu, p_len > 0 && p_start == start);
    const int covered = __reduce_add_sync(0xFFFFFFFFu, (same >> lane) & 1 ? p_len : 0), n_e = __popc(same);
    todo &= ~same;
    const Piece& pc = (&sm.piece[0][0])[e0];
    const int base = __popc(all & ((1u << e0) - 1));   // a tile's pieces follow one another
    const Req r = get_req(pc.b);
    const int row0 = pc.tile * S::kRows, rows = min(S::kRows, r.rows - row0);
    const bool whole = covered == pc.n;
    const int64_t mine_at = slot_of(pc, cta);
    if (!whole) {
      if (shared_tiles[0] < 0) shared_tiles[0] = e0;
      else shared_tiles[1] = e0;
    }
    join<D, S::kWarps, 8>(
        a, n_e, rows, (warp + S::kWarps - turn % S::kWarps) % S::kWarps, [&](int e, int row) { return sm.entry_ml[base + e][row]; },
        [&](int e, int row, int d) { return *reinterpret_cast<const float4*>(sm.entry_o[base + e] + row * D + d); }, whole, pc.h, r.qs,
        row0, a.part_o + mine_at * D, a.part_ml + mine_at);
    turn += rows;
  }
  if (shared_tiles[0] < 0) return;
  // ---- the last of a tile's blocks to arrive joins their parts
  __threadfence();
  __syncthreads();
  if (tid < 2 && (tid ? shared_tiles[1] : shared_tiles[0]) >= 0) {
    const Piece& pc = (&sm.piece[0][0])[tid ? shared_tiles[1] : shared_tiles[0]];
    int c0, c1;
    blocks_of(pc, c0, c1);
    const int old = atomicAdd(a.counters + c0, 1);
    sm.last[tid] = old == c1 - c0;
    if (old == c1 - c0) a.counters[c0] = 0;
    __threadfence();
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (shared_tiles[i] < 0 || !sm.last[i]) continue;
    const Piece& pc = (&sm.piece[0][0])[shared_tiles[i]];
    int c0, c1;
    blocks_of(pc, c0, c1);
    const Req r = get_req(pc.b);
    const int row0 = pc.tile * S::kRows, rows = min(S::kRows, r.rows - row0);
    // written by other blocks during this launch: read past L1
    join<D, S::kWarps, 20>(
        a, c1 - c0 + 1, rows, warp, [&](int e, int row) { return __ldcg(a.part_ml + slot_of(pc, c0 + e) + row); },
        [&](int e, int row, int d) { return __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot_of(pc, c0 + e) + row) * D + d)); },
        true, pc.h, r.qs, row0, nullptr, nullptr);
  }
}

template <int D, int TYPE, int N, int R, bool MODS>
int launch(const Args& a, int blocks, cudaStream_t s) {
  using S = Shape<D, N, R>;
  const void* f = reinterpret_cast<const void*>(attend_kernel<D, TYPE, N, R, MODS>);
  int per_sm = 0;
  int rc = kernel_fit(f, S::kThreads, sizeof(Smem<D, N, R>), &per_sm);
  if (rc) return rc;
  Args copy = a;
  void* args[] = {&copy};
  cudaError_t e = kv8::launch_early(f, dim3(blocks), S::kThreads, args, sizeof(Smem<D, N, R>), s);
  if (e != cudaSuccess) return cuda_fail(e, "kv8_attend launch");
  return QMV_OK;
}

// One translation unit per (D, type): rows is the row tile (8, 16 or 32).
int launch_64_int8(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);
int launch_64_e4m3(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);
int launch_128_int8(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);
int launch_128_e4m3(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);

template <int D, int TYPE>
int launch_rows(const Args& a, int rows, bool mods, int blocks, cudaStream_t s) {
  switch (rows) {
    case 8: return mods ? launch<D, TYPE, 1, 1, true>(a, blocks, s) : launch<D, TYPE, 1, 1, false>(a, blocks, s);
    case 16: return mods ? launch<D, TYPE, 2, 1, true>(a, blocks, s) : launch<D, TYPE, 2, 1, false>(a, blocks, s);
    default: return mods ? launch<D, TYPE, 2, 2, true>(a, blocks, s) : launch<D, TYPE, 2, 2, false>(a, blocks, s);
  }
}

}  // namespace attend
}  // namespace qmv

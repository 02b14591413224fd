// Attention over the paged 8-bit KV cache for decode and verification steps
// (kv8_attend), on the warp-level tensor cores.
//
// Work. The query rows of a (request, KV head) are its new tokens times the G
// query heads that share the KV head; they are cut into tiles of 16 * R rows. A
// unit is one page of one (request, row tile, KV head); all units of a call, in
// that order with the pages innermost, form one line that is cut into equal
// pieces, one per stream. A block has 8 / R streams of R warps each; every warp
// of a stream holds 16 rows and all of them read the stream's pages. So the
// blocks' loads differ by one page at most, whatever the mix of lengths, and no
// schedule has to be made on the host: a block sums the units of all requests
// (one load per request, a block scan) and finds its streams' starts.
//
// A stream walks its piece of the line with the running maximum and sum of a
// softmax per row. Where it covers all pages of a tile it writes the result;
// else it leaves (sum p v, maximum, sum p) in the workspace. The block joins its
// streams' partial tiles, and the last block to arrive at a tile that is cut
// between blocks joins the blocks' in their order: the result does not depend
// on timing.
//
// Data. A page's K or V tile is one contiguous piece of 64 * D bytes, fetched by
// one bulk copy into the stream's ring. The tiles are stored in the order of the
// m16n8k16 fragments: a lane's 16 bytes of K are four k-steps of one token, its
// 16 bytes of V four k-steps (sixteen tokens) of one d, so both are read with
// conflict-free 16-byte loads and the scores' accumulators are, in place, the
// fragments of the product with V. Codes become fp16 exactly: int8 as 1024 + byte
// by a byte permute and a subtraction, e4m3 by the conversion instruction. q is
// scaled per row by a power of two into fp16, so q . k is exact up to its fp32
// sum. The page's K scale multiplies the scores, its V scale the page's product
// with V: in fp32 both, after the sum over the page.
#pragma once

#include "gemv_core.cuh"
#include "kv8.cuh"

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
  float* part_o;         // [blocks][streams][2][rows][D] partial tiles of streams, then [blocks][2][rows][D] of blocks
  float2* part_ml;       // the same with one (maximum, sum) per row
  int* counters;         // [blocks], zero between calls
  int min_units;         // units a block takes at least before another block is used
  int* err;
};

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRingBytes = 192 * 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Partial rows of a block in the workspace: 8 / R streams x 2 x 16 R rows, then 2 x 16 R rows.
constexpr int kStreamRows = 256, kBlockRows = 256;

struct Req {
  int b, qs, qlen, ctx, pfx, rows, tiles;
};
__device__ __forceinline__ Req load_req(const Args& a, int b, int tile_rows) {
  Req r;
  r.b = b;
  const int q0 = min(max(a.q_start[b], 0), a.T), q1 = min(max(a.q_start[b + 1], 0), a.T);
  r.qs = q0;
  r.qlen = max(q1 - q0, 0);
  r.ctx = (int)min((int64_t)max(a.ctx[b], 0), (int64_t)a.max_pages * kPage);
  r.pfx = a.prefix ? a.prefix[b] : 0;
  r.rows = r.qlen * a.G;
  r.tiles = (r.rows + tile_rows - 1) / tile_rows;
  return r;
}
// Pages [p0, p0 + n) that hold the keys seen by a row tile; p0 = -1, n = 1 where it sees none.
__device__ __forceinline__ void tile_pages(const Args& a, const Req& r, int tile, int tile_rows, int& p0, int& n) {
  const int first = tile * tile_rows / a.G, last = (min(r.rows, (tile + 1) * tile_rows) - 1) / a.G;
  const int base = r.ctx - r.qlen;
  const int hi = min(max(base + last + 1, r.pfx), r.ctx);
  const int lo = a.window > 0 ? max(0, base + first - a.window + 1) : 0;
  if (hi <= lo) {
    p0 = -1;
    n = 1;
    return;
  }
  p0 = lo / kPage;
  n = (hi + kPage - 1) / kPage - p0;
}
__device__ __forceinline__ long long req_units(const Args& a, const Req& r, int tile_rows) {
  long long u = 0;
  for (int k = 0; k < r.tiles; ++k) {
    int p0, n;
    tile_pages(a, r, k, tile_rows, p0, n);
    u += n;
  }
  return u * a.H;
}

// A place on the line of units: a tile of a request, a KV head, and its pages.
struct Walk {
  Req r;
  int tile, h, p0, n;
  long long start;  // first unit of this (request, tile, head) on the line
};
__device__ __forceinline__ void walk_next(const Args& a, Walk& w, int tile_rows) {
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
      w.r = load_req(a, b, tile_rows);
    } while (w.r.tiles == 0);
  }
  tile_pages(a, w.r, w.tile, tile_rows, w.p0, w.n);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__device__ __forceinline__ void store_as(int type, void* base, int64_t i, float x, float y) {
  if (type == QMV_F32) *reinterpret_cast<float2*>(static_cast<float*>(base) + i) = make_float2(x, y);
  else if (type == QMV_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(base) + i) = h;
  } else {
    *reinterpret_cast<__half2*>(static_cast<__half*>(base) + i) = __floats2half2_rn(x, y);
  }
}
__device__ __forceinline__ void load8_as(int type, const void* base, int64_t i, float (&v)[8]) {
  if (type == QMV_F32) kv8::load8(static_cast<const float*>(base) + i, v);
  else if (type == QMV_BF16) kv8::load8(static_cast<const __nv_bfloat16*>(base) + i, v);
  else kv8::load8(static_cast<const __half*>(base) + i, v);
}

template <int D, int R>
struct Shape {
  static constexpr int kStreams = kWarps / R;
  static constexpr int kTile = kPage * D;                        // bytes of a K or V tile
  static constexpr int kStages = kRingBytes / kStreams / kTile;  // 3 R tiles of 128, 6 R of 64
  static constexpr int kRows = 16 * R;
};

// A stream's partial tile, as its block joins it.
struct Piece {
  long long start;  // of its tile on the line
  int n, len;       // pages of the tile, pages covered here (0: no piece)
  int b, tile, h;
};

template <int D, int R>
struct Smem {
  using S = Shape<D, R>;
  alignas(128) unsigned char ring[S::kStreams][S::kStages][S::kTile];
  alignas(8) uint64_t full[S::kStreams][S::kStages];
  alignas(8) uint64_t empty[S::kStreams][S::kStages];
  float scale[S::kStreams][S::kStages];
  long long start_base[S::kStreams];
  int start_b[S::kStreams];
  long long start_off[S::kStreams];
  Piece piece[S::kStreams][2];
  long long warp_sum[kWarps];
  int last;
};

// Join E partial tiles of `rows` rows (entry e: o_of(e), ml_of(e)) into the output or into (dst_o, dst_ml).
// `weights` (shared, E * rows floats) and all threads of the block.
template <int D, typename EntryFn>
__device__ __forceinline__ void join(const Args& a, int E, int rows, EntryFn entry, float* weights, bool to_out, const Piece& pc,
                                     const Req& r, int row0, float* dst_o, float2* dst_ml) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int row = warp; row < rows; row += kWarps) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, __ldcg(a.part_ml + entry(e) + row).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float use = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int e = lane; e < E; e += 32) {
      const float2 ml = __ldcg(a.part_ml + entry(e) + row);
      const float w = ex2(ml.x - use);
      weights[e * rows + row] = w;
      l += w * ml.y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (to_out) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      __syncwarp();
      for (int e = lane; e < E; e += 32) weights[e * rows + row] *= inv;
      if (lane == 0 && a.lse) {
        const int rr = row0 + row;
        a.lse[(int64_t)(r.qs + rr / a.G) * a.Hq + pc.h * a.G + rr % a.G] = l == 0.f ? -INFINITY : (use + log2f(l)) * kLn2;
      }
    } else if (lane == 0) {
      dst_ml[row] = make_float2(m, l);
    }
  }
  __syncthreads();
  constexpr int Q = D / 4;
  for (int u = tid; u < rows * Q; u += kThreads) {
    const int row = u / Q, d = (u % Q) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int e = 0; e < E; ++e) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (int64_t)(entry(e) + row) * D + d));
      const float w = weights[e * rows + row];
      s.x += w * v.x;
      s.y += w * v.y;
      s.z += w * v.z;
      s.w += w * v.w;
    }
    if (to_out) {
      const int rr = row0 + row;
      const int64_t o = (int64_t)(r.qs + rr / a.G) * a.ldo + (int64_t)(pc.h * a.G + rr % a.G) * D + d;
      store_as(a.out_type, a.out, o, s.x, s.y);
      store_as(a.out_type, a.out, o + 2, s.z, s.w);
    } else {
      *reinterpret_cast<float4*>(dst_o + (int64_t)row * D + d) = s;
    }
  }
  __syncthreads();
}

template <int D, int TYPE, int R, bool MODS>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ Args a) {
  using S = Shape<D, R>;
  constexpr int NT = D / 8;     // 8-wide tiles of d
  constexpr int KH = D / 64;    // 64-wide pieces of d
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem<D, R>& sm = *reinterpret_cast<Smem<D, R>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stream = warp / R, wr = warp % R;
  const int g = lane >> 2, t = lane & 3;

  if (tid == 0) {
    for (int i = 0; i < S::kStreams * S::kStages; ++i) {
      core::mbar_init(&sm.full[0][0] + i, 1);
      core::mbar_init(&sm.empty[0][0] + i, R);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < S::kStreams * 2) (&sm.piece[0][0] + tid)->len = 0;

  // ---- the line of units, and where this block's streams begin
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += req_units(a, load_req(a, b, S::kRows), S::kRows);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, W = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.warp_sum[w];
    W += sm.warp_sum[w];
  }
  if (W == 0) return;
  const long long most = (W + a.min_units - 1) / a.min_units;
  const int A = most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
  const int cta = blockIdx.x;
  if (cta >= A) return;
  const long long u0 = cta * W / A, u1 = (cta + 1) * W / A;
  {
    long long P = before + incl - mine;
    for (int b = b0; b < b1 && P < u1; ++b) {
      const long long ub = req_units(a, load_req(a, b, S::kRows), S::kRows);
      for (int i = 0; i < S::kStreams; ++i) {
        const long long x = u0 + (u1 - u0) * i / S::kStreams;
        if (P <= x && x < P + ub) {
          sm.start_b[i] = b;
          sm.start_off[i] = x - P;
          sm.start_base[i] = P;
        }
      }
      P += ub;
    }
  }
  __syncthreads();
  const long long s0 = u0 + (u1 - u0) * stream / S::kStreams, s1 = u0 + (u1 - u0) * (stream + 1) / S::kStreams;
  int left = (int)(s1 - s0);

  if (left > 0) {
    Walk cw;   // the piece being computed
    int cp;    // page within its tile
    {
      long long off = sm.start_off[stream], base = sm.start_base[stream];
      cw.r = load_req(a, sm.start_b[stream], S::kRows);
      cw.tile = 0;
      for (;;) {
        tile_pages(a, cw.r, cw.tile, S::kRows, cw.p0, cw.n);
        const long long units = (long long)cw.n * a.H;
        if (off < units || cw.tile + 1 >= cw.r.tiles) break;
        off -= units;
        base += units;
        ++cw.tile;
      }
      cw.h = (int)(off / cw.n);
      cp = (int)(off - (long long)cw.h * cw.n);
      cw.start = base + (long long)cw.h * cw.n;
    }
    Walk iw = cw;   // the piece being fetched
    int ip = cp, ileft = left;
    int win_page = -1, win_at = 0, win_n = 0;   // this lane's page of a window of up to 32 units
    float win_k = 0.f, win_v = 0.f;
    bool fetch_v = false;
    int istage = 0;
    uint32_t iphase = 1;   // parity of the empty barrier's phase that a first use passes at once

    auto fetch = [&]() {
      if (ileft == 0) return;
      if (!fetch_v && win_at == win_n) {
        win_at = 0;
        win_n = min(32, min(iw.n - ip, ileft));
        win_page = -1;
        if (lane < win_n && iw.p0 >= 0) {
          const int id = a.table[(int64_t)iw.r.b * a.ld_table + iw.p0 + ip + lane];
          if (id >= 0 && id < a.n_pages) {
            const float2 sc = reinterpret_cast<const float2*>(a.cache + a.scale_off)[(int64_t)id * a.H + iw.h];
            win_page = id;
            win_k = sc.x;
            win_v = sc.y;
          } else {
            atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
          }
        }
      }
      const int page = __shfl_sync(0xFFFFFFFFu, win_page, win_at);
      const float sc = __shfl_sync(0xFFFFFFFFu, fetch_v ? win_v : win_k, win_at);
      if (lane == 0) {
        if (R > 1) core::mbar_wait(&sm.empty[stream][istage], iphase, a.err);
        sm.scale[stream][istage] = page >= 0 ? sc : -1.f;
        uint64_t* bar = &sm.full[stream][istage];
        if (page >= 0) {
          const unsigned char* src = a.cache + ((int64_t)page * a.H + iw.h) * (2 * S::kTile) + (fetch_v ? S::kTile : 0);
          core::mbar_arrive_expect_tx(bar, S::kTile);
          core::bulk_g2s(sm.ring[stream][istage], src, S::kTile, bar);
        } else {
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(core::smem_addr(bar)) : "memory");
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
          walk_next(a, iw, S::kRows);
        }
      }
      fetch_v = !fetch_v;
    };
    const bool leader = wr == 0;
    // with several warps per stream a slot is refilled one item late, so that the leader seldom waits for the others
    if (leader)
      for (int i = 0; i < S::kStages - (R > 1 ? 1 : 0); ++i) fetch();

    int cstage = 0;
    uint32_t cphase = 0;
    auto release = [&]() {
      __syncwarp();
      if (R > 1 && lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(core::smem_addr(&sm.empty[stream][cstage])) : "memory");
      if (++cstage == S::kStages) {
        cstage = 0;
        cphase ^= 1;
      }
      if (leader) fetch();
    };

    bool first_piece = true;
    while (left > 0) {
      const int len = min(cw.n - cp, left);
      // ---- the 16 query rows of this warp
      const int row0 = cw.tile * S::kRows, nrows = min(S::kRows, cw.r.rows - row0);
      const int nr = min(max(nrows - wr * 16, 0), 16);   // of this warp
      uint32_t qf[KH * 4][4];
      float mult[2];      // product to score, without the page's scale
      int lo[2], hi[2];   // keys seen
      float slope[2];
      int pos[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = min(row0 + wr * 16 + g + 8 * half, cw.r.rows - 1);
        const int tok = row / a.G, hq = cw.h * a.G + row % a.G;
        const bool real = g + 8 * half < nr;
        const int64_t at = (int64_t)(cw.r.qs + tok) * a.ldq + (int64_t)hq * D;
        float v[KH * 2][8];
        float m = 0.f;
#pragma unroll
        for (int p = 0; p < KH * 2; ++p) {
          if (real) {
            load8_as(a.x_type, a.q, at + (p >> 1) * 64 + t * 16 + (p & 1) * 8, v[p]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[p][i]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        // the row's largest magnitude goes to [2^13, 2^14)
        const int e = min(max(13 + 127 - (int)(__float_as_uint(m) >> 23), -126), 126);
        const float f = core::exp2i(e);
        mult[half] = core::exp2i(-e) * a.scale;
#pragma unroll
        for (int p = 0; p < KH * 2; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            qf[(p >> 1) * 4 + (p & 1) * 2 + (i >> 1)][(i & 1) * 2 + half] = pack_h2(v[p][2 * i] * f, v[p][2 * i + 1] * f);
        pos[half] = cw.r.ctx - cw.r.qlen + tok;
        hi[half] = min(max(pos[half] + 1, cw.r.pfx), cw.r.ctx);
        lo[half] = a.window > 0 ? pos[half] - a.window + 1 : 0;
        slope[half] = 0.f;
        if (MODS) {
          if (a.slopes) slope[half] = a.slopes[hq] * kLog2e;
        } else {
          mult[half] *= kLog2e;
        }
      }
      int lo_all = max(lo[0], lo[1]), hi_all = min(hi[0], hi[1]);   // keys that every row of the warp sees
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        lo_all = max(lo_all, __shfl_xor_sync(0xFFFFFFFFu, lo_all, o));
        hi_all = min(hi_all, __shfl_xor_sync(0xFFFFFFFFu, hi_all, o));
      }

      float o[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      for (int u = 0; u < len; ++u) {
        const int key0 = (cw.p0 + cp + u) * kPage;
        core::mbar_wait(&sm.full[stream][cstage], cphase, a.err);
        const float sk = sm.scale[stream][cstage];
        const bool there = sk >= 0.f && nr > 0;
        uint32_t pf[4][4];
        float corr[2] = {1.f, 1.f};
        bool cut = false;
        if (there) {
          float s[8][4];
          const uint4* kt = reinterpret_cast<const uint4*>(sm.ring[stream][cstage]) + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int hh = 0; hh < KH; ++hh) {
              const uint4 w = kt[(j * KH + hh) * 32];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t k0, k1;
                codes_to_half<TYPE>(word4(w, i), k0, k1);
                mma16816(s[j], qf[hh * 4 + i], k0, k1);
              }
            }
          }
          // scores in units of log2
          cut = key0 < lo_all || key0 + kPage > hi_all;
          float f[2] = {fmaxf(mult[0] * sk, 1e-37f), fmaxf(mult[1] * sk, 1e-37f)};
          if (MODS) {
            const float k2 = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float x = s[j][i] * f[i >> 1];
                // cap * tanh(x / cap) = cap - 2 cap / (exp(2 x / cap) + 1)
                if (a.softcap > 0.f) x = a.softcap - __fdividef(2.f * a.softcap, ex2(x * k2) + 1.f);
                const int gap = pos[i >> 1] - (key0 + 16 * t + 2 * j + (i & 1));
                s[j][i] = x * kLog2e - slope[i >> 1] * (float)abs(gap);
              }
            f[0] = f[1] = 1.f;
          }
          if (cut) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key0 + 16 * t + 2 * j + (i & 1);
                if (key < lo[i >> 1] || key >= hi[i >> 1]) s[j][i] = -INFINITY;
              }
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * half], s[j][2 * half + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const float mn = fmaxf(m[half], mx * f[half]);
            const float use = mn == -INFINITY ? 0.f : mn;
            corr[half] = ex2(m[half] - use);
            m[half] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float p0 = ex2(fmaf(s[j][2 * half], f[half], -use)), p1 = ex2(fmaf(s[j][2 * half + 1], f[half], -use));
              sum += p0 + p1;
              pf[j >> 1][(j & 1) * 2 + half] = pack_h2(p0, p1);
            }
            l[half] = l[half] * corr[half] + sum;
          }
        }
        release();
        core::mbar_wait(&sm.full[stream][cstage], cphase, a.err);
        const float sv = sm.scale[stream][cstage];
        if (there) {
          const uint4* vt = reinterpret_cast<const uint4*>(sm.ring[stream][cstage]) + lane;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint4 w = vt[nt * 32];
            if (TYPE == QMV_KV_E4M3 && cut) {
              // slots past the request's end may hold any byte: a NaN code there would not be hidden by p = 0
              w.x &= ~__vcmpeq4(w.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              w.y &= ~__vcmpeq4(w.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              w.z &= ~__vcmpeq4(w.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              w.w &= ~__vcmpeq4(w.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            }
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t v0, v1;
              codes_to_half<TYPE>(word4(w, i), v0, v1);
              mma16816(c, pf[i], v0, v1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][i] = fmaf(c[i], sv, o[nt][i] * corr[i >> 1]);
          }
        }
        release();
      }

      // ---- end of the piece
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 1);
        l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 2);
      }
      const int which = first_piece ? 0 : 1;
      if (len == cw.n) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (g + 8 * half >= nr) continue;
          const int row = row0 + wr * 16 + g + 8 * half;
          const int64_t token = cw.r.qs + row / a.G;
          const int hq = cw.h * a.G + row % a.G;
          const float inv = l[half] == 0.f ? 0.f : 1.f / l[half];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            store_as(a.out_type, a.out, token * a.ldo + (int64_t)hq * D + nt * 8 + 2 * t, o[nt][2 * half] * inv, o[nt][2 * half + 1] * inv);
          if (a.lse && t == 0) a.lse[token * a.Hq + hq] = l[half] == 0.f ? -INFINITY : (m[half] + log2f(l[half])) * kLn2;
        }
      } else {
        const int64_t at = (int64_t)cta * (kStreamRows * 2) + (stream * 2 + which) * S::kRows + wr * 16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (g + 8 * half >= nr) continue;
          const int64_t row = at + g + 8 * half;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<float2*>(a.part_o + row * D + nt * 8 + 2 * t) = make_float2(o[nt][2 * half], o[nt][2 * half + 1]);
          if (t == 0) a.part_ml[row] = make_float2(m[half], l[half]);
        }
        if (leader && lane == 0) sm.piece[stream][which] = Piece{cw.start, cw.n, len, cw.r.b, cw.tile, cw.h};
      }
      first_piece = false;
      left -= len;
      cp = 0;
      if (left > 0) walk_next(a, cw, S::kRows);
    }
  }
  __syncthreads();

  // ---- join the partial tiles of this block's streams, tile by tile
  float* weights = reinterpret_cast<float*>(sm.ring);
  for (int e0 = 0; e0 < S::kStreams * 2;) {
    const Piece pc = (&sm.piece[0][0])[e0];
    if (pc.len == 0) {
      ++e0;
      continue;
    }
    int e1 = e0 + 1, covered = pc.len;
    for (; e1 < S::kStreams * 2; ++e1) {
      const Piece& p = (&sm.piece[0][0])[e1];
      if (p.len == 0) continue;
      if (p.start != pc.start) break;
      covered += p.len;
    }
    int n_e = 0;
    unsigned mask = 0;   // entries of this tile
    for (int e = e0; e < e1; ++e)
      if ((&sm.piece[0][0])[e].len > 0) {
        mask |= 1u << e;
        ++n_e;
      }
    const Req r = load_req(a, pc.b, S::kRows);
    const int row0 = pc.tile * S::kRows, rows = min(S::kRows, r.rows - row0);
    const int64_t base = (int64_t)cta * (kStreamRows * 2);
    auto stream_entry = [&](int e) { return base + (int64_t)__fns(mask, 0, e + 1) * S::kRows; };
    const bool whole = covered == pc.n;
    const int64_t mine_at = base + kStreamRows + (pc.start < u0 ? 0 : 1) * S::kRows;
    join<D>(a, n_e, rows, stream_entry, weights, whole, pc, r, row0, a.part_o + mine_at * D, a.part_ml + mine_at);
    if (!whole) {
      // blocks that hold a part of this tile
      const int c0 = (int)(((pc.start + 1) * A - 1) / W), c1 = (int)(((pc.start + pc.n) * A - 1) / W);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int old = atomicAdd(a.counters + c0, 1);
        sm.last = old == c1 - c0;
        if (sm.last) a.counters[c0] = 0;
      }
      __syncthreads();
      if (sm.last) {
        __threadfence();
        auto block_entry = [&](int e) {
          const long long c = c0 + e;
          return (int64_t)c * (kStreamRows * 2) + kStreamRows + (pc.start < c * W / A ? 0 : 1) * S::kRows;
        };
        join<D>(a, c1 - c0 + 1, rows, block_entry, weights, true, pc, r, row0, nullptr, nullptr);
      }
    }
    e0 = e1;
  }
}

template <int D, int TYPE, int R, bool MODS>
int launch(const Args& a, int blocks, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(attend_kernel<D, TYPE, R, MODS>);
  int per_sm = 0;
  int rc = kernel_fit(f, kThreads, sizeof(Smem<D, R>), &per_sm);
  if (rc) return rc;
  attend_kernel<D, TYPE, R, MODS><<<blocks, kThreads, sizeof(Smem<D, R>), s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv8_attend launch");
  return QMV_OK;
}

// One translation unit per (D, type): rows is the row tile (16, 32, 64 or 128).
int launch_64_int8(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);
int launch_64_e4m3(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);
int launch_128_int8(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);
int launch_128_e4m3(const Args& a, int rows, bool mods, int blocks, cudaStream_t s);

template <int D, int TYPE>
int launch_rows(const Args& a, int rows, bool mods, int blocks, cudaStream_t s) {
  switch (rows) {
    case 16: return mods ? launch<D, TYPE, 1, true>(a, blocks, s) : launch<D, TYPE, 1, false>(a, blocks, s);
    case 32: return mods ? launch<D, TYPE, 2, true>(a, blocks, s) : launch<D, TYPE, 2, false>(a, blocks, s);
    case 64: return mods ? launch<D, TYPE, 4, true>(a, blocks, s) : launch<D, TYPE, 4, false>(a, blocks, s);
    default: return mods ? launch<D, TYPE, 8, true>(a, blocks, s) : launch<D, TYPE, 8, false>(a, blocks, s);
  }
}

}  // namespace attend
}  // namespace qmv

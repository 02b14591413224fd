// Writing new keys and values into the paged 8-bit cache (kv8_append) and
// reading values back (kv8_read).
//
// One block takes one run (new tokens that share a page, at most 64) of one KV
// head, because the page's scale is a maximum over exactly these values: a
// thread holds up to two pieces of sixteen K and sixteen V values in registers
// from the load, through the rotation and the block's maximum, to the codes, so
// that each value is read once and each code written once. The cache's K tile
// takes the codes eight at a time straight from the registers; V is transposed
// through a byte tile in shared memory (word column swapped by the piece's
// number, so that the 32 lanes' byte stores meet 8 different banks) and leaves in
// 16-byte pieces of sixteen tokens. Codes already in the page are touched only
// where the scale grows: then they are read, rounded again and written in the
// same 16-byte pieces, and the piece that holds both old and new tokens merges
// them.
//
// The blocks after those of the runs rotate the query heads (the code of
// rope_run), so that a layer's rotation and cache write are one launch.
#include "kv8.cuh"

#include <cstring>

namespace qmv {
namespace {

using namespace kv8;

constexpr int kThreads8 = 256;

struct AppendArgs {
  qmv_rope r;
  int has_rope;
  const void *k, *v, *q;
  void* q_out;
  int64_t ldk, ldv, ldq, ldqo, ldp;
  int q_out_type, n_tokens, n_q_heads, n_runs;
  const int32_t *slots, *runs, *positions;
  unsigned char* cache;
  int64_t scale_off, n_pages;
  int H;
  int q_blocks;            // blocks that rotate query heads
  int q_heads_per_block;   // heads that one of them takes of a token
  int* err;
};

__device__ __forceinline__ uint32_t byte_of(const uint4& w, int i) {
  const uint32_t x = (i >> 2) == 0 ? w.x : (i >> 2) == 1 ? w.y : (i >> 2) == 2 ? w.z : w.w;
  return (x >> ((i & 3) * 8)) & 255u;
}

template <int TYPE>
__device__ __forceinline__ uint4 round_again(const uint4& w, float ratio) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i] |= encode<TYPE>(decode<TYPE>((in[i] >> (8 * j)) & 255u) * ratio) << (8 * j);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float amax8(const float (&v)[8], float m, bool& odd) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = fabsf(v[i]);
    if (x <= 3.402823466e38f) m = fmaxf(m, x);
    else odd = true;
  }
  return m;
}

template <typename TI, int D, int TYPE>
__global__ void __launch_bounds__(kThreads8) kv8_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int C = D / 16;                        // pieces of sixteen values per token
  constexpr int U = kPage * C / kThreads8;         // pieces per thread of a full page
  __shared__ __align__(16) uint32_t vt[D][kPage / 4];   // V codes, transposed
  __shared__ float red[2][kThreads8 / 32];
  const int tid = threadIdx.x;
  const int n_run_blocks = a.n_runs * a.H;
  if ((int)blockIdx.x >= n_run_blocks) {
    // query rotation: blocks stride over (token, group of heads)
    const int groups = (a.n_q_heads + a.q_heads_per_block - 1) / a.q_heads_per_block;
    const int c = tid % C, y = tid / C, rows = kThreads8 / C;
    for (int64_t w = blockIdx.x - n_run_blocks; w < (int64_t)a.n_tokens * groups; w += a.q_blocks) {
      const int64_t t = w / groups;
      const int h0 = (int)(w % groups) * a.q_heads_per_block;
      rope_tokens<TI>(a.r, static_cast<const TI*>(a.q), a.ldq, t, t + 1, h0, min(a.n_q_heads, h0 + a.q_heads_per_block),
                      a.positions, a.ldp, a.q_out, a.q_out_type, a.ldqo, 1.f, c, y, rows);
    }
    return;
  }
  const int run = blockIdx.x / a.H, head = blockIdx.x % a.H;
  const int2 rn = reinterpret_cast<const int2*>(a.runs)[run];
  const int t0 = rn.x, n = rn.y;
  if (n == 0) return;
  if (t0 < 0 || n < 0 || n > kPage || t0 > a.n_tokens - n) {
    if (tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    return;
  }
  const int slot = a.slots[t0];
  if (slot < 0) return;
  const int64_t page = slot / kPage;
  const int off = slot % kPage;
  if (page >= a.n_pages || off + n > kPage) {
    if (tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    return;
  }
  unsigned char* tile = a.cache + (page * a.H + head) * (int64_t)(2 * kPage * D);
  float* scale = reinterpret_cast<float*>(a.cache + a.scale_off) + (page * a.H + head) * 2;
  const float2 was = off > 0 ? *reinterpret_cast<const float2*>(scale) : make_float2(0.f, 0.f);

  // new values: piece u of this thread is sixteen values of token t0 + i
  float ka[U][8], kb[U][8], va[U][8], vb[U][8];
  float mk = 0.f, mv = 0.f;
  bool odd = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = tid + u * kThreads8, i = p / C, c = p % C;
    if (i >= n) continue;
    const TI* pk = static_cast<const TI*>(a.k) + (int64_t)(t0 + i) * a.ldk + (int64_t)head * D;
    const TI* pv = static_cast<const TI*>(a.v) + (int64_t)(t0 + i) * a.ldv + (int64_t)head * D;
    const RopeChunk ch = a.has_rope ? rope_chunk(a.r, c) : RopeChunk{16 * c, 16 * c + 8, false};
    load8(pk + ch.d0, ka[u]);
    load8(pk + ch.d1, kb[u]);
    load8(pv + 16 * c, va[u]);
    load8(pv + 16 * c + 8, vb[u]);
    if (ch.turned) {
      float cs[8], sn[8];
      rope_angles(a.r, c, a.positions + t0 + i, a.ldp, 1.f, cs, sn);
      rope_turn(a.r.interleaved != 0, cs, sn, ka[u], kb[u]);
    }
    mk = amax8(kb[u], amax8(ka[u], mk, odd), odd);
    mv = amax8(vb[u], amax8(va[u], mv, odd), odd);
  }
  if (odd) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xFFFFFFFFu, mk, o));
    mv = fmaxf(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, o));
  }
  if ((tid & 31) == 0) {
    red[0][tid >> 5] = mk;
    red[1][tid >> 5] = mv;
  }
  __syncthreads();  // every thread has read `was` too
#pragma unroll
  for (int w = 0; w < kThreads8 / 32; ++w) {
    mk = fmaxf(mk, red[0][w]);
    mv = fmaxf(mv, red[1][w]);
  }
  const float top = code_top<TYPE>();
  const float sk = fmaxf(was.x, __fdiv_rn(mk, top)), sv = fmaxf(was.y, __fdiv_rn(mv, top));
  const float ik = sk > 0.f ? __frcp_rn(sk) : 0.f, iv = sv > 0.f ? __frcp_rn(sv) : 0.f;
  if (tid == 0) *reinterpret_cast<float2*>(scale) = make_float2(sk, sv);

  // K: codes eight at a time, and V into the transposing tile
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = tid + u * kThreads8, i = p / C, c = p % C;
    if (i >= n) continue;
    const RopeChunk ch = a.has_rope ? rope_chunk(a.r, c) : RopeChunk{16 * c, 16 * c + 8, false};
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[j] |= encode<TYPE>((j < 2 ? ka[u][(4 * j + b) & 7] : kb[u][(4 * j + b) & 7]) * ik) << (8 * b);
    }
    *reinterpret_cast<uint2*>(tile + k_byte(off + i, ch.d0, D)) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(tile + k_byte(off + i, ch.d1, D)) = make_uint2(w[2], w[3]);
    const int tok = off + i, column = (tok >> 2) ^ ((2 * c) & 15);
#pragma unroll
    for (int d = 0; d < 16; ++d)
      reinterpret_cast<unsigned char*>(&vt[16 * c + d][column])[tok & 3] =
          (unsigned char)encode<TYPE>((d < 8 ? va[u][d & 7] : vb[u][d & 7]) * iv);
  }
  // K codes already in the page
  if (off > 0 && sk > was.x && was.x > 0.f) {
    const float ratio = was.x * ik;
    for (int p = tid; p < off * C; p += kThreads8) {
      uint4* at = reinterpret_cast<uint4*>(tile + k_byte(p / C, (p % C) * 16, D));
      *at = round_again<TYPE>(*at, ratio);
    }
  }
  __syncthreads();
  // V: pieces of sixteen tokens that hold a new token, and those before them where the scale has grown
  const bool grown = off > 0 && sv > was.y && was.y > 0.f;
  const float ratio = was.y * iv;
  const int g0 = grown ? 0 : off / 16, g1 = (off + n + 15) / 16;
  for (int p = tid; p < D * (g1 - g0); p += kThreads8) {
    const int d = p % D, g = g0 + p / D, first = off - 16 * g;   // tokens from `first` on are new
    uint4* at = reinterpret_cast<uint4*>(tile + kPage * D + v_byte(16 * g, d));
    const int swap = (2 * (d / 16)) & 15;
    uint4 fresh;
    fresh.x = vt[d][(4 * g) ^ swap];
    fresh.y = vt[d][(4 * g + 1) ^ swap];
    fresh.z = vt[d][(4 * g + 2) ^ swap];
    fresh.w = vt[d][(4 * g + 3) ^ swap];
    if (first <= 0) {
      // slots past the run's end are not in use yet, so their bytes may be anything
      *at = fresh;
    } else if (grown) {
      uint4 old = round_again<TYPE>(*at, ratio);
      uint32_t* o = reinterpret_cast<uint32_t*>(&old);
      const uint32_t* f = reinterpret_cast<const uint32_t*>(&fresh);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int keep = min(max(first - 4 * j, 0), 4);   // bytes of the word that are old
        const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        o[j] = (o[j] & mask) | (f[j] & ~mask);
      }
      *at = old;
    } else {
      // old codes stay as they are: only the new bytes are written
      for (int i = first; i < min(16, first + n); ++i) reinterpret_cast<unsigned char*>(at)[i] = (unsigned char)byte_of(fresh, i);
    }
  }
}

// ---- reading back

struct ReadArgs {
  const unsigned char* cache;
  int64_t scale_off, n_pages, n, ldo;
  const int32_t* slots;
  void *k_out, *v_out;
  int H, out_type;
  int* err;
};

// A block takes 64 entries of the slot list and one head. Entries that follow
// one another in one page (the usual case) go through shared memory: the page's
// 2 x 64 x D codes are read in 16-byte pieces and every output row leaves in
// 16-byte pieces. Pieces of eight values of V are gathered from eight rows of
// the transposed tile, whose words lie 64 bytes apart: the tile's rows are
// swapped by d / 8 so that the lanes of a warp meet different banks.
template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads8) kv8_read_kernel(const __grid_constant__ ReadArgs a) {
  __shared__ __align__(16) unsigned char kt[kPage * D];
  __shared__ __align__(16) uint32_t vt[D][kPage / 4];
  __shared__ int slot[kPage];
  const int tid = threadIdx.x, head = blockIdx.y;
  const int64_t e0 = (int64_t)blockIdx.x * kPage;
  const int n = (int)min((int64_t)kPage, a.n - e0);
  if (tid < n) slot[tid] = a.slots[e0 + tid];
  __syncthreads();
  constexpr int P = D / 8;
  for (int first = 0; first < n;) {
    const int s0 = slot[first];
    const int64_t page = s0 < 0 ? -1 : s0 / kPage;
    int last = first + 1;  // entries [first, last) lie in one page, in any order
    while (last < n && (slot[last] < 0 ? -1 : slot[last] / kPage) == page) ++last;
    const bool there = page >= 0 && page < a.n_pages;
    if (page >= a.n_pages && tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    float2 sc = make_float2(0.f, 0.f);
    if (there) {
      const unsigned char* tile = a.cache + (page * a.H + head) * (int64_t)(2 * kPage * D);
      sc = reinterpret_cast<const float2*>(a.cache + a.scale_off)[page * a.H + head];
      for (int p = tid; p < kPage * D / 16; p += kThreads8) {
        reinterpret_cast<uint4*>(kt)[p] = reinterpret_cast<const uint4*>(tile)[p];
        const uint4 w = reinterpret_cast<const uint4*>(tile + kPage * D)[p];
        const int d = p / 4, q = (p % 4) * 4, swap = (d / 8) & 15;
        vt[d][q ^ swap] = w.x;
        vt[d][(q + 1) ^ swap] = w.y;
        vt[d][(q + 2) ^ swap] = w.z;
        vt[d][(q + 3) ^ swap] = w.w;
      }
    }
    __syncthreads();
    for (int p = tid; p < (last - first) * P; p += kThreads8) {
      const int e = first + p / P, d0 = (p % P) * 8;
      float k[8], v[8];
      if (there) {
        const int tok = slot[e] % kPage;
        const uint2 w = *reinterpret_cast<const uint2*>(kt + k_byte(tok, d0, D));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          k[i] = decode<TYPE>(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 255u) * sc.x;
          v[i] = decode<TYPE>((vt[d0 + i][(tok >> 2) ^ ((d0 / 8) & 15)] >> (8 * (tok & 3))) & 255u) * sc.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.f;
      }
      const int64_t o = (e0 + e) * a.ldo + (int64_t)head * D + d0;
      store8_as(a.out_type, a.k_out, o, k);
      store8_as(a.out_type, a.v_out, o, v);
    }
    __syncthreads();
    first = last;
  }
}

template <typename TI>
const void* append_kernel(int D, int type) {
  if (D == 64) return type == QMV_KV_INT8 ? (const void*)kv8_append_kernel<TI, 64, QMV_KV_INT8> : (const void*)kv8_append_kernel<TI, 64, QMV_KV_E4M3>;
  return type == QMV_KV_INT8 ? (const void*)kv8_append_kernel<TI, 128, QMV_KV_INT8> : (const void*)kv8_append_kernel<TI, 128, QMV_KV_E4M3>;
}

}  // namespace

namespace kv8 {
int check_kv_desc(const qmv_kv_desc* d) {
  if (!d) return fail(QMV_ERR_ARG, "desc is NULL");
  if (d->abi_version != QMV_ABI_VERSION) return fail(QMV_ERR_ARG, "desc abi_version %u, library %d", d->abi_version, QMV_ABI_VERSION);
  qmv_kv_desc ref;
  int rc = kv8_desc((int)d->type, d->n_pages, d->n_kv_heads, d->head_dim, &ref);
  if (rc) return rc;
  if (memcmp(ref.off, d->off, sizeof(ref.off)) || memcmp(ref.bytes, d->bytes, sizeof(ref.bytes)) || ref.total_bytes != d->total_bytes)
    return fail(QMV_ERR_ARG, "desc sections do not match the layout of %lld pages", (long long)d->n_pages);
  return QMV_OK;
}
}  // namespace kv8
}  // namespace qmv

using namespace qmv;
using namespace qmv::kv8;

extern "C" {

int kv8_desc(int type, int64_t n_pages, int32_t n_kv_heads, int32_t head_dim, qmv_kv_desc* out) {
  if (!out) return fail(QMV_ERR_ARG, "out is NULL");
  if (type != QMV_KV_INT8 && type != QMV_KV_E4M3) return fail(QMV_ERR_ARG, "unknown cache type %d", type);
  if (n_pages < 1 || n_kv_heads < 1 || n_kv_heads > 1024) return fail(QMV_ERR_ARG, "n_pages=%lld n_kv_heads=%d", (long long)n_pages, n_kv_heads);
  if (n_pages > INT32_MAX / kPage) return fail(QMV_ERR_UNSUPPORTED, "n_pages=%lld: slots must fit 31 bits", (long long)n_pages);
  if (head_dim != 64 && head_dim != 128) return fail(QMV_ERR_UNSUPPORTED, "head_dim=%d (64 and 128 are served)", head_dim);
  memset(out, 0, sizeof(*out));
  out->abi_version = QMV_ABI_VERSION;
  out->type = (uint32_t)type;
  out->n_kv_heads = n_kv_heads;
  out->head_dim = head_dim;
  out->n_pages = n_pages;
  out->bytes[0] = n_pages * n_kv_heads * 2 * kPage * head_dim;
  out->bytes[1] = n_pages * n_kv_heads * 2 * (int64_t)sizeof(float);
  out->off[1] = (out->bytes[0] + 255) / 256 * 256;
  out->total_bytes = (out->off[1] + out->bytes[1] + 255) / 256 * 256;
  return QMV_OK;
}

int kv8_append(const qmv_kv_desc* desc, void* cache, const qmv_rope* rope, const kv8_append_args* g, void* stream) {
  int rc = check_kv_desc(desc);
  if (rc) return rc;
  if (!g) return fail(QMV_ERR_ARG, "args is NULL");
  const int xs = dtype_size(g->x_type);
  if (!xs) return fail(QMV_ERR_ARG, "x_type=%d", g->x_type);
  if (g->n_tokens < 0 || g->n_runs < 0) return fail(QMV_ERR_ARG, "n_tokens=%d n_runs=%d", g->n_tokens, g->n_runs);
  const int64_t row = (int64_t)desc->n_kv_heads * desc->head_dim;
  if (g->ldk < row || g->ldv < row) return fail(QMV_ERR_ARG, "ldk=%lld ldv=%lld below %lld", (long long)g->ldk, (long long)g->ldv, (long long)row);
  if (g->ldk * xs % 16 || g->ldv * xs % 16) return fail(QMV_ERR_ALIGN, "rows of k and v must be 16-byte aligned");
  if (rope) {
    rc = check_rope(rope);
    if (rc) return rc;
    if (rope->head_dim != desc->head_dim) return fail(QMV_ERR_ARG, "rope head_dim=%d, cache %d", rope->head_dim, desc->head_dim);
    if (g->ldp < g->n_tokens) return fail(QMV_ERR_ARG, "ldp=%lld below n_tokens", (long long)g->ldp);
  }
  if (g->q) {
    if (!rope) return fail(QMV_ERR_ARG, "q without rope: there is nothing to do for it");
    const int os = dtype_size(g->q_out_type);
    if (!os) return fail(QMV_ERR_ARG, "q_out_type=%d", g->q_out_type);
    const int64_t qrow = (int64_t)g->n_q_heads * desc->head_dim;
    if (g->n_q_heads < 1 || g->n_q_heads > 65536 || g->ldq < qrow || g->ldqo < qrow)
      return fail(QMV_ERR_ARG, "n_q_heads=%d ldq=%lld ldqo=%lld", g->n_q_heads, (long long)g->ldq, (long long)g->ldqo);
    if (g->ldq * xs % 16 || g->ldqo * os % 16) return fail(QMV_ERR_ALIGN, "rows of q and q_out must be 16-byte aligned");
    if (!g->q_out) return fail(QMV_ERR_ARG, "NULL q_out");
    if (!aligned16(g->q) || !aligned16(g->q_out)) return fail(QMV_ERR_ALIGN, "q and q_out must be 16-byte aligned");
    if (g->q == g->q_out && (g->x_type != g->q_out_type || g->ldq != g->ldqo))
      return fail(QMV_ERR_ARG, "in place needs one type and one stride");
  }
  if (g->n_tokens == 0) return QMV_OK;
  if (!cache || !g->k || !g->v || !g->slots || (g->n_runs > 0 && !g->runs) || (rope && !g->positions))
    return fail(QMV_ERR_ARG, "NULL cache, k, v, slots, runs or positions");
  if (!aligned16(cache) || !aligned16(g->k) || !aligned16(g->v)) return fail(QMV_ERR_ALIGN, "cache, k and v must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(g->slots) & 3u) || (reinterpret_cast<uintptr_t>(g->runs) & 7u) ||
      (rope && (reinterpret_cast<uintptr_t>(g->positions) & 3u)))
    return fail(QMV_ERR_ALIGN, "slots and positions must be 4-byte aligned, runs 8-byte");
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");

  AppendArgs a;
  memset(&a, 0, sizeof(a));
  if (rope) a.r = *rope;
  a.has_rope = rope != nullptr;
  a.k = g->k;
  a.v = g->v;
  a.q = g->q;
  a.q_out = g->q_out;
  a.ldk = g->ldk;
  a.ldv = g->ldv;
  a.ldq = g->ldq;
  a.ldqo = g->ldqo;
  a.ldp = g->ldp;
  a.q_out_type = g->q_out_type;
  a.n_tokens = g->n_tokens;
  a.n_q_heads = g->n_q_heads;
  a.n_runs = g->n_runs;
  a.slots = g->slots;
  a.runs = g->runs;
  a.positions = g->positions;
  a.cache = static_cast<unsigned char*>(cache);
  a.scale_off = desc->off[1];
  a.n_pages = desc->n_pages;
  a.H = desc->n_kv_heads;
  a.err = err;
  int64_t blocks = (int64_t)g->n_runs * desc->n_kv_heads;
  if (g->q) {
    // as rope_run: few tokens are split over the heads, many take all heads of a token in one block
    const int rows = kThreads8 / (desc->head_dim / 16);
    const bool split = g->n_tokens < 4 * sm_count();
    a.q_heads_per_block = split && rows < g->n_q_heads ? rows : g->n_q_heads;
    const int64_t groups = (g->n_q_heads + a.q_heads_per_block - 1) / a.q_heads_per_block;
    const int64_t work = groups * g->n_tokens;
    a.q_blocks = (int)(work < (1 << 16) ? work : (1 << 16));
    blocks += a.q_blocks;
  }
  if (blocks == 0) return QMV_OK;
  if (blocks > INT32_MAX) return fail(QMV_ERR_UNSUPPORTED, "too many runs");
  const void* f = g->x_type == QMV_F32 ? append_kernel<float>(desc->head_dim, (int)desc->type)
                  : g->x_type == QMV_BF16 ? append_kernel<__nv_bfloat16>(desc->head_dim, (int)desc->type)
                                          : append_kernel<__half>(desc->head_dim, (int)desc->type);
  void* args[] = {&a};
  cudaError_t e = cudaLaunchKernel(f, dim3((unsigned)blocks), dim3(kThreads8), args, 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv8_append launch");
  return QMV_OK;
}

int kv8_read(const qmv_kv_desc* desc, const void* cache, const int32_t* slots, int64_t n, void* k_out, void* v_out,
             int out_type, int64_t ldo, void* stream) {
  int rc = check_kv_desc(desc);
  if (rc) return rc;
  const int os = dtype_size(out_type);
  if (!os) return fail(QMV_ERR_ARG, "out_type=%d", out_type);
  if (n < 0 || n > INT32_MAX) return fail(QMV_ERR_ARG, "n=%lld", (long long)n);
  if (ldo < (int64_t)desc->n_kv_heads * desc->head_dim) return fail(QMV_ERR_ARG, "ldo=%lld", (long long)ldo);
  if (ldo * os % 16) return fail(QMV_ERR_ALIGN, "output rows must be 16-byte aligned");
  if (n == 0) return QMV_OK;
  if (!cache || !slots || !k_out || !v_out) return fail(QMV_ERR_ARG, "NULL cache, slots or outputs");
  if (!aligned16(cache) || !aligned16(k_out) || !aligned16(v_out) || (reinterpret_cast<uintptr_t>(slots) & 3u))
    return fail(QMV_ERR_ALIGN, "cache and outputs must be 16-byte aligned, slots 4-byte");
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");
  ReadArgs a{static_cast<const unsigned char*>(cache), desc->off[1], desc->n_pages, n, ldo, slots, k_out, v_out,
             desc->n_kv_heads, out_type, err};
  const dim3 grid((unsigned)((n + kPage - 1) / kPage), (unsigned)desc->n_kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool i8 = desc->type == QMV_KV_INT8;
  if (desc->head_dim == 64) {
    if (i8) kv8_read_kernel<64, QMV_KV_INT8><<<grid, kThreads8, 0, s>>>(a);
    else kv8_read_kernel<64, QMV_KV_E4M3><<<grid, kThreads8, 0, s>>>(a);
  } else {
    if (i8) kv8_read_kernel<128, QMV_KV_INT8><<<grid, kThreads8, 0, s>>>(a);
    else kv8_read_kernel<128, QMV_KV_E4M3><<<grid, kThreads8, 0, s>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv8_read launch");
  return QMV_OK;
}

}  // extern "C"

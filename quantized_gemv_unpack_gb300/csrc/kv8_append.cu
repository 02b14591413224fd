// Writing new keys and values into the paged 8-bit cache (kv8_append) and
// reading values back (kv8_read).
//
// One block takes one run (new tokens that share a page, at most 64) of one or a
// few KV heads, because a page's scale is a maximum over exactly these values of a
// head: a thread holds its pieces of sixteen K and sixteen V values in registers
// from the load, through the rotation and the block's maximum, to the codes, so
// that each value is read once and each code written once. The cache's K tile
// takes the codes eight at a time straight from the registers; V is transposed,
// four tokens by exchanges between lanes and sixteen through shared memory, and
// leaves in 16-byte pieces of sixteen tokens. Codes already in the page are touched only
// where the scale grows: then they are read, rounded again and written in the
// same 16-byte pieces, and the piece that holds both old and new tokens merges
// them.
//
// A decode step's runs are one token each: they go to a kernel of one warp per run
// and head, whose further blocks rotate the query heads, so that a layer's
// rotation and cache write are one launch there.
//
// Measured (40 query and 8 KV heads of 128): 8190 prompt tokens, bf16 to e4m3, 18 us
// behind the 32 of the rotation of q, 50 together; reading them back 14 us. Neither
// the write nor the read reaches a limit of the machine: block-wide steps and the
// transposition of V leave issue 52 and 63 % busy, DRAM 18 and 13 %. A step of 64
// tokens: 4.5 us, and 5.6 to read them back, launch and dependent loads.
#include "kv8.cuh"

#include <cstring>

namespace qmv {
namespace {

using namespace kv8;

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
  int head_group, head_groups;   // KV heads of one block, blocks per run
  int q_heads;                   // heads of a block that rotates query heads (few tokens)
  int* err;
};

__device__ __forceinline__ uint32_t byte_of(const uint4& w, int i) {
  const uint32_t x = (i >> 2) == 0 ? w.x : (i >> 2) == 1 ? w.y : (i >> 2) == 2 ? w.z : w.w;
  return (x >> ((i & 3) * 8)) & 255u;
}

// Sixteen codes rounded again at ratio <= 1 of their scale.
template <int TYPE>
__device__ __forceinline__ uint4 round_again(const uint4& w, float ratio) {
  float a[8], b[8];
  decode8<TYPE>(make_uint2(w.x, w.y), a);
  decode8<TYPE>(make_uint2(w.z, w.w), b);
  const uint2 lo = encode8<TYPE>(a, ratio), hi = encode8<TYPE>(b, ratio);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// Largest finite magnitude among sixteen values and m.
__device__ __forceinline__ float amax16(const float (&a)[8], const float (&b)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = fabsf(a[i]), y = fabsf(b[i]);
    m = fmaxf(m, fmaxf(x <= 3.402823466e38f ? x : 0.f, y <= 3.402823466e38f ? y : 0.f));
  }
  return m;
}

// Four words of four bytes in each of four lanes (lane bits `one` and `two` of the lane number), transposed: word j of
// lane k comes out as byte k of word j of lanes 0..3, in that order.
__device__ __forceinline__ void transpose_bytes(uint32_t (&w)[4], bool hi1, bool hi2, int one, int two) {
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    // lanes that differ in `two` exchange: the lower keeps bytes 0, 1 of both and takes the other's
    const uint32_t give = hi2 ? __byte_perm(w[j], w[j + 1], 0x5410) : __byte_perm(w[j], w[j + 1], 0x7632);
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, two);
    w[j] = hi2 ? __byte_perm(got, w[j], 0x7610) : __byte_perm(w[j], got, 0x5410);
    w[j + 1] = hi2 ? __byte_perm(got, w[j + 1], 0x7632) : __byte_perm(w[j + 1], got, 0x7610);
  }
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t give = hi1 ? __byte_perm(w[j], w[j + 1], 0x6420) : __byte_perm(w[j], w[j + 1], 0x7531);
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, one);
    w[j] = hi1 ? __byte_perm(got, w[j], 0x7150) : __byte_perm(w[j], got, 0x5240);
    w[j + 1] = hi1 ? __byte_perm(got, w[j + 1], 0x7352) : __byte_perm(w[j + 1], got, 0x7260);
  }
}

// Word columns of the transposing tile's row d are swapped by this, so that the lanes' words meet different banks.
__device__ __forceinline__ int v_swap(int d) { return (2 * (d / 16) + ((d >> 1) & 1)) & 15; }

// BLOCK threads hold a full page's 64 * D / 16 pieces, U per thread.
template <typename TI, int D, int TYPE, int BLOCK>
__device__ __forceinline__ void append_run(const AppendArgs& a) {
  constexpr int C = D / 16;                        // pieces of sixteen values per token
  constexpr int U = kPage * C / BLOCK;             // pieces per thread of a full page
  __shared__ __align__(16) uint32_t vt[D][kPage / 4];   // V codes, transposed
  __shared__ float red[2][BLOCK / 32];
  __shared__ float4 set;                           // new scales of K and V, and their reciprocals
  __shared__ float2 before;                        // the scales before
  extern __shared__ __align__(16) float2 angles[]; // of the run's tokens, with rope; read two pairs at a time
  const int tid = threadIdx.x;
  const int run = blockIdx.x / a.head_groups, first_head = (blockIdx.x % a.head_groups) * a.head_group;
  const int last_head = min(a.H, first_head + a.head_group);
  const int2 rn = reinterpret_cast<const int2*>(a.runs)[run];
  const int t0 = rn.x, n = rn.y;
  if (n == 0) return;
  if (t0 < 0 || n < 0 || n > kPage || t0 > a.n_tokens - n) {
    if (tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    return;
  }
  // piece u of this thread is sixteen values of token t0 + i (chunk c); the first head's loads are in flight while the
  // angles are computed
  Raw16<TI> rk[U], rv[U];
  auto fetch = [&](int head) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = tid + u * BLOCK, i = p / C, c = p % C;
      if (i >= n) continue;
      const RopeChunk ch = a.has_rope ? rope_chunk(a.r, c) : RopeChunk{16 * c, 16 * c + 8, false};
      rk[u] = load_raw(static_cast<const TI*>(a.k) + (int64_t)(t0 + i) * a.ldk + (int64_t)head * D, ch.d0, ch.d1);
      rv[u] = load_raw(static_cast<const TI*>(a.v) + (int64_t)(t0 + i) * a.ldv + (int64_t)head * D, 16 * c, 16 * c + 8);
    }
  };
  fetch(first_head);
  const int slot = a.slots[t0];
  if (a.has_rope) rope_angles(a.r, n, a.positions + t0, a.ldp, 1.f, angles, tid, BLOCK);
  if (slot < 0) return;
  const int64_t page = slot / kPage;
  const int off = slot % kPage;
  if (page >= a.n_pages || off + n > kPage) {
    if (tid == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    return;
  }
  __syncthreads();  // the angles are there

  for (int head = first_head; head < last_head; ++head) {
    if (head > first_head) fetch(head);
    unsigned char* tile = a.cache + (page * a.H + head) * (int64_t)(2 * kPage * D);
    float* scale = reinterpret_cast<float*>(a.cache + a.scale_off) + (page * a.H + head) * 2;

    // K rotated in fp32; V stays as it came until it is encoded
    float ka[U][8], kb[U][8];
    float mk = 0.f, mv = 0.f;
    bool odd = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = tid + u * BLOCK, i = p / C, c = p % C;
      if (i >= n) {
#pragma unroll
        for (int j = 0; j < 2 * Raw16<TI>::W; ++j) rv[u].w[j] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) ka[u][j] = kb[u][j] = 0.f;
        continue;
      }
      unpack(rk[u], ka[u], kb[u]);
      if (a.has_rope && c * 16 < a.r.rot_dim) {
        float cs[8], sn[8];
        chunk_angles(angles, i, c, C, cs, sn);
        rope_turn(a.r.interleaved != 0, cs, sn, ka[u], kb[u]);
      }
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(ka[u][j]), fabsf(kb[u][j])));
      const uint32_t tv = raw_top(rv[u]);
      if (raw_top(rk[u]) >= odd_bits<TI>() || tv >= odd_bits<TI>() || m > 3.402823466e38f) {
        odd = true;
        float x[8], y[8];
        unpack(rv[u], x, y);
        mk = amax16(ka[u], kb[u], mk);
        mv = amax16(x, y, mv);
      } else {
        mk = fmaxf(mk, m);
        mv = fmaxf(mv, top_value<TI>(tv));
      }
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
    __syncthreads();  // the previous head's V tile has been read too
    if (tid < 32) {
      // one warp joins the maxima and takes the quotients for all
      constexpr int W = BLOCK / 32;
      mk = red[0][tid & (W - 1)];
      mv = red[1][tid & (W - 1)];
#pragma unroll
      for (int o = W / 2; o; o >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xFFFFFFFFu, mk, o));
        mv = fmaxf(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, o));
      }
      const float2 old = off > 0 ? *reinterpret_cast<const float2*>(scale) : make_float2(0.f, 0.f);
      const float top = code_top<TYPE>();
      const float sk = grown_scale(old.x, mk, top), sv = grown_scale(old.y, mv, top);
      __syncwarp();
      if (tid == 0) {
        set = make_float4(sk, sv, sk > 0.f ? __frcp_rn(sk) : 0.f, sv > 0.f ? __frcp_rn(sv) : 0.f);
        before = old;
        *reinterpret_cast<float2*>(scale) = make_float2(sk, sv);
      }
    }
    __syncthreads();
    const float2 was = before;
    const float sk = set.x, sv = set.y, ik = set.z, iv = set.w;

    // K: codes eight at a time, and V into the transposing tile
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = tid + u * BLOCK, i = p / C, c = p % C;
      const RopeChunk ch = a.has_rope ? rope_chunk(a.r, c) : RopeChunk{16 * c, 16 * c + 8, false};
      float va[8], vb[8];
      unpack(rv[u], va, vb);
      uint2 w0, w1, x0, x1;
      if (!odd) {
        w0 = encode8<TYPE>(ka[u], ik);
        w1 = encode8<TYPE>(kb[u], ik);
        x0 = encode8<TYPE>(va, iv);
        x1 = encode8<TYPE>(vb, iv);
      } else {
        w0 = encode8_any<TYPE>(ka[u], ik);
        w1 = encode8_any<TYPE>(kb[u], ik);
        x0 = encode8_any<TYPE>(va, iv);
        x1 = encode8_any<TYPE>(vb, iv);
      }
      if (i < n) {
        *reinterpret_cast<uint2*>(tile + k_byte(off + i, ch.d0, D)) = w0;
        *reinterpret_cast<uint2*>(tile + k_byte(off + i, ch.d1, D)) = w1;
      }
      uint32_t v4[4] = {x0.x, x0.y, x1.x, x1.y};
      const int tok = off + i;
      if ((off & 3) == 0) {
        // the lanes of four neighbouring tokens exchange bytes, so that each holds words of four tokens of one d
        transpose_bytes(v4, (i & 1) != 0, (i & 2) != 0, C, 2 * C);
        if (tok < kPage)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = 16 * c + 4 * j + (i & 3);
            vt[d][(tok >> 2) ^ v_swap(d)] = v4[j];
          }
      } else if (i < n) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int d = 16 * c + j;
          reinterpret_cast<unsigned char*>(&vt[d][(tok >> 2) ^ v_swap(d)])[tok & 3] = (unsigned char)(v4[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
    // K codes already in the page
    if (off > 0 && sk > was.x && was.x > 0.f) {
      const float ratio = was.x * ik;
      for (int p = tid; p < off * C; p += BLOCK) {
        uint4* at = reinterpret_cast<uint4*>(tile + k_byte(p / C, (p % C) * 16, D));
        *at = round_again<TYPE>(*at, ratio);
      }
    }
    __syncthreads();
    // V: pieces of sixteen tokens that hold a new token, and those before them where the scale has grown
    const bool grown = off > 0 && sv > was.y && was.y > 0.f;
    const float ratio = was.y * iv;
    const int g0 = grown ? 0 : off / 16, groups = (off + n + 15) / 16 - g0;
    for (int p = tid; p < D * groups; p += BLOCK) {
      // neighbouring threads take the groups of one d: a full page's row of 64 bytes in four pieces
      const int d = groups == 4 ? p >> 2 : p / groups, g = g0 + p - d * groups, first = off - 16 * g;   // from `first` on: new
      uint4* at = reinterpret_cast<uint4*>(tile + kPage * D + v_byte(16 * g, d));
      const int swap = v_swap(d);
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
}

template <typename TI, int D, int TYPE, int BLOCK>
__global__ void __launch_bounds__(BLOCK, 1024 / BLOCK) kv8_append_kernel(const __grid_constant__ AppendArgs a) {
  follow_previous();
  append_run<TI, D, TYPE, BLOCK>(a);
}

// Runs of a few tokens (a decode step: one). One warp takes a run of one head, a lane the two values of D / 64 pairs of K
// and as many of V: no block-wide step, and the chain of loads (run, slot, values, scale) is the time.
// Values are read again for the codes where the run has more than one token.
constexpr int kFewThreads = 128;

template <typename TI, int D, int TYPE>
__global__ void __launch_bounds__(kFewThreads) kv8_append_few_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int V = D / 64;                    // values per lane from each half of a chunk
  constexpr int C = D / 16, L = 8 / V;         // chunks, lanes per chunk
  __shared__ __align__(16) float2 angles[D / 2];   // read two pairs at a time, like all tables of angles
  const int tid = threadIdx.x, lane = tid & 31;
  follow_previous();
  const int n_runs = a.n_runs * a.H, run_blocks = (n_runs + kFewThreads / 32 - 1) / (kFewThreads / 32);
  if ((int)blockIdx.x >= run_blocks) {
    const int w = blockIdx.x - run_blocks, groups = (a.n_q_heads + a.q_heads - 1) / a.q_heads;
    const int h0 = (w % groups) * a.q_heads;
    rope_tokens<TI>(a.r, static_cast<const TI*>(a.q), a.ldq, w / groups, 1, h0, min(a.n_q_heads, h0 + a.q_heads), a.positions,
                    a.ldp, a.q_out, a.q_out_type, a.ldqo, 1.f, angles, tid, kFewThreads);
    return;
  }
  const int index = blockIdx.x * (kFewThreads / 32) + (tid >> 5);
  if (index >= n_runs) return;
  const int run = index / a.H, head = index - run * a.H;
  const int2 rn = reinterpret_cast<const int2*>(a.runs)[run];
  const int t0 = rn.x, n = rn.y;
  if (n == 0) return;
  if (t0 < 0 || n < 0 || n > kPage || t0 > a.n_tokens - n) {
    if (lane == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    return;
  }
  const int c = lane / L, sub = (lane % L) * V;   // pairs sub, .. of chunk c
  const RopeChunk ch = a.has_rope ? rope_chunk(a.r, c) : RopeChunk{16 * c, 16 * c + 8, false};
  const bool side = ch.turned && a.r.interleaved != 0;   // a pair's values lie side by side
  auto k_at = [&](int half, int j) { return side ? 16 * c + 2 * (sub + j) + half : (half ? ch.d1 : ch.d0) + sub + j; };
  uint64_t turn[V];
  const int32_t* pos[V];
  if (ch.turned) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int pair = 8 * c + sub + j;
      turn[j] = a.r.turn[pair];
      pos[j] = a.positions + (int64_t)a.r.axis[pair] * a.ldp + t0;
    }
  }
  float k[2][V], v[2][V];
  auto load = [&](int i) {
    const TI* pk = static_cast<const TI*>(a.k) + (int64_t)(t0 + i) * a.ldk + (int64_t)head * D;
    const TI* pv = static_cast<const TI*>(a.v) + (int64_t)(t0 + i) * a.ldv + (int64_t)head * D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      k[0][j] = (float)pk[k_at(0, j)];
      k[1][j] = (float)pk[k_at(1, j)];
      v[0][j] = (float)pv[16 * c + sub + j];
      v[1][j] = (float)pv[16 * c + 8 + sub + j];
    }
    if (!ch.turned) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint64_t ph = (uint64_t)(int64_t)pos[j][i] * turn[j];
      float cs, sn;
      sincospif((float)(int32_t)(ph >> 32) * 4.656612873077393e-10f, &sn, &cs);
      rope_pair(cs, sn, k[0][j], k[1][j]);
    }
  };
  load(0);
  const int slot = a.slots[t0];
  if (slot < 0) return;
  const int64_t page = slot / kPage;
  const int off = slot % kPage;
  if (page >= a.n_pages || off + n > kPage) {
    if (lane == 0) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
    return;
  }
  unsigned char* tile = a.cache + (page * a.H + head) * (int64_t)(2 * kPage * D);
  float* scale = reinterpret_cast<float*>(a.cache + a.scale_off) + (page * a.H + head) * 2;
  const float2 was = off > 0 ? *reinterpret_cast<const float2*>(scale) : make_float2(0.f, 0.f);
  float mk = 0.f, mv = 0.f;
  bool odd = false;
  for (int i = 0; i < n; ++i) {
    if (i > 0) load(i);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (fabsf(k[e][j]) <= 3.402823466e38f) mk = fmaxf(mk, fabsf(k[e][j]));
        else odd = true;
        if (fabsf(v[e][j]) <= 3.402823466e38f) mv = fmaxf(mv, fabsf(v[e][j]));
        else odd = true;
      }
  }
  if (odd) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xFFFFFFFFu, mk, o));
    mv = fmaxf(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, o));
  }
  const float top = code_top<TYPE>();
  const float sk = grown_scale(was.x, mk, top), sv = grown_scale(was.y, mv, top);
  const float ik = sk > 0.f ? __frcp_rn(sk) : 0.f, iv = sv > 0.f ? __frcp_rn(sv) : 0.f;
  __syncwarp();  // every lane has read `was`
  if (lane == 0) *reinterpret_cast<float2*>(scale) = make_float2(sk, sv);
  // codes already in the page
  if (off > 0 && sk > was.x && was.x > 0.f) {
    const float ratio = was.x * ik;
    for (int p = lane; p < off * C; p += 32) {
      uint4* at = reinterpret_cast<uint4*>(tile + k_byte(p / C, (p % C) * 16, D));
      *at = round_again<TYPE>(*at, ratio);
    }
  }
  if (off > 0 && sv > was.y && was.y > 0.f) {
    const float ratio = was.y * iv;
    const int groups = (off + 15) / 16;
    for (int p = lane; p < D * groups; p += 32) {
      uint4* at = reinterpret_cast<uint4*>(tile + kPage * D + v_byte(16 * (p % groups), p / groups));
      *at = round_again<TYPE>(*at, ratio);   // bytes of tokens past `off` are written below, or not in use
    }
  }
  __syncwarp();
  for (int i = 0; i < n; ++i) {
    if (n > 1) load(i);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        tile[k_byte(off + i, k_at(e, j), D)] = (unsigned char)encode<TYPE>(k[e][j] * ik);
        tile[kPage * D + v_byte(off + i, 16 * c + 8 * e + sub + j)] = (unsigned char)encode<TYPE>(v[e][j] * iv);
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

// A block takes 32 entries of the slot list and one head. K goes straight from its
// 8-byte pieces to the output. V is stored transposed, so entries that follow one
// another in one page (the usual case) take the 16-token groups they touch through
// shared memory, two such stretches at a time; pieces of eight values are then
// gathered from eight rows there, whose word columns are swapped by d / 8 so that
// the lanes of a warp meet different banks.
constexpr int kReadEntries = 32, kReadThreads = 256;

template <int D, int TYPE>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const __grid_constant__ ReadArgs a) {
  __shared__ __align__(16) uint32_t vt[2][D][kPage / 4];
  constexpr int P = D / 8, PER = kReadEntries * P / kReadThreads;   // pieces of eight per entry, per thread
  const int tid = threadIdx.x, lane = tid & 31, head = blockIdx.y;
  const int64_t e0 = (int64_t)blockIdx.x * kReadEntries;
  const int n = (int)min((int64_t)kReadEntries, a.n - e0);
  follow_previous();
  // every warp finds the stretches: entries of one page that follow one another
  const int mine = lane < n ? a.slots[e0 + lane] : -1;
  const int page = mine < 0 ? -1 : mine / kPage;
  if (page >= a.n_pages && tid < 32) atomicCAS(a.err, 0, (int)QMV_ERR_CORRUPT);
  const bool there = page >= 0 && page < a.n_pages;
  float2 sc = make_float2(0.f, 0.f);
  if (there) sc = reinterpret_cast<const float2*>(a.cache + a.scale_off)[(int64_t)page * a.H + head];
  const int before = __shfl_up_sync(0xFFFFFFFFu, page, 1);   // by all lanes: not inside the condition
  const unsigned heads = __ballot_sync(0xFFFFFFFFu, lane == 0 || page != before);
  const int stretch = __popc(heads & (0xFFFFFFFFu >> (31 - lane))) - 1, stretches = __popc(heads);

  for (int s0 = 0; s0 < stretches; s0 += 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned in = __ballot_sync(0xFFFFFFFFu, stretch == s0 + j && there);
      if (in == 0) continue;
      const int tok = mine % kPage;
      const int g0 = __reduce_min_sync(0xFFFFFFFFu, (in >> lane) & 1 ? tok : kPage) / 16;
      const int groups = __reduce_max_sync(0xFFFFFFFFu, (in >> lane) & 1 ? tok : -1) / 16 + 1 - g0;
      const int pg = __shfl_sync(0xFFFFFFFFu, page, __ffs(in) - 1);
      const unsigned char* tile = a.cache + ((int64_t)pg * a.H + head) * (2 * kPage * D) + kPage * D;
      for (int p = tid; p < D * groups; p += kReadThreads) {
        const int d = p / groups, g = g0 + p % groups, swap = (d / 8) & 15;
        const uint4 w = *reinterpret_cast<const uint4*>(tile + v_byte(16 * g, d));
        vt[j][d][(4 * g) ^ swap] = w.x;
        vt[j][d][(4 * g + 1) ^ swap] = w.y;
        vt[j][d][(4 * g + 2) ^ swap] = w.z;
        vt[j][d][(4 * g + 3) ^ swap] = w.w;
      }
    }
    if (s0 == 0) {   // K, while the first groups of V arrive
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int p = tid + u * kReadThreads, e = p / P, d0 = (p % P) * 8;
        const int slot = __shfl_sync(0xFFFFFFFFu, mine, e);
        const bool ok = __shfl_sync(0xFFFFFFFFu, (int)there, e) != 0;
        const float s = __shfl_sync(0xFFFFFFFFu, sc.x, e);
        if (e >= n) continue;
        uint2 w = make_uint2(0, 0);
        if (ok) w = *reinterpret_cast<const uint2*>(a.cache + ((int64_t)(slot / kPage) * a.H + head) * (2 * kPage * D) + k_byte(slot % kPage, d0, D));
        float k[8];
        decode8<TYPE>(w, k);
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = ok ? k[i] * s : 0.f;
        store8_as(a.out_type, a.k_out, (e0 + e) * a.ldo + (int64_t)head * D + d0, k);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int p = tid + u * kReadThreads, e = p / P, d0 = (p % P) * 8;
      const int slot = __shfl_sync(0xFFFFFFFFu, mine, e), j = __shfl_sync(0xFFFFFFFFu, stretch, e) - s0;
      const bool ok = __shfl_sync(0xFFFFFFFFu, (int)there, e) != 0;
      const float s = __shfl_sync(0xFFFFFFFFu, sc.y, e);
      if (e >= n || j < 0 || j > 1) continue;
      const int tok = ok ? slot % kPage : 0;   // a slot that is not there has no place in the tile (and gives zeros)
      uint32_t x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = vt[j][d0 + i][(tok >> 2) ^ ((d0 / 8) & 15)];
      const uint32_t two = (tok & 3) | ((4 + (tok & 3)) << 4);   // the token's byte of two words
      const uint2 w = make_uint2(__byte_perm(__byte_perm(x[0], x[1], two), __byte_perm(x[2], x[3], two), 0x5410),
                                 __byte_perm(__byte_perm(x[4], x[5], two), __byte_perm(x[6], x[7], two), 0x5410));
      float v[8];
      decode8<TYPE>(w, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = ok ? v[i] * s : 0.f;
      store8_as(a.out_type, a.v_out, (e0 + e) * a.ldo + (int64_t)head * D + d0, v);
    }
    __syncthreads();
  }
}

template <typename TI, int D, int TYPE>
const void* append_variant(bool few) {
  return few ? (const void*)kv8_append_few_kernel<TI, D, TYPE> : (const void*)kv8_append_kernel<TI, D, TYPE, 4 * D>;
}
template <typename TI>
const void* append_kernel(int D, int type, bool few) {
  const bool i8 = type == QMV_KV_INT8;
  if (D == 64) return i8 ? append_variant<TI, 64, QMV_KV_INT8>(few) : append_variant<TI, 64, QMV_KV_E4M3>(few);
  return i8 ? append_variant<TI, 128, QMV_KV_INT8>(few) : append_variant<TI, 128, QMV_KV_E4M3>(few);
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
  const int64_t per_head = (int64_t)g->n_runs * desc->n_kv_heads;   // runs times heads: numbered in 31 bits
  if (per_head > INT32_MAX / 2) return fail(QMV_ERR_UNSUPPORTED, "n_runs=%d of %d heads", g->n_runs, desc->n_kv_heads);
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
  const int D = desc->head_dim, sms = sm_count();
  // Fewer than eight tokens per entry of the run list go to the kernel of one warp per run and head. A plan's list ends in
  // empty entries (it has room for about two runs per request), so that its bound is 16 to 18 tokens per request. The choice is
  // one for the call: 63 decode tokens beside a prompt chunk of 1000 (40 and 8 heads of 128, fp32) take 67 us so, a warp to a
  // page, and 20 as two calls.
  const bool few = g->n_tokens < 8 * (int64_t)g->n_runs;
  // The heads of a block share the angles of its run's tokens: the fewest heads (a power of two, up to 8) with which all
  // blocks are resident at once. 8190 tokens of 40 and 8 heads of 128, rotation included: 50 us with 4 heads a block (the
  // rule's choice), 59, 55 and 60 with 1, 2 and 8; 512 tokens: 11.6 with 1, 13.7, 19 and 30 with 2, 4 and 8.
  const int64_t resident = (int64_t)sms * (1024 / (4 * D));
  a.head_group = 1;
  while (rope && a.head_group < 8 && per_head > a.head_group * resident) a.head_group *= 2;
  a.head_groups = (desc->n_kv_heads + a.head_group - 1) / a.head_group;
  int64_t blocks = few ? (per_head + kFewThreads / 32 - 1) / (kFewThreads / 32) : (int64_t)g->n_runs * a.head_groups;
  if (g->q && few) {
    a.q_heads = g->n_q_heads > 16 ? 16 : g->n_q_heads;
    blocks += (int64_t)g->n_tokens * ((g->n_q_heads + a.q_heads - 1) / a.q_heads);
    if (blocks > INT32_MAX) return fail(QMV_ERR_UNSUPPORTED, "n_tokens=%d of %d query heads", g->n_tokens, g->n_q_heads);
  }
  const void* f = g->x_type == QMV_F32 ? append_kernel<float>(D, (int)desc->type, few)
                  : g->x_type == QMV_BF16 ? append_kernel<__nv_bfloat16>(D, (int)desc->type, few)
                                          : append_kernel<__half>(D, (int)desc->type, few);
  const int threads = few ? kFewThreads : 4 * D;
  const size_t smem = rope && !few ? (size_t)kPage * D / 2 * sizeof(float2) : 0;
  int per_sm = 0;
  rc = kernel_fit(f, threads, smem, &per_sm);
  if (rc) return rc;
  if (g->q && !few) {
    // long runs: the query heads are rotated by a launch of their own (measured on 8190 tokens of 40 and 8 heads: 50
    // us, and 65 us as blocks of one launch, where the cache write's registers halve the rotation's loads in flight)
    rc = rope_launch(rope, g->q, g->x_type, g->n_tokens, g->n_q_heads, g->ldq, g->positions, g->ldp, g->q_out, g->q_out_type,
                     g->ldqo, 0, static_cast<cudaStream_t>(stream));
    if (rc) return rc;
  }
  if (blocks == 0) return QMV_OK;
  void* args[] = {&a};
  cudaError_t e = launch_early(f, dim3((unsigned)blocks), threads, args, smem, static_cast<cudaStream_t>(stream));
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
  const dim3 grid((unsigned)((n + kReadEntries - 1) / kReadEntries), (unsigned)desc->n_kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool i8 = desc->type == QMV_KV_INT8;
  const void* f = desc->head_dim == 64 ? (i8 ? (const void*)kv8_read_kernel<64, QMV_KV_INT8> : (const void*)kv8_read_kernel<64, QMV_KV_E4M3>)
                                       : (i8 ? (const void*)kv8_read_kernel<128, QMV_KV_INT8> : (const void*)kv8_read_kernel<128, QMV_KV_E4M3>);
  void* args[] = {&a};
  cudaError_t e = launch_early(f, grid, kReadThreads, args, 0, s);
  if (e != cudaSuccess) return cuda_fail(e, "kv8_read launch");
  return QMV_OK;
}

}  // extern "C"

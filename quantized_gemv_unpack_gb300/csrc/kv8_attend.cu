// kv8_attend: checks of arguments, workspace and choice of the kernel.
#include <cmath>
#include <cstring>

#include "kv8_prompt.cuh"

using namespace qmv;
using namespace qmv::kv8;

namespace {

constexpr size_t kCounterBytes = 16384;  // one int per block, or two and two per item of a wave (prompts)

struct Layout {
  int blocks;
  size_t ml_off, o_off, total;
};
Layout layout(const qmv_kv_desc* d) {
  Layout l;
  l.blocks = sm_count();
  if (l.blocks > 1024) l.blocks = 1024;
  const size_t rows = (size_t)l.blocks * attend::kPartRows;
  l.ml_off = kCounterBytes;
  l.o_off = l.ml_off + rows * sizeof(float2);
  l.total = l.o_off + rows * d->head_dim * sizeof(float);
  return l;
}

int check_workspace(const qmv_kv_desc* desc, const void* workspace, size_t ws_bytes, const Layout& l) {
  (void)desc;
  if (!workspace) return fail(QMV_ERR_ARG, "NULL workspace");
  if (!aligned16(workspace)) return fail(QMV_ERR_ALIGN, "workspace must be 16-byte aligned");
  if (ws_bytes < l.total) return fail(QMV_ERR_ARG, "workspace %zu < %zu bytes", ws_bytes, l.total);
  return QMV_OK;
}

// The kernel of a call, by the query rows per (request, KV head) that max_new bounds. Measured when the rule was set (times in us, warp-level
// tensor cores / tcgen05; both have gained 5 to 20 % since): 30 rows of 40 query and 8 KV heads of 128, 1 request of 16384 tokens 38 / 46, 4 of them 48 / 72,
// 16 of 2048 31 / 34; 48 rows of one KV head, 34 / 35 over 4 requests of 4096 tokens, 66 / 49 over 4 of 16384, 30 / 26 over
// 4 of 1200; with 65 and 130 rows of 8 heads the first takes 1.5 to 4 times as long. Few rows are bound by the cache's
// bytes and by joins, which the first has more streams for; many rows by the products. The choice is one for the call: 63
// requests of one token over 4096 beside a chunk of 1000 tokens (40 and 8 heads of 128) take 301 us so, and 155 as two calls; over
// 16384 tokens 954 and 387.
enum Kernel { kWarps, kPrompt, kPromptParts };
Kernel choose(int64_t rows, int64_t all_rows, int requests, int H) {
  if (rows <= 32 || (all_rows / 256 + 1) * requests * H > INT32_MAX / 2) return kWarps;  // items are numbered in 31 bits
  // items of 256 rows for half the blocks or fewer: their keys are cut into parts
  return (rows + 255) / 256 * requests * H > sm_count() / 2 ? kPrompt : kPromptParts;
}

}  // namespace

extern "C" {

size_t kv8_attend_workspace_size(const qmv_kv_desc* desc) {
  if (check_kv_desc(desc)) return 0;
  return layout(desc).total;
}

int kv8_attend_init(const qmv_kv_desc* desc, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_kv_desc(desc);
  if (rc) return rc;
  rc = check_workspace(desc, workspace, ws_bytes, layout(desc));
  if (rc) return rc;
  cudaError_t e = cudaMemsetAsync(workspace, 0, kCounterBytes, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  return QMV_OK;
}

int kv8_attend(const qmv_kv_desc* desc, const void* cache, const kv8_attend_args* g, void* stream) {
  int rc = check_kv_desc(desc);
  if (rc) return rc;
  if (!g) return fail(QMV_ERR_ARG, "args is NULL");
  const int xs = dtype_size(g->x_type), os = dtype_size(g->out_type);
  if (!xs || !os) return fail(QMV_ERR_ARG, "x_type=%d out_type=%d", g->x_type, g->out_type);
  const int H = desc->n_kv_heads, D = desc->head_dim;
  if (g->n_q_heads < 1 || g->n_q_heads % H || g->n_q_heads > 65536)
    return fail(QMV_ERR_ARG, "n_q_heads=%d must be a multiple of the cache's %d heads", g->n_q_heads, H);
  if (g->n_requests < 1 || g->n_requests > QMV_KV_MAX_REQUESTS)
    return fail(QMV_ERR_ARG, "n_requests=%d outside 1..%d", g->n_requests, QMV_KV_MAX_REQUESTS);
  if (g->n_tokens < 0 || g->max_new < 1) return fail(QMV_ERR_ARG, "n_tokens=%d max_new=%d", g->n_tokens, g->max_new);
  if ((int64_t)g->n_tokens * (g->n_q_heads / H) > INT32_MAX / 2) return fail(QMV_ERR_UNSUPPORTED, "too many query rows");
  if (g->max_pages < 1 || g->ld_table < g->max_pages || g->max_pages > INT32_MAX / kPage - 1)
    return fail(QMV_ERR_ARG, "max_pages=%d ld_table=%lld", g->max_pages, (long long)g->ld_table);
  if (g->window < 0) return fail(QMV_ERR_ARG, "window=%d", g->window);
  if (!(g->scale > 0.f) || !std::isfinite(g->scale)) return fail(QMV_ERR_ARG, "scale must be positive and finite");
  if (!(g->softcap >= 0.f) || !std::isfinite(g->softcap)) return fail(QMV_ERR_ARG, "softcap must be 0 (none) or positive and finite");
  const int64_t row = (int64_t)g->n_q_heads * D;
  if (g->ldq < row || g->ldo < row) return fail(QMV_ERR_ARG, "ldq=%lld ldo=%lld below %lld", (long long)g->ldq, (long long)g->ldo, (long long)row);
  if (g->ldq * xs % 16 || g->ldo * os % 16) return fail(QMV_ERR_ALIGN, "rows of q and out must be 16-byte aligned");
  if (!cache || !g->q || !g->out || !g->q_start || !g->ctx || !g->table) return fail(QMV_ERR_ARG, "NULL cache, q, out, q_start, ctx or table");
  if (!aligned16(cache) || !aligned16(g->q) || !aligned16(g->out)) return fail(QMV_ERR_ALIGN, "cache, q and out must be 16-byte aligned");
  const void* words[] = {g->q_start, g->ctx, g->table, g->slopes, g->prefix, g->lse};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(QMV_ERR_ALIGN, "index arrays, slopes and lse must be 4-byte aligned");
  const Layout l = layout(desc);
  rc = check_workspace(desc, g->workspace, g->ws_bytes, l);
  if (rc) return rc;
  if (g->n_tokens == 0) return QMV_OK;
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");

  attend::Args a;
  memset(&a, 0, sizeof(a));
  a.cache = static_cast<const unsigned char*>(cache);
  a.scale_off = desc->off[1];
  a.n_pages = desc->n_pages;
  a.q = g->q;
  a.out = g->out;
  a.lse = g->lse;
  a.ldq = g->ldq;
  a.ldo = g->ldo;
  a.ld_table = g->ld_table;
  a.x_type = g->x_type;
  a.out_type = g->out_type;
  a.B = g->n_requests;
  a.T = g->n_tokens;
  a.Hq = g->n_q_heads;
  a.H = H;
  a.G = g->n_q_heads / H;
  int log_g = 0;
  while ((1 << log_g) < a.G) ++log_g;
  a.g_shift = 31 + log_g;
  a.g_mul = (uint32_t)(((1ull << a.g_shift) + a.G - 1) / a.G);   // 2^31 for G = 1
  a.q_start = g->q_start;
  a.ctx = g->ctx;
  a.table = g->table;
  a.prefix = g->prefix;
  a.slopes = g->slopes;
  a.max_pages = g->max_pages;
  a.window = g->window;
  a.scale = g->scale;
  a.softcap = g->softcap;
  unsigned char* ws = static_cast<unsigned char*>(g->workspace);
  a.counters = reinterpret_cast<int*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml_off);
  a.part_o = reinterpret_cast<float*>(ws + l.o_off);
  a.err = err;
  const int64_t rows = (int64_t)(g->max_new < g->n_tokens ? g->max_new : g->n_tokens) * a.G;
  const int tile = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  const bool mods = g->softcap > 0.f || g->slopes;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool i8 = desc->type == QMV_KV_INT8;
  const Kernel kernel = choose(rows, (int64_t)g->n_tokens * a.G, g->n_requests, H);
  if (kernel != kWarps) {
    const bool split = kernel == kPromptParts;
    if (D == 64) return i8 ? prompt::launch_64_int8(a, mods, split, l.blocks, s) : prompt::launch_64_e4m3(a, mods, split, l.blocks, s);
    return i8 ? prompt::launch_128_int8(a, mods, split, l.blocks, s) : prompt::launch_128_e4m3(a, mods, split, l.blocks, s);
  }
  if (D == 64) return i8 ? attend::launch_64_int8(a, tile, mods, l.blocks, s) : attend::launch_64_e4m3(a, tile, mods, l.blocks, s);
  return i8 ? attend::launch_128_int8(a, tile, mods, l.blocks, s) : attend::launch_128_e4m3(a, tile, mods, l.blocks, s);
}

}  // extern "C"

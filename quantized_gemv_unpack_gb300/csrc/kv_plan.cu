// Block tables, slot maps and run lists of one serving step, built on the GPU
// from the requests' lengths (kv_plan).
//
// Per request the step needs three exclusive sums: of new tokens (q_start), of
// new pages (place in the ring of free pages) and of runs or returned pages. A
// block takes them over all requests with warp scans: 1 to 8 requests per
// thread, a few hundred cycles. Then every token finds its request by binary
// search in the sums (shared memory) and writes its slot, its position, its
// table entry if it opens a page and its run if it heads one. Nothing here is
// worth bandwidth: a step of 64 requests moves 6 KB, and the time is that of the
// launch and of three dependent loads (lengths; ring state; table or ring).
//
// Many tokens (admission of prompts) are spread over a cluster of 8 blocks. Each
// block takes the sums for itself, which costs less than handing them round, and
// the cluster's barrier separates the last read of lens, the ring's state and
// the table's returned rows from the first write, so that outputs may alias
// inputs.
#include "kv8.cuh"

namespace qmv {
namespace {

constexpr int kMaxPlanThreads = 1024;
constexpr int kPlanCluster = 8;

struct Scratch {   // per request, in dynamic shared memory
  int32_t* start;  // first token (at most T)
  int32_t* len;    // tokens in the cache before the step
  int32_t* page;   // place of its first new page among the step's new pages
  int32_t* run;    // place of its first run, or of its first returned page
  int32_t* status;
};

// Exclusive sum over the block's threads of one value per thread; *total gets the sum.
__device__ long long block_scan(long long v, long long* total, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[warps - 1];
  return (warp ? warp_sums[warp - 1] : 0) + s - v;
}

__global__ void __launch_bounds__(kMaxPlanThreads) kv_plan_kernel(const __grid_constant__ kv_plan_args a, int n_blocks,
                                                                  int* err) {
  extern __shared__ int32_t plan_smem[];
  __shared__ long long warp_sums[32];
  const int B = a.n_requests, T = a.n_tokens, N = a.n_pages;
  const Scratch s{plan_smem, plan_smem + B, plan_smem + 2 * B, plan_smem + 3 * B, plan_smem + 4 * B};
  const int tid = threadIdx.x, nt = blockDim.x;
  const int block = blockIdx.x;
  const int per = (B + nt - 1) / nt;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);

  int head = a.ring_state[0], count = a.ring_state[1];
  if (head < 0 || head >= N || count < 0 || count > N) {
    if (block == 0 && tid == 0) atomicCAS(err, 0, (int)QMV_ERR_CORRUPT);
    head = 0;
    count = 0;
  }

  // tokens
  long long sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += max(a.add[b], 0);
  long long at = block_scan(sum, &total, warp_sums);
  const int n_tokens = (int)min((long long)T, total);
  long long need_sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.lens[b], add = a.add[b];
    const long long tok = max(add, 0);
    const long long held = ((long long)len + 63) >> 6, after = ((long long)len + tok + 63) >> 6;
    const bool bad = len < 0 || held > a.max_pages || after > a.max_pages || at + tok > T;
    s.start[b] = (int)min(at, (long long)T);
    s.len[b] = len;
    s.status[b] = bad ? 2 : (add < 0 ? 3 : 0);
    if (!bad && add > 0) need_sum += after - held;
    at += tok;
  }
  // new pages: a request is short of pages where the needs up to its own exceed what is free
  long long need_at = block_scan(need_sum, &total, warp_sums);
  long long run_sum = 0, back_sum = 0, taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = s.len[b], add = max(a.add[b], 0);
    const int held = (int)(((long long)len + 63) >> 6);
    if (s.status[b] == 3) back_sum += held;
    if (s.status[b] != 0) continue;
    const int need = (int)(((long long)len + add + 63) >> 6) - held;
    s.page[b] = (int)min(need_at, (long long)INT32_MAX);
    need_at += need;
    if (need > 0 && need_at > count) {
      s.status[b] = 1;
      continue;
    }
    taken += need;
    if (add > 0) run_sum += ((len + add - 1) >> 6) - (len >> 6) + 1;
  }
  // runs (low half, at most T in all) and pages taken (high half, at most count) in one scan
  const long long both = block_scan(run_sum | (taken << 32), &total, warp_sums);
  const int n_runs = (int)(total & 0x7FFFFFFFll), popped = (int)(total >> 32);
  long long n_back;
  long long back_at = block_scan(back_sum, &n_back, warp_sums), run_at = both & 0x7FFFFFFFll;
  for (int b = b0; b < b1; ++b) {
    if (s.status[b] == 3) {
      s.run[b] = (int)min(back_at, (long long)N);
      back_at += (s.len[b] + 63) >> 6;
    } else if (s.status[b] == 0) {
      s.run[b] = (int)run_at;
      const int len = s.len[b], add = max(a.add[b], 0);
      if (add > 0) run_at += ((len + add - 1) >> 6) - (len >> 6) + 1;
    }
  }
  const int room = N - count;  // returned pages go behind the `count` free ones
  __syncthreads();
  if (n_blocks > 1) {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }

  const int gtid = block * nt + tid, gnt = n_blocks * nt;
  for (int b = gtid; b <= B; b += gnt) {
    if (b == B) {
      a.q_start[B] = n_tokens;
      break;
    }
    const int st = s.status[b], len = s.len[b];
    const int start = s.start[b], end = b + 1 < B ? s.start[b + 1] : n_tokens;
    a.q_start[b] = start;
    a.status[b] = st;
    const int after = len + (end - start);
    a.lens_out[b] = st == 0 ? after : (st == 3 ? 0 : len);
    a.ctx[b] = st == 0 ? after : 0;
  }
  if (gtid == 0) {
    const int kept = (int)min(n_back, (long long)room);
    int h = head + popped;
    a.ring_state_out[0] = h >= N ? h - N : h;
    a.ring_state_out[1] = count - popped + kept;
    if (n_back > room) atomicCAS(err, 0, (int)QMV_ERR_CORRUPT);
  }
  for (int t = gtid; t < T; t += gnt) {
    int slot = -1, pos = -1;
    if (t < n_tokens) {
      int lo = 0, hi = B;  // the last request that starts at or before t: the one that has it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.start[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int b = lo;
      if (s.status[b] == 0) {
        const int len = s.len[b], i = t - s.start[b];
        const int end = b + 1 < B ? s.start[b + 1] : n_tokens;
        pos = len + i;
        const int held = (len + 63) >> 6, index = pos >> 6;
        int page;
        if (index < held) {
          page = a.table[(int64_t)b * a.ld_table + index];
        } else {
          int k = head + s.page[b] + index - held;
          if (k >= N) k -= N;
          page = a.ring[k];
          if ((pos & 63) == 0) a.table[(int64_t)b * a.ld_table + index] = page;
        }
        slot = page * 64 + (pos & 63);
        if ((pos & 63) == 0 || i == 0) {
          const int r = s.run[b] + index - (len >> 6);
          if (r < a.max_runs)
            reinterpret_cast<int2*>(a.runs)[r] = make_int2(t, min(64 - (pos & 63), end - t));
        }
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  for (int r = n_runs + gtid; r < a.max_runs; r += gnt) reinterpret_cast<int2*>(a.runs)[r] = make_int2(0, 0);
  // returned pages: one warp per leaving request
  const int lane = tid & 31;
  for (int b = gtid >> 5; b < B; b += gnt >> 5) {
    if (s.status[b] != 3) continue;
    const int held = (s.len[b] + 63) >> 6;
    for (int i = lane; i < held; i += 32) {
      const long long k = (long long)s.run[b] + i;
      if (k >= room) break;
      long long at_ring = (long long)head + count + k;
      if (at_ring >= N) at_ring -= N;
      a.ring[at_ring] = a.table[(int64_t)b * a.ld_table + i];
    }
  }
}

}  // namespace
}  // namespace qmv

using namespace qmv;

extern "C" {

int64_t kv_max_runs(int64_t n_requests, int64_t n_tokens) {
  if (n_requests <= 0 || n_tokens <= 0) return 0;
  const int64_t with = n_requests < n_tokens ? n_requests : n_tokens;
  const int64_t most = n_tokens / 64 + 2 * with;
  return most < n_tokens ? most : n_tokens;
}

int kv_plan(const kv_plan_args* a, void* stream) {
  if (!a) return fail(QMV_ERR_ARG, "args is NULL");
  if (a->n_requests < 1 || a->n_requests > QMV_KV_MAX_REQUESTS)
    return fail(QMV_ERR_ARG, "n_requests=%d outside 1..%d", a->n_requests, QMV_KV_MAX_REQUESTS);
  if (a->n_tokens < 0 || a->n_pages < 1 || a->max_pages < 1 || a->ld_table < a->max_pages)
    return fail(QMV_ERR_ARG, "n_tokens=%d n_pages=%d max_pages=%d ld_table=%lld", a->n_tokens, a->n_pages, a->max_pages,
                (long long)a->ld_table);
  if (a->n_pages > INT32_MAX / 64) return fail(QMV_ERR_UNSUPPORTED, "n_pages=%d: slots must fit 31 bits", a->n_pages);
  if (a->max_pages > INT32_MAX / 64) return fail(QMV_ERR_UNSUPPORTED, "max_pages=%d: positions must fit 31 bits", a->max_pages);
  if (a->max_runs < kv_max_runs(a->n_requests, a->n_tokens))
    return fail(QMV_ERR_ARG, "max_runs=%d below kv_max_runs=%lld", a->max_runs,
                (long long)kv_max_runs(a->n_requests, a->n_tokens));
  const void* need[] = {a->lens, a->add, a->table, a->ring, a->ring_state, a->ring_state_out, a->lens_out, a->ctx,
                        a->status, a->q_start};
  for (const void* p : need) {
    if (!p) return fail(QMV_ERR_ARG, "NULL pointer");
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(QMV_ERR_ALIGN, "int32 arrays must be 4-byte aligned");
  }
  if (a->n_tokens > 0) {
    if (!a->slots || !a->positions || !a->runs) return fail(QMV_ERR_ARG, "NULL slots, positions or runs");
    if ((reinterpret_cast<uintptr_t>(a->slots) | reinterpret_cast<uintptr_t>(a->positions)) & 3u)
      return fail(QMV_ERR_ALIGN, "int32 arrays must be 4-byte aligned");
  }
  if (a->max_runs > 0 && (reinterpret_cast<uintptr_t>(a->runs) & 7u)) return fail(QMV_ERR_ALIGN, "runs must be 8-byte aligned");
  int* err = device_error_word();
  if (!err) return fail(QMV_ERR_CUDA, "cannot locate the device error word");

  const int B = a->n_requests, T = a->n_tokens;
  const int most = B > T ? B : T;
  // one block while its threads see at most 4 tokens each: more blocks only add the cluster barrier
  const int n_blocks = most > 4 * kMaxPlanThreads ? kPlanCluster : 1;
  const int threads = most <= 256 ? 256 : kMaxPlanThreads;
  const size_t smem = (size_t)B * 5 * sizeof(int32_t);
  int per_sm = 0;
  int rc = kernel_fit(reinterpret_cast<const void*>(kv_plan_kernel), threads, smem, &per_sm);
  if (rc) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n_blocks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_plan_kernel, *a, n_blocks, err);
  if (e != cudaSuccess) return cuda_fail(e, "kv_plan launch");
  return QMV_OK;
}

}  // extern "C"

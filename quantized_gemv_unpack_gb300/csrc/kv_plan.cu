// Block tables, slot maps and run lists of one serving step, built on the GPU
// from the requests' lengths (kv_plan).
//
// Per request the step needs exclusive sums of new tokens (q_start), of new pages
// (place in the ring of free pages), of runs and of returned pages. A block takes
// them over all requests with three scans: 1 to 8 requests per thread. Then every
// thread finds the request of its four tokens by binary search in the sums
// (shared memory) and writes their slots and positions, the table's entry of a
// page that one of them opens and the run that one of them heads. Nothing here is
// worth bandwidth: a step of 64 requests moves 6 KB, and the time (4.9 us; 9.9 for
// 512 requests with 65536 tokens) is that of the launch, of the scans and of three
// dependent loads (lengths; ring state; table or ring).
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
constexpr int kPlanCluster = 8;   // blocks: the largest cluster that every device of this kind schedules

struct Scratch {   // per request, in dynamic shared memory
  int32_t* start;  // first token (at most T)
  int32_t* len;    // tokens in the cache before the step
  int32_t* held;   // pages in its row before the step
  int32_t* page;   // place of its first new page among the step's new pages
  int32_t* run;    // place of its first run, or of its first returned page
  int32_t* status;
};
constexpr int kScratchWords = sizeof(Scratch) / sizeof(int32_t*);

// Sums stop at kMost: past any count of tokens or pages that a call can serve (2^30 tokens at most), so that a sum that has
// stopped is over every limit. Two of them come to 2^31 + 2, which does not fit an int: they are added without sign.
constexpr int kMost = (1 << 30) + 1;
__device__ __forceinline__ int add_most(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)kMost); }

// Exclusive sums over the block's threads of K values per thread, with the totals. Every warp sums the warps' sums for
// itself, so a scan has one barrier; `sums` is not used again by the next one.
template <int K>
__device__ __forceinline__ void block_scan(int (&v)[K], int (&total)[K], int (*sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int s[K], w[K];
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = v[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, s[k], o);
      if (lane >= o) s[k] = add_most(s[k], u);
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < K; ++k) sums[k][warp] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = lane < warps ? sums[k][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, w[k], o);
      if (lane >= o) w[k] = add_most(w[k], u);
    }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    total[k] = __shfl_sync(0xFFFFFFFFu, w[k], 31);
    const int before_warp = __shfl_sync(0xFFFFFFFFu, w[k], (warp + 31) & 31);
    int before_lane = __shfl_up_sync(0xFFFFFFFFu, s[k], 1);   // a stopped sum cannot be undone by subtraction
    if (lane == 0) before_lane = 0;
    v[k] = add_most(warp ? before_warp : 0, before_lane);
  }
}

__global__ void __launch_bounds__(kMaxPlanThreads) kv_plan_kernel(const __grid_constant__ kv_plan_args a, int n_blocks,
                                                                  int* err) {
  extern __shared__ int32_t plan_smem[];
  __shared__ int warp_sums[5][32];
  const int B = a.n_requests, T = a.n_tokens, N = a.n_pages;
  const Scratch s{plan_smem, plan_smem + B, plan_smem + 2 * B, plan_smem + 3 * B, plan_smem + 4 * B, plan_smem + 5 * B};
  const int tid = threadIdx.x, nt = blockDim.x;
  const int block = blockIdx.x;
  const int per = (B + nt - 1) / nt;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);

  kv8::let_next_begin();
  kv8::follow_previous();
  int head = a.ring_state[0], count = a.ring_state[1];
  if (head < 0 || head >= N || count < 0 || count > N) {
    if (block == 0 && tid == 0) atomicCAS(err, 0, (int)QMV_ERR_CORRUPT);
    head = 0;
    count = 0;
  }

  // tokens
  int sum[1] = {0}, total[1];
  for (int b = b0; b < b1; ++b) sum[0] = add_most(sum[0], min(max(a.add[b], 0), kMost));
  block_scan<1>(sum, total, warp_sums);
  const int n_tokens = min(T, total[0]);
  int at = sum[0], need[1] = {0};
  for (int b = b0; b < b1; ++b) {
    const int len = a.lens[b], add = a.add[b];
    const int tok = min(max(add, 0), kMost);
    const int full = (int)(((long long)len + 63) >> 6), held = a.held ? a.held[b] : full;
    const long long after = ((long long)len + tok + 63) >> 6;
    const bool bad = len < 0 || held < full || held > a.max_pages || after > a.max_pages || (unsigned)at + (unsigned)tok > (unsigned)T;
    s.start[b] = min(at, T);
    s.len[b] = len;
    s.held[b] = held;
    s.status[b] = bad ? 2 : (add < 0 ? 3 : 0);
    if (!bad && add > 0) need[0] = add_most(need[0], max((int)after - held, 0));
    at = add_most(at, tok);
  }
  // new pages: a request is short of pages where the needs up to its own exceed what is free
  block_scan<1>(need, total, warp_sums + 1);
  int need_at = need[0];
  int sums3[3] = {0, 0, 0}, total3[3];   // runs, returned pages, pages taken
  for (int b = b0; b < b1; ++b) {
    const int len = s.len[b];
    if (s.status[b] == 3) sums3[1] = add_most(sums3[1], s.held[b]);
    if (s.status[b] != 0) continue;
    const int add = max(a.add[b], 0);   // served so far: at most T
    const int want = max(((len + add + 63) >> 6) - s.held[b], 0);
    s.page[b] = need_at;
    need_at = add_most(need_at, want);
    if (want > 0 && need_at > count) {
      s.status[b] = 1;
      continue;
    }
    sums3[2] += want;   // at most count in all
    if (add > 0) sums3[0] += ((len + add - 1) >> 6) - (len >> 6) + 1;   // at most T in all
  }
  block_scan<3>(sums3, total3, warp_sums + 2);
  const int n_runs = total3[0], n_back = total3[1], popped = total3[2];
  int run_at = sums3[0], back_at = sums3[1];
  for (int b = b0; b < b1; ++b) {
    const int len = s.len[b];
    if (s.status[b] == 3) {
      s.run[b] = back_at;
      back_at = add_most(back_at, s.held[b]);
    } else if (s.status[b] == 0) {
      s.run[b] = run_at;
      const int add = max(a.add[b], 0);
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
    if (a.held) a.held_out[b] = st == 0 ? max(s.held[b], (after + 63) >> 6) : (st == 3 ? 0 : s.held[b]);
  }
  if (gtid == 0) {
    const int kept = min(n_back, room);
    int h = head + popped;
    a.ring_state_out[0] = h >= N ? h - N : h;
    a.ring_state_out[1] = count - popped + kept;
    if (n_back > room) atomicCAS(err, 0, (int)QMV_ERR_CORRUPT);
  }
  // tokens, one per thread or four neighbours: a search in shared memory, then from token to token. (Neighbours of a decode
  // step are tokens of different requests, whose loads would follow one another.)
  const int each = T > gnt ? 4 : 1;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  int search = 1;   // steps that halve B requests to one
  while ((1 << search) < B) ++search;
  for (int t0 = gtid * each; t0 < T; t0 += gnt * each) {
    // the last request that starts at or before the token: the one that has it
    int b = 0;
    for (int step = 1 << (search - 1); step; step >>= 1)
      if (b + step < B && s.start[b + step] <= t0) b += step;
    int start = s.start[b], end = b + 1 < B ? s.start[b + 1] : n_tokens, len = s.len[b], held = s.held[b], page_index = -1, page = 0;
    bool served = s.status[b] == 0;
    int slot[4], pos[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u;
      slot[u] = pos[u] = -1;
      if (u >= each || t >= n_tokens) continue;
      while (t >= end) {   // on to the next request with tokens
        ++b;
        start = end;
        end = b + 1 < B ? s.start[b + 1] : n_tokens;
        len = s.len[b];
        held = s.held[b];
        served = s.status[b] == 0;
        page_index = -1;
      }
      if (!served) continue;
      pos[u] = len + t - start;
      const int index = pos[u] >> 6;
      const bool opens = (pos[u] & 63) == 0;
      if (index != page_index) {
        page_index = index;
        if (index < held) {
          page = a.table[(int64_t)b * a.ld_table + index];
        } else {
          int k = head + s.page[b] + index - held;
          if (k >= N) k -= N;
          page = a.ring[k];
        }
      }
      slot[u] = page * 64 + (pos[u] & 63);
      if (opens && index >= held) a.table[(int64_t)b * a.ld_table + index] = page;
      if (opens || t == start) {
        const int r = s.run[b] + index - (len >> 6);
        if (r < a.max_runs) reinterpret_cast<int2*>(a.runs)[r] = make_int2(t, min(64 - (pos[u] & 63), end - t));
      }
    }
    if (wide && each == 4 && t0 + 3 < T) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (u < each && t0 + u < T) {
          a.slots[t0 + u] = slot[u];
          a.positions[t0 + u] = pos[u];
        }
    }
  }
  for (int r = n_runs + gtid; r < a.max_runs; r += gnt) reinterpret_cast<int2*>(a.runs)[r] = make_int2(0, 0);
  // returned pages: the warps share out groups of 32 requests, and within a group its leaving requests, whose rows they copy
  const int lane = tid & 31, warps = gnt >> 5, groups = (B + 31) >> 5;
  const int sharers = warps > groups ? warps / groups : 1;
  for (int w = gtid >> 5; w < groups * sharers; w += warps) {
    const int first = (w % groups) * 32;
    int turn = w / groups;   // leaving requests until this warp's next
    unsigned gone = __ballot_sync(0xFFFFFFFFu, first + lane < B && s.status[min(first + lane, B - 1)] == 3);
    for (; gone; gone &= gone - 1) {
      if (turn-- != 0) continue;
      turn = sharers - 1;
      const int b = first + __ffs(gone) - 1;
      const int held = s.held[b], place = s.run[b], n = min(held, room - place);
      const int32_t* row = a.table + (int64_t)b * a.ld_table;
#pragma unroll 4
      for (int i = lane; i < n; i += 32) {
        int k = head + count + place + i - N;   // below N: place + i < N - count
        if (k < 0) k += N;
        a.ring[k] = row[i];
      }
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
  if (a->n_tokens > (1 << 30)) return fail(QMV_ERR_UNSUPPORTED, "n_tokens=%d over 2^30", a->n_tokens);
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
  if ((a->held != nullptr) != (a->held_out != nullptr)) return fail(QMV_ERR_ARG, "held and held_out: both or neither");
  if ((reinterpret_cast<uintptr_t>(a->held) | reinterpret_cast<uintptr_t>(a->held_out)) & 3u)
    return fail(QMV_ERR_ALIGN, "int32 arrays must be 4-byte aligned");
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
  // one block while its threads see at most four requests or four tokens each: more blocks only add the cluster barrier
  const int n_blocks = most > 4 * kMaxPlanThreads ? kPlanCluster : 1;
  const int threads = most <= 256 ? 256 : kMaxPlanThreads;
  const size_t smem = (size_t)B * kScratchWords * sizeof(int32_t);
  int per_sm = 0;
  // asked for the most requests: the library keeps an answer per size asked for, and B differs from step to step
  int rc = kernel_fit(reinterpret_cast<const void*>(kv_plan_kernel), threads, (size_t)QMV_KV_MAX_REQUESTS * kScratchWords * sizeof(int32_t), &per_sm);
  if (rc) return rc;
  kv_plan_args copy = *a;
  int blocks = n_blocks;
  void* args[] = {&copy, &blocks, &err};
  cudaError_t e = kv8::launch_early(reinterpret_cast<const void*>(kv_plan_kernel), dim3(n_blocks), threads, args, smem,
                                    static_cast<cudaStream_t>(stream), n_blocks);
  if (e != cudaSuccess) return cuda_fail(e, "kv_plan launch");
  return QMV_OK;
}

}  // extern "C"

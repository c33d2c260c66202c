// Upkeep of the paged cache on the device: pages are given to sequences, shared
// with branches, taken back and moved together, in stream order and without the
// host.
//
// The integers (which page goes where) are the work of one CTA, since each answer
// hangs on those before it: free pages are found in order by counting them per
// warp over equal segments of page_refs, a scan over the 32 counts, and a second
// pass that lists them; the calls' entries get theirs by a scan of what they need.
// Bound by latency: a few dependent reads of L2 and barriers (the 4-byte counts of
// 65,536 pages are 256 KB).  The bytes that a fork or a compaction moves are
// copied by a second kernel over the whole device, 16 bytes a thread and eight of
// them in flight, launched to be resident when the list is ready.
// Sources and targets of the copies of one call are disjoint by construction
// (targets are free pages), so their order does not matter.
// Measured, 6 layers, 2 KV heads of 256, pages of 64: 64 sequences of 2048, a quarter of
// them freed, the pool compacted and as many grown again: 86 us, 73% of a copy's rate for
// the pages that move; keeping the pages in flight with bulk copies through shared memory
// instead took as long.  Four sequences freed and forked into 8 each: 18 us on the device.
#include "kv8.cuh"
#include "../pdl.cuh"

namespace cmr {
namespace kv8 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kFreeThreads = 128;

// Words of the workspace: a head of 16, then lists.
enum Head { kJobs = 0, kLive = 1 };
constexpr int kHead = 16;

__device__ __forceinline__ void flag(const PagesArgs& a, int bit) {
  if (a.status != nullptr) atomicOr(a.status, bit);
}

// Exclusive sum over the CTA's threads, and the total.
__device__ int64_t block_scan(int v, int64_t* total) {
  __shared__ int64_t s_warp[kPlanWarps + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int64_t w = s_warp[lane];
    int64_t z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, z, o);
      if (lane >= o) z += y;
    }
    s_warp[lane] = z - w;
    if (lane == 31) s_warp[kPlanWarps] = z;
  }
  __syncthreads();
  *total = s_warp[kPlanWarps];
  return s_warp[warp] + x - v;
}

// This warp's share [s0, s1) of pages [lo, hi): equal segments of whole lines.
__device__ __forceinline__ void warp_segment(int lo, int hi, int& s0, int& s1) {
  const int64_t span = (static_cast<int64_t>(hi) - lo + kPlanWarps - 1) / kPlanWarps;
  const int64_t seg = (span + 31) / 32 * 32, at = lo + (threadIdx.x / 32) * seg;
  s0 = static_cast<int>(at < hi ? at : hi);
  s1 = static_cast<int>(at + seg < hi ? at + seg : hi);
}

// Lists in `out`, lowest first, the pages of [lo, hi) that are free (or in use),
// at most `limit` of them; returns how many there are in all.
__device__ int select_pages(const int32_t* refs, int lo, int hi, bool want_free, int limit,
                            int32_t* out) {
  const int lane = threadIdx.x & 31;
  int s0, s1;
  warp_segment(lo, hi, s0, s1);
  int count = 0;
#pragma unroll 8
  for (int i = s0 + lane; i < s1; i += 32) count += (__ldcg(refs + i) <= 0) == want_free;
  count = __reduce_add_sync(~0u, count);
  int64_t total;
  const int before = static_cast<int>(block_scan(lane == 0 ? count : 0, &total));
  int at = __shfl_sync(~0u, before, 0);  // lane 0 has the sum of the earlier warps
#pragma unroll 4
  for (int i0 = s0; i0 < s1 && at < limit; i0 += 32) {
    const int i = i0 + lane;
    const bool hit = i < s1 && (__ldcg(refs + i) <= 0) == want_free;
    const uint32_t hits = __ballot_sync(~0u, hit);
    const int k = at + __popc(hits & ((1u << lane) - 1));
    if (hit && k < limit) out[k] = i;
    at += __popc(hits);
  }
  __syncthreads();
  return static_cast<int>(total);
}

// Whether an entry before i names the same row (asked by a whole warp).
__device__ bool named_before(const int32_t* slots, int i, int32_t slot) {
  bool same = false;
  for (int j = threadIdx.x & 31; j < i; j += 32) same |= __ldg(slots + j) == slot;
  return __any_sync(~0u, same);
}

// Looks through a row, every `parts`-th run of kRowRun entries from run `part` on: the places
// of the first negative one and of the first page id outside the pool that it comes upon,
// or max_pages (asked by a whole warp).
constexpr int kRowAhead = 8;
constexpr int kRowRun = 32 * kRowAhead;
__device__ void look_through_row(const PagesArgs& a, int32_t slot, int part, int parts, int& end,
                                 int& odd) {
  const int lane = threadIdx.x & 31;
  const int32_t* row = a.table + static_cast<int64_t>(slot) * a.max_pages;
  end = odd = a.max_pages;
  for (int64_t k0 = static_cast<int64_t>(part) * kRowRun; k0 < a.max_pages && end == a.max_pages;
       k0 += static_cast<int64_t>(parts) * kRowRun) {
    int32_t id[kRowAhead];
#pragma unroll
    for (int j = 0; j < kRowAhead; ++j) {
      const int64_t k = k0 + 32 * j + lane;
      id[j] = k < a.max_pages ? __ldcg(row + k) : 0;
    }
#pragma unroll
    for (int j = 0; j < kRowAhead; ++j) {
      const int at = static_cast<int>(k0 + 32 * j + lane);
      if (id[j] < 0) end = min(end, at);
      if (id[j] >= a.pool.num_pages) odd = min(odd, at);
    }
    end = __reduce_min_sync(~0u, end);
  }
  odd = __reduce_min_sync(~0u, odd);
}

__device__ __forceinline__ int64_t pages_for(int32_t tokens, int32_t page_tokens) {
  return (static_cast<int64_t>(tokens) + page_tokens - 1) / page_tokens;
}

__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const PagesArgs a) {
  pdl::wait();
  pdl::launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int32_t* need = a.workspace + kHead;  // [n]
  int32_t* have = need + a.n;           // [n]
  int32_t* first = have + a.n;          // [n]: where its pages start in the list, or -1
  int32_t* list = first + a.n;          // free pages
  // A warp to an entry, or several where there are few: each looks through its part of the
  // row.  64 rows of 128 pages, of which each gets one more: 14 us; 8 of 4096: 23, 64: 107.
  __shared__ int s_end[kPlanWarps], s_odd[kPlanWarps];
  const int parts = a.n < kPlanWarps ? kPlanWarps / a.n : 1;
  const int first_i = warp / parts;
  if (parts > 1) {
    if (warp == 0) s_end[lane] = s_odd[lane] = a.max_pages;
    __syncthreads();
    const int32_t slot = first_i < a.n ? __ldg(a.dst + first_i) : -1;
    if (slot >= 0 && slot < a.rows) {
      int end, odd;
      look_through_row(a, slot, warp - first_i * parts, parts, end, odd);
      if (lane == 0) {
        atomicMin(&s_end[first_i], end);
        atomicMin(&s_odd[first_i], odd);
      }
    }
    __syncthreads();
  }
  for (int i = first_i; i < a.n && warp == first_i * parts; i += kPlanWarps) {
    const int32_t slot = __ldg(a.dst + i), len = __ldg(a.lens + i);
    const bool known = slot >= 0 && slot < a.rows && !named_before(a.dst, i, slot);
    int held = 0, odd = 0;
    if (known) {
      if (parts > 1) {
        held = s_end[i];
        odd = s_odd[i];
      } else {
        look_through_row(a, slot, 0, 1, held, odd);
      }
    }
    if (lane == 0) {
      int more = 0;
      if (!known || len < 0) {
        flag(a, CMR_DEVICE_CACHE_RANGE);
      } else {
        if (odd < held) flag(a, CMR_DEVICE_CACHE_RANGE);
        const int64_t want = pages_for(len, a.page_tokens);
        if (want > a.max_pages)
          flag(a, CMR_DEVICE_CACHE_RANGE);
        else
          more = max(0, static_cast<int>(want) - held);
      }
      need[i] = more;
      have[i] = held;
    }
  }
  __syncthreads();
  int64_t total = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    int64_t sum;
    const int i = i0 + threadIdx.x;
    block_scan(i < a.n ? need[i] : 0, &sum);
    total += sum;
  }
  if (total == 0) return;
  const int limit = static_cast<int>(min(total, static_cast<int64_t>(a.pool.num_pages)));
  const int free = min(limit, select_pages(a.refs, 0, a.pool.num_pages, true, limit, list));
  int64_t before = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    int64_t sum;
    const int i = i0 + threadIdx.x;
    const int mine = i < a.n ? need[i] : 0;
    const int64_t at = before + block_scan(mine, &sum);
    before += sum;
    // an entry without enough pages left, and those behind it, get none
    const bool given = at + mine <= free;
    if (mine > 0 && !given) flag(a, CMR_DEVICE_PAGES_FULL);
    if (i < a.n) first[i] = given ? static_cast<int32_t>(at) : -1;
  }
  __syncthreads();
  for (int i = warp; i < a.n; i += kPlanWarps) {
    const int count = need[i], at = first[i];
    if (count == 0 || at < 0) continue;
    int32_t* row = a.table + static_cast<int64_t>(__ldg(a.dst + i)) * a.max_pages + have[i];
    for (int k = lane; k < count; k += 32) {
      const int32_t id = list[at + k];
      row[k] = id;
      a.refs[id] = 1;
    }
    // what stood behind the row's end stays behind it
    if (lane == 0 && have[i] + count < a.max_pages) row[count] = -1;
  }
}

// Which entries of a fork hold, their shared pages and their own last page; the
// copies are left as jobs (from, to, rows) in the workspace.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PagesArgs a) {
  pdl::wait();
  pdl::launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int P = a.page_tokens;
  int32_t* jobs = a.workspace + kHead;  // [n][3]
  int32_t* state = jobs + 3 * a.n;      // [n]: -1 skipped, else whether it needs a page
  int32_t* list = state + a.n;
  for (int i = warp; i < a.n; i += kPlanWarps) {
    const int32_t src = __ldg(a.src + i), dst = __ldg(a.dst + i), len = __ldg(a.lens + i);
    bool ok = src >= 0 && src < a.rows && dst >= 0 && dst < a.rows && src != dst && len >= 0;
    ok = ok && !named_before(a.dst, i, dst);
    const int64_t pages = ok ? pages_for(len, P) : 0;
    ok = ok && pages <= a.max_pages &&
         __ldcg(a.table + static_cast<int64_t>(dst) * a.max_pages) < 0;
    if (ok) {
      const int32_t* row = a.table + static_cast<int64_t>(src) * a.max_pages;
      bool bad = false;
      for (int k = lane; k < pages; k += 32) {
        const int32_t id = __ldcg(row + k);
        bad |= id < 0 || id >= a.pool.num_pages || __ldcg(a.refs + id) <= 0;
      }
      ok = !__any_sync(~0u, bad);
    }
    if (lane == 0) {
      state[i] = ok ? (len % P != 0 ? 1 : 0) : -1;
      if (!ok) flag(a, CMR_DEVICE_CACHE_RANGE);
    }
  }
  __syncthreads();
  int total = 0;  // at most n
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    int64_t sum;
    const int i = i0 + threadIdx.x;
    block_scan(i < a.n && state[i] == 1, &sum);
    total += static_cast<int>(sum);
  }
  int free = 0;
  if (total > 0) {
    const int limit = min(total, a.pool.num_pages);
    free = min(limit, select_pages(a.refs, 0, a.pool.num_pages, true, limit, list));
  }
  int before = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    int64_t sum;
    const int i = i0 + threadIdx.x;
    const int kind = i < a.n ? state[i] : -1;
    const int at = before + static_cast<int>(block_scan(kind == 1, &sum));
    before += static_cast<int>(sum);
    const bool given = kind == 0 || (kind == 1 && at < free);
    if (kind == 1 && !given) flag(a, CMR_DEVICE_PAGES_FULL);
    if (i < a.n) state[i] = !given ? -1 : (kind == 1 ? at : a.n);
  }
  __syncthreads();
  for (int i = warp; i < a.n; i += kPlanWarps) {
    const int rank = state[i];  // among the entries that get a page; n: needs none
    if (rank < 0) continue;
    const int len = __ldg(a.lens + i);
    const int32_t* srow = a.table + static_cast<int64_t>(__ldg(a.src + i)) * a.max_pages;
    int32_t* drow = a.table + static_cast<int64_t>(__ldg(a.dst + i)) * a.max_pages;
    for (int k = lane; k < len / P; k += 32) {
      const int32_t id = __ldcg(srow + k);
      drow[k] = id;
      atomicAdd(a.refs + id, 1);
    }
    if (rank < a.n && lane == 0) {
      const int32_t id = list[rank];
      drow[len / P] = id;
      a.refs[id] = 1;
      jobs[3 * rank] = __ldcg(srow + len / P);
      jobs[3 * rank + 1] = id;
      jobs[3 * rank + 2] = len % P;
    }
    const int pages = len / P + (len % P != 0);
    if (lane == 0 && pages > 0 && pages < a.max_pages) drow[pages] = -1;
  }
  if (threadIdx.x == 0) a.workspace[kJobs] = min(total, free);
}

// n16 chunks of 16 bytes, by the whole CTA, eight loads in flight per thread.
__device__ __forceinline__ void copy_chunks(uint4* dst, const uint4* src, int n16) {
  constexpr int kBatch = 8;
  for (int i0 = threadIdx.x; i0 < n16; i0 += kCopyThreads * kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k * kCopyThreads < n16) x[k] = __ldcs(src + i0 + k * kCopyThreads);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k * kCopyThreads < n16) __stcs(dst + i0 + k * kCopyThreads, x[k]);
  }
}

// Copies the first rows of each job's page, a (layer, K or V, head) to a CTA at a
// time, and its scale.
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const PagesArgs a) {
  pdl::wait();
  pdl::launch_dependents();
  const int32_t* jobs = a.workspace + kHead;
  const int hk = a.pool.hk, D = a.pool.head_dim;
  const int64_t page = static_cast<int64_t>(a.page_tokens) * D;
  const int64_t units = static_cast<int64_t>(a.pool.num_layers) * hk * 2;
  const int64_t all = units * __ldcg(a.workspace + kJobs);
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    const int64_t job = w / units;
    const int u = static_cast<int>(w - job * units);
    const int h = (u >> 1) % hk, l = (u >> 1) / hk;
    const int32_t from = __ldcg(jobs + 3 * job), to = __ldcg(jobs + 3 * job + 1);
    const int rows = __ldcg(jobs + 3 * job + 2);
    const int64_t s = (static_cast<int64_t>(l) * a.pool.num_pages + from) * hk + h;
    const int64_t d = (static_cast<int64_t>(l) * a.pool.num_pages + to) * hk + h;
    uint8_t* codes = (u & 1) ? a.pool.v : a.pool.k;
    float* scales = (u & 1) ? a.pool.vs : a.pool.ks;
    copy_chunks(reinterpret_cast<uint4*>(codes + d * page),
                reinterpret_cast<const uint4*>(codes + s * page), rows * (D / 16));
    if (threadIdx.x == 0) scales[d] = scales[s];
  }
}

// A CTA per named row.
__global__ void __launch_bounds__(kFreeThreads) free_kernel(const PagesArgs a) {
  pdl::wait();
  pdl::launch_dependents();
  __shared__ int s_end;
  const int i = blockIdx.x;
  const int32_t slot = __ldg(a.dst + i);
  bool same = slot < 0 || slot >= a.rows;
  for (int j = threadIdx.x; j < i && !same; j += kFreeThreads) same = __ldg(a.dst + j) == slot;
  if (__syncthreads_or(same)) {
    if (threadIdx.x == 0) flag(a, CMR_DEVICE_CACHE_RANGE);
    return;
  }
  int32_t* row = a.table + static_cast<int64_t>(slot) * a.max_pages;
  for (int k0 = 0; k0 < a.max_pages; k0 += kFreeThreads) {
    const int k = k0 + threadIdx.x;
    if (threadIdx.x == 0) s_end = a.max_pages;
    __syncthreads();
    const int32_t id = k < a.max_pages ? row[k] : -1;
    if (id < 0 && k < a.max_pages) atomicMin(&s_end, k);
    __syncthreads();
    const int end = s_end;
    if (k < end && id >= 0) {
      if (id >= a.pool.num_pages) {
        flag(a, CMR_DEVICE_CACHE_RANGE);
      } else if (atomicSub(a.refs + id, 1) <= 0) {  // it was free already
        atomicAdd(a.refs + id, 1);
        flag(a, CMR_DEVICE_CACHE_RANGE);
      }
      row[k] = -1;
    }
    if (end < a.max_pages) return;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagesArgs a) {
  __shared__ int s_below;  // pages in use among the first `live`
  pdl::wait();
  pdl::launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n = a.pool.num_pages;
  int32_t* to = a.workspace + kHead;
  int32_t* from = to + n;
  // pages in use, of each warp's segment and before it
  int s0, s1;
  warp_segment(0, n, s0, s1);
  int used = 0;
#pragma unroll 8
  for (int i = s0 + lane; i < s1; i += 32) used += __ldcg(a.refs + i) > 0;
  used = __reduce_add_sync(~0u, used);
  int64_t sum;
  int before = static_cast<int>(block_scan(lane == 0 ? used : 0, &sum));
  before = __shfl_sync(~0u, before, 0);
  const int live = static_cast<int>(sum);
  // those below `live`: the segment that the border falls into counts up to it
  if (live >= s0 && (live < s1 || (live == n && s1 == n && s0 < s1))) {
    int below = 0;
    for (int i = s0 + lane; i < min(s1, live); i += 32) below += __ldcg(a.refs + i) > 0;
    below = __reduce_add_sync(~0u, below);
    if (lane == 0) s_below = before + below;
  }
  __syncthreads();
  // the free ones below the border and the used ones from it on, both in order
  const int below = s_below;
  int at = before;
#pragma unroll 4
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < s1, use = in && __ldcg(a.refs + i) > 0;
    const uint32_t uses = __ballot_sync(~0u, use);
    const int u = at + __popc(uses & ((1u << lane) - 1));  // used ones before page i
    if (in && !use && i < live) to[i - u] = i;
    if (use && i >= live) from[u - below] = i;
    at += __popc(uses);
  }
  __syncthreads();
  const int holes = live - below;
  for (int i = threadIdx.x; i < holes; i += kPlanThreads) {
    a.refs[to[i]] = a.refs[from[i]];
    a.refs[from[i]] = 0;
  }
  if (threadIdx.x == 0) {
    a.workspace[kJobs] = holes;
    a.workspace[kLive] = live;
  }
}

// Copies the moved pages, one (page, layer, K or V) to a CTA at a time, and
// renames them in the table.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const PagesArgs a) {
  pdl::wait();
  pdl::launch_dependents();
  const int32_t* to = a.workspace + kHead;
  const int32_t* from = to + a.pool.num_pages;
  const int moves = __ldcg(a.workspace + kJobs);
  const int live = __ldcg(a.workspace + kLive);
  const int hk = a.pool.hk;
  const int64_t bytes = static_cast<int64_t>(hk) * a.page_tokens * a.pool.head_dim;
  const int units = a.pool.num_layers * 2;
  const int64_t all = static_cast<int64_t>(moves) * units;
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    const int64_t m = w / units;
    const int u = static_cast<int>(w - m * units);
    const int64_t s = static_cast<int64_t>(u >> 1) * a.pool.num_pages + __ldcg(from + m);
    const int64_t d = static_cast<int64_t>(u >> 1) * a.pool.num_pages + __ldcg(to + m);
    uint8_t* codes = (u & 1) ? a.pool.v : a.pool.k;
    float* scales = (u & 1) ? a.pool.vs : a.pool.ks;
    copy_chunks(reinterpret_cast<uint4*>(codes + d * bytes),
                reinterpret_cast<const uint4*>(codes + s * bytes), static_cast<int>(bytes / 16));
    for (int h = threadIdx.x; h < hk; h += kCopyThreads) scales[d * hk + h] = scales[s * hk + h];
  }
  const int64_t entries = static_cast<int64_t>(a.rows) * a.max_pages;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < entries;
       i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    const int32_t id = a.table[i];
    if (id < live) continue;
    int lo = 0, hi = moves;  // its place among the pages moved
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(from + mid) < id)
        lo = mid + 1;
      else
        hi = mid;
    }
    if (lo < moves && __ldcg(from + lo) == id) {
      a.table[i] = __ldcg(to + lo);
      continue;
    }
    // no page in use: a fault where it is one of its row's pages
    int64_t k = i - i % a.max_pages;
    while (k < i && __ldcg(a.table + k) >= 0) ++k;
    if (k == i) flag(a, CMR_DEVICE_CACHE_RANGE);
  }
}

// CTAs of the copying kernels: eight per SM keep about 256 KB per SM in flight.
unsigned copy_grid(int64_t units) {
  const int64_t most = static_cast<int64_t>(sm_count()) * 8;
  return static_cast<unsigned>(units < 1 ? 1 : (units < most ? units : most));
}

}  // namespace

size_t pages_workspace_bytes(int32_t rows, int32_t num_pages, int32_t n) {
  (void)rows;
  return sizeof(int32_t) * (kHead + 2 * static_cast<size_t>(num_pages) + 4 * static_cast<size_t>(n));
}

cudaError_t launch_extend(const PagesArgs& a, cudaStream_t stream) {
  return pdl::launch(extend_kernel, dim3(1), dim3(kPlanThreads), 0, stream, true, a);
}

cudaError_t launch_fork(const PagesArgs& a, cudaStream_t stream) {
  const cudaError_t e =
      pdl::launch(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, true, a);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.n) * a.pool.num_layers * a.pool.hk * 2;
  return pdl::launch(fork_copy_kernel, dim3(copy_grid(units)), dim3(kCopyThreads), 0, stream, true, a);
}

cudaError_t launch_free(const PagesArgs& a, cudaStream_t stream) {
  return pdl::launch(free_kernel, dim3(a.n), dim3(kFreeThreads), 0, stream, true, a);
}

cudaError_t launch_compact(const PagesArgs& a, cudaStream_t stream) {
  const cudaError_t e =
      pdl::launch(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, true, a);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.pool.num_pages / 2 + 1) * a.pool.num_layers * 2;
  return pdl::launch(compact_move_kernel, dim3(copy_grid(units)), dim3(kCopyThreads), 0, stream, true, a);
}

}  // namespace kv8
}  // namespace cmr

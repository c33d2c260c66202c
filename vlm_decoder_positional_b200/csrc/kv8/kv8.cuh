// Declarations shared by the kernels and the C-ABI layer of libcmr_kv8: the
// paged 8-bit cache as the kernels see it, and e4m3 helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "../cmr_internal.cuh"
#include "cmr_kv8.h"

// All kernels here are launched with programmatic stream serialization: their CTAs
// may be placed while the kernel before them in the stream drains.  Every CTA of
// every one of them waits (pdl::wait) before it touches memory that another kernel
// could have written, whoever launched that kernel, so a launch never sees unfinished
// work; what overlaps is the launch itself, which took 2 of the 58 us of a decode
// step's attention (64 x 4,096 tokens).
namespace cmr {
namespace kv8 {

constexpr int kMinScaleExp = -60;
constexpr int kMaxScaleExp = 60;

struct Pool {
  uint8_t* k;  // e4m3 [L, pages, hk, P, D]
  uint8_t* v;
  float* ks;  // [L, pages, hk]
  float* vs;
  int32_t num_pages;
  int32_t page_shift;  // log2 of the tokens of a page
  int32_t num_layers, hk, head_dim;
};

struct Table {
  const int32_t* pages;  // [rows, max_pages]
  int32_t rows;
  int32_t max_pages;
  const int32_t* slot;  // [num_seqs], or nullptr: sequence b uses row b
};

// The tokens of a call: sequence b holds packed tokens cu[b] .. cu[b + 1), at
// absolute indices from pos_offset[b] on.
struct Batch {
  const int32_t* cu;          // nullptr: one token each
  const int32_t* pos_offset;  // nullptr: zeros
  int32_t num_seqs;
  int64_t n_tokens;
};

struct WriteArgs {
  uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* start;
  const int32_t* amount;
  int32_t hq, rot_dim;
  Batch batch;
  Pool pool;
  Table table;
  int32_t* status;
};

struct AttendArgs {
  const uint16_t* q;
  uint16_t* out;
  int32_t hq, group;  // group = hq / hk
  float scale_log2;   // softmax scale * log2(e)
  Batch batch;
  Pool pool;
  Table table;
  void* workspace;
  int32_t* status;
  int64_t min_rows, max_rows;  // the sequences to take: those of so many query rows
};

cudaError_t launch_write(const WriteArgs& a, const FreqTable& table, cudaStream_t stream);

// The attention kernels and the rule between them (attend_rows.cu).
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t stream);
size_t attend_workspace_bytes(int32_t num_seqs, int64_t n_tokens, int32_t num_layers, int32_t hq,
                              int32_t hk, int32_t head_dim);

struct PagesArgs {
  Pool pool;  // null pointers for the calls that move nothing
  int32_t page_tokens;
  int32_t* table;
  int32_t rows, max_pages;
  int32_t* refs;
  const int32_t* src;
  const int32_t* dst;  // the slots of extend and free
  const int32_t* lens;
  int32_t n;
  int32_t* workspace;
  int32_t* status;
};
size_t pages_workspace_bytes(int32_t rows, int32_t num_pages, int32_t n);
cudaError_t launch_extend(const PagesArgs& a, cudaStream_t stream);
cudaError_t launch_fork(const PagesArgs& a, cudaStream_t stream);
cudaError_t launch_free(const PagesArgs& a, cudaStream_t stream);
cudaError_t launch_compact(const PagesArgs& a, cudaStream_t stream);

// SMs of the current device (cached; 0 if it cannot be read).
int sm_count();

// Lets a kernel use `bytes` of dynamic shared memory, the most it is launched with; *done
// has a bit for each device on which that was said (it costs a tenth of a launch).
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done);

#ifdef __CUDACC__

// Whether a scale is one that the cache may hold (false for NaN).
__device__ __forceinline__ bool scale_ok(float s) {
  return s >= 0x1p-60f && s <= 0x1p60f;
}

// Bounds of sequence b's packed tokens; false (and an empty range) when
// cu_seqlens is malformed there.
__device__ __forceinline__ bool seq_range(const Batch& b, int32_t i, int64_t& lo, int64_t& hi) {
  if (b.cu == nullptr) {
    lo = i;
    hi = i + 1;
    return true;
  }
  lo = __ldg(b.cu + i);
  hi = __ldg(b.cu + i + 1);
  if (lo >= 0 && lo <= hi && hi <= b.n_tokens) return true;
  lo = hi = 0;
  return false;
}

// The last i < n with holds(i), holds being true up to some i and false behind it, or
// 0: asked by a whole warp, 32 places at a time.
template <typename F>
__device__ __forceinline__ int32_t last_true(int32_t n, F holds) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(threadIdx.x & 31) * step;
    const uint32_t yes = __ballot_sync(~0u, i < hi && holds(static_cast<int32_t>(i)));
    const int32_t last = yes ? 31 - __clz(yes) : 0;
    const int64_t next = lo + static_cast<int64_t>(last + 1) * step;
    lo += last * step;
    hi = static_cast<int32_t>(next < hi ? next : hi);
  }
  return lo;
}

// Table row of sequence b, or -1 when its slot lies outside the table.
__device__ __forceinline__ int32_t table_row(const Table& t, int32_t b) {
  const int32_t s = t.slot ? __ldg(t.slot + b) : b;
  return s >= 0 && s < t.rows ? s : -1;
}

// Page id that holds page index j of a row, or -1 when there is none.
__device__ __forceinline__ int32_t page_id(const Table& t, int32_t num_pages, int32_t row,
                                           int64_t j) {
  if (row < 0 || j < 0 || j >= t.max_pages) return -1;
  const int32_t id = __ldg(t.pages + static_cast<int64_t>(row) * t.max_pages + j);
  return id >= 0 && id < num_pages ? id : -1;
}

// Two e4m3 codes of a 16-bit word to f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// lo and hi to two e4m3 codes, rounded to nearest even; beyond +-448 saturates,
// NaN gives 0x7f.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

#endif  // __CUDACC__

}  // namespace kv8
}  // namespace cmr

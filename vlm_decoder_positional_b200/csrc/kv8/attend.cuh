// What the two attention kernels share: their launches and workspaces, and how
// a call's query rows are cut into row tiles.  The rows of a KV head are the
// (token, query head) pairs of its group, token by token; an item is a tile of at
// most R of them that belong to one sequence.
#pragma once

#include "kv8.cuh"

namespace cmr {
namespace kv8 {

size_t attend_rows_workspace(int32_t num_seqs, int64_t n_tokens, int32_t hq, int32_t hk,
                             int32_t head_dim);
cudaError_t launch_attend_rows(const AttendArgs& a, cudaStream_t stream);

// The tcgen05 kernel for many rows (attend_tiles.cu).
size_t attend_tiles_workspace(int32_t num_seqs, int32_t num_layers, int32_t hk, int32_t head_dim);
cudaError_t launch_attend_tiles(const AttendArgs& a, cudaStream_t stream);

// Tensor maps of the pool's codes, [unit = (layer, page, head)][row of the page][dim],
// for boxes of `rows` rows of up to 128 dims, swizzled by as many bytes.
bool encode_pool_maps(const Pool& pool, uint32_t rows, CUtensorMap* k, CUtensorMap* v);

// Item slots per (layer, KV head) that the tokens of a call can need.
inline int64_t item_slots(int32_t num_seqs, int64_t n_tokens, int group, int R, bool step) {
  return step ? static_cast<int64_t>(num_seqs) * ((group + R - 1) / R)
              : n_tokens * group / R + num_seqs;
}

#ifdef __CUDACC__

// Byte offset of 16-byte chunk c of row r in a panel.
template <int W>
__device__ __forceinline__ int swizzled(int r, int c) {
  return W == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void load_3d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                             int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                        int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

struct Item {
  int32_t b, row;      // sequence and its table row (-1: none)
  int32_t rows;        // query rows (0: no such item)
  int32_t first_row;   // index of the first among the sequence's token x group rows
  int64_t tok;         // first packed token of the sequence
  int64_t p0;
  int64_t vis_first;   // tokens that the first and the last row see, within the table
  int64_t vis_last;
  bool cut;            // the last row would see beyond the table
};

// The first slot of sequence b: room enough for the partial tiles before it.
template <int R>
__device__ __forceinline__ int64_t item_base(const AttendArgs& a, int64_t b) {
  return static_cast<int64_t>(__ldg(a.batch.cu + b)) * a.group / R + b;
}

// Tokens that a query at position pos - 1 of sequence b sees, within the table; *cut
// when it would see more.
__device__ __forceinline__ int64_t visible(const AttendArgs& a, int32_t row, int64_t pos, bool* cut) {
  const int64_t cap = row < 0 ? 0 : static_cast<int64_t>(a.table.max_pages) << a.pool.page_shift;
  *cut = pos > cap;
  return max(static_cast<int64_t>(0), min(pos, cap));
}

// Row tile rt of sequence b, which has packed tokens [t0, t1) and rows in that tile.
template <int R>
__device__ __forceinline__ Item make_item(const AttendArgs& a, int32_t b, int64_t t0, int64_t t1,
                                          int32_t rt) {
  Item it{};
  const int64_t all = (t1 - t0) * a.group;
  it.b = b;
  it.first_row = rt * R;
  it.rows = static_cast<int32_t>(min(static_cast<int64_t>(R), all - it.first_row));
  it.tok = t0;
  it.p0 = a.batch.pos_offset ? __ldg(a.batch.pos_offset + b) : 0;
  it.row = table_row(a.table, b);
  it.vis_first = visible(a, it.row, it.p0 + it.first_row / a.group + 1, &it.cut);
  it.vis_last = visible(a, it.row, it.p0 + (it.first_row + it.rows - 1) / a.group + 1, &it.cut);
  return it;
}

__device__ __forceinline__ bool takes(const AttendArgs& a, int64_t rows) {
  return rows >= a.min_rows && rows <= a.max_rows;
}

template <int R>
__device__ __forceinline__ Item find_item(const AttendArgs& a, int32_t bi, bool* bad) {
  if (a.batch.cu == nullptr) {
    const int32_t per = (a.group + R - 1) / R;
    const int32_t b = bi / per;
    return make_item<R>(a, b, b, b + 1, bi - b * per);
  }
  int32_t lo = 0, hi = a.batch.num_seqs;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (item_base<R>(a, mid) <= bi)
      lo = mid;
    else
      hi = mid;
  }
  int64_t t0, t1;
  if (!seq_range(a.batch, lo, t0, t1)) {
    *bad = true;
    return Item{};
  }
  if (!takes(a, (t1 - t0) * a.group)) return Item{};
  const int64_t rt = bi - item_base<R>(a, lo);
  if (rt < 0 || rt * R >= (t1 - t0) * a.group) return Item{};
  return make_item<R>(a, lo, t0, t1, static_cast<int32_t>(rt));
}

#endif  // __CUDACC__

}  // namespace kv8
}  // namespace cmr

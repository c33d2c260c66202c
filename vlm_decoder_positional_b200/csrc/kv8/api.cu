// The C ABI of libcmr_kv8 (declared in include/cmr_kv8.h): host-side argument
// checks and the kernel launches.  Nothing here allocates device memory or
// synchronises.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "kv8.cuh"

namespace {

thread_local char g_message[320] = "no error";
thread_local const char* g_last_kernel = nullptr;
thread_local bool g_known = false;  // the caller knows where its addresses lie

cmr_status fail(cmr_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_message, sizeof g_message, fmt, ap);
  va_end(ap);
  return s;
}

cmr_status cuda_fail(cudaError_t e, const char* what) {
  return fail(CMR_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// A required pointer (or, `optional`, a null one): device or managed memory of the
// current device, aligned to `align` bytes.
cmr_status check(const void* p, const char* name, size_t align = 4, bool optional = false) {
  if (p == nullptr)
    return optional ? CMR_OK : fail(CMR_EINVAL, "%s is required", name);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return fail(CMR_EINVAL, "%s must be %zu-byte aligned", name, align);
  return CMR_OK;
}

cmr_status on_device(const void* p, const char* name, int dev) {
  if (p == nullptr) return CMR_OK;
  cudaPointerAttributes attr;
  cudaError_t e = cudaPointerGetAttributes(&attr, p);
  if (e != cudaSuccess) {
    cudaGetLastError();  // clear the error this query may have set
    return fail(CMR_EINVAL, "%s: not a CUDA pointer (%s)", name, cudaGetErrorName(e));
  }
  if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
    return fail(CMR_EINVAL, "%s: not device memory (memory type %d)", name,
                static_cast<int>(attr.type));
  if (attr.type == cudaMemoryTypeDevice && attr.device != dev)
    return fail(CMR_EINVAL, "%s: lives on device %d but device %d is current", name,
                attr.device, dev);
  return CMR_OK;
}

struct Named {
  const void* p;
  const char* name;
};

template <size_t N>
cmr_status all_on_device(const Named (&list)[N]) {
  if (g_known) return CMR_OK;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();  // no pointer will pass then
  for (const Named& x : list) {
    const cmr_status s = on_device(x.p, x.name, dev);
    if (s != CMR_OK) return s;
  }
  return CMR_OK;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

int page_shift(int32_t page_tokens) {
  switch (page_tokens) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

// Checks of the pool's shape and pointers; fills *pool.
cmr_status check_pool(const void* k_pages, const void* v_pages, const float* k_scales,
                      const float* v_scales, int32_t num_layers, int32_t hk, int32_t head_dim,
                      int32_t num_pages, int32_t page_tokens, cmr::kv8::Pool* pool) {
  if (num_layers < 0) return fail(CMR_EINVAL, "negative num_layers");
  if (hk < 1) return fail(CMR_EINVAL, "hk must be >= 1");
  if (num_pages < 1) return fail(CMR_EINVAL, "num_pages must be >= 1");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(CMR_EUNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", head_dim);
  if (page_shift(page_tokens) < 0)
    return fail(CMR_EUNSUPPORTED, "page_tokens must be 16, 32, 64 or 128, got %d", page_tokens);
  if (static_cast<int64_t>(hk) * num_layers > 65535)  // a dimension of a grid
    return fail(CMR_EUNSUPPORTED, "hk * num_layers exceeds 65535");
  if (static_cast<int64_t>(hk) * num_layers > INT32_MAX / num_pages)
    return fail(CMR_EUNSUPPORTED, "num_layers * num_pages * hk exceeds INT32_MAX");
  if (hk > (1 << 23) / head_dim)
    return fail(CMR_EUNSUPPORTED, "hk * head_dim exceeds 2^23");
  cmr_status s;
  if ((s = check(k_pages, "k_pages", 16)) != CMR_OK) return s;
  if ((s = check(v_pages, "v_pages", 16)) != CMR_OK) return s;
  if ((s = check(k_scales, "k_scales")) != CMR_OK) return s;
  if ((s = check(v_scales, "v_scales")) != CMR_OK) return s;
  pool->k = static_cast<uint8_t*>(const_cast<void*>(k_pages));
  pool->v = static_cast<uint8_t*>(const_cast<void*>(v_pages));
  pool->ks = const_cast<float*>(k_scales);
  pool->vs = const_cast<float*>(v_scales);
  pool->num_pages = num_pages;
  pool->page_shift = page_shift(page_tokens);
  pool->num_layers = num_layers;
  pool->hk = hk;
  pool->head_dim = head_dim;
  return CMR_OK;
}

cmr_status check_table(const int32_t* page_table, int32_t table_rows, int32_t max_pages) {
  if (table_rows < 1 || max_pages < 1)
    return fail(CMR_EINVAL, "table_rows and max_pages must be >= 1");
  return check(page_table, "page_table");
}

// Checks of a batch's shape; CMR_OK with *empty set when it has no tokens.
cmr_status check_batch(const int32_t* cu_seqlens, int32_t num_seqs, const int32_t* pos_offset,
                       int64_t n_tokens, cmr::kv8::Batch* b, bool* empty) {
  *empty = false;
  if (n_tokens < 0 || num_seqs < 0) return fail(CMR_EINVAL, "negative n_tokens or num_seqs");
  if (n_tokens > INT32_MAX) return fail(CMR_EINVAL, "n_tokens exceeds int32 indexing");
  if (n_tokens == 0) {
    *empty = true;
    return CMR_OK;
  }
  if (num_seqs == 0) return fail(CMR_EINVAL, "num_seqs must be > 0 when there are tokens");
  if (!cu_seqlens && num_seqs != n_tokens)
    return fail(CMR_EINVAL, "without cu_seqlens every sequence holds one token (num_seqs == n_tokens)");
  cmr_status s;
  if ((s = check(cu_seqlens, "cu_seqlens", 4, true)) != CMR_OK) return s;
  if ((s = check(pos_offset, "pos_offset", 4, true)) != CMR_OK) return s;
  b->cu = cu_seqlens;
  b->pos_offset = pos_offset;
  b->num_seqs = num_seqs;
  b->n_tokens = n_tokens;
  return CMR_OK;
}

cmr_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (need == 0) return CMR_OK;
  if (!workspace || have < need)
    return fail(CMR_EINVAL, "workspace must hold at least %zu bytes, has %zu", need,
                workspace ? have : static_cast<size_t>(0));
  return check(workspace, "workspace", 16);
}

// Frequencies and their planes, as in cmr_rotate_qk.
cmr_status check_rotation(double theta, const int32_t sections[3], int32_t rot_dim,
                          int32_t head_dim, cmr::FreqTable* table) {
  if (rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > head_dim)
    return fail(CMR_EINVAL, "rot_dim must be a multiple of 16 in [16, head_dim]");
  if (!(theta > 0.0) || !std::isfinite(theta)) return fail(CMR_EINVAL, "theta must be finite and > 0");
  if (!sections) return fail(CMR_EINVAL, "sections is required");
  const int F = rot_dim / 2;
  // a model calls with one theta and rot_dim: their powers cost as much as the launch
  thread_local struct {
    double theta;
    int32_t rot_dim;
    double inv_freq[cmr::kMaxFreqs];
  } last = {};
  if (last.theta != theta || last.rot_dim != rot_dim) {
    for (int j = 0; j < cmr::kMaxFreqs; ++j)
      last.inv_freq[j] = j < F ? std::pow(theta, -2.0 * j / rot_dim) : 0.0;
    last.theta = theta;
    last.rot_dim = rot_dim;
  }
  for (int j = 0; j < cmr::kMaxFreqs; ++j) {
    table->plane[j] = 0;
    table->inv_freq[j] = last.inv_freq[j];
  }
  if (sections[0] < 0 || sections[1] < 0 || sections[2] < 0 ||
      static_cast<int64_t>(sections[0]) + sections[1] + sections[2] != F)
    return fail(CMR_EINVAL, "sections must be >= 0 and sum to rot_dim / 2");
  for (int plane = 1; plane <= 2; ++plane)
    for (int m = 0; m < sections[plane]; ++m) {
      const int j = 3 * m + plane;
      if (j >= F)
        return fail(CMR_EINVAL, "sections[%d] = %d does not fit the interleave", plane, sections[plane]);
      table->plane[j] = plane;
    }
  return CMR_OK;
}

// Shared by the page calls: table, counts, list of rows.
cmr_status check_pages(int32_t* page_table, int32_t table_rows, int32_t max_pages,
                       int32_t* page_refs, int32_t num_pages, int32_t n,
                       cmr::kv8::PagesArgs* a) {
  if (n < 0) return fail(CMR_EINVAL, "negative n");
  if (num_pages < 1) return fail(CMR_EINVAL, "num_pages must be >= 1");
  cmr_status s;
  if ((s = check_table(page_table, table_rows, max_pages)) != CMR_OK) return s;
  if ((s = check(page_refs, "page_refs")) != CMR_OK) return s;
  a->pool.num_pages = num_pages;
  a->table = page_table;
  a->rows = table_rows;
  a->max_pages = max_pages;
  a->refs = page_refs;
  a->n = n;
  return CMR_OK;
}

cmr_status check_pages_workspace(void* workspace, size_t workspace_bytes,
                                 cmr::kv8::PagesArgs* a) {
  a->workspace = static_cast<int32_t*>(workspace);
  return check_workspace(workspace, workspace_bytes,
                         cmr::kv8::pages_workspace_bytes(a->rows, a->pool.num_pages, a->n));
}

// The words of cmr_kv8_call.
struct Words {
  const char* at;
  int64_t i64(int k) const {
    int64_t v;
    memcpy(&v, at + 8 * k, 8);
    return v;
  }
  double f64(int k) const {
    double v;
    memcpy(&v, at + 8 * k, 8);
    return v;
  }
  // what does not fit becomes a negative number, which every call refuses
  int32_t i32(int k) const {
    const int64_t v = i64(k);
    return v >= INT32_MIN && v <= INT32_MAX ? static_cast<int32_t>(v) : INT32_MIN;
  }
  size_t size(int k) const { return static_cast<size_t>(i64(k)); }
  void* ptr(int k) const { return reinterpret_cast<void*>(i64(k)); }
  int32_t* ints(int k) const { return reinterpret_cast<int32_t*>(i64(k)); }
  float* flt(int k) const { return reinterpret_cast<float*>(i64(k)); }
  cmr_stream_t stream(int k) const { return reinterpret_cast<cmr_stream_t>(i64(k)); }
};

}  // namespace

namespace cmr {

// tensor_map.cu and the shared headers name the kernel that ran through this.
void note_kernel(const char* name) { g_last_kernel = name; }

namespace kv8 {

int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  int c = cached[dev & 63].load(std::memory_order_relaxed);
  if (c == 0) {
    if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cached[dev & 63].store(c, std::memory_order_relaxed);
  }
  return c;
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace kv8
}  // namespace cmr

extern "C" {

const char* cmr_kv8_last_error_message(void) { return g_message; }

const char* cmr_kv8_last_attend_kernel(void) { return g_last_kernel ? g_last_kernel : ""; }

cmr_status cmr_kv8_rotate_qk(void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                             int32_t num_seqs, const int32_t* pos_offset, const int32_t* start,
                             const int32_t* amount, int64_t n_tokens, int32_t num_layers,
                             int32_t hq, int32_t hk, int32_t head_dim, double theta,
                             const int32_t sections[3], int32_t rot_dim, void* k_pages,
                             void* v_pages, float* k_scales, float* v_scales, int32_t num_pages,
                             int32_t page_tokens, const int32_t* page_table, int32_t table_rows,
                             int32_t max_pages, const int32_t* slot, int32_t* device_status,
                             cmr_stream_t stream) {
  cmr::kv8::WriteArgs a{};
  cmr::FreqTable table;
  bool empty;
  cmr_status s;
  if (hq < 0) return fail(CMR_EINVAL, "negative hq");
  if ((s = check_pool(k_pages, v_pages, k_scales, v_scales, num_layers, hk, head_dim, num_pages,
                      page_tokens, &a.pool)) != CMR_OK)
    return s;
  if ((s = check_rotation(theta, sections, rot_dim, head_dim, &table)) != CMR_OK) return s;
  if ((static_cast<int64_t>(hq) + hk) * num_layers > INT32_MAX)
    return fail(CMR_EUNSUPPORTED, "(hq + hk) * num_layers exceeds INT32_MAX");
  if ((s = check_table(page_table, table_rows, max_pages)) != CMR_OK) return s;
  if ((s = check_batch(cu_seqlens, num_seqs, pos_offset, n_tokens, &a.batch, &empty)) != CMR_OK)
    return s;
  if (empty || num_layers == 0) return CMR_OK;
  if ((s = check(q, "q", 16, hq == 0)) != CMR_OK) return s;
  if ((s = check(k, "k", 16)) != CMR_OK) return s;
  if ((s = check(v, "v", 16)) != CMR_OK) return s;
  if ((s = check(start, "start")) != CMR_OK) return s;
  if ((s = check(amount, "amount")) != CMR_OK) return s;
  if ((s = check(slot, "slot", 4, true)) != CMR_OK) return s;
  const int64_t per_head = static_cast<int64_t>(num_layers) * n_tokens * head_dim * 2;
  const int64_t pool = static_cast<int64_t>(num_layers) * num_pages * hk * page_tokens * head_dim;
  const struct {
    const void* p;
    int64_t bytes;
  } made[] = {{q, hq * per_head}, {k_pages, pool}, {v_pages, pool}},
    given[] = {{k, hk * per_head}, {v, hk * per_head}, {k_pages, pool}, {v_pages, pool}};
  for (int i = hq > 0 ? 0 : 1; i < 3; ++i)  // of the pages: only k and v
    for (int j = 0; j < (i == 0 ? 4 : 2); ++j)
      if (overlap(made[i].p, made[i].bytes, given[j].p, given[j].bytes))
        return fail(CMR_EINVAL, "q, k or v overlaps what the call writes");
  const Named list[] = {{hq ? q : nullptr, "q"}, {k, "k"}, {v, "v"}, {cu_seqlens, "cu_seqlens"},
                        {pos_offset, "pos_offset"}, {start, "start"}, {amount, "amount"},
                        {k_pages, "k_pages"}, {v_pages, "v_pages"}, {k_scales, "k_scales"},
                        {v_scales, "v_scales"}, {page_table, "page_table"}, {slot, "slot"},
                        {device_status, "device_status"}};
  if ((s = all_on_device(list)) != CMR_OK) return s;
  a.q = static_cast<uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.start = start;
  a.amount = amount;
  a.hq = hq;
  a.rot_dim = rot_dim;
  a.table = {page_table, table_rows, max_pages, slot};
  a.status = device_status;
  const cudaError_t e = cmr::kv8::launch_write(a, table, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CMR_OK : cuda_fail(e, "kv8_rotate_qk launch");
}

size_t cmr_kv8_attend_workspace_bytes(int32_t num_seqs, int64_t n_tokens, int32_t num_layers,
                                      int32_t hq, int32_t hk, int32_t head_dim) {
  if (num_seqs <= 0 || n_tokens <= 0 || n_tokens > INT32_MAX || num_layers <= 0 || hk <= 0 ||
      hq <= 0 || hq % hk != 0 || hq / hk > 128 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  return cmr::kv8::attend_workspace_bytes(num_seqs, n_tokens, num_layers, hq, hk, head_dim);
}

cmr_status cmr_kv8_attend(const void* q, void* out, const int32_t* cu_seqlens, int32_t num_seqs,
                          const int32_t* pos_offset, int64_t n_tokens, int32_t num_layers,
                          int32_t hq, int32_t hk, int32_t head_dim, double scale,
                          const void* k_pages, const void* v_pages, const float* k_scales,
                          const float* v_scales, int32_t num_pages, int32_t page_tokens,
                          const int32_t* page_table, int32_t table_rows, int32_t max_pages,
                          const int32_t* slot, void* workspace, size_t workspace_bytes,
                          int32_t* device_status, cmr_stream_t stream) {
  cmr::kv8::AttendArgs a{};
  bool empty;
  cmr_status s;
  if ((s = check_pool(k_pages, v_pages, k_scales, v_scales, num_layers, hk, head_dim, num_pages,
                      page_tokens, &a.pool)) != CMR_OK)
    return s;
  if (hq < 1 || hq % hk != 0 || hq / hk > 128)
    return fail(CMR_EINVAL, "hq must be a positive multiple of hk, at most 128 of it");
  const double log2e = 1.4426950408889634074;
  if (!std::isfinite(scale) || !std::isfinite(static_cast<float>(scale * log2e)))
    return fail(CMR_EINVAL, "scale must be finite");
  if ((s = check_table(page_table, table_rows, max_pages)) != CMR_OK) return s;
  if (static_cast<int64_t>(max_pages) * page_tokens > INT32_MAX - 256)
    return fail(CMR_EINVAL, "max_pages * page_tokens exceeds int32 indexing");
  if ((s = check_batch(cu_seqlens, num_seqs, pos_offset, n_tokens, &a.batch, &empty)) != CMR_OK)
    return s;
  if (empty || num_layers == 0) return CMR_OK;
  if ((s = check(q, "q", 16)) != CMR_OK) return s;
  if ((s = check(out, "out", 16)) != CMR_OK) return s;
  if ((s = check(slot, "slot", 4, true)) != CMR_OK) return s;
  const int64_t bytes = static_cast<int64_t>(num_layers) * n_tokens * hq * head_dim * 2;
  const int64_t pool = static_cast<int64_t>(num_layers) * num_pages * hk * page_tokens * head_dim;
  if (overlap(q, bytes, out, bytes) || overlap(k_pages, pool, out, bytes) ||
      overlap(v_pages, pool, out, bytes))
    return fail(CMR_EINVAL, "out must not overlap q or the cache");
  if ((s = check_workspace(workspace, workspace_bytes,
                           cmr_kv8_attend_workspace_bytes(num_seqs, n_tokens, num_layers, hq, hk,
                                                          head_dim))) != CMR_OK)
    return s;
  const Named list[] = {{q, "q"}, {out, "out"}, {cu_seqlens, "cu_seqlens"},
                        {pos_offset, "pos_offset"}, {k_pages, "k_pages"}, {v_pages, "v_pages"},
                        {k_scales, "k_scales"}, {v_scales, "v_scales"},
                        {page_table, "page_table"}, {slot, "slot"}, {workspace, "workspace"},
                        {device_status, "device_status"}};
  if ((s = all_on_device(list)) != CMR_OK) return s;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.hq = hq;
  a.group = hq / hk;
  a.scale_log2 = static_cast<float>(scale * log2e);
  a.table = {page_table, table_rows, max_pages, slot};
  a.workspace = workspace;
  a.status = device_status;
  const cudaError_t e = cmr::kv8::launch_attend(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CMR_OK : cuda_fail(e, "kv8_attend launch");
}

size_t cmr_kv8_pages_workspace_bytes(int32_t table_rows, int32_t num_pages, int32_t n) {
  if (table_rows < 1 || num_pages < 1 || n < 0) return 0;
  return cmr::kv8::pages_workspace_bytes(table_rows, num_pages, n);
}

cmr_status cmr_kv8_extend(int32_t* page_table, int32_t table_rows, int32_t max_pages,
                          int32_t* page_refs, int32_t num_pages, int32_t page_tokens,
                          const int32_t* slots, const int32_t* lens, int32_t n, void* workspace,
                          size_t workspace_bytes, int32_t* device_status, cmr_stream_t stream) {
  cmr::kv8::PagesArgs a{};
  cmr_status s;
  if (page_shift(page_tokens) < 0)
    return fail(CMR_EUNSUPPORTED, "page_tokens must be 16, 32, 64 or 128, got %d", page_tokens);
  if ((s = check_pages(page_table, table_rows, max_pages, page_refs, num_pages, n, &a)) != CMR_OK)
    return s;
  if ((s = check_pages_workspace(workspace, workspace_bytes, &a)) != CMR_OK) return s;
  if (n == 0) return CMR_OK;
  if ((s = check(slots, "slots")) != CMR_OK) return s;
  if ((s = check(lens, "lens")) != CMR_OK) return s;
  const Named list[] = {{page_table, "page_table"}, {page_refs, "page_refs"}, {slots, "slots"},
                        {lens, "lens"}, {workspace, "workspace"},
                        {device_status, "device_status"}};
  if ((s = all_on_device(list)) != CMR_OK) return s;
  a.page_tokens = page_tokens;
  a.dst = slots;
  a.lens = lens;
  a.status = device_status;
  const cudaError_t e = cmr::kv8::launch_extend(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CMR_OK : cuda_fail(e, "kv8_extend launch");
}

cmr_status cmr_kv8_fork(void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                        int32_t num_layers, int32_t hk, int32_t head_dim, int32_t num_pages,
                        int32_t page_tokens, int32_t* page_table, int32_t table_rows,
                        int32_t max_pages, int32_t* page_refs, const int32_t* src,
                        const int32_t* dst, const int32_t* lens, int32_t n, void* workspace,
                        size_t workspace_bytes, int32_t* device_status, cmr_stream_t stream) {
  cmr::kv8::PagesArgs a{};
  cmr_status s;
  if ((s = check_pages(page_table, table_rows, max_pages, page_refs, num_pages, n, &a)) != CMR_OK)
    return s;
  if ((s = check_pages_workspace(workspace, workspace_bytes, &a)) != CMR_OK) return s;
  if ((s = check_pool(k_pages, v_pages, k_scales, v_scales, num_layers, hk, head_dim, num_pages,
                      page_tokens, &a.pool)) != CMR_OK)
    return s;
  if (n == 0) return CMR_OK;
  if ((s = check(src, "src")) != CMR_OK) return s;
  if ((s = check(dst, "dst")) != CMR_OK) return s;
  if ((s = check(lens, "lens")) != CMR_OK) return s;
  const Named list[] = {{k_pages, "k_pages"}, {v_pages, "v_pages"}, {k_scales, "k_scales"},
                        {v_scales, "v_scales"}, {page_table, "page_table"},
                        {page_refs, "page_refs"}, {src, "src"}, {dst, "dst"}, {lens, "lens"},
                        {workspace, "workspace"}, {device_status, "device_status"}};
  if ((s = all_on_device(list)) != CMR_OK) return s;
  a.page_tokens = page_tokens;
  a.src = src;
  a.dst = dst;
  a.lens = lens;
  a.status = device_status;
  const cudaError_t e = cmr::kv8::launch_fork(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CMR_OK : cuda_fail(e, "kv8_fork launch");
}

cmr_status cmr_kv8_free(int32_t* page_table, int32_t table_rows, int32_t max_pages,
                        int32_t* page_refs, int32_t num_pages, const int32_t* slots, int32_t n,
                        int32_t* device_status, cmr_stream_t stream) {
  cmr::kv8::PagesArgs a{};
  cmr_status s;
  if ((s = check_pages(page_table, table_rows, max_pages, page_refs, num_pages, n, &a)) != CMR_OK)
    return s;
  if (n == 0) return CMR_OK;
  if ((s = check(slots, "slots")) != CMR_OK) return s;
  const Named list[] = {{page_table, "page_table"}, {page_refs, "page_refs"}, {slots, "slots"},
                        {device_status, "device_status"}};
  if ((s = all_on_device(list)) != CMR_OK) return s;
  a.dst = slots;
  a.status = device_status;
  const cudaError_t e = cmr::kv8::launch_free(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CMR_OK : cuda_fail(e, "kv8_free launch");
}

cmr_status cmr_kv8_compact(void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                           int32_t num_layers, int32_t hk, int32_t head_dim, int32_t num_pages,
                           int32_t page_tokens, int32_t* page_table, int32_t table_rows,
                           int32_t max_pages, int32_t* page_refs, void* workspace,
                           size_t workspace_bytes, int32_t* device_status, cmr_stream_t stream) {
  cmr::kv8::PagesArgs a{};
  cmr_status s;
  if ((s = check_pages(page_table, table_rows, max_pages, page_refs, num_pages, 0, &a)) != CMR_OK)
    return s;
  if ((s = check_pages_workspace(workspace, workspace_bytes, &a)) != CMR_OK) return s;
  if ((s = check_pool(k_pages, v_pages, k_scales, v_scales, num_layers, hk, head_dim, num_pages,
                      page_tokens, &a.pool)) != CMR_OK)
    return s;
  const Named list[] = {{k_pages, "k_pages"}, {v_pages, "v_pages"}, {k_scales, "k_scales"},
                        {v_scales, "v_scales"}, {page_table, "page_table"},
                        {page_refs, "page_refs"}, {workspace, "workspace"},
                        {device_status, "device_status"}};
  if ((s = all_on_device(list)) != CMR_OK) return s;
  a.page_tokens = page_tokens;
  a.status = device_status;
  const cudaError_t e = cmr::kv8::launch_compact(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CMR_OK : cuda_fail(e, "kv8_compact launch");
}

cmr_status cmr_kv8_call(int32_t call, const void* words, int32_t count) {
  if (!words) return fail(CMR_EINVAL, "words is required");
  const Words w{static_cast<const char*>(words)};
  struct Known {
    explicit Known(bool known) { g_known = known; }
    ~Known() { g_known = false; }
  } known((call & CMR_KV8_KNOWN_ADDRESSES) != 0);
  switch (call & ~CMR_KV8_KNOWN_ADDRESSES) {
    case 0:
      if (count != 28) break;
      return cmr_kv8_rotate_qk(w.ptr(0), w.ptr(1), w.ptr(2), w.ints(3), w.i32(4), w.ints(5),
                               w.ints(6), w.ints(7), w.i64(8), w.i32(9), w.i32(10), w.i32(11),
                               w.i32(12), w.f64(13), w.ints(14), w.i32(15), w.ptr(16), w.ptr(17),
                               w.flt(18), w.flt(19), w.i32(20), w.i32(21), w.ints(22), w.i32(23),
                               w.i32(24), w.ints(25), w.ints(26), w.stream(27));
    case 1:
      if (count != 25) break;
      return cmr_kv8_attend(w.ptr(0), w.ptr(1), w.ints(2), w.i32(3), w.ints(4), w.i64(5),
                            w.i32(6), w.i32(7), w.i32(8), w.i32(9), w.f64(10), w.ptr(11),
                            w.ptr(12), w.flt(13), w.flt(14), w.i32(15), w.i32(16), w.ints(17),
                            w.i32(18), w.i32(19), w.ints(20), w.ptr(21), w.size(22), w.ints(23),
                            w.stream(24));
    case 2:
      if (count != 13) break;
      return cmr_kv8_extend(w.ints(0), w.i32(1), w.i32(2), w.ints(3), w.i32(4), w.i32(5),
                            w.ints(6), w.ints(7), w.i32(8), w.ptr(9), w.size(10), w.ints(11),
                            w.stream(12));
    case 3:
      if (count != 21) break;
      return cmr_kv8_fork(w.ptr(0), w.ptr(1), w.flt(2), w.flt(3), w.i32(4), w.i32(5), w.i32(6),
                          w.i32(7), w.i32(8), w.ints(9), w.i32(10), w.i32(11), w.ints(12),
                          w.ints(13), w.ints(14), w.ints(15), w.i32(16), w.ptr(17), w.size(18),
                          w.ints(19), w.stream(20));
    case 4:
      if (count != 9) break;
      return cmr_kv8_free(w.ints(0), w.i32(1), w.i32(2), w.ints(3), w.i32(4), w.ints(5), w.i32(6),
                          w.ints(7), w.stream(8));
    case 5:
      if (count != 17) break;
      return cmr_kv8_compact(w.ptr(0), w.ptr(1), w.flt(2), w.flt(3), w.i32(4), w.i32(5), w.i32(6),
                             w.i32(7), w.i32(8), w.ints(9), w.i32(10), w.i32(11), w.ints(12),
                             w.ptr(13), w.size(14), w.ints(15), w.stream(16));
    default:
      return fail(CMR_EINVAL, "no call has the number %d", call);
  }
  return fail(CMR_EINVAL, "call %d does not have %d words", call, count);
}

}  // extern "C"

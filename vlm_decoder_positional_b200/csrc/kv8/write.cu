// Rotate Q in place and write the rotated K and the V rows of the same tokens
// into the paged 8-bit cache, in one launch.
//
// A page's scale is s = 2^e, the smallest with max |x| <= 448 s over the rows
// written (at least the page's old scale when it held rows), and a code is
// e4m3(x / s), x / s being exact.  448 = 1.75 * 2^8, so e follows from the
// exponent and mantissa bits of the largest bf16 magnitude alone.
//
// Bound by memory: K, V and Q's rotated dims are read once from DRAM, the codes
// (half of the bf16 bytes) and Q's rotated dims are written once.  A scale needs
// all rows of its page before the first code can be written, so a page's rows
// stay in registers from the load to the store.
//
// write_pages_kernel (prompts and chunks): a CTA owns a page and a group of
// layers and walks over their (layer, K or V, head) tiles of at most P x D
// values, with the loads of the next tile in flight while it reduces and
// encodes the present one; the cos/sin of the page's tokens are computed once
// and kept in shared memory for all heads and layers.  A page's tokens and the
// units before it are found from cu_seqlens alone (sequence b's pages start at
// unit cu[b] / P + 2 b, room enough for its first and last partial pages), so no
// list of pages is built.  Q's rows go to the CTAs behind, eight frequencies of
// a token to a thread as in the other rotation kernels.
// write_step_kernel (one token per sequence): a warp per K and V row, since a
// page gets one row and the rest of the work is latency.
#include <mutex>

#include "kv8.cuh"
#include "../rotate_common.cuh"

namespace cmr {
namespace kv8 {
namespace {

using namespace rot;

constexpr int kThreads = 256;
constexpr int kQBatch = 4;  // Q head rows in flight per thread

// Exponent of the scale for a largest bf16 magnitude of these bits (finite).
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return bits == 0 ? kMinScaleExp : min(max(e, kMinScaleExp), kMaxScaleExp);
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Largest magnitude bits of the two halves of a packed running maximum.
__device__ __forceinline__ uint32_t halves_max(uint32_t m) { return max(m & 0xffffu, m >> 16); }

__device__ __forceinline__ uint32_t magnitudes(uint32_t m, const uint4& x) {
  m = __vmaxs2(m, x.x & 0x7fff7fffu);
  m = __vmaxs2(m, x.y & 0x7fff7fffu);
  m = __vmaxs2(m, x.z & 0x7fff7fffu);
  return __vmaxs2(m, x.w & 0x7fff7fffu);
}

// The same with infinities and NaN left out.
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t m, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    m = __vmaxs2(m, (lo < 0x7f80u ? lo : 0u) | (hi < 0x7f80u ? hi << 16 : 0u));
  }
  return m;
}

__device__ __forceinline__ float inf_to_nan(float x) {
  return fabsf(x) == __int_as_float(0x7f800000) ? __int_as_float(0x7fffffff) : x;
}

// Eight bf16 values over the scale, as codes.
template <bool kCheck>
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
    if (kCheck) {
      lo = inf_to_nan(lo);
      hi = inf_to_nan(hi);
    }
    r[i] = f32_to_e4m3x2(lo * inv, hi * inv);
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Four codes under another scale: code * ratio, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const uint32_t a = e4m3x2_to_f16x2(w & 0xffffu), b = e4m3x2_to_f16x2(w >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return f32_to_e4m3x2(x.x * ratio, x.y * ratio) | (f32_to_e4m3x2(y.x * ratio, y.y * ratio) << 16);
}

// The scale of a page whose new rows need exponent e and which held rows under
// `old` (held) or none: sets *ratio to old / new where those have to be encoded
// again, else to 1.
__device__ __forceinline__ float page_scale(int e, bool held, float old, float* ratio,
                                            int32_t* status) {
  float s = pow2f(e);
  *ratio = 1.f;
  if (held) {
    if (!scale_ok(old)) {
      if (status != nullptr) atomicOr(status, CMR_DEVICE_BAD_SCALE);
    } else if (old >= s) {
      s = old;
    } else {
      *ratio = old / s;
    }
  }
  return s;
}

// This lane's chunk of 8 values of a K row, rotated: chunk c < F / 8 holds the
// first halves of pairs whose second halves lie F / 8 chunks on.
__device__ __forceinline__ uint4 rotate_chunk(const uint4& x, int lane, int c, int half8,
                                              const float2* cs) {
  const bool first = c < half8;
  const bool rotated = c < 2 * half8;
  const int partner = first ? lane + half8 : lane - half8;
  const int from = rotated ? partner : lane;
  uint4 y;
  y.x = __shfl_sync(~0u, x.x, from);
  y.y = __shfl_sync(~0u, x.y, from);
  y.z = __shfl_sync(~0u, x.z, from);
  y.w = __shfl_sync(~0u, x.w, from);
  if (!rotated) return x;
  const uint32_t* own = reinterpret_cast<const uint32_t*>(&x);
  const uint32_t* oth = reinterpret_cast<const uint32_t*>(&y);
  const float2* f = cs + 8 * (first ? c : c - half8);
  uint4 r;
  uint32_t* out = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float2 f0 = f[2 * m], f1 = f[2 * m + 1];
    const float o0 = bf16_lo(own[m]), o1 = bf16_hi(own[m]);
    const float p0 = bf16_lo(oth[m]), p1 = bf16_hi(oth[m]);
    out[m] = first ? pack_bf16x2(o0 * f0.x - p0 * f0.y, o1 * f1.x - p1 * f1.y)
                   : pack_bf16x2(o0 * f0.x + p0 * f0.y, o1 * f1.x + p1 * f1.y);
  }
  return r;
}

__device__ __forceinline__ float2 cos_sin_of(const WriteArgs& a, int32_t b, int64_t p, int plane,
                                             double inv) {
  const Planes r = canvas_row(p, __ldg(a.start + b), __ldg(a.amount + b));
  float c, s;
  cos_sin(plane == 0 ? r.t : (plane == 1 ? r.h : r.w), inv, c, s);
  return make_float2(c, s);
}

// Where page id's tile of (layer, head) starts, and its scale's place.
__device__ __forceinline__ int64_t unit_index(const Pool& p, int l, int32_t id, int h) {
  return (static_cast<int64_t>(l) * p.num_pages + id) * p.hk + h;
}

// Rotates rows of Q: item v = group of (layer, head) rows x token; thread u of an
// item owns frequencies [8u, 8u + 8).
__device__ __forceinline__ void rotate_q_items(const WriteArgs& a, const double* s_inv,
                                               const int32_t* s_plane, int64_t block,
                                               int32_t groups, int32_t per_group) {
  const int F = a.rot_dim / 2, U = F / 8;
  const int per_cta = kThreads / U;
  const int local = threadIdx.x / U, u = threadIdx.x - local * U;
  if (local >= per_cta) return;
  const int64_t N = a.batch.n_tokens;
  const int64_t v = block * per_cta + local;
  if (v >= N * groups) return;
  const int64_t g = groups == 1 ? 0 : v / N;
  const int64_t t = v - g * N;
  // the last sequence with cu[b] <= t
  int32_t b = static_cast<int32_t>(t);
  int64_t p = 0;
  if (a.batch.cu != nullptr) {
    if (t >= __ldg(a.batch.cu + a.batch.num_seqs)) return;
    int32_t lo = 0, hi = a.batch.num_seqs;
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (__ldg(a.batch.cu + mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    int64_t t0, t1;
    if (!seq_range(a.batch, b, t0, t1) || t < t0 || t >= t1) return;
    p = t - t0;
  }
  p += a.batch.pos_offset ? __ldg(a.batch.pos_offset + b) : 0;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 f = cos_sin_of(a, b, p, s_plane[8 * u + e], s_inv[8 * u + e]);
    c[e] = f.x;
    s[e] = f.y;
  }
  const int64_t D = a.pool.head_dim, q_tok = a.hq * D, q_layer = N * q_tok;
  const int j_lo = static_cast<int>(g) * per_group;
  const int j_hi = min(a.hq * a.pool.num_layers, j_lo + per_group);
  const int step = F / 8;
  int h = j_lo % a.hq, l = j_lo / a.hq;
  for (int j0 = j_lo; j0 < j_hi; j0 += kQBatch) {
    uint4 x1[kQBatch], x2[kQBatch];
    uint4* ptr[kQBatch];
#pragma unroll
    for (int i = 0; i < kQBatch; ++i) {
      ptr[i] = nullptr;
      if (j0 + i < j_hi) {
        ptr[i] = reinterpret_cast<uint4*>(a.q + l * q_layer + t * q_tok + h * D + 8 * u);
        x1[i] = __ldcs(ptr[i]);
        x2[i] = __ldcs(ptr[i] + step);
        if (++h == a.hq) {
          h = 0;
          ++l;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kQBatch; ++i)
      if (ptr[i] != nullptr) {
        rotate_unit(x1[i], x2[i], c, s);
        __stcs(ptr[i], x1[i]);
        __stcs(ptr[i] + step, x2[i]);
      }
  }
}

template <int D, int P>
__global__ void __launch_bounds__(kThreads, P * D <= 64 * 256 ? 2 : 1)
    write_pages_kernel(const WriteArgs a, const FreqTable table, int32_t units, int32_t groups,
                       int32_t layers_per_group, int32_t q_groups, int32_t q_per_group) {
  constexpr int D8 = D / 8;                       // 16-byte chunks of a row
  constexpr int kRows = kThreads / D8;            // rows of one pass
  constexpr int kPasses = P / kRows > 0 ? P / kRows : 1;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ float2 s_cs[];                // [rows written][F]
  __shared__ double s_inv[kMaxFreqs];
  __shared__ int32_t s_plane[kMaxFreqs];
  __shared__ uint32_t s_max[2][kWarps];
  const int F = a.rot_dim / 2;
  for (int j = threadIdx.x; j < F; j += kThreads) {
    s_inv[j] = table.inv_freq[j];
    s_plane[j] = table.plane[j];
  }
  __syncthreads();

  const int64_t kv_blocks = static_cast<int64_t>(units) * groups;
  if (blockIdx.x >= kv_blocks) {
    rotate_q_items(a, s_inv, s_plane, blockIdx.x - kv_blocks, q_groups, q_per_group);
    return;
  }
  const int32_t unit = blockIdx.x / groups;
  const int l_lo = (blockIdx.x - unit * groups) * layers_per_group;
  const int l_hi = min(a.pool.num_layers, l_lo + layers_per_group);

  // The sequence of this unit: the last b with cu[b] / P + 2 b <= unit.
  int32_t b = 0;
  {
    int32_t hi = a.batch.num_seqs;
    while (hi - b > 1) {
      const int32_t mid = (b + hi) >> 1;
      if (__ldg(a.batch.cu + mid) / P + 2 * static_cast<int64_t>(mid) <= unit)
        b = mid;
      else
        hi = mid;
    }
  }
  int64_t t0, t1;
  if (!seq_range(a.batch, b, t0, t1)) {
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, CMR_DEVICE_BAD_CU_SEQLENS);
    return;
  }
  const int64_t p0 = a.batch.pos_offset ? __ldg(a.batch.pos_offset + b) : 0;
  const int64_t end = p0 + (t1 - t0);
  const int64_t i = unit - (t0 / P + 2 * static_cast<int64_t>(b));
  if (i == 0 && p0 < 0 && end > p0 && threadIdx.x == 0 && a.status != nullptr)
    atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
  const int64_t j = (p0 > 0 ? p0 : 0) / P + i;
  const int64_t first = max(max(p0, static_cast<int64_t>(0)), j * P);
  const int64_t last = min(end, (j + 1) * P);
  if (first >= last) return;
  const int32_t id = page_id(a.table, a.pool.num_pages, table_row(a.table, b), j);
  if (id < 0) {
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
    return;
  }
  const int row0 = static_cast<int>(first - j * P);  // rows the page held before
  const int n = static_cast<int>(last - first);      // rows to write
  const int64_t tok = t0 + (first - p0);
  for (int m = threadIdx.x; m < n * F; m += kThreads) {
    const int r = m / F, f = m - r * F;
    s_cs[m] = cos_sin_of(a, b, first + r, s_plane[f], s_inv[f]);
  }
  __syncthreads();

  const int lane = threadIdx.x & 31;
  const int c = threadIdx.x % D8, r0 = threadIdx.x / D8;
  const int half8 = F / 8;
  const int hk = a.pool.hk;
  const int64_t tok_stride = static_cast<int64_t>(hk) * D;
  const int64_t layer = a.batch.n_tokens * tok_stride;
  const int tiles = (l_hi - l_lo) * hk * 2;
  // tile m: layer l_lo + m / (2 hk), K (even) or V (odd) of head (m / 2) % hk
  auto load = [&](int m, uint4(&x)[kPasses], float& old) {
    const int l = l_lo + m / (2 * hk), h = (m >> 1) % hk;
    const uint16_t* src = (m & 1) ? a.v : a.k;
    const uint4* p = reinterpret_cast<const uint4*>(src + l * layer + tok * tok_stride + h * D) + c;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int r = r0 + k * kRows;
      x[k] = make_uint4(0, 0, 0, 0);
      if (r < n) x[k] = __ldcs(p + r * (tok_stride / 8));
    }
    old = row0 > 0 ? __ldcg(((m & 1) ? a.pool.vs : a.pool.ks) + unit_index(a.pool, l, id, h)) : 0.f;
  };

  uint4 x[kPasses], next[kPasses];
  float old, next_old = 0.f;
  load(0, x, old);
  for (int m = 0; m < tiles; ++m) {
    if (m + 1 < tiles) load(m + 1, next, next_old);
    if ((m & 1) == 0) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = r0 + k * kRows;  // rows of zeros turn to zeros
        x[k] = rotate_chunk(x[k], lane, c, half8, s_cs + (r < n ? r : 0) * F);
      }
    }
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) mx = magnitudes(mx, x[k]);
    mx = __reduce_max_sync(~0u, halves_max(mx));
    if (lane == 0) s_max[m & 1][threadIdx.x / 32] = mx;
    __syncthreads();  // the next tile's maxima go to the other half
    uint32_t bits = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) bits = max(bits, s_max[m & 1][w]);
    const bool odd_values = bits >= 0x7f80u;  // an infinity or a NaN
    if (odd_values) {
      mx = 0;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) mx = finite_magnitudes(mx, x[k]);
      mx = __reduce_max_sync(~0u, halves_max(mx));
      __syncthreads();
      if (lane == 0) s_max[m & 1][threadIdx.x / 32] = mx;
      __syncthreads();
      bits = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) bits = max(bits, s_max[m & 1][w]);
    }
    const int l = l_lo + m / (2 * hk), h = (m >> 1) % hk;
    const int64_t at = unit_index(a.pool, l, id, h);
    float ratio;
    const float s = page_scale(scale_exp(bits), row0 > 0, old, &ratio, a.status);
    const float inv = 1.f / s;
    uint8_t* page = ((m & 1) ? a.pool.v : a.pool.k) + at * (P * D);
    uint2* dst = reinterpret_cast<uint2*>(page + row0 * D) + c;
    if (!odd_values) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = r0 + k * kRows;
        if (r < n) __stcs(dst + r * D8, encode8<false>(x[k], inv));
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = r0 + k * kRows;
        if (r < n) __stcs(dst + r * D8, encode8<true>(x[k], inv));
      }
    }
    if (ratio != 1.f) {
      uint32_t* held = reinterpret_cast<uint32_t*>(page);
      for (int k = threadIdx.x; k < row0 * (D / 4); k += kThreads)
        held[k] = rescale4(held[k], ratio);
    }
    if (threadIdx.x == 0) ((m & 1) ? a.pool.vs : a.pool.ks)[at] = s;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) x[k] = next[k];
    old = next_old;
  }
}

constexpr int kStepThreads = 128;
constexpr int kStepWarps = kStepThreads / 32;

// One token per sequence: a warp per (sequence, layer, KV head), which writes the K
// and the V row, and a warp per (sequence, layer) for Q's rows.
template <int D>
__global__ void __launch_bounds__(kStepThreads)
    write_step_kernel(const WriteArgs a, const FreqTable table) {
  constexpr int D8 = D / 8;
  __shared__ float2 s_cs[kStepWarps][kMaxFreqs];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int F = a.rot_dim / 2, U = F / 8;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kStepWarps + warp;
  const int64_t B = a.batch.num_seqs;
  const int L = a.pool.num_layers, hk = a.pool.hk;
  const int64_t n_kv = B * L * hk;
  const bool is_q = item >= n_kv;
  const int64_t w = is_q ? item - n_kv : item;
  if (is_q && (a.hq == 0 || w >= B * L)) return;
  const int64_t rows = w / B;  // layer (Q), or layer x head
  const int32_t b = static_cast<int32_t>(w - rows * B);
  const int64_t p = a.batch.pos_offset ? __ldg(a.batch.pos_offset + b) : 0;

  // the loads that need no position go out before cos/sin are computed
  const int l = static_cast<int>(is_q ? rows : rows / hk);
  const int h = static_cast<int>(rows - static_cast<int64_t>(l) * hk);  // KV items
  const int64_t kv_at = ((l * B + b) * hk + h) * D;
  uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
  if (!is_q && lane < D8) {
    xk = __ldcs(reinterpret_cast<const uint4*>(a.k + kv_at) + lane);
    xv = __ldcs(reinterpret_cast<const uint4*>(a.v + kv_at) + lane);
  }
  for (int f = lane; f < F; f += 32)
    s_cs[warp][f] = cos_sin_of(a, b, p, table.plane[f], table.inv_freq[f]);
  __syncwarp();

  if (is_q) {
    for (int m = lane; m < a.hq * U; m += 32) {
      const int head = m / U, u = m - head * U;
      uint4* q = reinterpret_cast<uint4*>(a.q + ((l * B + b) * a.hq + head) * D + 8 * u);
      uint4 x1 = __ldcs(q), x2 = __ldcs(q + U);
      float c[8], s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = s_cs[warp][8 * u + e].x;
        s[e] = s_cs[warp][8 * u + e].y;
      }
      rotate_unit(x1, x2, c, s);
      __stcs(q, x1);
      __stcs(q + U, x2);
    }
    return;
  }

  const int32_t id = p < 0 ? -1
                           : page_id(a.table, a.pool.num_pages, table_row(a.table, b),
                                     p >> a.pool.page_shift);
  if (id < 0) {
    if (lane == 0 && a.status != nullptr) atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
    return;
  }
  const int P = 1 << a.pool.page_shift;
  const int row0 = static_cast<int>(p) & (P - 1);
  const int64_t at = unit_index(a.pool, l, id, h);
  const float old_k = row0 > 0 ? __ldcg(a.pool.ks + at) : 0.f;
  const float old_v = row0 > 0 ? __ldcg(a.pool.vs + at) : 0.f;
  xk = rotate_chunk(xk, lane, lane, U, s_cs[warp]);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint4 x = which ? xv : xk;
    uint32_t bits = __reduce_max_sync(~0u, halves_max(magnitudes(0u, x)));
    if (bits >= 0x7f80u)
      bits = __reduce_max_sync(~0u, halves_max(finite_magnitudes(0u, x)));
    float ratio;
    const float s = page_scale(scale_exp(bits), row0 > 0, which ? old_v : old_k, &ratio, a.status);
    uint8_t* page = (which ? a.pool.v : a.pool.k) + at * (P * D);
    if (lane < D8)
      reinterpret_cast<uint2*>(page + row0 * D)[lane] = encode8<true>(x, 1.f / s);
    if (ratio != 1.f) {
      uint32_t* held = reinterpret_cast<uint32_t*>(page);
#pragma unroll 4
      for (int k = lane; k < row0 * (D / 4); k += 32) held[k] = rescale4(held[k], ratio);
    }
    if (lane == 0) (which ? a.pool.vs : a.pool.ks)[at] = s;
  }
}

template <int D, int P>
cudaError_t launch_pages(const WriteArgs& a, const FreqTable& table, cudaStream_t stream) {
  const int F = a.rot_dim / 2;
  const int64_t N = a.batch.n_tokens;
  const int64_t units = N / P + 2 * static_cast<int64_t>(a.batch.num_seqs);
  const size_t smem = static_cast<size_t>(P) * F * sizeof(float2);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(write_pages_kernel<D, P>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int L = a.pool.num_layers;
  const int groups = L;  // one layer to a CTA
  int32_t q_groups = 0, q_per = 1;
  int64_t q_blocks = 0;
  if (a.hq > 0) {
    // a token's (layer, head) rows are split while there are too few threads for
    // two waves of the device
    const int64_t rows = static_cast<int64_t>(a.hq) * L;
    const int64_t per_cta = kThreads / (F / 8);
    const int64_t want = (2 * static_cast<int64_t>(sm_count()) * 4 * per_cta + N - 1) / N;
    const int64_t g = want < 1 ? 1 : (want > rows ? rows : want);
    q_per = static_cast<int32_t>((rows + g - 1) / g);
    q_groups = static_cast<int32_t>((rows + q_per - 1) / q_per);
    q_blocks = (N * q_groups + per_cta - 1) / per_cta;
  }
  const int64_t blocks = units * groups + q_blocks;
  if (units > INT32_MAX || blocks > INT32_MAX) return cudaErrorInvalidValue;
  write_pages_kernel<D, P><<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(
      a, table, static_cast<int32_t>(units), groups, (L + groups - 1) / groups, q_groups, q_per);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_pages_d(const WriteArgs& a, const FreqTable& table, cudaStream_t stream) {
  switch (a.pool.page_shift) {
    case 4: return launch_pages<D, 16>(a, table, stream);
    case 5: return launch_pages<D, 32>(a, table, stream);
    case 6: return launch_pages<D, 64>(a, table, stream);
    default: return launch_pages<D, 128>(a, table, stream);
  }
}

template <int D>
cudaError_t launch_step(const WriteArgs& a, const FreqTable& table, cudaStream_t stream) {
  const int64_t B = a.batch.num_seqs, L = a.pool.num_layers;
  const int64_t items = B * L * a.pool.hk + (a.hq > 0 ? B * L : 0);
  const int64_t blocks = (items + kStepWarps - 1) / kStepWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  write_step_kernel<D><<<static_cast<unsigned>(blocks), kStepThreads, 0, stream>>>(a, table);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_write(const WriteArgs& a, const FreqTable& table, cudaStream_t stream) {
  const bool step = a.batch.cu == nullptr;
  switch (a.pool.head_dim) {
    case 64: return step ? launch_step<64>(a, table, stream) : launch_pages_d<64>(a, table, stream);
    case 128:
      return step ? launch_step<128>(a, table, stream) : launch_pages_d<128>(a, table, stream);
    default:
      return step ? launch_step<256>(a, table, stream) : launch_pages_d<256>(a, table, stream);
  }
}

}  // namespace kv8
}  // namespace cmr

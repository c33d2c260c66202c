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
// write_pages_kernel (prompts and chunks): a CTA takes up to eight of a page's
// (K or V, layer, head) tiles of at most P x D values one after the other.  A
// thread holds a tile's pairs of chunks in registers, all loads of a tile are in
// flight at once, and the other CTAs of the SM (three of 64 x 256) fill the time
// that one spends on its maximum and its codes.  The cos/sin of the page's tokens
// are computed once and kept in shared memory for the CTA's K tiles (with few
// pages a CTA takes fewer tiles, down to one).  A page's tokens and the
// units before it are found from cu_seqlens alone (sequence b's pages start at
// unit cu[b] / P + 2 b, room enough for its first and last partial pages), so no
// list of pages is built.  Q's rows go to the CTAs behind, eight frequencies of
// a token to a thread as in the other rotation kernels.
// write_step_kernel (one token per sequence): a warp per K and V row, since a
// page gets one row and the rest of the work is latency.
// Measured, 6 layers, 8 query and 2 KV heads of 256, pages of 64: 8 prompts of 4096
// 181 us, 86% of a copy's rate; 12 ragged chunks 17 us; a step of 256 sequences 7 us
// and of one 4 us on the device (12 with the host's part of the call).
#include "kv8.cuh"
#include "../pdl.cuh"
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

// The larger of two packed pairs of bf16 magnitudes; a NaN stays.
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t m, uint32_t x) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t magnitudes(uint32_t m, const uint4& x) {
  m = max_magnitudes(m, x.x);
  m = max_magnitudes(m, x.y);
  m = max_magnitudes(m, x.z);
  return max_magnitudes(m, x.w);
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

__device__ __forceinline__ uint4 infs_to_nan(const uint4& x) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7fffu) == 0x7f80u) w[i] |= 0x40u;
    if ((w[i] & 0x7fff0000u) == 0x7f800000u) w[i] |= 0x400000u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight bf16 values over the scale, as codes.
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = f32_to_e4m3x2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Four codes under another scale: code * ratio, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const uint32_t a = e4m3x2_to_f16x2(w & 0xffffu), b = e4m3x2_to_f16x2(w >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return f32_to_e4m3x2(x.x * ratio, x.y * ratio) | (f32_to_e4m3x2(y.x * ratio, y.y * ratio) << 16);
}

// n16 chunks of 16 codes under another scale, by threads tid of `threads`, four
// chunks in flight.
__device__ __forceinline__ void rescale_rows(uint8_t* codes, int n16, float ratio, int tid,
                                             int threads) {
  uint4* p = reinterpret_cast<uint4*>(codes);
  for (int k0 = tid; k0 < n16; k0 += 4 * threads) {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i * threads < n16) x[i] = p[k0 + i * threads];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i * threads < n16)
        p[k0 + i * threads] = make_uint4(rescale4(x[i].x, ratio), rescale4(x[i].y, ratio),
                                         rescale4(x[i].z, ratio), rescale4(x[i].w, ratio));
  }
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

__device__ __forceinline__ Planes planes_of(const WriteArgs& a, int32_t b, int64_t p) {
  return canvas_row(p, __ldg(a.start + b), __ldg(a.amount + b));
}

__device__ __forceinline__ float2 cos_sin_of(const Planes& r, int plane, double inv) {
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
  const Planes at = planes_of(a, b, p);
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 f = cos_sin_of(at, s_plane[8 * u + e], s_inv[8 * u + e]);
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

// Where a CTA's tiles are read and written.
struct PageWork {
  const uint16_t* src;  // K or V at the page's first new token, layer 0, head 0
  uint8_t* codes;       // the pool
  float* scales;
  int32_t id, row0, n;  // page, rows it held before, rows to write
  int64_t tok_stride, layer;  // elements
  const float2* cs;     // [n][F] (keys)
};

// Tiles [lo, hi) of K (or of V), a tile being layer t / hk and head t % hk.  A thread
// holds pairs of 16-byte chunks.  Those that rotation pairs, U = rot_dim / 16 of each
// row, come first for all rows, so that whole warps rotate or do not; the others are
// chunks (2 U + c, 2 U + c + left), c < left.  kFull: the whole page is written.
template <int D, int P, bool kKey, bool kFull>
__device__ __forceinline__ void write_tiles(const WriteArgs& a, const PageWork& w, int lo, int hi,
                                            uint32_t (*s_max)[kThreads / 32]) {
  constexpr int kHalf = D / 16;
  constexpr int kPairs = P * kHalf / kThreads > 0 ? P * kHalf / kThreads : 1;
  constexpr int kWarps = kThreads / 32;
  constexpr bool kAll = kFull && P * kHalf >= kThreads;  // every thread has all its pairs
  const int lane = threadIdx.x & 31;
  const int hk = a.pool.hk;
  const int F = a.rot_dim / 2;
  const int U = kKey ? F / 8 : 0, left = kHalf - U;
  const int turned = w.n * U;  // rotated pairs
  int from[kPairs];            // element offset of the first chunk, -1: no pair
  uint32_t to[kPairs];         // byte offset in the page
  int cs[kPairs];              // of the pair's cos/sin
  if constexpr (kKey) {
    const int reciprocal = left > 0 ? ((1 << 20) + left - 1) / left : 0;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int idx = threadIdx.x + k * kThreads, rest = idx - turned;
      // rest < 2,048 and left <= 16: the product is below 2^31 and the quotient exact
      const int r = idx < turned ? idx / max(U, 1) : (rest * reciprocal) >> 20;
      const int c = idx < turned ? idx - r * U : 2 * U + rest - r * left;
      from[k] = kAll || idx < w.n * kHalf ? static_cast<int>(r * w.tok_stride) + 8 * c : -1;
      to[k] = (w.row0 + r) * D + 8 * c;
      cs[k] = r * F + 8 * c;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int idx = threadIdx.x + k * kThreads, r = idx / kHalf, c = idx % kHalf;
      from[k] = kAll || r < w.n ? static_cast<int>(r * w.tok_stride) + 8 * c : -1;
      to[k] = (w.row0 + r) * D + 8 * c;
      cs[k] = 0;
    }
  }
  const bool held = w.row0 > 0;
  for (int m = lo; m < hi; ++m) {
    const int l = m / hk, h = m - l * hk;
    const uint16_t* src = w.src + l * w.layer + h * D;
    const int64_t at = unit_index(a.pool, l, w.id, h);
    const float old = held ? __ldcg(w.scales + at) : 0.f;
    uint4 x[kPairs][2];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int apart = kKey && threadIdx.x + k * kThreads < turned ? U : left;
      if (kAll || from[k] >= 0) {
        const uint4* p = reinterpret_cast<const uint4*>(src + from[k]);
        x[k][0] = __ldcs(p);
        x[k][1] = __ldcs(p + apart);
      } else {
        x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
      }
    }
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      if (kKey && threadIdx.x + k * kThreads < turned) {
        const float4* f = reinterpret_cast<const float4*>(w.cs + cs[k]);
        float c[8], s[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 y = f[e];
          c[2 * e] = y.x;
          s[2 * e] = y.y;
          c[2 * e + 1] = y.z;
          s[2 * e + 1] = y.w;
        }
        rotate_unit(x[k][0], x[k][1], c, s);
      }
      mx = magnitudes(magnitudes(mx, x[k][0]), x[k][1]);
    }
    mx = __reduce_max_sync(~0u, halves_max(mx));
    if (lane == 0) s_max[m & 1][threadIdx.x / 32] = mx;
    __syncthreads();  // the next tile's maxima go to the other half
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) bits = max(bits, s_max[m & 1][i]);
    const bool odd_values = bits >= 0x7f80u;  // an infinity or a NaN
    if (odd_values) {
      mx = 0;
#pragma unroll
      for (int k = 0; k < kPairs; ++k)
        mx = finite_magnitudes(finite_magnitudes(mx, x[k][0]), x[k][1]);
      mx = __reduce_max_sync(~0u, halves_max(mx));
      __syncthreads();
      if (lane == 0) s_max[m & 1][threadIdx.x / 32] = mx;
      __syncthreads();
      bits = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) bits = max(bits, s_max[m & 1][i]);
    }
    float ratio;
    const float s = page_scale(scale_exp(bits), held, old, &ratio, a.status);
    const float inv = 1.f / s;
    uint8_t* page = w.codes + at * (P * D);
    if (odd_values) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        x[k][0] = infs_to_nan(x[k][0]);
        x[k][1] = infs_to_nan(x[k][1]);
      }
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int apart = kKey && threadIdx.x + k * kThreads < turned ? U : left;
      if (kAll || from[k] >= 0) {
        uint2* dst = reinterpret_cast<uint2*>(page + to[k]);
        __stcs(dst, encode8(x[k][0], inv));
        __stcs(dst + apart, encode8(x[k][1], inv));
      }
    }
    if (ratio != 1.f) rescale_rows(page, w.row0 * (D / 16), ratio, threadIdx.x, kThreads);
    if (threadIdx.x == 0) w.scales[at] = s;
  }
}

template <int D, int P, bool kKey>
__device__ __forceinline__ void write_tiles(const WriteArgs& a, const PageWork& w, int lo, int hi,
                                            uint32_t (*s_max)[kThreads / 32]) {
  if (w.n == P)
    write_tiles<D, P, kKey, true>(a, w, lo, hi, s_max);
  else
    write_tiles<D, P, kKey, false>(a, w, lo, hi, s_max);
}

// Tiles of a page: its K, then its V, each layer by layer, head by head.
template <int D, int P>
__global__ void __launch_bounds__(kThreads, P * D <= 64 * 256 ? 3 : 2)
    write_pages_kernel(const WriteArgs a, const FreqTable table, int32_t units, int32_t groups,
                       int32_t tiles_per_group, int32_t q_groups, int32_t q_per_group) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ float4 s_cs4[];               // [rows written][F] of (cos, sin)
  __shared__ double s_inv[kMaxFreqs];
  __shared__ int32_t s_plane[kMaxFreqs];
  __shared__ uint32_t s_max[2][kWarps];
  __shared__ Planes s_at[P];                      // of the rows written
  float2* s_cs = reinterpret_cast<float2*>(s_cs4);
  const int F = a.rot_dim / 2;
  for (int j = threadIdx.x; j < F; j += kThreads) {
    s_inv[j] = table.inv_freq[j];
    s_plane[j] = table.plane[j];
  }
  __syncthreads();
  pdl::wait();
  pdl::launch_dependents();

  const int64_t kv_blocks = static_cast<int64_t>(units) * groups;
  if (blockIdx.x >= kv_blocks) {
    rotate_q_items(a, s_inv, s_plane, blockIdx.x - kv_blocks, q_groups, q_per_group);
    return;
  }
  const int32_t unit = blockIdx.x / groups;
  const int hk = a.pool.hk;
  const int k_tiles = a.pool.num_layers * hk;
  const int m_lo = (blockIdx.x - unit * groups) * tiles_per_group;
  const int m_hi = min(2 * k_tiles, m_lo + tiles_per_group);

  // The sequence of this unit: the last b with cu[b] / P + 2 b <= unit.
  const int32_t b = last_true(a.batch.num_seqs, [&](int32_t i) {
    return __ldg(a.batch.cu + i) / P + 2 * static_cast<int64_t>(i) <= unit;
  });
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
  if (m_lo < k_tiles) {
    for (int r = threadIdx.x; r < n; r += kThreads) s_at[r] = planes_of(a, b, first + r);
    __syncthreads();
    for (int m = threadIdx.x; m < n * F; m += kThreads) {
      const int r = m / F, f = m - r * F;
      s_cs[m] = cos_sin_of(s_at[r], s_plane[f], s_inv[f]);
    }
    __syncthreads();
  }

  PageWork w;
  w.tok_stride = static_cast<int64_t>(hk) * D;
  w.layer = a.batch.n_tokens * w.tok_stride;
  w.id = id;
  w.row0 = row0;
  w.n = n;
  w.cs = s_cs;
  if (m_lo < k_tiles) {
    w.src = a.k + tok * w.tok_stride;
    w.codes = a.pool.k;
    w.scales = a.pool.ks;
    write_tiles<D, P, true>(a, w, m_lo, min(m_hi, k_tiles), s_max);
    __syncthreads();  // the maxima of the last tile have been read
  }
  if (m_hi > k_tiles) {
    w.src = a.v + tok * w.tok_stride;
    w.codes = a.pool.v;
    w.scales = a.pool.vs;
    write_tiles<D, P, false>(a, w, max(m_lo, k_tiles) - k_tiles, m_hi - k_tiles, s_max);
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
  pdl::wait();
  pdl::launch_dependents();
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
  const Planes planes = planes_of(a, b, p);
  for (int f = lane; f < F; f += 32)
    s_cs[warp][f] = cos_sin_of(planes, table.plane[f], table.inv_freq[f]);
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
      reinterpret_cast<uint2*>(page + row0 * D)[lane] = encode8(infs_to_nan(x), 1.f / s);
    if (ratio != 1.f) rescale_rows(page, row0 * (D / 16), ratio, lane, 32);
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
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void*>(write_pages_kernel<D, P>),
                   static_cast<int>(P * (D / 2) * sizeof(float2)), &done);
    if (e != cudaSuccess) return e;
  }
  const int L = a.pool.num_layers;
  // Up to eight tiles to a CTA, whose K tiles share their cos/sin, while that leaves
  // two waves of CTAs; one tile each when there are few pages.
  const int tiles = 2 * L * a.pool.hk;
  const int64_t wanted = 2 * 4 * static_cast<int64_t>(sm_count());
  int per = 8;
  while (per > 1 && units * ((tiles + per - 1) / per) < wanted) per /= 2;
  const int groups = (tiles + per - 1) / per;
  int32_t q_groups = 0, q_per = 1;
  int64_t q_blocks = 0;
  if (a.hq > 0) {
    // a token's (layer, head) rows are split while there are too few threads for
    // two waves of the device, but eight share a cos/sin, which costs as much as
    // ten rotated rows
    const int64_t rows = static_cast<int64_t>(a.hq) * L;
    const int64_t per_cta = kThreads / (F / 8);
    const int64_t want = (2 * static_cast<int64_t>(sm_count()) * 4 * per_cta + N - 1) / N;
    const int64_t most = (rows + 7) / 8;
    const int64_t g = want < 1 ? 1 : (want > most ? most : want);
    q_per = static_cast<int32_t>((rows + g - 1) / g);
    q_groups = static_cast<int32_t>((rows + q_per - 1) / q_per);
    q_blocks = (N * q_groups + per_cta - 1) / per_cta;
  }
  const int64_t blocks = units * groups + q_blocks;
  if (units > INT32_MAX || blocks > INT32_MAX) return cudaErrorInvalidValue;
  return pdl::launch(write_pages_kernel<D, P>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                     smem, stream, true, a, table, static_cast<int32_t>(units), groups, per,
                     q_groups, q_per);
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
  return pdl::launch(write_step_kernel<D>, dim3(static_cast<unsigned>(blocks)),
                     dim3(kStepThreads), 0, stream, true, a, table);
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

// Attention over the paged 8-bit cache for calls with few query rows per
// sequence: decode steps and short chunks.
//
// With a page's scales 2^a (keys) and 2^e (values) and codes k, v in e4m3,
//   out = sum_i p_i v_i / sum_i p_i 2^-e_i,   p_i = 2^(c 2^a_i (q . k_i) + e_i - r),
// c = softmax scale * log2(e) and r a running maximum of the exponent: the value
// scale enters the weight, so codes are never multiplied by a scale, and a page
// of large values cannot push the weights of the others out of range.  e4m3
// codes are exact in f16; q is brought to f16 exactly by a power of two per row
// (bits below 2^-24 of the row's largest value are lost), p is rounded to f16
// (at most 2^-11 relative, unbiased, against the 2^-9 of the bf16 result), and all
// sums, maxima and the accumulator are fp32.
//
// Bound by reading the cache once (1 byte per value).  The rows of a KV head's
// query group, 8 or 16 of them, share each key and value that is read.  The work
// is the list of 64-token tiles of all (layer, KV head, sequence, row tile) items,
// cut into equal runs, one per resident CTA, so that sequences of any lengths
// load the device evenly; a CTA keeps the running maximum and sum for the item
// at hand, writes items that lie in its run whole, and leaves a partial result
// of those that do not (at most two) in the workspace, which a second kernel
// joins.  No atomics: the same call gives the same bits.
// In a CTA a producer warp keeps a ring of tiles in flight with bulk copies, and
// four warps take 16 tokens of a tile each: S^T = K Q^T with the tokens as the
// rows of mma.m16n8k16, whose fragments are then consecutive bytes of a key, and
// O^T += V^T P^T, whose fragments are bytes of two tokens woven together by prmt.
// The tensor work is a few percent of the time, so tcgen05 would gain nothing.
#include "kv8.cuh"
#include "attend.cuh"
#include "../pdl.cuh"
#include "../rotate_common.cuh"
#include "../tma.cuh"

namespace cmr {
namespace kv8 {
namespace {

using rot::bf16_hi;
using rot::bf16_lo;
using rot::pack_bf16x2;

constexpr int kTile = 64;       // tokens of a tile
constexpr int kWarps = 4;       // consumer warps, 16 tokens of a tile each
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kMaxSplitItems = 2048;  // items per (layer, head) that are split evenly
constexpr int kMaxCtas = 1024;        // of the split form
constexpr float kLazy = 8.f;    // the reference moves once weights pass 2^8

struct StageInfo {
  float k_scale[4];    // per 16 tokens
  float v_log2[4];     // log2 of the value scale
  float v_inv[4];      // 1 / value scale
  uint32_t valid;      // bit g: tokens [16g, 16g + 16) have a page
};

template <int D, int NQ>
struct Smem {
  static constexpr int R = 8 * NQ;
  static constexpr int kStages = NQ == 1 ? 3 : 2;
  static constexpr int kStage = 2 * kTile * D;
  static constexpr int kQ = kStages * kStage;                      // f16 fragments of Q
  static constexpr int kO = kQ + (D / 16) * NQ * 32 * 8;           // [R][D + 4] floats
  static constexpr int kNan = kO + R * (D + 4) * 4;                // [D] ints
  static constexpr int kRow = kNan + D * 4;                        // per row: see below
  static constexpr int kInfo = kRow + 4 * (2 * R + 2 * kWarps * R);
  static constexpr int kBars = (kInfo + kStages * static_cast<int>(sizeof(StageInfo)) + 7) / 8 * 8;
  static constexpr int kPrefix = (kBars + 16 * kStages + 15) / 16 * 16;  // [items + 1] ints
};

struct RowsArgs {
  AttendArgs a;
  int32_t items;       // row-tile slots per (layer, head): NB
  int32_t ctas;        // CTAs of the split form; 0: one CTA per item
  float* partial;      // [ctas][2][R][D + 2]
  int32_t* prefix;     // [NB + 1], written by CTA 0 for the joining kernel
};

__device__ __forceinline__ int32_t item_tiles(const Item& it) {
  if (it.rows == 0) return 0;
  return max(1, static_cast<int32_t>((it.vis_last + kTile - 1) / kTile));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// The run of tiles [lo, hi) of this CTA, and the walk over the items in it.
struct Run {
  int64_t lo, hi;
  int32_t total;  // tiles per (layer, head)
};

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? 2 : 1) attend_rows_kernel(const RowsArgs ra) {
  using S = Smem<D, NQ>;
  constexpr int R = S::R;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const AttendArgs& a = ra.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  uint2* s_q = reinterpret_cast<uint2*>(smem + S::kQ);
  float* s_o = reinterpret_cast<float*>(smem + S::kO);
  int* s_nan = reinterpret_cast<int*>(smem + S::kNan);
  float* s_mult = reinterpret_cast<float*>(smem + S::kRow);        // [R] score to log2 weight
  int* s_vis = reinterpret_cast<int*>(s_mult + R);                 // [R] tokens seen
  float* s_ref = reinterpret_cast<float*>(s_vis + R);              // [warps][R]
  float* s_sum = s_ref + kWarps * R;                               // [warps][R]
  StageInfo* s_info = reinterpret_cast<StageInfo*>(smem + S::kInfo);
  int* s_prefix = reinterpret_cast<int*>(smem + S::kPrefix);
  const uint32_t stage0 = tma::smem_addr(smem);
  const uint32_t full0 = tma::smem_addr(smem + S::kBars);
  const uint32_t empty0 = full0 + 8 * NS;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      tma::mbar_init(full0 + 8 * s, 1);
      tma::mbar_init(empty0 + 8 * s, kWarps);
    }
    tma::mbar_init_fence();
  }
  bool bad = false;
  const int NB = ra.items;
  Run run;
  int32_t only = -1;  // the item of a CTA that has one
  int64_t item0 = 0;  // (layer, head) of it
  if (ra.ctas > 0) {
    for (int i = tid; i < NB; i += kThreads) {
      const Item it = find_item<R>(a, i, &bad);
      s_prefix[i] = item_tiles(it);
      if (blockIdx.x == 0 && it.rows > 0 && it.cut && a.status != nullptr)
        atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
    }
    if (bad && blockIdx.x == 0 && a.status != nullptr)
      atomicOr(a.status, CMR_DEVICE_BAD_CU_SEQLENS);
    __syncthreads();
    if (warp == 0) {  // exclusive scan in place
      int carry = 0;
      for (int i0 = 0; i0 < NB; i0 += 32) {
        const int i = i0 + lane;
        const int v = i < NB ? s_prefix[i] : 0;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(~0u, x, o);
          if (lane >= o) x += y;
        }
        if (i < NB) s_prefix[i] = carry + x - v;
        carry += __shfl_sync(~0u, x, 31);
      }
      if (lane == 0) s_prefix[NB] = carry;
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = tid; i <= NB; i += kThreads) ra.prefix[i] = s_prefix[i];
    run.total = s_prefix[NB];
    const int64_t all = static_cast<int64_t>(run.total) * a.pool.num_layers * a.pool.hk;
    const int64_t per = (all + ra.ctas - 1) / ra.ctas;
    run.lo = min(all, blockIdx.x * per);
    run.hi = min(all, run.lo + per);
  } else {
    only = blockIdx.x;
    item0 = blockIdx.y;
    const Item it = find_item<R>(a, only, &bad);
    if (tid == 0 && a.status != nullptr && item0 == 0) {
      if (bad) atomicOr(a.status, CMR_DEVICE_BAD_CU_SEQLENS);
      if (it.rows > 0 && it.cut) atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
    }
    run.total = item_tiles(it);
    run.lo = 0;
    run.hi = run.total;
    __syncthreads();
  }
  pdl::launch_dependents();

  // The segment of the run that starts at tile w: its (layer, head), item, first
  // tile and tile count, and whether it is the whole item.
  auto segment = [&](int64_t w, int64_t& lh, int32_t& bi, int32_t& t0, int32_t& nt, bool& whole) {
    if (only >= 0) {
      lh = item0;
      bi = only;
      t0 = 0;
      nt = run.total;
      whole = true;
      return;
    }
    lh = w / run.total;
    const int32_t r = static_cast<int32_t>(w - lh * run.total);
    int32_t lo = 0, hi = NB;
    while (hi - lo > 1) {  // the last item that starts at or before r
      const int32_t mid = (lo + hi) >> 1;
      if (s_prefix[mid] <= r)
        lo = mid;
      else
        hi = mid;
    }
    bi = lo;
    t0 = r - s_prefix[lo];
    const int32_t left = s_prefix[lo + 1] - r;
    nt = static_cast<int32_t>(min(static_cast<int64_t>(left), run.hi - w));
    whole = t0 == 0 && nt == left;
  };

  const int P = 1 << a.pool.page_shift;
  if (warp == kWarps) {
    // ---- producer: lane 4 i + g looks after tokens [16g, 16g + 16) of tile i of
    // a batch of eight tiles
    int stage = 0, phase = 0, issued = 0;
    bool dead = false;
    uint32_t problems = 0;
    for (int64_t w = run.lo; w < run.hi && !dead;) {
      int64_t lh;
      int32_t bi, t0, nt;
      bool whole;
      segment(w, lh, bi, t0, nt, whole);
      w += nt;
      bool ignored = false;
      const Item it = find_item<R>(a, bi, &ignored);
      const int l = static_cast<int>(lh / a.pool.hk), h = static_cast<int>(lh - l * a.pool.hk);
      const int g = lane & 3;
      for (int tb = 0; tb < nt && !dead; tb += 8) {
        const int tile = tb + (lane >> 2);
        const int64_t tok = static_cast<int64_t>(t0 + tile) * kTile + 16 * g;
        int32_t id = -1;
        float ks = 0.f, vs = 1.f;
        int64_t unit = 0;
        const bool wanted = tile < nt && tok < it.vis_last;
        if (wanted) {
          id = page_id(a.table, a.pool.num_pages, it.row, tok >> a.pool.page_shift);
          if (id >= 0) {
            unit = (static_cast<int64_t>(l) * a.pool.num_pages + id) * a.pool.hk + h;
            ks = __ldg(a.pool.ks + unit);
            vs = __ldg(a.pool.vs + unit);
            if (!scale_ok(ks) || !scale_ok(vs)) {
              problems |= CMR_DEVICE_BAD_SCALE;
              id = -1;
              vs = 1.f;
            }
          } else {
            problems |= CMR_DEVICE_CACHE_RANGE;
          }
        }
        const uint32_t valid = __ballot_sync(~0u, id >= 0);
        // the lane that copies for a page (or for 64 tokens of a larger one) takes
        // the rows up to the last one seen, in whole groups of 16
        const int span = min(P, kTile);
        int rows = 0;
        if (id >= 0 && (16 * g) % span == 0) {
          const int64_t left = it.vis_last - tok;
          rows = static_cast<int>(min(static_cast<int64_t>(span), (left + 15) / 16 * 16));
        }
        int quad_rows = rows + __shfl_xor_sync(~0u, rows, 1);
        quad_rows += __shfl_xor_sync(~0u, quad_rows, 2);
        const int tiles = min(8, nt - tb);
        for (int i = 0; i < tiles; ++i) {
          if (issued >= NS && !tma::mbar_wait(empty0 + 8 * stage, phase ^ 1)) dead = true;
          dead = __any_sync(~0u, dead);
          if (dead) break;
          if ((lane >> 2) == i) {
            StageInfo& info = s_info[stage];
            info.k_scale[g] = ks;
            info.v_log2[g] = __log2f(vs);
            info.v_inv[g] = 1.f / vs;
            if (g == 0) info.valid = (valid >> (4 * i)) & 15u;
          }
          __syncwarp();
          const uint32_t bar = full0 + 8 * stage;
          if (lane == 4 * i) tma::mbar_arrive_expect_tx(bar, 2u * quad_rows * D);
          __syncwarp();
          if ((lane >> 2) == i && rows > 0) {
            const int64_t src = unit * (static_cast<int64_t>(P) * D) + (tok & (P - 1)) * D;
            const uint32_t dst = stage0 + stage * S::kStage + 16 * g * D;
            bulk_load(dst, a.pool.k + src, rows * D, bar);
            bulk_load(dst + kTile * D, a.pool.v + src, rows * D, bar);
          }
          ++issued;
          if (++stage == NS) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    // no copy is left in flight when the CTA ends
    const int last = min(issued, NS);
    for (int i = 0; i < last; ++i) {
      const int n = issued - 1 - i;
      if (!tma::mbar_wait(full0 + 8 * (n % NS), (n / NS) & 1)) dead = true;
    }
    if (a.status != nullptr) {
      if (problems) atomicOr(a.status, static_cast<int>(problems));
      if (dead && lane == 0) atomicOr(a.status, CMR_DEVICE_WAIT_TIMEOUT);
    }
    return;
  }

  // ---- consumers
  const int g = lane >> 2, t = lane & 3;
  int stage = 0, phase = 0;
  bool dead = false;
  for (int64_t w = run.lo; w < run.hi;) {
    int64_t lh;
    int32_t bi, t0, nt;
    bool whole;
    segment(w, lh, bi, t0, nt, whole);
    const bool at_start = w == run.lo;
    w += nt;
    bool ignored = false;
    const Item it = find_item<R>(a, bi, &ignored);
    const int l = static_cast<int>(lh / a.pool.hk), h = static_cast<int>(lh - l * a.pool.hk);
    const int vis_first = static_cast<int>(it.vis_first), vis_last = static_cast<int>(it.vis_last);
    auto row_at = [&](int r) {  // element offset of query row r of the item
      const int f = it.first_row + r;
      const int64_t tok = it.tok + f / a.group;
      const int head = h * a.group + f % a.group;
      return ((l * a.batch.n_tokens + tok) * a.hq + head) * D;
    };

    // Q to f16, each row over a power of two, in the order of the B fragments
    {
      constexpr int kPer = kConsumers / R;       // threads of a row
      constexpr int kChunks = D / 8 / kPer;      // 16-byte chunks of a thread (>= 1)
      constexpr int kHave = kChunks > 0 ? kChunks : 1;
      const int r = tid / kPer, c0 = tid % kPer;
      uint4 x[kHave];
      uint32_t mx = 0;
#pragma unroll
      for (int k = 0; k < kHave; ++k) {
        x[k] = make_uint4(0, 0, 0, 0);
        const int c = c0 + k * kPer;
        if (r < it.rows && c < D / 8)
          x[k] = __ldg(reinterpret_cast<const uint4*>(a.q + row_at(r)) + c);
        const uint32_t ww[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = __vmaxs2(mx, ww[i] & 0x7fff7fffu);
      }
      mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
      for (int o = kPer / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(~0u, mx, o));
      const bool finite = mx < 0x7f80u;
      int e = static_cast<int>(mx >> 7) - 127;
      e = mx == 0 ? 0 : max(-126, min(e, 126));
      const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int k = 0; k < kHave; ++k) {
        const int c = c0 + k * kPer;
        if (c < D / 8) {
          const uint32_t ww[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = finite ? pack_f16x2(bf16_lo(ww[i]) * inv, bf16_hi(ww[i]) * inv) : 0x7fff7fffu;
          const int d = 8 * c;
          const int m = d / 64 * 4 + (d % 16) / 4, tt = (d % 64) / 16;
          const int nq = r / 8, gq = r % 8;
          s_q[(m * NQ + nq) * 32 + gq * 4 + tt] = make_uint2(f[0], f[1]);
          s_q[((m + 1) * NQ + nq) * 32 + gq * 4 + tt] = make_uint2(f[2], f[3]);
        }
      }
      if (c0 == 0) {
        s_mult[r] = a.scale_log2 * __int_as_float((127 + e) << 23);
        const int64_t seen = it.p0 + (it.first_row + r) / a.group + 1;
        s_vis[r] = r < it.rows ? static_cast<int>(max(static_cast<int64_t>(0),
                                                      min(seen, it.vis_last)))
                               : 0;
      }
      for (int d = tid; d < D; d += kConsumers) s_nan[d] = 0x7fffffff;
    }
    tma::named_sync(1, kConsumers);

    float o[D / 16][NQ][4];
    float ref[NQ][2], sum[NQ][2], mult[NQ][2];
    int vis[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ref[n][i] = -INFINITY;
        sum[n][i] = 0.f;
        mult[n][i] = s_mult[8 * n + 2 * t + i];
        vis[n][i] = s_vis[8 * n + 2 * t + i];
      }
#pragma unroll
      for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
    }

    for (int tile = 0; tile < nt; ++tile) {
      if (!dead && !tma::mbar_wait(full0 + 8 * stage, phase, tma::kConsumerWaitLimitNs)) dead = true;
      const uint8_t* kt = smem + stage * S::kStage + warp * 16 * D;
      const uint8_t* vt = kt + kTile * D;
      const StageInfo& info = s_info[stage];
      const float k_scale = info.k_scale[warp], v_log2 = info.v_log2[warp];
      const float v_inv = info.v_inv[warp];
      const bool valid = (info.valid >> warp) & 1u;
      const int tok0 = (t0 + tile) * kTile + warp * 16;

      // scores of tokens tok0 + g and + g + 8 against queries 2t, 2t + 1
      float s[NQ][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
      if (valid && tok0 < vis_last) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint4 lo = *reinterpret_cast<const uint4*>(kt + g * D + j * 64 + t * 16);
          const uint4 hi = *reinterpret_cast<const uint4*>(kt + (g + 8) * D + j * 64 + t * 16);
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = e4m3x2_to_f16x2(wl[i] & 0xffffu), a2 = e4m3x2_to_f16x2(wl[i] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(wh[i] & 0xffffu), a3 = e4m3x2_to_f16x2(wh[i] >> 16);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const uint2 q = s_q[((j * 4 + i) * NQ + n) * 32 + lane];
              mma_f16(s[n], a0, a1, a2, a3, q.x, q.y);
            }
          }
        }
      }
      uint32_t pb[NQ][2];
      bool move = false;
      float mx[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = tok0 + g + (i >= 2 ? 8 : 0);
          const float x = fmaf(s[n][i], mult[n][i & 1] * k_scale, v_log2);
          s[n][i] = valid && tok < vis[n][i & 1] ? x : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(s[n][i], s[n][i + 2]);
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 4));
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
          mx[n][i] = m;
          move |= m > ref[n][i] + kLazy;
        }
      }
      if (__any_sync(~0u, move)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float r = fmaxf(ref[n][i], mx[n][i]);
            f[i] = r == -INFINITY ? 1.f : exp2_approx(ref[n][i] - r);
            ref[n][i] = r;
            sum[n][i] *= f[i];
          }
#pragma unroll
          for (int m = 0; m < D / 16; ++m) {
            o[m][n][0] *= f[0];
            o[m][n][1] *= f[1];
            o[m][n][2] *= f[0];
            o[m][n][3] *= f[1];
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float r = ref[n][i & 1] == -INFINITY ? 0.f : ref[n][i & 1];
          p[i] = exp2_approx(s[n][i] - r);
          sum[n][i & 1] = fmaf(p[i], v_inv, sum[n][i & 1]);
        }
        pb[n][0] = transpose_8x8(pack_f16x2(p[0], p[1]));
        pb[n][1] = transpose_8x8(pack_f16x2(p[2], p[3]));
      }

      // O^T += V^T P^T over the 16 tokens
      if (valid && tok0 < vis_last) {
        constexpr int VW = D >= 128 ? 4 : 2;  // words of a token that a thread reads at once
        constexpr int H = D / (32 * VW);
        const bool edge = tok0 + 16 > vis_first;  // some row does not see all of them
#pragma unroll
        for (int hh = 0; hh < H; ++hh) {
          uint32_t v[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tk = 2 * t + (i & 1) + (i >= 2 ? 8 : 0);
            const uint8_t* src = vt + tk * D + hh * 32 * VW + g * 4 * VW;
            if constexpr (VW == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(src);
              v[i][0] = x.x;
              v[i][1] = x.y;
              v[i][2] = x.z;
              v[i][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(src);
              v[i][0] = x.x;
              v[i][1] = x.y;
            }
          }
          if (edge) {
            // A weight of zero does not make a NaN vanish: rows that nobody sees are
            // cleared, and a NaN that some rows see and some do not is taken out and
            // given back, at the end, to the rows that see it.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = tok0 + 2 * t + (i & 1) + (i >= 2 ? 8 : 0);
#pragma unroll
              for (int x = 0; x < VW; ++x) {
                if (tok >= vis_last) {
                  v[i][x] = 0;
                } else if (tok >= vis_first) {
                  const uint32_t nan = ((v[i][x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                  if (nan) {
                    for (int y = 0; y < 4; ++y)
                      if (nan & (0x80u << (8 * y)))
                        atomicMin(&s_nan[hh * 32 * VW + g * 4 * VW + 4 * x + y], tok);
                    v[i][x] &= ~((nan >> 7) * 0xffu);
                  }
                }
              }
            }
          }
#pragma unroll
          for (int x = 0; x < VW; ++x) {
            const uint32_t lo01 = __byte_perm(v[0][x], v[1][x], 0x5140);
            const uint32_t hi01 = __byte_perm(v[0][x], v[1][x], 0x7362);
            const uint32_t lo23 = __byte_perm(v[2][x], v[3][x], 0x5140);
            const uint32_t hi23 = __byte_perm(v[2][x], v[3][x], 0x7362);
            const int m = (hh * VW + x) * 2;
            {
              const uint32_t a0 = e4m3x2_to_f16x2(lo01 & 0xffffu), a1 = e4m3x2_to_f16x2(lo01 >> 16);
              const uint32_t a2 = e4m3x2_to_f16x2(lo23 & 0xffffu), a3 = e4m3x2_to_f16x2(lo23 >> 16);
#pragma unroll
              for (int n = 0; n < NQ; ++n) mma_f16(o[m][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
            {
              const uint32_t a0 = e4m3x2_to_f16x2(hi01 & 0xffffu), a1 = e4m3x2_to_f16x2(hi01 >> 16);
              const uint32_t a2 = e4m3x2_to_f16x2(hi23 & 0xffffu), a3 = e4m3x2_to_f16x2(hi23 >> 16);
#pragma unroll
              for (int n = 0; n < NQ; ++n) mma_f16(o[m + 1][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(empty0 + 8 * stage);
      if (++stage == NS) {
        stage = 0;
        phase ^= 1;
      }
    }

    // join the four warps, one after another
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = sum[n][i];
        x += __shfl_xor_sync(~0u, x, 4);
        x += __shfl_xor_sync(~0u, x, 8);
        x += __shfl_xor_sync(~0u, x, 16);
        if (g == 0) {
          s_ref[warp * R + 8 * n + 2 * t + i] = ref[n][i];
          s_sum[warp * R + 8 * n + 2 * t + i] = x;
        }
      }
    tma::named_sync(1, kConsumers);
    float f[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * n + 2 * t + i;
        float top = s_ref[r];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, s_ref[k * R + r]);
        f[n][i] = top == -INFINITY ? 0.f : exp2_approx(ref[n][i] - top);
      }
    for (int turn = 0; turn < kWarps; ++turn) {
      if (warp == turn) {
        constexpr int VW = D >= 128 ? 4 : 2;
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
          const int d = (m / (2 * VW)) * 32 * VW + g * 4 * VW + 2 * (m % (2 * VW));
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* dst = s_o + (8 * n + 2 * t + (i & 1)) * (D + 4) + d + (i >> 1);
              const float x = o[m][n][i] * f[n][i & 1];
              *dst = turn == 0 ? x : *dst + x;
            }
        }
      }
      tma::named_sync(1, kConsumers);
    }
    for (int idx = tid; idx < R * (D / 4); idx += kConsumers) {
      const int r = idx / (D / 4), d = (idx - r * (D / 4)) * 4;
      if (r >= it.rows) continue;
      float top = s_ref[r];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) top = fmaxf(top, s_ref[k * R + r]);
      float total = 0.f;
      if (top != -INFINITY)
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
          total += s_sum[k * R + r] * exp2_approx(s_ref[k * R + r] - top);
      float4 x = *reinterpret_cast<const float4*>(s_o + r * (D + 4) + d);
      const int4 from = *reinterpret_cast<const int4*>(s_nan + d);
      const int seen = s_vis[r];
      const float nan = __int_as_float(0x7fffffff);
      if (from.x < seen) x.x = nan;
      if (from.y < seen) x.y = nan;
      if (from.z < seen) x.z = nan;
      if (from.w < seen) x.w = nan;
      if (whole) {
        const float inv = total == 0.f ? 0.f : 1.f / total;
        *reinterpret_cast<uint2*>(a.out + row_at(r) + d) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
      } else {
        float* rec = ra.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (at_start ? 0 : 1)) *
                                      (R * (D + 2));
        *reinterpret_cast<float4*>(rec + r * D + d) = x;
        if (d == 0) {
          rec[R * D + r] = top;
          rec[R * D + R + r] = total;
        }
      }
    }
    tma::named_sync(1, kConsumers);  // Q, rows and O are rewritten for the next segment
  }
  if (dead && lane == 0 && a.status != nullptr) atomicOr(a.status, CMR_DEVICE_WAIT_TIMEOUT);
}

constexpr int kJoinThreads = 256;

// Joins the partial results of an item's row: grid (items x layers x heads, R).
template <int D, int NQ>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const RowsArgs ra) {
  constexpr int R = 8 * NQ;
  constexpr int kLanes = D / 4;                    // threads of a row of a partial result
  constexpr int kGroups = kJoinThreads / kLanes;
  __shared__ float s_w[kMaxCtas];
  __shared__ float s_red[2][kJoinThreads / 32];
  __shared__ float4 s_o[kJoinThreads];
  const AttendArgs& a = ra.a;
  pdl::wait();
  const int tid = threadIdx.x;
  const int32_t NB = ra.items;
  const int32_t bi = static_cast<int32_t>(blockIdx.x % NB);
  const int64_t lh = blockIdx.x / NB;
  const int64_t total = __ldcg(ra.prefix + NB);
  const int64_t lo = lh * total + __ldcg(ra.prefix + bi);
  const int64_t hi = lh * total + __ldcg(ra.prefix + bi + 1);
  if (lo >= hi) return;
  const int64_t all = total * a.pool.num_layers * a.pool.hk;
  const int64_t per = (all + ra.ctas - 1) / ra.ctas;
  const int64_t c0 = lo / per, c1 = (hi - 1) / per;
  if (c0 == c1) return;  // written whole
  bool bad = false;
  const Item it = find_item<R>(a, bi, &bad);
  const int r = blockIdx.y;
  if (r >= it.rows) return;
  const int n = static_cast<int>(c1 - c0 + 1);
  constexpr int kRec = R * (D + 2);
  auto record = [&](int k) {  // the item starts inside CTA c0's run unless at its start
    const int64_t c = c0 + k;
    return ra.partial + (c * 2 + (c * per >= lo ? 0 : 1)) * kRec;
  };
  float top = -INFINITY;
  for (int k = tid; k < n; k += kJoinThreads) {
    const float m = __ldcg(record(k) + R * D + r);
    s_w[k] = m;
    top = fmaxf(top, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if ((tid & 31) == 0) s_red[0][tid / 32] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinThreads / 32; ++k) top = fmaxf(top, s_red[0][k]);
  float sum = 0.f;
  for (int k = tid; k < n; k += kJoinThreads) {
    const float w = top == -INFINITY ? 0.f : exp2_approx(s_w[k] - top);
    s_w[k] = w;
    sum += w * __ldcg(record(k) + R * D + R + r);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if ((tid & 31) == 0) s_red[1][tid / 32] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinThreads / 32; ++k) sum += s_red[1][k];
  const int ln = tid % kLanes, gr = tid / kLanes;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = gr; k < n; k += kGroups) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(record(k) + r * D) + ln);
    const float w = s_w[k];
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
  }
  s_o[tid] = acc;
  __syncthreads();
  if (gr == 0) {
#pragma unroll
    for (int k = 1; k < kGroups; ++k) {
      const float4 x = s_o[k * kLanes + ln];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int l = static_cast<int>(lh / a.pool.hk), h = static_cast<int>(lh - l * a.pool.hk);
    const int f = it.first_row + r;
    uint16_t* dst = a.out + ((l * a.batch.n_tokens + it.tok + f / a.group) * a.hq + h * a.group +
                             f % a.group) * D + 4 * ln;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                                pack_bf16x2(acc.z * inv, acc.w * inv));
  }
}

// Rows of a tile: 8 where a decode step's group fits them, else 16.
int rows_of(int group, bool step) { return step && group <= 8 ? 8 : 16; }

int max_ctas(int R) {
  const int n = sm_count() * (R == 8 ? 2 : 1);
  return n < kMaxCtas ? n : kMaxCtas;
}

size_t align16(size_t x) { return (x + 15) / 16 * 16; }

template <int D, int NQ>
cudaError_t launch(RowsArgs ra, cudaStream_t stream) {
  using S = Smem<D, NQ>;
  const AttendArgs& a = ra.a;
  const int64_t lh = static_cast<int64_t>(a.pool.num_layers) * a.pool.hk;
  const size_t smem = S::kPrefix + (ra.ctas > 0 ? (ra.items + 1) * sizeof(int) : 0);
  cudaError_t e = cudaFuncSetAttribute(
      attend_rows_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      static_cast<int>(S::kPrefix + (kMaxSplitItems + 1) * sizeof(int)));
  if (e != cudaSuccess) return e;
  if (ra.ctas == 0) {
    if (lh > 65535) return cudaErrorInvalidValue;
    attend_rows_kernel<D, NQ><<<dim3(ra.items, static_cast<unsigned>(lh)), kThreads, smem, stream>>>(ra);
    return cudaGetLastError();
  }
  attend_rows_kernel<D, NQ><<<ra.ctas, kThreads, smem, stream>>>(ra);
  e = cudaGetLastError();
  if (e != cudaSuccess || ra.ctas == 1) return e;
  return pdl::launch(attend_join_kernel<D, NQ>, dim3(static_cast<unsigned>(ra.items * lh), 8 * NQ),
                     dim3(kJoinThreads), 0, stream, true, ra);
}

}  // namespace

size_t attend_rows_workspace(int32_t num_seqs, int64_t n_tokens, int32_t hq, int32_t hk,
                             int32_t head_dim) {
  // both forms of a call (with and without cu_seqlens) fit
  size_t most = 0;
  const int group = hq / hk;
  for (const bool step : {false, true}) {
    const int R = rows_of(group, step);
    const int64_t nb = item_slots(num_seqs, n_tokens, group, R, step);
    if (nb > kMaxSplitItems) continue;
    const size_t bytes = align16((nb + 1) * sizeof(int32_t)) +
                         static_cast<size_t>(max_ctas(R)) * 2 * R * (head_dim + 2) * sizeof(float);
    most = bytes > most ? bytes : most;
  }
  return most;
}

cudaError_t launch_attend_rows(const AttendArgs& a, cudaStream_t stream) {
  const bool step = a.batch.cu == nullptr;
  const int R = rows_of(a.group, step);
  const int64_t nb = item_slots(a.batch.num_seqs, a.batch.n_tokens, a.group, R, step);
  if (nb > INT32_MAX) return cudaErrorInvalidValue;
  RowsArgs ra{};
  ra.a = a;
  ra.items = static_cast<int32_t>(nb);
  const int64_t cap = static_cast<int64_t>(a.table.max_pages) << a.pool.page_shift;
  const int64_t most_tiles = (cap + kTile - 1) / kTile * nb;  // per layer and head
  if (nb <= kMaxSplitItems && most_tiles <= INT32_MAX) {
    ra.prefix = static_cast<int32_t*>(a.workspace);
    ra.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                          align16((nb + 1) * sizeof(int32_t)));
    // no more CTAs than there can be tiles
    const int64_t tiles = most_tiles * a.pool.num_layers * a.pool.hk;
    const int most = max_ctas(R);
    ra.ctas = tiles < most ? static_cast<int32_t>(tiles) : most;
    // the joining grid has a block for every item and row
    if (nb * a.pool.num_layers * a.pool.hk > INT32_MAX) return cudaErrorInvalidValue;
  }
  switch (a.pool.head_dim) {
    case 64: return R == 8 ? launch<64, 1>(ra, stream) : launch<64, 2>(ra, stream);
    case 128: return R == 8 ? launch<128, 1>(ra, stream) : launch<128, 2>(ra, stream);
    default: return R == 8 ? launch<256, 1>(ra, stream) : launch<256, 2>(ra, stream);
  }
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t stream) {
  // More than 16 rows per sequence, on average: the tcgen05 kernel, which reads the
  // cache once for 128 rows.
  if (a.batch.n_tokens * a.group > 16 * static_cast<int64_t>(a.batch.num_seqs)) {
    bool launched = false;
    const cudaError_t e = launch_attend_tiles(a, stream, &launched);
    if (launched && e == cudaSuccess) note_kernel("attend_tiles_kernel");
    if (e != cudaSuccess || launched) return e;
  }
  const cudaError_t e = launch_attend_rows(a, stream);
  if (e == cudaSuccess) note_kernel("attend_rows_kernel");
  return e;
}

size_t attend_workspace_bytes(int32_t num_seqs, int64_t n_tokens, int32_t num_layers, int32_t hq,
                              int32_t hk, int32_t head_dim) {
  const size_t rows = attend_rows_workspace(num_seqs, n_tokens, hq, hk, head_dim);
  const size_t tiles = attend_tiles_workspace(num_seqs, n_tokens, num_layers, hq, hk, head_dim);
  return rows > tiles ? rows : tiles;
}

}  // namespace kv8
}  // namespace cmr

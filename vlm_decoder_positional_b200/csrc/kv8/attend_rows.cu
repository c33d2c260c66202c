// Attention over the paged 8-bit cache for calls with few query rows per
// sequence: decode steps and short chunks.
//
// With a page's scales 2^a (keys) and 2^e (values) and codes k, v in e4m3,
//   out = sum_i p_i v_i / sum_i p_i 2^-e_i,   p_i = 2^(c 2^a_i (q . k_i) + e_i - r),
// c = softmax scale * log2(e) and r a running maximum of the exponent: the value
// scale enters the weight, so codes are never multiplied by a scale, and a page
// of large values cannot push the weights of the others out of range.  e4m3
// codes are exact in f16; q is brought to f16 exactly by a power of two per row
// (bits below 2^-24 of the row's largest value are lost).  p is rounded to f16 for the
// product: r is placed so that the row's largest p lies between 2^13 and 2^15, so a
// weight of 2^-27 of it or more is off by 2^-11 of itself at most (the bf16 result by
// 2^-8), a smaller one by 2^-38 of the largest: tokens behind a strong one keep their
// part, however many they are.  The sum of weights takes p as it is; all sums, maxima and
// the accumulator are fp32.
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
// The tensor pipe is busy in 16 % of the cycles, so tcgen05 would gain nothing.
// Measured, 8 query and 2 KV heads of 256, pages of 64: 64 sequences of 4096 53 us
// (5.1 TB/s, 79% of a copy's rate), one of 262144 55 us, 128 of 1 to 8192 29 us where
// the bytes alone take 15: what is left is the start of the two kernels and the last
// tile's way through them, about 8 us, which one sequence of 700 takes as well.
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
// Items of fewer tiles are not split, which saves the joining kernel: a call for 16
// sequences of 100 or 300 tokens takes 12.8 us instead of 15.0, of 700 16.9 instead of
// 15.5 (in tables of no more pages than they need).
constexpr int kMinSplitTiles = 6;
// Weights are at most 2^kBase when the reference moves, and 2^(kBase + kLazy) before it
// does, which f16 holds; the less it is let drift, the smaller the weights that f16 still
// tells apart.  O is in registers, so moving it costs little: 8 and 7, 4 and 11, 2 and 13,
// 1 and 14 all take 53.0 us for 64 sequences of 4096.
constexpr float kBase = 13.f;
constexpr float kLazy = 2.f;

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
  static constexpr int W = D < 128 ? D : 128;                      // bytes of a swizzled row
  static constexpr int kPanel = kTile * W;                         // W dims of a tile
  static constexpr int kStage = 2 * kTile * D;
  static constexpr int kQ = kStages * kStage;                      // f16 fragments of Q
  static constexpr int kNan = kQ + (D / 16) * NQ * 32 * 8;         // [2][D] ints
  static constexpr int kRow = kNan + 2 * D * 4;                    // [2] of the rows' words
  static constexpr int kRowWords = 2 * R + 2 * kWarps * R;
  static constexpr int kInfo = kRow + 2 * 4 * kRowWords;
  static constexpr int kBars = (kInfo + kStages * static_cast<int>(sizeof(StageInfo)) + 7) / 8 * 8;
  static constexpr int kItems = (kBars + 16 * kStages + 15) / 16 * 16;  // 3 ints an item, and 1
};

struct RowsArgs {
  AttendArgs a;
  int32_t items;       // row-tile slots per (layer, head): NB
  int32_t ctas;        // CTAs of the split form; 0: one CTA per item
  float* partial;      // [ctas][2][R][D + 2]
  int32_t* prefix;     // [NB + 1], written by CTA 0 for the joining kernel
  int4* left;          // [ctas]: the item that a run starts and leaves to others to end
                       // (layer x head, item, last CTA, place of the first piece), or -1
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

// The token of a warp's 16 that row m < 8 of S^T stands for (m + 8: 8 further).  Any
// order will do, as long as P^T and V^T follow it; with this one, and rows swizzled
// as TMA leaves them, the eight lanes that read shared memory together hit different
// banks, both for keys (lanes of rows m, m + 1) and for values (even or odd m).
__device__ __forceinline__ int token_of(int m) { return m ^ ((m & 1) << 2); }

// Work is counted in tiles, and kLead more for each item: what it costs to start
// and to finish one.  Places [start, start + kLead) of an item's stretch hold no
// tile.  128 sequences of 1 to 7,698 tokens: 54 us without, 33 with 2, 26.6 with 4,
// 28 with 6; 64 of 4,096: 54.7, 54.6, 53.2, 52.6.
constexpr int kLead = 4;

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? 2 : 1)
    attend_rows_kernel(const RowsArgs ra, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map) {
  using S = Smem<D, NQ>;
  constexpr int R = S::R;
  constexpr int NS = S::kStages;
  constexpr int M = D / 16;  // O^T's row blocks
  constexpr int W = S::W;
  constexpr int kPanels = D / W;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (tma::smem_addr(smem_raw) & 1023)) & 1023);
  const AttendArgs& a = ra.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  uint2* s_q = reinterpret_cast<uint2*>(smem + S::kQ);
  StageInfo* s_info = reinterpret_cast<StageInfo*>(smem + S::kInfo);
  const int NB = ra.items;
  const int kept = ra.ctas > 0 ? NB : 1;                              // items of this CTA's list
  int* s_prefix = reinterpret_cast<int*>(smem + S::kItems);           // [kept + 1]
  int* s_seen = s_prefix + kept + 1;                                  // [kept] vis_last
  int* s_row = s_seen + kept;                                         // [kept] table row
  const uint32_t stage0 = tma::smem_addr(smem);
  const uint32_t full0 = tma::smem_addr(smem + S::kBars);
  const uint32_t empty0 = full0 + 8 * NS;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      tma::mbar_init(full0 + 8 * s, 2);
      tma::mbar_init(empty0 + 8 * s, kWarps);
    }
    tma::mbar_init_fence();
  }
  pdl::wait();
  // What the first copies will wait for, one after another, is asked for at once: the
  // tensor maps, and the page table, a line to a thread of the grid.
  if (tid == 32) {
    tma::prefetch_map(&k_map);
    tma::prefetch_map(&v_map);
  }
  {
    const int64_t line = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + tid;
    const int64_t entry = line * 32;
    if (entry < static_cast<int64_t>(a.table.rows) * a.table.max_pages)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table.pages + entry));
  }
  // ---- the items and this CTA's run [lo, hi) of the work
  bool bad = false;
  const int first = ra.ctas > 0 ? 0 : blockIdx.x;  // item number of list entry 0
  for (int i = tid; i < kept; i += kThreads) {
    const Item it = find_item<R>(a, first + i, &bad);
    const int tiles = item_tiles(it);
    s_prefix[i] = tiles > 0 ? tiles + kLead : 0;
    s_seen[i] = static_cast<int>(it.vis_last);
    s_row[i] = it.row;
    if ((ra.ctas > 0 ? blockIdx.x == 0 : blockIdx.y == 0) && it.rows > 0 && it.cut &&
        a.status != nullptr)
      atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
  }
  if (bad && (ra.ctas > 0 ? blockIdx.x == 0 : blockIdx.y == 0) && a.status != nullptr)
    atomicOr(a.status, CMR_DEVICE_BAD_CU_SEQLENS);
  __syncthreads();
  if (warp == 0) {  // exclusive scan in place
    int carry = 0;
    for (int i0 = 0; i0 < kept; i0 += 32) {
      const int i = i0 + lane;
      const int v = i < kept ? s_prefix[i] : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      __syncwarp();
      if (i < kept) s_prefix[i] = carry + x - v;
      carry += __shfl_sync(~0u, x, 31);
    }
    if (lane == 0) s_prefix[kept] = carry;
  }
  __syncthreads();
  // per (layer, head); all of the work fits 31 bits, which the launch has seen to
  const uint32_t total = s_prefix[kept];
  uint32_t run_lo, run_hi, lh0 = 0;
  if (ra.ctas > 0) {
    if (blockIdx.x == 0)
      for (int i = tid; i <= NB; i += kThreads) ra.prefix[i] = s_prefix[i];
    const uint32_t all = total * a.pool.num_layers * a.pool.hk;
    const uint32_t per = (all + ra.ctas - 1) / ra.ctas;
    run_lo = min(all, blockIdx.x * per);
    run_hi = min(all, run_lo + per);
  } else {
    lh0 = blockIdx.y;
    run_lo = 0;
    run_hi = total;
  }
  pdl::launch_dependents();

  // Entry of the list at place r of a (layer, head)'s work.
  auto entry_at = [&](uint32_t r) {
    int32_t lo = 0, hi = kept;
    while (hi - lo > 1) {  // the last that starts at or before r
      const int32_t mid = (lo + hi) >> 1;
      if (static_cast<uint32_t>(s_prefix[mid]) <= r)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };

  const int P = 1 << a.pool.page_shift;
  if (warp == kWarps) {
    // ---- producer: lane 4 i + g looks after tokens [16g, 16g + 16) of place i of a
    // batch of eight
    const int g = lane & 3;
    uint32_t problems = 0;
    struct Look {
      bool tile;      // the place holds a tile
      int64_t unit;   // its page's (layer, page, head), or -1
      int64_t tok;
      float ks, vs;
    };
    auto look = [&](uint32_t w0) {
      Look k{false, -1, 0, 0.f, 1.f};
      const uint32_t w = w0 + (lane >> 2);
      if (w >= run_hi) return k;
      const uint32_t lh = w / total;
      const uint32_t r = w - lh * total;
      const int32_t e = entry_at(r);
      const int32_t tile = static_cast<int32_t>(r) - s_prefix[e] - kLead;
      if (tile < 0) return k;
      k.tile = true;
      k.tok = static_cast<int64_t>(tile) * kTile + 16 * g;
      const int seen = s_seen[e];
      if (k.tok >= seen) return k;
      const int32_t id = page_id(a.table, a.pool.num_pages, s_row[e], k.tok >> a.pool.page_shift);
      if (id < 0) {
        problems |= CMR_DEVICE_CACHE_RANGE;
        return k;
      }
      const uint32_t l = (lh + lh0) / a.pool.hk, h = lh + lh0 - l * a.pool.hk;
      k.unit = (static_cast<int64_t>(l) * a.pool.num_pages + id) * a.pool.hk + h;
      k.ks = __ldg(a.pool.ks + k.unit);
      k.vs = __ldg(a.pool.vs + k.unit);
      return k;
    };
    int stage = 0, phase = 0, issued = 0;
    bool dead = false;
    // A sequence's pages are read once and marked so in L2, where tables, scales and partial
    // results stay: 53 us instead of 57 for 64 sequences of 4096, 54.5 instead of 59 for one
    // of 262144.  Pages that branches share are read by each of them: 64 branches of 4000
    // tokens or of 500 take the same either way (51 and 22.5 us), 8 of 20000 41 us marked
    // and 39 not, 16 of 100000 262 and 231; the call does not know which pages are shared.
    const uint64_t policy = tma::l2_evict_first_policy();
    Look now = look(run_lo);
    for (uint32_t w = run_lo; w < run_hi && !dead; w += 8) {
      const uint32_t tiles = __ballot_sync(~0u, now.tile);
      const uint32_t pages = __ballot_sync(~0u, now.unit >= 0);
      for (int i = 0; i < 8; ++i) {
        if (!((tiles >> (4 * i)) & 1u)) continue;
        if (issued >= NS && !tma::mbar_wait(empty0 + 8 * stage, phase ^ 1)) dead = true;
        dead = __any_sync(~0u, dead);
        if (dead) break;
        const uint32_t bar = full0 + 8 * stage;
        if (lane == 4 * i)
          tma::mbar_arrive_expect_tx(bar, __popc((pages >> (4 * i)) & 15u) * 2 * 16 * D);
        __syncwarp();
        const bool mine = (lane >> 2) == i;
        if (mine && now.unit >= 0) {
          const uint32_t dst = stage0 + stage * S::kStage + 16 * g * W;
          const int row = static_cast<int>(now.tok) & (P - 1), unit = static_cast<int>(now.unit);
#pragma unroll
          for (int x = 0; x < kPanels; ++x)
            load_3d_hint(dst + x * S::kPanel, &k_map, bar, x * W, row, unit, policy);
#pragma unroll
          for (int x = 0; x < kPanels; ++x)
            load_3d_hint(dst + kTile * D + x * S::kPanel, &v_map, bar, x * W, row, unit, policy);
        }
        // the scales, under the copies
        const bool good = now.unit >= 0 && scale_ok(now.ks) && scale_ok(now.vs);
        if (mine && now.unit >= 0 && !good) problems |= CMR_DEVICE_BAD_SCALE;
        const uint32_t valid = __ballot_sync(~0u, good);
        if (mine) {
          StageInfo& info = s_info[stage];
          info.k_scale[g] = good ? now.ks : 0.f;
          info.v_log2[g] = good ? __log2f(now.vs) : 0.f;
          info.v_inv[g] = good ? 1.f / now.vs : 1.f;
          if (g == 0) info.valid = (valid >> (4 * i)) & 15u;
        }
        __syncwarp();
        if (lane == 4 * i) tma::mbar_arrive(bar);
        ++issued;
        if (++stage == NS) {
          stage = 0;
          phase ^= 1;
        }
      }
      now = look(w + 8);  // with this batch's last copies in flight
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
  constexpr int VW = D >= 128 ? 4 : 2;  // words of a token's values that a thread reads at once
  constexpr int H = D / (32 * VW);

  struct Segment {
    uint32_t w;       // where the next begins
    uint32_t lh;
    int32_t entry;
    int32_t t0, nt;   // tiles
    bool whole, late; // the whole item; the item started before this run
  };
  // The first segment at or behind place w; nt = 0 behind the last.
  auto segment = [&](uint32_t w) {
    Segment sg{w, 0, 0, 0, 0, false, false};
    while (sg.w < run_hi) {
      const uint32_t lh = sg.w / total;
      const int32_t e = entry_at(sg.w - lh * total);
      const uint32_t start = lh * total + s_prefix[e], end = lh * total + s_prefix[e + 1];
      const uint32_t lo = max(sg.w, start + kLead), hi = min(end, run_hi);
      if (lo < hi) {
        sg.lh = lh + lh0;
        sg.entry = e;
        sg.t0 = static_cast<int32_t>(lo - start) - kLead;
        sg.nt = static_cast<int32_t>(hi - lo);
        sg.whole = sg.t0 == 0 && hi == end;
        sg.late = start < run_lo;
        sg.w = hi;
        return sg;
      }
      sg.w = min(end, run_hi);
    }
    return sg;
  };
  // Element offset of query row r of an item.
  auto row_at = [&](const Item& it, int l, int h, int r) {
    const int f = it.first_row + r;
    const int64_t tok = it.tok + f / a.group;
    return ((l * a.batch.n_tokens + tok) * a.hq + h * a.group + f % a.group) * D;
  };
  constexpr int kPer = kConsumers / R;                            // threads of a row of Q
  constexpr int kHave = D / 8 / kPer > 0 ? D / 8 / kPer : 1;      // 16-byte chunks of a thread
  const int q_row = tid / kPer, q_chunk = tid % kPer;
  auto load_q = [&](const Item& it, int l, int h, uint4 (&x)[kHave]) {
#pragma unroll
    for (int k = 0; k < kHave; ++k) {
      x[k] = make_uint4(0, 0, 0, 0);
      const int c = q_chunk + k * kPer;
      if (q_row < it.rows && c < D / 8)
        x[k] = __ldg(reinterpret_cast<const uint4*>(a.q + row_at(it, l, h, q_row)) + c);
    }
  };

  int stage = 0, phase = 0, turn = 0;
  bool dead = false, ignored = false;
  Segment sg = segment(run_lo);
  int4 left = make_int4(-1, 0, 0, 0);
  Item it{};
  int l = 0, h = 0;
  uint4 xq[kHave];
  if (sg.nt > 0) {
    l = static_cast<int>(sg.lh / a.pool.hk);
    h = static_cast<int>(sg.lh) - l * a.pool.hk;
    it = find_item<R>(a, first + sg.entry, &ignored);
    load_q(it, l, h, xq);
  }
  while (sg.nt > 0) {
    const int vis_first = static_cast<int>(it.vis_first), vis_last = static_cast<int>(it.vis_last);
    turn ^= 1;  // the rows' words have two places: the last segment's may still be read
    int* s_nan = reinterpret_cast<int*>(smem + S::kNan) + turn * D;
    float* s_mult = reinterpret_cast<float*>(smem + S::kRow) + turn * S::kRowWords;  // [R]
    int* s_vis = reinterpret_cast<int*>(s_mult + R);  // [R] tokens seen
    float* s_ref = reinterpret_cast<float*>(s_vis + R);  // [warps][R]
    float* s_sum = s_ref + kWarps * R;                   // [warps][R]

    // Q to f16, each row over a power of two, in the order of the B fragments
    {
      uint32_t mx = 0;
#pragma unroll
      for (int k = 0; k < kHave; ++k) {
        const uint32_t ww[4] = {xq[k].x, xq[k].y, xq[k].z, xq[k].w};
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
        const int c = q_chunk + k * kPer;
        if (c < D / 8) {
          const uint32_t ww[4] = {xq[k].x, xq[k].y, xq[k].z, xq[k].w};
          uint32_t f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = finite ? pack_f16x2(bf16_lo(ww[i]) * inv, bf16_hi(ww[i]) * inv) : 0x7fff7fffu;
          const int d = 8 * c;
          const int m = d / 64 * 4 + (d % 16) / 4, tt = (d % 64) / 16;
          const int nq = q_row / 8, gq = q_row % 8;
          s_q[(m * NQ + nq) * 32 + gq * 4 + tt] = make_uint2(f[0], f[1]);
          s_q[((m + 1) * NQ + nq) * 32 + gq * 4 + tt] = make_uint2(f[2], f[3]);
        }
      }
      if (q_chunk == 0) {
        s_mult[q_row] = a.scale_log2 * __int_as_float((127 + e) << 23);
        const int64_t seen = it.p0 + (it.first_row + q_row) / a.group + 1;
        s_vis[q_row] = q_row < it.rows ? static_cast<int>(max(static_cast<int64_t>(0),
                                                              min(seen, it.vis_last)))
                                       : 0;
      }
      for (int d = tid; d < D; d += kConsumers) s_nan[d] = 0x7fffffff;
    }
    // the next segment's Q is on its way during this one's tiles
    const Segment next = segment(sg.w);
    Item next_it{};
    int next_l = 0, next_h = 0;
    if (next.nt > 0) {
      next_l = static_cast<int>(next.lh / a.pool.hk);
      next_h = static_cast<int>(next.lh) - next_l * a.pool.hk;
      next_it = find_item<R>(a, first + next.entry, &ignored);
      load_q(next_it, next_l, next_h, xq);
    }
    tma::named_sync(1, kConsumers);

    float o[M][NQ][4];
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
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
    }

    uint8_t* used = nullptr;  // the last tile's stage
    for (int tile = 0; tile < sg.nt; ++tile) {
      if (!dead && !tma::mbar_wait(full0 + 8 * stage, phase, tma::kConsumerWaitLimitNs)) dead = true;
      used = smem + stage * S::kStage;
      const StageInfo& info = s_info[stage];
      const float k_scale = info.k_scale[warp], v_log2 = info.v_log2[warp];
      const float v_inv = info.v_inv[warp];
      const int tok0 = (sg.t0 + tile) * kTile + warp * 16;
      const bool live = ((info.valid >> warp) & 1u) && tok0 < vis_last;

      if (live) {
        // scores of two tokens against queries 2t, 2t + 1, summed over the dims in
        // two chains
        float part[2][NQ][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) part[i][n][x] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const int r = warp * 16 + token_of(g);
          const int c = j * 4 + t;  // 16-byte chunk of the keys
          const uint8_t* src = used + c / (W / 16) * S::kPanel;
          const uint4 lo = *reinterpret_cast<const uint4*>(src + swizzled<W>(r, c % (W / 16)));
          const uint4 hi = *reinterpret_cast<const uint4*>(src + swizzled<W>(r + 8, c % (W / 16)));
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = e4m3x2_to_f16x2(wl[i] & 0xffffu), a2 = e4m3x2_to_f16x2(wl[i] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(wh[i] & 0xffffu), a3 = e4m3x2_to_f16x2(wh[i] >> 16);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const uint2 q = s_q[((j * 4 + i) * NQ + n) * 32 + lane];
              mma_f16(part[i & 1][n], a0, a1, a2, a3, q.x, q.y);
            }
          }
        }
        float s[NQ][4];
        uint32_t pb[NQ][2];
        bool move = false;
        float mx[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = tok0 + token_of(g) + (i >= 2 ? 8 : 0);
            const float dot = part[0][n][i] + part[1][n][i];
            const float x = fmaf(dot, mult[n][i & 1] * k_scale, v_log2);
            s[n][i] = tok < vis[n][i & 1] ? x : -INFINITY;
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
            for (int m = 0; m < M; ++m) {
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
            const float r = (ref[n][i & 1] == -INFINITY ? 0.f : ref[n][i & 1]) - kBase;
            p[i] = exp2_approx(s[n][i] - r);
            sum[n][i & 1] = fmaf(p[i], v_inv, sum[n][i & 1]);
          }
          pb[n][0] = transpose_8x8(pack_f16x2(p[0], p[1]));
          pb[n][1] = transpose_8x8(pack_f16x2(p[2], p[3]));
        }

        // O^T += V^T P^T over the 16 tokens
        const bool edge = tok0 + 16 > vis_first;  // some row does not see all of them
#pragma unroll
        for (int hh = 0; hh < H; ++hh) {
          uint32_t v[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = warp * 16 + token_of(2 * t + (i & 1)) + (i >= 2 ? 8 : 0);
            const uint8_t* src = used + kTile * D + hh * S::kPanel;
            if constexpr (VW == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(src + swizzled<W>(r, g));
              v[i][0] = x.x;
              v[i][1] = x.y;
              v[i][2] = x.z;
              v[i][3] = x.w;
            } else {
              const uint2 x =
                  *reinterpret_cast<const uint2*>(src + swizzled<W>(r, g / 2) + (g & 1) * 8);
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
              const int tok = tok0 + token_of(2 * t + (i & 1)) + (i >= 2 ? 8 : 0);
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
      if (tile + 1 < sg.nt) {  // the last tile's stage is kept for the joining below
        if (lane == 0) tma::mbar_arrive(empty0 + 8 * stage);
        if (++stage == NS) {
          stage = 0;
          phase ^= 1;
        }
      }
    }

    // join the four warps through the last tile's stage
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
    tma::named_sync(1, kConsumers);  // the tile has been read by all
    float4* dump = reinterpret_cast<float4*>(used);
    constexpr int kSlots = M * NQ * 32;  // of a warp's O
    constexpr int kDumps = 8 / (2 * NQ);  // warps whose O a stage holds: 4 or 2
    {
      float f[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * n + 2 * t + i;
          float top = s_ref[r];
#pragma unroll
          for (int k = 1; k < kWarps; ++k) top = fmaxf(top, s_ref[k * R + r]);
          f[n][i] = top == -INFINITY ? 1.f : exp2_approx(ref[n][i] - top);
        }
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          o[m][n][0] *= f[n][0];
          o[m][n][1] *= f[n][1];
          o[m][n][2] *= f[n][0];
          o[m][n][3] *= f[n][1];
        }
    }
    if constexpr (kDumps < kWarps) {  // the upper warps' first, into the lower ones
      if (warp >= kDumps)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            dump[(warp - kDumps) * kSlots + (m * NQ + n) * 32 + lane] =
                make_float4(o[m][n][0], o[m][n][1], o[m][n][2], o[m][n][3]);
      tma::named_sync(1, kConsumers);
      if (warp < kDumps)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const float4 x = dump[warp * kSlots + (m * NQ + n) * 32 + lane];
            o[m][n][0] += x.x;
            o[m][n][1] += x.y;
            o[m][n][2] += x.z;
            o[m][n][3] += x.w;
          }
      tma::named_sync(1, kConsumers);
    }
    if (warp < kDumps)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          dump[warp * kSlots + (m * NQ + n) * 32 + lane] =
              make_float4(o[m][n][0], o[m][n][1], o[m][n][2], o[m][n][3]);
    tma::named_sync(1, kConsumers);
    // thread (warp, lane) finishes blocks m of its warp's quarter: consecutive dims
    // of queries 2t and 2t + 1
    constexpr int kMine = M / kWarps;
    float* rec = ra.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (sg.late ? 0 : 1)) *
                                  (R * (D + 2));
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float y[2][2 * kMine];
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int slot = ((warp * kMine + k) * NQ + n) * 32 + lane;
        float4 x = dump[slot];
#pragma unroll
        for (int w = 1; w < kDumps; ++w) {
          const float4 z = dump[w * kSlots + slot];
          x.x += z.x;
          x.y += z.y;
          x.z += z.z;
          x.w += z.w;
        }
        y[0][2 * k] = x.x;
        y[1][2 * k] = x.y;
        y[0][2 * k + 1] = x.z;
        y[1][2 * k + 1] = x.w;
      }
      const int m0 = warp * kMine;
      const int d = m0 / (2 * VW) * 32 * VW + g * 4 * VW + 2 * (m0 % (2 * VW));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * n + 2 * t + i;
        if (r >= it.rows) continue;
        float top = s_ref[r];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, s_ref[k * R + r]);
        float all = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
          all += s_sum[k * R + r] * (top == -INFINITY ? 1.f : exp2_approx(s_ref[k * R + r] - top));
        const int seen = s_vis[r];
#pragma unroll
        for (int k = 0; k < 2 * kMine; ++k)
          if (s_nan[d + k] < seen) y[i][k] = __int_as_float(0x7fffffff);
        if (sg.whole) {
          const float inv = all == 0.f ? 0.f : 1.f / all;
          uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row_at(it, l, h, r) + d);
          uint32_t w[kMine];
#pragma unroll
          for (int k = 0; k < kMine; ++k) w[k] = pack_bf16x2(y[i][2 * k] * inv, y[i][2 * k + 1] * inv);
          if constexpr (kMine == 4)
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          else
#pragma unroll
            for (int k = 0; k < kMine; ++k) dst[k] = w[k];
        } else {
#pragma unroll
          for (int k = 0; k < kMine; ++k)
            *reinterpret_cast<float2*>(rec + r * D + d + 2 * k) =
                make_float2(y[i][2 * k], y[i][2 * k + 1]);
          if (d == 0) {
            rec[R * D + r] = top;
            rec[R * D + R + r] = all;
          }
        }
      }
    }
    if (!sg.whole && sg.t0 == 0) {  // the run's last: it goes on in the next
      const uint32_t end = (sg.lh - lh0) * total + s_prefix[sg.entry + 1];
      left = make_int4(static_cast<int>(sg.lh), sg.entry,
                       static_cast<int>((end - 1) / max(run_hi - run_lo, 1u)), sg.late ? 0 : 1);
    }
    // the stage goes back: plain accesses before the next copy into it
    tma::fence_async_shared();
    __syncwarp();
    if (lane == 0) tma::mbar_arrive(empty0 + 8 * stage);
    if (++stage == NS) {
      stage = 0;
      phase ^= 1;
    }
    sg = next;
    it = next_it;
    l = next_l;
    h = next_h;
  }
  if (tid == 0 && ra.ctas > 0) ra.left[blockIdx.x] = left;
  if (dead && lane == 0 && a.status != nullptr) atomicOr(a.status, CMR_DEVICE_WAIT_TIMEOUT);
}

constexpr int kJoinThreads = 256;
constexpr int kJoinLanes = 16;                          // threads of 64 dims of a row
constexpr int kJoinGroups = kJoinThreads / kJoinLanes;  // partial results read at once
constexpr int kJoinAhead = 8;                           // and ahead by each thread

// Joins the partial results of 64 dims of an item's row: grid (items x layers x
// heads, R, D / 64).
template <int D, int NQ>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const RowsArgs ra) {
  constexpr int R = 8 * NQ;
  __shared__ float s_w[kMaxCtas];
  __shared__ float s_red[2][kJoinThreads / 32];
  __shared__ float4 s_o[kJoinThreads];
  const AttendArgs& a = ra.a;
  const int tid = threadIdx.x;
  const int32_t NB = ra.items;
  const int32_t bi = static_cast<int32_t>(blockIdx.x % NB);
  const uint32_t lh = blockIdx.x / NB;
  const int r = blockIdx.y;
  pdl::wait();
  pdl::launch_dependents();
  bool bad = false;
  const Item it = find_item<R>(a, bi, &bad);
  if (r >= it.rows) return;
  const uint32_t total = __ldcg(ra.prefix + NB);
  const uint32_t start = lh * total + __ldcg(ra.prefix + bi);
  const uint32_t end = lh * total + __ldcg(ra.prefix + bi + 1);
  const uint32_t all = total * a.pool.num_layers * a.pool.hk;
  const uint32_t per = (all + ra.ctas - 1) / ra.ctas;
  const uint32_t c0 = (start + kLead) / per, c1 = (end - 1) / per;
  if (c0 == c1) return;  // written whole
  const int n = static_cast<int>(c1 - c0 + 1);
  constexpr int kRec = R * (D + 2);
  auto record = [&](int k) {  // in the second place where the item starts within the run
    const uint32_t c = c0 + k;
    return ra.partial + (static_cast<int64_t>(c) * 2 + (start >= c * per ? 1 : 0)) * kRec;
  };
  const int ln = tid % kJoinLanes, gr = tid / kJoinLanes;
  const int d = blockIdx.z * 4 * kJoinLanes + 4 * ln;
  // the first values are on their way while their weights are found
  float4 x[kJoinAhead];
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i) {
    const int k = gr + i * kJoinGroups;
    x[i] = k < n ? __ldcg(reinterpret_cast<const float4*>(record(k) + r * D + d))
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
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
    const float w = top == -INFINITY ? 1.f : exp2_approx(s_w[k] - top);
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
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4& y) {
    acc.x = fmaf(w, y.x, acc.x);
    acc.y = fmaf(w, y.y, acc.y);
    acc.z = fmaf(w, y.z, acc.z);
    acc.w = fmaf(w, y.w, acc.w);
  };
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i) {
    const int k = gr + i * kJoinGroups;
    if (k < n) add(s_w[k], x[i]);
  }
  for (int k = gr + kJoinAhead * kJoinGroups; k < n; k += kJoinGroups)
    add(s_w[k], __ldcg(reinterpret_cast<const float4*>(record(k) + r * D + d)));
  s_o[tid] = acc;
  __syncthreads();
  if (gr == 0) {
#pragma unroll
    for (int k = 1; k < kJoinGroups; ++k) {
      const float4 y = s_o[k * kJoinLanes + ln];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int l = static_cast<int>(lh / a.pool.hk);
    const int h = static_cast<int>(lh) - l * a.pool.hk;
    const int f = it.first_row + r;
    uint16_t* dst = a.out + ((l * a.batch.n_tokens + it.tok + f / a.group) * a.hq + h * a.group +
                             f % a.group) * D + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                                pack_bf16x2(acc.z * inv, acc.w * inv));
  }
}

// The same with a CTA for each run, for calls of many items: each run leaves at
// most one item to be joined, of a few pieces.
template <int D, int NQ>
__global__ void __launch_bounds__(kJoinThreads) attend_join_runs_kernel(const RowsArgs ra) {
  constexpr int R = 8 * NQ;
  constexpr int kRec = R * (D + 2);
  const AttendArgs& a = ra.a;
  pdl::wait();
  pdl::launch_dependents();
  const int4 left = __ldcg(ra.left + blockIdx.x);
  if (left.x < 0) return;
  const int64_t lh = left.x;
  const int c0 = blockIdx.x, c1 = left.z;
  const float* rec0 = ra.partial + (static_cast<int64_t>(c0) * 2 + left.w) * kRec;
  bool bad = false;
  const Item it = find_item<R>(a, left.y, &bad);
  const int l = static_cast<int>(lh / a.pool.hk);
  const int h = static_cast<int>(lh - static_cast<int64_t>(l) * a.pool.hk);
  for (int idx = threadIdx.x; idx < it.rows * (D / 4); idx += kJoinThreads) {
    const int r = idx / (D / 4), d = (idx - r * (D / 4)) * 4;
    float top = __ldcg(rec0 + R * D + r);
    float sum = __ldcg(rec0 + R * D + R + r);
    float4 acc = __ldcg(reinterpret_cast<const float4*>(rec0 + r * D + d));
#pragma unroll 4
    for (int c = c0 + 1; c <= c1; ++c) {
      const float* rec = ra.partial + static_cast<int64_t>(c) * 2 * kRec;
      const float ref = __ldcg(rec + R * D + r);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + r * D + d));
      const float to = fmaxf(top, ref);
      const float f = to == -INFINITY ? 1.f : exp2_approx(top - to);
      const float w = to == -INFINITY ? 1.f : exp2_approx(ref - to);
      top = to;
      sum = fmaf(sum, f, w * __ldcg(rec + R * D + R + r));
      acc.x = fmaf(acc.x, f, w * x.x);
      acc.y = fmaf(acc.y, f, w * x.y);
      acc.z = fmaf(acc.z, f, w * x.z);
      acc.w = fmaf(acc.w, f, w * x.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int f = it.first_row + r;
    uint16_t* dst = a.out + ((l * a.batch.n_tokens + it.tok + f / a.group) * a.hq + h * a.group +
                             f % a.group) * D + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                                pack_bf16x2(acc.z * inv, acc.w * inv));
  }
}

// Rows of a tile: 8 where sequences have no more on average, else 16.  Two CTAs of 8 rows
// share an SM: 64 sequences of 2 tokens (4 heads a group) behind 4000 take 66 us in
// tiles of 8 and 92 in tiles of 16; with 3 tokens each, which need two tiles of 8, 107
// and 94.
int rows_of(int32_t num_seqs, int64_t n_tokens, int group) {
  return n_tokens * group <= 8 * static_cast<int64_t>(num_seqs) ? 8 : 16;
}

int max_ctas(int R) {
  const int n = sm_count() * (R == 8 ? 2 : 1);
  return n < kMaxCtas ? n : kMaxCtas;
}

size_t align16(size_t x) { return (x + 15) / 16 * 16; }

template <int D, int NQ>
cudaError_t launch(const RowsArgs& ra, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t stream) {
  using S = Smem<D, NQ>;
  const AttendArgs& a = ra.a;
  const int64_t lh = static_cast<int64_t>(a.pool.num_layers) * a.pool.hk;
  const size_t smem = 1024 + S::kItems + (3 * (ra.ctas > 0 ? ra.items : 1) + 1) * sizeof(int);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(
      reinterpret_cast<const void*>(attend_rows_kernel<D, NQ>),
      static_cast<int>(1024 + S::kItems + (3 * kMaxSplitItems + 1) * sizeof(int)), &done);
  if (e != cudaSuccess) return e;
  if (ra.ctas == 0) {
    return pdl::launch(attend_rows_kernel<D, NQ>, dim3(ra.items, static_cast<unsigned>(lh)),
                       dim3(kThreads), smem, stream, true, ra, k, v);
  }
  e = pdl::launch(attend_rows_kernel<D, NQ>, dim3(ra.ctas), dim3(kThreads), smem, stream, true, ra,
                  k, v);
  if (e != cudaSuccess || ra.ctas == 1) return e;
  // With one item to four runs or more, an item is cut into a few pieces: a CTA
  // joins them all.  With fewer items there are many pieces, and the CTAs share
  // an item's rows and dims.  By the first way and by the second (one token each, two KV
  // heads, replayed from a graph with cold caches): one sequence of 700 18.4 and 14.3 us,
  // one of 20000 55 and 20, 8 of 4000 29 and 26, 16 of 4000 31 and 31, 36 43 and 47, 64 61
  // and 70, 128 104 and 121.
  if (ra.items * lh * 4 >= ra.ctas)
    return pdl::launch(attend_join_runs_kernel<D, NQ>, dim3(ra.ctas), dim3(kJoinThreads), 0, stream,
                       true, ra);
  const int rows = a.batch.cu == nullptr && a.group < 8 * NQ ? a.group : 8 * NQ;
  return pdl::launch(attend_join_kernel<D, NQ>,
                     dim3(static_cast<unsigned>(ra.items * lh), rows, D / 64), dim3(kJoinThreads),
                     0, stream, true, ra);
}

}  // namespace

size_t attend_rows_workspace(int32_t num_seqs, int64_t n_tokens, int32_t hq, int32_t hk,
                             int32_t head_dim) {
  // both forms of a call (with and without cu_seqlens) fit
  size_t most = 0;
  const int group = hq / hk;
  for (const bool step : {false, true}) {
    if (step && num_seqs != n_tokens) continue;
    const int R = rows_of(num_seqs, n_tokens, group);
    const int64_t nb = item_slots(num_seqs, n_tokens, group, R, step);
    if (nb > kMaxSplitItems) continue;
    const size_t bytes = align16((nb + 1) * sizeof(int32_t)) +
                         static_cast<size_t>(max_ctas(R)) * sizeof(int4) +
                         static_cast<size_t>(max_ctas(R)) * 2 * R * (head_dim + 2) * sizeof(float);
    most = bytes > most ? bytes : most;
  }
  return most;
}

cudaError_t launch_attend_rows(const AttendArgs& a, cudaStream_t stream) {
  const bool step = a.batch.cu == nullptr;
  const int R = rows_of(a.batch.num_seqs, a.batch.n_tokens, a.group);
  const int64_t nb = item_slots(a.batch.num_seqs, a.batch.n_tokens, a.group, R, step);
  if (nb > INT32_MAX) return cudaErrorInvalidValue;
  RowsArgs ra{};
  ra.a = a;
  ra.items = static_cast<int32_t>(nb);
  const int64_t cap = static_cast<int64_t>(a.table.max_pages) << a.pool.page_shift;
  const int64_t most_tiles = ((cap + kTile - 1) / kTile + kLead) * nb;  // per layer and head
  const int64_t lh = static_cast<int64_t>(a.pool.num_layers) * a.pool.hk;
  if (nb <= kMaxSplitItems && cap > (kMinSplitTiles - 1) * kTile && most_tiles <= INT32_MAX / lh) {
    ra.prefix = static_cast<int32_t*>(a.workspace);
    ra.left = reinterpret_cast<int4*>(static_cast<uint8_t*>(a.workspace) +
                                      align16((nb + 1) * sizeof(int32_t)));
    ra.partial = reinterpret_cast<float*>(ra.left + max_ctas(R));
    // no more CTAs than there can be tiles
    const int64_t tiles = most_tiles * lh;
    const int most = max_ctas(R);
    ra.ctas = tiles < most ? static_cast<int32_t>(tiles) : most;
  }
  CUtensorMap k, v;
  if (!encode_pool_maps(a.pool, 16, &k, &v)) return cudaErrorNotSupported;
  switch (a.pool.head_dim) {
    case 64: return R == 8 ? launch<64, 1>(ra, k, v, stream) : launch<64, 2>(ra, k, v, stream);
    case 128: return R == 8 ? launch<128, 1>(ra, k, v, stream) : launch<128, 2>(ra, k, v, stream);
    default: return R == 8 ? launch<256, 1>(ra, k, v, stream) : launch<256, 2>(ra, k, v, stream);
  }
}

bool encode_pool_maps(const Pool& pool, uint32_t rows, CUtensorMap* k, CUtensorMap* v) {
  const int64_t units = static_cast<int64_t>(pool.num_layers) * pool.hk * pool.num_pages;
  if (units > INT32_MAX) return false;
  const uint32_t P = 1u << pool.page_shift;
  const uint32_t W = pool.head_dim < 128 ? pool.head_dim : 128;
  const uint64_t D = static_cast<uint64_t>(pool.head_dim);
  const uint64_t dims[3] = {D, P, static_cast<uint64_t>(units)};
  const uint64_t strides[2] = {D, D * P};
  const uint32_t box[3] = {W, rows, 1};
  return encode_u8_tensor_map(k, pool.k, 3, dims, strides, box, static_cast<int>(W)) &&
         encode_u8_tensor_map(v, pool.v, 3, dims, strides, box, static_cast<int>(W));
}

namespace {

// Which kernels a call needs.  The tcgen05 kernel reads the cache once for 128 rows: for
// more than 16 rows per sequence on average (64 sequences behind 4000, 4 query heads a
// group: 96 us by rows and 93 by tiles for 4 tokens each, 166 and 93 for 5; one behind
// 200000: 69 and 77 us for 4 tokens, 120 and 77 for 8; one behind 100: 17 and 22 us for
// 4), and for more than 8 where the tokens, whose shares only the device knows, may be
// one sequence's.  Up to 8, such a call is shared out: the sequences of more than
// kFewRows rows go to the one kernel, the others to the other.  63 sequences of one
// token behind 2000 and one of 60 behind 100000 take 120 us so and 428 by rows alone, one
// of 128 179 and 876.  Where there was nothing to share out that costs a second launch,
// with a CTA for each row tile that there might be: 8 us for 64 sequences of one token
// behind 4000 (55 to 63), 12 for 64 behind 500 (27 to 39), 27 for 256 (45 to 72), 82 for 1024
// (184 to 266).
// Above 8 rows on average the tcgen05 kernel has the single tokens too, each in a tile of
// 128 rows: 63 of them behind 4000 and a prompt of 2048 take 121 us, and 154 by both.
// A call of up to kSmallCall rows is not shared out.  64 rows, of 13 tokens and three
// single ones: behind 200 tokens 16 us by rows and 26 by tiles, behind 2000 25 and 27, behind
// 20000 57 and 45; of 5 tokens and seven single ones, by rows and by both: 16 and 27, 25
// and 32, 55 and 63.
constexpr int kSmallCall = 64;
constexpr int kFewRows = 32;

struct Kernels {
  bool rows, tiles;
};

Kernels kernels_of(int32_t num_seqs, int64_t n_tokens, int group, bool step) {
  const int64_t rows = n_tokens * group;
  const bool uneven = !step && num_seqs > 1 && rows > kSmallCall;
  const bool tiles = rows > (uneven ? 8 : 16) * static_cast<int64_t>(num_seqs);
  return {!tiles, tiles || uneven};
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& args, cudaStream_t stream) {
  AttendArgs a = args;
  const Kernels k = kernels_of(a.batch.num_seqs, a.batch.n_tokens, a.group, a.batch.cu == nullptr);
  a.min_rows = 0;
  a.max_rows = k.rows && k.tiles ? kFewRows : INT64_MAX;
  if (k.rows) {
    const cudaError_t e = launch_attend_rows(a, stream);
    if (e != cudaSuccess) return e;
    a.min_rows = kFewRows + 1;
    a.max_rows = INT64_MAX;
  }
  if (k.tiles) {
    const cudaError_t e = launch_attend_tiles(a, stream);
    if (e != cudaSuccess) return e;
  }
  note_kernel(!k.tiles ? "attend_rows_kernel"
                       : (k.rows ? "attend_rows_kernel, attend_tiles_kernel" : "attend_tiles_kernel"));
  return cudaSuccess;
}

size_t attend_workspace_bytes(int32_t num_seqs, int64_t n_tokens, int32_t num_layers, int32_t hq,
                              int32_t hk, int32_t head_dim) {
  // both forms of a call (with and without cu_seqlens) fit; of two kernels the second
  // begins when the first has ended
  size_t most = 0;
  for (const bool step : {false, true}) {
    if (step && num_seqs != n_tokens) continue;
    const Kernels k = kernels_of(num_seqs, n_tokens, hq / hk, step);
    const size_t rows = k.rows ? attend_rows_workspace(num_seqs, n_tokens, hq, hk, head_dim) : 0;
    const size_t tiles = k.tiles ? attend_tiles_workspace(num_seqs, num_layers, hk, head_dim) : 0;
    most = rows > most ? rows : most;
    most = tiles > most ? tiles : most;
  }
  return most;
}

}  // namespace kv8
}  // namespace cmr

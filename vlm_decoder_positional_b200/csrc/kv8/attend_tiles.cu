// Attention over the paged 8-bit cache for calls with many query rows: prompts and
// chunks, on tcgen05.
//
// A CTA takes 128 query rows of a KV head (token x query group) and walks over
// tiles of 128 cached tokens.  Both products run in kind::f8f6f4 on the codes as
// they lie in the cache: TMA brings pages into swizzled shared memory, keys are a
// K-major operand, values an MN-major one, and no code is ever converted.  What
// is not 8 bits wide is written as a sum of 8-bit numbers:
//   q = q1 + q2, e4m3, over a power of two per row that brings the row's largest
//       value into (224, 448]: q1 keeps 4 significant bits, q2 those of the rest,
//       together bf16's 8 (values below 2^-8 of the largest lose bits under
//       2^-19 of it);
//   p = p1 + p2 + p3, e5m2: e5m2 is the upper byte of f16, so p1 is the upper byte of
//       p in f16, p2 that of what is left, and p3 that of the rest, rounded: 9
//       significant bits, down to e5m2's smallest number 2^-16.  The row's largest p
//       lies between 2^9 and 2^15, so a weight of 2^-17 of it or more keeps its 9 bits,
//       a smaller one is off by 2^-26 of the largest.  Letting the reference drift less
//       would leave more room below: 2^-28 (base 11, drift 4) takes 2.5 % more time for
//       4 prompts of 8192, 2^-29 5 %, 2^-30 10 %.
// A p that keeps its 9 bits carries about half the rounding of a bf16 weight (2^-9 and the
// 2^-11 of f16 before it, for 2^-8), and S and O are fp32 accumulators in tensor memory.
// The scales enter as in attend_rows.cu: keys' in the exponent's factor, values' in the
// exponent, and 2^-e in the sum of weights, which takes p as it is.
//
// Bound by the tensor cores: 2 x D steps of QK and 3 x 128 of PV at the 8-bit rate
// (twice bf16's) are 1.25 x the time of the same product in bf16.  Converting V
// to f16 in shared memory instead (2 x 128 steps' worth) would pay 96 KB of shared
// memory traffic per tile, more than the third term costs.
//
// Warps: 0 loads, 1 issues the products, 2-3 clear values that must not be seen,
// 4-11 do the softmax: two threads to a row, 64 of a tile's tokens each.  S has two
// buffers, so QK of the next tile runs while this one's softmax does; p's terms take
// the place of S.  The reference of the running softmax moves only when weights pass
// 2^6 times it, and O is scaled again only then.
// Measured, 8 query and 2 KV heads of 256: 4 prompts of 8192 1.0 ms in a short run and
// 1.16 ms in a long one, in which the clock falls to 1.6 GHz under the power limit: 0.95
// PFLOP/s of the plain product's operations, 2.4 of those issued, 8 bits wide.  In copies
// of the kernel with a part left out, 0.70 ms without the products, 1.03 without the
// softmax, 1.11 with the loads of the first tiles only: the products bound it.  8 ragged
// chunks take 16 us of the device.
#include "attend.cuh"
#include "kv8.cuh"
#include "tcgen05.cuh"
#include "../pdl.cuh"
#include "../rotate_common.cuh"
#include "../tma.cuh"

namespace cmr {
namespace kv8 {
namespace {

using rot::bf16_hi;
using rot::bf16_lo;
using rot::pack_bf16x2;

constexpr int kRows = 128;     // query rows of a CTA
constexpr int kTile = 128;     // tokens of a tile
constexpr int kStages = 2;     // K and V tiles in flight
constexpr int kInfos = 4;      // a tile's scales outlive its keys by the softmax
constexpr int kSoftmax = 256;  // threads
constexpr int kCleaners = 64;
constexpr int kFirstWarp = 4;  // of the softmax
constexpr int kThreads = kSoftmax + 32 * kFirstWarp;
constexpr int kPlanned = 256;   // sequences of a call whose items are split
constexpr float kBase = 9.f;   // weights are at most 2^9 when the reference moves
constexpr float kLazy = 6.f;   // and 2^15 before it does
constexpr uint32_t kColumns = 512;

struct TileInfo {
  float k_scale[8];  // per 16 tokens
  float v_log2[8];
  float v_inv[8];
  uint32_t valid;
};

// An item's share of the device: it is walked by n CTAs of `tiles` tiles each, the
// last one of fewer.
struct Piece {
  Item it;
  int32_t lh;    // layer x heads + head, or -1: none
  int32_t all;   // tiles that the item's last row sees
  int32_t tiles;
  int32_t z, n;  // this one's number, of n
  int32_t rec;   // record of the item's first piece, in the head's part; in the kernel, this one's
  int32_t split; // number of the item among the head's split ones; of no piece: how many they are
};

template <int D>
struct Smem {
  static constexpr int W = D < 128 ? D : 128;  // bytes of a swizzled row
  static constexpr int kPanel = kTile * W;     // rows x W: also Q's, of 128 rows
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kQ = 0;  // two terms
  static constexpr int kK = 2 * kRows * D;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kNan = kV + kStages * kTileBytes;
  static constexpr int kMax = kNan + D * 4;             // [2][2][128] floats
  static constexpr int kSum = kMax + 4 * kRows * 4;     // [2][128]
  static constexpr int kAt = kSum + 2 * kRows * 4;      // [128] element offsets, 8 bytes
  static constexpr int kInfo = kAt + kRows * 8;
  static constexpr int kBars = (kInfo + kInfos * static_cast<int>(sizeof(TileInfo)) + 7) / 8 * 8;
  static constexpr int kMisc = kBars + 8 * (5 * kStages + 7);
  static constexpr int kPiece = kMisc + 16;
  static constexpr int kBytes = kPiece + static_cast<int>(sizeof(Piece)) + 1024;  // and room to align
};

struct TilesArgs {
  AttendArgs a;
  int32_t items;    // slots per (layer, head)
  int32_t sms;      // multiprocessors among which items are split; 0: no item is split
  int32_t* count;   // split items of a head in this call
  int32_t room;     // for split items, of a head
  int4* split;      // [heads][room]: what the joining kernel has to know of each
  float* partial;   // [sms] records of a piece: [128][D], then the rows' ref and sum
};

// Items of sequence b, or 0, and the tiles that its last row sees.
__device__ __forceinline__ void weigh(const AttendArgs& a, int32_t b, uint32_t& m, uint32_t& tiles,
                                      bool& odd) {
  m = tiles = 0;
  if (b >= a.batch.num_seqs) return;
  int64_t lo, hi;
  bool cut;
  odd |= !seq_range(a.batch, b, lo, hi);
  if (!takes(a, (hi - lo) * a.group)) return;
  const int64_t p0 = a.batch.pos_offset ? __ldg(a.batch.pos_offset + b) : 0;
  const int64_t vis = visible(a, table_row(a.table, b), p0 + hi - lo, &cut);
  m = static_cast<uint32_t>(((hi - lo) * a.group + kRows - 1) / kRows);
  tiles = static_cast<uint32_t>(max(static_cast<int64_t>(1), (vis + kTile - 1) / kTile));
}

// Piece x of the call; asked by whole warps.  With T tiles in all items (those of a
// sequence's last row tile counted for each of its items) and S multiprocessors, an item
// of t tiles is cut in t S / T pieces, rounded down: the items that are cut have S pieces
// at most, S / heads in each head, and no piece is twice as long as what each
// multiprocessor has to do on average.  Short code: it is fetched anew by every call.
__device__ __forceinline__ Piece find_piece(const TilesArgs& ta, uint32_t x, bool* bad) {
  const AttendArgs& a = ta.a;
  const int lane = threadIdx.x & 31;
  const uint32_t heads = static_cast<uint32_t>(a.pool.num_layers) * a.pool.hk;
  const uint32_t at = x / heads;
  Piece p{};
  p.lh = -1;
  uint32_t m, n;
  bool odd = false;
  unsigned long long tiles = 0;
#pragma unroll 1
  for (int32_t b = lane; b - lane < a.batch.num_seqs; b += 32) {
    weigh(a, b, m, n, odd);
    tiles += static_cast<unsigned long long>(m) * n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(~0u, tiles, o);
  // sequences out of order may overlap: nothing is split then
  odd = __any_sync(~0u, odd);
  *bad |= odd;
  // a little less than S / T, so that rounding adds no piece
  const float per_tile = odd ? 0.f : ta.sms * (1.f - 0x1p-16f) /
                                         (static_cast<float>(tiles) * static_cast<float>(heads));
  uint32_t base = 0, rec = 0;  // pieces, and records + 2^16 x split items, of the sequences before
#pragma unroll 1
  for (int32_t b = lane; b - lane < a.batch.num_seqs; b += 32) {
    if (a.batch.num_seqs > 32) weigh(a, b, m, n, odd);
    n = max(1u, min(n, static_cast<uint32_t>(n * per_tile)));
    const uint32_t mine = m * n, recs = n > 1 ? mine + (m << 16) : 0u;
    uint32_t end = mine, rec_end = recs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(~0u, end, o), v = __shfl_up_sync(~0u, rec_end, o);
      if (lane >= o) {
        end += u;
        rec_end += v;
      }
    }
    end += base;
    rec_end += rec;
    const uint32_t here = __ballot_sync(~0u, at >= end - mine && at < end);
    if (here) {
      const int from = __ffs(here) - 1;
      const uint32_t pieces = __shfl_sync(~0u, n, from);
      const uint32_t k = at - __shfl_sync(~0u, end - mine, from);
      const uint32_t first = __shfl_sync(~0u, rec_end - recs, from);
      const uint32_t last = __shfl_sync(~0u, m, from) - 1;
      b += from - lane;
      int64_t lo, hi;
      seq_range(a.batch, b, lo, hi);
      // the last row tiles, which see most, come first
      const uint32_t item = k / pieces;
      p.it = make_item<kRows>(a, b, lo, hi, static_cast<int32_t>(last - item));
      p.lh = static_cast<int32_t>(x - at * heads);
      p.n = static_cast<int32_t>(pieces);
      p.z = static_cast<int32_t>(k - item * pieces);
      p.all = max(1, (static_cast<int>(p.it.vis_last) + kTile - 1) / kTile);
      p.tiles = (p.all + p.n - 1) / p.n;
      p.rec = static_cast<int32_t>((first & 0xffffu) + item * pieces);
      p.split = static_cast<int32_t>((first >> 16) + item);
      return p;
    }
    base = __shfl_sync(~0u, end, 31);
    rec = __shfl_sync(~0u, rec_end, 31);
  }
  p.split = static_cast<int32_t>(rec >> 16);
  return p;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two fp32 operations in an instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 parts(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The bytes of a word that are e4m3's NaN, as their upper bits.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tiles_kernel(const TilesArgs ta, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map) {
  using S = Smem<D>;
  constexpr int W = S::W;
  constexpr int kPanels = D / W;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (tma::smem_addr(smem_raw) & 1023)) & 1023);
  const AttendArgs& a = ta.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  int* s_nan = reinterpret_cast<int*>(smem + S::kNan);
  float* s_max = reinterpret_cast<float*>(smem + S::kMax);
  float* s_sum = reinterpret_cast<float*>(smem + S::kSum);
  int64_t* s_at = reinterpret_cast<int64_t*>(smem + S::kAt);  // of the query rows, in Q and out
  TileInfo* s_info = reinterpret_cast<TileInfo*>(smem + S::kInfo);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* s_dead = reinterpret_cast<volatile int*>(s_tmem + 1);
  volatile int* s_nan_taken = s_dead + 1;
  Piece* s_piece = reinterpret_cast<Piece*>(smem + S::kPiece);
  const uint32_t q_smem = tma::smem_addr(smem + S::kQ);
  const uint32_t k_smem = tma::smem_addr(smem + S::kK);
  const uint32_t v_smem = tma::smem_addr(smem + S::kV);
  const uint32_t bars = tma::smem_addr(smem + S::kBars);
  const uint32_t k_full = bars, k_empty = bars + 8 * kStages;
  const uint32_t v_full = bars + 16 * kStages, v_empty = bars + 24 * kStages;
  const uint32_t s_full = bars + 32 * kStages, p_full = s_full + 16;
  const uint32_t o_done = s_full + 32, q_ready = s_full + 40, drained = s_full + 48;
  const uint32_t v_clean = s_full + 56;

  if (tid == 0) {
    tma::prefetch_map(&k_map);
    tma::prefetch_map(&v_map);
  }
  pdl::wait();
  // Not before the wait: the kernel ahead may be another's, which signals before it takes
  // tensor memory of its own; it would wait for these columns and this CTA for its end.
  if (warp == 1) tc::alloc(tma::smem_addr(s_tmem), kColumns);
  if (warp == 0) {
    // ---- the item: heavy (late) row tiles first
    bool bad = false;
    Piece piece;
    if (ta.sms > 0) {
      piece = find_piece(ta, blockIdx.x, &bad);
    } else {
      const int32_t lh = static_cast<int32_t>(blockIdx.x) / ta.items;
      piece.it = find_item<kRows>(
          a, ta.items - 1 - (static_cast<int32_t>(blockIdx.x) - lh * ta.items), &bad);
      piece.lh = piece.it.rows > 0 ? lh : -1;
      piece.all = piece.tiles = max(1, (static_cast<int>(piece.it.vis_last) + kTile - 1) / kTile);
      piece.z = 0;
      piece.n = 1;
    }
    if (lane == 0) {
      if (ta.sms > 0) {
        // the last slot is never a piece, unless sequences overlap
        if (blockIdx.x == gridDim.x - 1) *ta.count = piece.lh < 0 ? piece.split : 0;
        if (piece.n > 1 && piece.z == 0) {
          const int n = (piece.all + piece.tiles - 1) / piece.tiles;
          ta.split[piece.lh * ta.room + piece.split] =
              make_int4((n > 1 ? n << 8 : 0) + piece.it.rows, piece.it.first_row,
                        static_cast<int>(piece.it.tok), piece.rec);
        }
        piece.rec += piece.lh * (ta.sms / (a.pool.num_layers * a.pool.hk)) + piece.z;
      }
      *s_piece = piece;
      if (a.status != nullptr) {
        if (bad) atomicOr(a.status, CMR_DEVICE_BAD_CU_SEQLENS);
        if (piece.lh == 0 && piece.z == 0 && piece.it.cut)
          atomicOr(a.status, CMR_DEVICE_CACHE_RANGE);
      }
    }
  } else if (tid == 64) {
    for (int s = 0; s < kStages; ++s) {
      tma::mbar_init(k_full + 8 * s, 1);
      tma::mbar_init(k_empty + 8 * s, 1);
      tma::mbar_init(v_full + 8 * s, 1);
      tma::mbar_init(v_empty + 8 * s, 1);
      tma::mbar_init(v_clean + 8 * s, kCleaners / 32);
    }
    for (int s = 0; s < 2; ++s) {
      tma::mbar_init(s_full + 8 * s, 2);
      tma::mbar_init(p_full + 8 * s, kSoftmax / 32);
    }
    tma::mbar_init(o_done, 1);
    tma::mbar_init(drained, 1);
    tma::mbar_init(q_ready, kSoftmax / 32);
    tma::mbar_init_fence();
    *s_dead = 0;
    *s_nan_taken = 0;
  }
  for (int d = tid; d < D; d += kThreads) s_nan[d] = 0x7fffffff;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const Item it = s_piece->it;
  const int vis_first = static_cast<int>(it.vis_first), vis_last = static_cast<int>(it.vis_last);
  const int t0 = s_piece->z * s_piece->tiles;
  const int nt = min(s_piece->tiles, s_piece->all - t0);
  if (s_piece->lh < 0 || nt <= 0) {
    if (warp == 1) tc::dealloc(*s_tmem, kColumns);
    return;
  }
  const int l = s_piece->lh / a.pool.hk, h = s_piece->lh - l * a.pool.hk;
  const uint32_t tmem = *s_tmem;
  const uint32_t tmem_s[2] = {tmem + 256, tmem + 384};

  // A wait that gives up after its limit ends all later waits of the CTA.
  auto wait = [&](uint32_t bar, int parity) {
    if (tma::mbar_try_wait(bar, static_cast<uint32_t>(parity) & 1u) || *s_dead) return;
    if (!tma::mbar_wait(bar, static_cast<uint32_t>(parity) & 1u)) *s_dead = 1;
  };

  const int P = 1 << a.pool.page_shift;
  if (warp == 0) {
    // ---- loads: lane g < 8 looks after tokens [16g, 16g + 16) of a tile
    uint32_t problems = 0;
    auto look = [&](int i, int32_t& unit, float& ks, float& vs) {
      unit = -1;
      ks = 0.f;
      vs = 1.f;
      const int64_t tok = static_cast<int64_t>(t0 + i) * kTile + 16 * lane;
      if (lane >= 8 || i >= nt || tok >= vis_last) return;
      const int32_t id = page_id(a.table, a.pool.num_pages, it.row, tok >> a.pool.page_shift);
      if (id < 0) {
        problems |= CMR_DEVICE_CACHE_RANGE;
        return;
      }
      const int64_t u = (static_cast<int64_t>(l) * a.pool.num_pages + id) * a.pool.hk + h;
      ks = __ldg(a.pool.ks + u);
      vs = __ldg(a.pool.vs + u);
      if (scale_ok(ks) && scale_ok(vs)) {
        unit = static_cast<int32_t>(u);
      } else {
        problems |= CMR_DEVICE_BAD_SCALE;
        vs = 1.f;
      }
    };
    int32_t unit;
    float ks, vs;
    look(0, unit, ks, vs);
    int keys = 0, values = 0;  // tiles whose loads were issued
    for (int i = 0; i < nt; ++i) {
      const int stage = i % kStages, parity = (i / kStages - 1) & 1;
      const uint32_t valid = __ballot_sync(~0u, unit >= 0) & 0xffu;
      const bool copies = unit >= 0 && (16 * lane) % P == 0;  // first 16 tokens of a page
      const uint32_t bytes = __popc(__ballot_sync(~0u, copies)) * P * D;
      // keys
      if (i >= kStages) wait(k_empty + 8 * stage, parity);
      __syncwarp();
      const bool alive = __all_sync(~0u, *s_dead == 0);
      if (lane < 8) {
        TileInfo& info = s_info[i % kInfos];
        info.k_scale[lane] = ks;
        info.v_log2[lane] = __log2f(vs);
        info.v_inv[lane] = 1.f / vs;
        if (lane == 0) info.valid = valid;
      }
      __syncwarp();
      if (!alive) break;
      if (lane == 0) tma::mbar_arrive_expect_tx(k_full + 8 * stage, bytes);
      __syncwarp();
      if (copies)
        for (int x = 0; x < kPanels; ++x)
          load_3d(k_smem + stage * S::kTileBytes + x * S::kPanel + 16 * lane * W, &k_map,
                  k_full + 8 * stage, x * W, 0, unit);
      ++keys;
      // values
      if (i >= kStages) wait(v_empty + 8 * stage, parity);
      __syncwarp();
      if (!__all_sync(~0u, *s_dead == 0)) break;
      if (lane == 0) tma::mbar_arrive_expect_tx(v_full + 8 * stage, bytes);
      __syncwarp();
      if (copies)
        for (int x = 0; x < kPanels; ++x)
          load_3d(v_smem + stage * S::kTileBytes + x * S::kPanel + 16 * lane * W, &v_map,
                  v_full + 8 * stage, x * W, 0, unit);
      ++values;
      look(i + 1, unit, ks, vs);
    }
    // no copy is left in flight when the CTA ends
    for (int n = max(0, keys - kStages); n < keys; ++n)
      tma::mbar_wait(k_full + 8 * (n % kStages), (n / kStages) & 1);
    for (int n = max(0, values - kStages); n < values; ++n)
      tma::mbar_wait(v_full + 8 * (n % kStages), (n / kStages) & 1);
    if (problems && a.status != nullptr) atomicOr(a.status, static_cast<int>(problems));
  } else if (warp == 1) {
    // ---- products
    if (lane == 0) {
      constexpr uint32_t kQkDesc = tc::instruction(tc::kE4M3, tc::kE4M3, false, kTile);
      constexpr uint32_t kPvDesc = tc::instruction(tc::kE5M2, tc::kE4M3, true, D);
      // The products are issued from straight code, with descriptors that differ by
      // constants: computed in a loop, each cost about 40 cycles of the tensor pipe.
      const uint64_t q_desc = tc::descriptor<W>(q_smem, 0, 8 * W);
      uint64_t k_desc[kStages], v_desc[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) {
        k_desc[s] = tc::descriptor<W>(k_smem + s * S::kTileBytes, 0, 8 * W);
        v_desc[s] = tc::descriptor<W>(v_smem + s * S::kTileBytes, S::kPanel, 8 * W);
      }
      auto keys = [&](int i, int stage, uint64_t kd) {
        wait(k_full + 8 * stage, i / kStages);
        tc::fence_after();
        if (*s_dead) return;
        // passes on what the loads wrote beside the keys; the buffer's last phase is over,
        // since its weights were waited for
        tma::mbar_arrive(s_full + 8 * (i & 1));
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint32_t at = (k * 32 / W) * S::kPanel + (k * 32) % W;
            tc::mma_ss(tmem_s[i & 1], q_desc + ((term * kRows * D + at) >> 4), kd + (at >> 4),
                       kQkDesc, term + k > 0);
          }
        tc::commit(k_empty + 8 * stage);
        tc::commit(s_full + 8 * (i & 1));
      };
      auto values = [&](int j, int stage, uint64_t vd) {
        wait(v_full + 8 * stage, j / kStages);
        wait(v_clean + 8 * stage, j / kStages);
        wait(p_full + 8 * (j & 1), j / 2);
        tc::fence_after();
        if (*s_dead) return;
        const uint32_t p = tmem_s[j & 1];
        // groups of 32 tokens that some row sees
        const int steps = min(kTile / 32, (vis_last - (t0 + j) * kTile + 31) / 32);
        if (steps == kTile / 32) {
#pragma unroll
          for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              tc::mma_ts(tmem, p + term * 32 + k * 8, vd + ((k * 32 * W) >> 4), kPvDesc,
                         term + k > 0 || j > 0);
        } else {
          for (int term = 0; term < 3; ++term)
            for (int k = 0; k < max(1, steps); ++k)
              tc::mma_ts(tmem, p + term * 32 + k * 8, vd + ((k * 32 * W) >> 4), kPvDesc,
                         term + k > 0 || j > 0);
        }
        tc::commit(v_empty + 8 * stage);
        tc::commit(o_done);
      };
      static_assert(kStages == 2, "the loop below takes the stages in turn");
      wait(q_ready, 0);
      tc::fence_after();
      keys(0, 0, k_desc[0]);
      for (int i = 1; i <= nt; i += 2) {
        if (i < nt) keys(i, 1, k_desc[1]);
        values(i - 1, 0, v_desc[0]);
        if (i < nt) {
          if (i + 1 < nt) keys(i + 1, 0, k_desc[0]);
          values(i, 1, v_desc[1]);
        }
      }
      // nothing of the tensor cores is in flight when tensor memory is freed
      if (*s_dead) {
        tc::commit(drained);
        tma::mbar_wait(drained, 0);
      }
    }
    __syncwarp();
  } else if (warp < kFirstWarp) {
    // ---- values that some row does not see.  A weight of zero does not make a NaN
    // vanish: rows that nobody sees are cleared, and a NaN that some query rows see
    // and some do not is taken out and given back, at the end, to those that see it.
    const int ct = tid - 64;
    for (int i = 0; i < nt; ++i) {
      const int tile = (t0 + i) * kTile, stage = i % kStages;
      wait(v_full + 8 * stage, i / kStages);
      const uint32_t valid = s_info[i % kInfos].valid;
      if (tile + kTile > vis_first || valid != 0xffu) {
        uint8_t* v = smem + S::kV + stage * S::kTileBytes;
        // rows before the first that somebody does not see are fine, and those behind
        // the last group of 32 that somebody sees take no part
        const int lo = valid == 0xffu ? max(0, vis_first - tile) : 0;
        const int hi = min(kTile, (max(vis_last - tile, 1) + 31) / 32 * 32);
        constexpr int kChunks = D / 16;  // of a row
        constexpr int kAhead = 8;
        for (int i0 = lo * kChunks + ct; i0 < hi * kChunks; i0 += kCleaners * kAhead) {
          uint4 y[kAhead];
          uint32_t nan = 0;  // chunks that hold one
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int idx = min(i0 + k * kCleaners, hi * kChunks - 1), r = idx / kChunks;
            y[k] = *reinterpret_cast<const uint4*>(
                v + idx % kChunks / (W / 16) * S::kPanel + r * W + idx % (W / 16) * 16);
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int idx = i0 + k * kCleaners, r = idx / kChunks;
            const bool gone = tile + r >= vis_last || !((valid >> (r / 16 & 7)) & 1u);
            const uint32_t any = nan_codes(y[k].x) | nan_codes(y[k].y) | nan_codes(y[k].z) |
                                 nan_codes(y[k].w);
            if (idx < hi * kChunks && gone)
              *reinterpret_cast<uint4*>(v + idx % kChunks / (W / 16) * S::kPanel + r * W +
                                        idx % (W / 16) * 16) = make_uint4(0, 0, 0, 0);
            else if (idx < hi * kChunks && any && tile + r >= vis_first)
              nan |= 1u << k;
          }
          while (nan) {
            const int idx = i0 + (__ffs(nan) - 1) * kCleaners, r = idx / kChunks;
            nan &= nan - 1;
            *s_nan_taken = 1;
            uint32_t* w = reinterpret_cast<uint32_t*>(
                v + idx % kChunks / (W / 16) * S::kPanel + r * W + idx % (W / 16) * 16);
            // logical chunk of this place: the swizzle is its own inverse
            const int c = (swizzled<W>(r, idx % (W / 16)) - r * W) / 16;
            const int d = idx % kChunks / (W / 16) * W + c * 16;
            for (int k = 0; k < 4; ++k) {
              const uint32_t bad = nan_codes(w[k]);
              for (int b = 0; b < 4; ++b)
                if (bad & (0x80u << (8 * b))) atomicMin(&s_nan[d + 4 * k + b], tile + r);
              w[k] &= ~((bad >> 7) * 0xffu);
            }
          }
        }
        tma::fence_async_shared();
      }
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(v_clean + 8 * stage);
    }
    tma::named_sync(6, kSoftmax + kCleaners);  // which NaNs were taken out is known
  } else {
    // ---- softmax: thread (row, half)
    const int st = tid - 32 * kFirstWarp;
    const int half = st / kRows, row = st % kRows;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if (half == 0) {
      const int f = it.first_row + row;
      const int64_t tok = it.tok + f / a.group;
      s_at[row] = ((l * a.batch.n_tokens + tok) * a.hq + h * a.group + f % a.group) * D;
    }
    tma::named_sync(1, kSoftmax);

    // Q over a power of two, as two e4m3 terms: a warp reads whole rows, a 16-byte
    // chunk (8 dims) to a lane
    {
      constexpr int kLanes = D / 8;         // lanes of a row
      constexpr int kAtOnce = 32 / kLanes;  // rows of a warp's load
      constexpr int kLoads = kRows / (kSoftmax / 32) / kAtOnce;
      constexpr int kAhead = kLoads < 16 ? kLoads : 16;
      const int c = lane % kLanes, first = (warp - kFirstWarp) * kAtOnce + lane / kLanes;
#pragma unroll
      for (int n0 = 0; n0 < kLoads; n0 += kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          const int r = first + (n0 + n) * (kSoftmax / 32) * kAtOnce;
          x[n] = r < it.rows ? __ldg(reinterpret_cast<const uint4*>(a.q + s_at[r]) + c)
                             : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          const int r = first + (n0 + n) * (kSoftmax / 32) * kAtOnce;
          const uint32_t w[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = __vmaxs2(mx, w[i] & 0x7fff7fffu);
          mx = max(mx & 0xffffu, mx >> 16);
          if constexpr (kLanes == 32) {
            mx = __reduce_max_sync(~0u, mx);
          } else {
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(~0u, mx, o));
          }
          // s = 2^e with max |q| in (224 s, 448 s]
          int e = static_cast<int>(mx >> 7) - 127 - 8 + ((mx & 0x7fu) > 0x60u ? 1 : 0);
          e = mx == 0 ? 0 : max(-126, e);
          // a negative softmax scale turns q around, so that scores only grow with S
          const float inv = copysignf(__int_as_float((127 - e) << 23), a.scale_log2);
          uint32_t t1[4], t2[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // exact in f16 down to 2^-14, where e4m3 has 2^-9 for its last bit
            const uint32_t q = pack_f16x2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
            t1[i] = f16x2_to_e4m3x2(q);
            t2[i] = f16x2_to_e4m3x2(sub_f16x2(q, e4m3x2_to_f16x2(t1[i])));
          }
          const int off = (8 * c / W) * S::kPanel + swizzled<W>(r, (8 * c % W) / 16) + (c & 1) * 8;
          *reinterpret_cast<uint2*>(smem + S::kQ + off) =
              make_uint2(t1[0] | (t1[1] << 16), t1[2] | (t1[3] << 16));
          *reinterpret_cast<uint2*>(smem + S::kQ + kRows * D + off) =
              make_uint2(t2[0] | (t2[1] << 16), t2[2] | (t2[3] << 16));
          if (c == 0)
            s_sum[r] = mx < 0x7f80u ? fabsf(a.scale_log2) * __int_as_float((127 + e) << 23)
                                    : __int_as_float(0x7fffffff);  // the row becomes NaN
        }
      }
      tma::fence_async_shared();
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(q_ready);
    }
    tma::named_sync(1, kSoftmax);
    const float mult = s_sum[row];  // of S, for the exponent (s_sum is free until the end)
    const int seen = row < it.rows
                         ? static_cast<int>(max(static_cast<int64_t>(0),
                                                min(it.p0 + (it.first_row + row) / a.group + 1,
                                                    it.vis_last)))
                         : 0;

    float ref = -INFINITY, sum = 0.f;
    for (int i = 0; i < nt; ++i) {
      const int tile = (t0 + i) * kTile;
      const TileInfo& info = s_info[i % kInfos];
      wait(s_full + 8 * (i & 1), i / 2);
      tc::fence_after();
      const uint32_t valid = info.valid;
      const bool edge = tile + kTile > vis_first || valid != 0xffu;
      uint32_t x[2][32];
      tc::ld32(x[0], tmem_s[i & 1] + lanes + 64 * half);
      tc::ld32(x[1], tmem_s[i & 1] + lanes + 64 * half + 32);
      tc::wait_ld();

      // the exponent of a weight is S f + c, with f and c of the token's page
      float f[4], c[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f[g] = mult * info.k_scale[4 * half + g];
        c[g] = info.v_log2[4 * half + g];
      }
      if (edge) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int tok = tile + 64 * half + 16 * g + j;
            const float y = fmaf(__uint_as_float(x[g / 2][g % 2 * 16 + j]), f[g], c[g]);
            x[g / 2][g % 2 * 16 + j] = __float_as_uint(
                tok < seen && ((valid >> (4 * half + g)) & 1u) ? y : -INFINITY);
          }
          f[g] = 1.f;
          c[g] = 0.f;
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t* y = x[g / 2] + g % 2 * 16;
        float top = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
#pragma unroll
        for (int j = 2; j < 16; j += 2)
          top = max3(top, __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
        mx = fmaxf(mx, fmaf(top, f[g], c[g]));
      }
      // the row's maximum over both halves; the two warps of these rows have read
      // their parts of S
      float* ex = s_max + (i & 1) * 2 * kRows;
      ex[half * kRows + row] = mx;
      tc::fence_before();
      tma::named_sync(2 + (warp & 3), 64);
      tc::fence_after();
      mx = fmaxf(mx, ex[(1 - half) * kRows + row]);
      const bool move = mx > ref + kLazy;
      if (__any_sync(~0u, move)) {
        const float to = fmaxf(ref, mx);
        const float down = to == -INFINITY ? 1.f : exp2_approx(ref - to);
        ref = to;
        sum *= down;
        if (i > 0) {
          wait(o_done, i - 1);  // S of this tile came after the product of tile i - 2
          tc::fence_after();
#pragma unroll
          for (int d = 0; d < D / 2; d += 32) {
            uint32_t o[32];
            tc::ld32(o, tmem + lanes + half * (D / 2) + d);
            tc::wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * down);
            tc::st32(tmem + lanes + half * (D / 2) + d, o);
          }
        }
      }

      const float shift = (ref == -INFINITY ? 0.f : ref) - kBase;
      uint32_t t1[16], t2[16], t3[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint64_t ff = pair(f[g], f[g]), less = pair(c[g] - shift, c[g] - shift);
        uint64_t part = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 4 tokens: a word of each term
          float p[4];
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const uint32_t* y = x[g / 2] + g % 2 * 16 + 4 * j + k;
            const float2 e = parts(fma2(pair(__uint_as_float(y[0]), __uint_as_float(y[1])), ff, less));
            p[k] = exp2_approx(e.x);
            p[k + 1] = exp2_approx(e.y);
            part = add2(part, pair(p[k], p[k + 1]));
          }
          // three times 3 significant bits, the last ones rounded
          const uint32_t a0 = pack_f16x2(p[0], p[1]), a1 = pack_f16x2(p[2], p[3]);
          const uint32_t b0 = sub_f16x2(a0, a0 & 0xff00ff00u), b1 = sub_f16x2(a1, a1 & 0xff00ff00u);
          const uint32_t c0 = sub_f16x2(b0, b0 & 0xff00ff00u), c1 = sub_f16x2(b1, b1 & 0xff00ff00u);
          t1[4 * g + j] = __byte_perm(a0, a1, 0x7531);
          t2[4 * g + j] = __byte_perm(b0, b1, 0x7531);
          t3[4 * g + j] = __byte_perm(c0 + 0x00800080u, c1 + 0x00800080u, 0x7531);
        }
        sum = fmaf(parts(part).x + parts(part).y, info.v_inv[4 * half + g], sum);
      }
      tc::st16(tmem_s[i & 1] + lanes + 16 * half, t1);
      tc::st16(tmem_s[i & 1] + lanes + 32 + 16 * half, t2);
      tc::st16(tmem_s[i & 1] + lanes + 64 + 16 * half, t3);

      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(p_full + 8 * (i & 1));
    }

    s_sum[half * kRows + row] = sum;
    tma::named_sync(6, kSoftmax + kCleaners);
    sum += s_sum[(1 - half) * kRows + row];
    // a phase's parity tells it from its neighbours only: the last product but one may
    // still be running here, since its keys' successors were multiplied before it
    if (nt > 1) wait(o_done, nt - 2);
    wait(o_done, nt - 1);
    tc::fence_after();
    const bool whole = s_piece->tiles == s_piece->all;
    const float inv = !whole ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);
    // Through shared memory, where Q and the keys have been used for the last time,
    // to rows that a warp writes whole: 16-byte chunks, their place turned by the
    // row so that neither side meets bank conflicts.
    const bool nan_taken = *s_nan_taken != 0;
    const int words = whole ? D / 2 : D;  // of a row: bf16 pairs, or floats
    const int mask = min(words / 4, 32) - 1;
    uint32_t* stage = reinterpret_cast<uint32_t*>(smem) + row * words;
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
      uint32_t o[32];
      const int d = half * (D / 2) + c;
      tc::ld32(o, tmem + lanes + d);
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * inv);
      if (nan_taken) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (s_nan[d + k] < seen) o[k] = 0x7fffffffu;
      }
      if (whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            w[m] = pack_bf16x2(__uint_as_float(o[8 * k + 2 * m]),
                               __uint_as_float(o[8 * k + 2 * m + 1]));
          *reinterpret_cast<uint4*>(stage + 4 * ((d / 8 + k) ^ (row & mask))) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(stage + 4 * ((d / 4 + k) ^ (row & mask))) =
              make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
    float* rec = ta.partial + static_cast<int64_t>(s_piece->rec) * (kRows * (D + 2));
    if (!whole && half == 0) {
      rec[kRows * D + row] = ref;
      rec[kRows * D + kRows + row] = sum;
    }
    tma::named_sync(1, kSoftmax);
    const uint4* from = reinterpret_cast<const uint4*>(smem);
    constexpr int kWarps = kSoftmax / 32;
    if (whole) {
      constexpr int kChunks = D / 8;        // of a row
      constexpr int kAtOnce = 32 / kChunks;  // rows of a warp's store
      const int c = lane % kChunks;
#pragma unroll 4
      for (int n = 0; n < kRows / kWarps / kAtOnce; ++n) {
        const int r = (n * kWarps + warp - kFirstWarp) * kAtOnce + lane / kChunks;
        if (r < it.rows)
          reinterpret_cast<uint4*>(a.out + s_at[r])[c] = from[r * kChunks + (c ^ (r & mask))];
      }
    } else {
      constexpr int kChunks = D / 4;
#pragma unroll 4
      for (int idx = st; idx < it.rows * kChunks; idx += kSoftmax) {
        const int r = idx / kChunks, c = idx % kChunks;
        reinterpret_cast<uint4*>(rec + r * D)[c] = from[r * kChunks + (c ^ (r & mask))];
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, kColumns);
  }
  if (tid == 0 && *s_dead && a.status != nullptr) atomicOr(a.status, CMR_DEVICE_WAIT_TIMEOUT);
}

constexpr int kJoinThreads = 256;

// Joins the pieces of split items: grid (room for split items, shares of the rows).  kSub
// threads share the pieces of four dims of a row.
template <int D, int kSub>
__global__ void __launch_bounds__(kJoinThreads) attend_tiles_join_kernel(const TilesArgs ta) {
  const AttendArgs& a = ta.a;
  pdl::wait();
  pdl::launch_dependents();
  const int per = ta.sms / (a.pool.num_layers * a.pool.hk);
  const int lh = blockIdx.x / ta.room;
  if (static_cast<int>(blockIdx.x) - lh * ta.room >= __ldcg(ta.count)) return;
  const int4 item = __ldcg(ta.split + blockIdx.x);
  const int n = item.x >> 8;  // 0: a row tile that sees one tile only
  const int r0 = blockIdx.y * (kJoinThreads / (D / 4) / kSub);
  if (n == 0 || r0 >= (item.x & 0xff)) return;
  const int l = lh / a.pool.hk, h = lh - l * a.pool.hk;
  constexpr int kLanes = D / 4;
  const int sub = threadIdx.x / kLanes % kSub;
  const int ln = threadIdx.x % kLanes;
  const int r = r0 + threadIdx.x / (kLanes * kSub);
  if (kSub == 1 && r >= (item.x & 0xff)) return;
  const float* rec0 = ta.partial + static_cast<int64_t>(lh * per + item.w) * (kRows * (D + 2));
  float top = -INFINITY;
#pragma unroll 4
  for (int k = sub; k < n; k += kSub)
    top = fmaxf(top, __ldcg(rec0 + k * (kRows * (D + 2)) + kRows * D + r));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  auto add = [&](float ref, float more, const float4& x) {
    const float w = top == -INFINITY ? 0.f : exp2_approx(ref - top);
    sum = fmaf(w, more, sum);
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
  };
#pragma unroll 4
  for (int k = sub; k < n; k += kSub) {
    const float* rec = rec0 + k * (kRows * (D + 2));
    add(__ldcg(rec + kRows * D + r), __ldcg(rec + kRows * D + kRows + r),
        __ldcg(reinterpret_cast<const float4*>(rec + r * D) + ln));
  }
  if constexpr (kSub > 1) {
    static_assert(kSub * kLanes == kJoinThreads, "the CTA's threads share a row");
    __shared__ float4 s_acc[kJoinThreads];
    __shared__ float2 s_ref[kJoinThreads];
    s_acc[threadIdx.x] = acc;
    s_ref[threadIdx.x] = make_float2(top, sum);
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int j = 1; j < kSub; ++j) top = fmaxf(top, s_ref[j * kLanes + ln].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll 4
    for (int j = 0; j < kSub; ++j) {
      const float2 part = s_ref[j * kLanes + ln];
      add(part.x, part.y, s_acc[j * kLanes + ln]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int f = item.y + r;
  uint16_t* dst = a.out + ((l * a.batch.n_tokens + item.z + f / a.group) * a.hq + h * a.group +
                           f % a.group) * D + 4 * ln;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                              pack_bf16x2(acc.z * inv, acc.w * inv));
}

// The multiprocessors that items are split among.  Each CTA works the plan out for itself,
// 32 sequences at a time: with it and without, 64 chunks of 6 tokens behind 500 take 35
// and 25 us, 256 108 and 82, 512 238 and 143, 1024 637 and 277; with one of 100 behind 20000
// among them 72 and 297, 131 and 352, 258 and 423, 661 and 557.  So up to kPlanned sequences;
// and with more heads than half of the multiprocessors no item has two pieces.
int split_among(int32_t num_seqs, int64_t heads) {
  return num_seqs <= kPlanned && 2 * heads <= sm_count() ? sm_count() : 0;
}

template <int D>
cudaError_t launch(const TilesArgs& ta, const CUtensorMap& k, const CUtensorMap& v, int64_t lh,
                   cudaStream_t stream) {
  using S = Smem<D>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(attend_tiles_kernel<D>), S::kBytes, &done);
  if (e != cudaSuccess) return e;
  const unsigned slots = static_cast<unsigned>(ta.items * lh) + ta.sms;
  e = pdl::launch(attend_tiles_kernel<D>, dim3(slots), dim3(kThreads), S::kBytes, stream, true, ta,
                  k, v);
  if (e != cudaSuccess || ta.sms == 0) return e;
  // With few items there are many pieces of each: the threads of a CTA share those of one
  // row.  So and without (two KV heads, replayed from a graph with cold caches): one chunk of
  // 40 tokens behind 20000, 4 slots, 35 and 47 us; two of 100 behind 6000, 16 slots, 43 and
  // 39; four, 32 slots, 57 and 51; eight of 60 behind 3000, 46 slots, 49 and 41.
  constexpr int kPer = kJoinThreads / (D / 4);
  const unsigned room = static_cast<unsigned>(ta.room * lh);
  if (ta.items * lh <= 16)
    return pdl::launch(attend_tiles_join_kernel<D, kPer>, dim3(room, kRows), dim3(kJoinThreads), 0,
                       stream, true, ta);
  return pdl::launch(attend_tiles_join_kernel<D, 1>, dim3(room, kRows / kPer), dim3(kJoinThreads),
                     0, stream, true, ta);
}

}  // namespace

size_t attend_tiles_workspace(int32_t num_seqs, int32_t num_layers, int32_t hk, int32_t head_dim) {
  const size_t sms = split_among(num_seqs, static_cast<int64_t>(num_layers) * hk);
  return sms == 0 ? 0 : 16 + sms * (sizeof(int4) + kRows * (head_dim + 2) * sizeof(float));
}

cudaError_t launch_attend_tiles(const AttendArgs& a, cudaStream_t stream) {
  const Pool& pool = a.pool;
  const int64_t lh = static_cast<int64_t>(pool.num_layers) * pool.hk;
  int64_t items = item_slots(a.batch.num_seqs, a.batch.n_tokens, a.group, kRows,
                             a.batch.cu == nullptr);
  if (items * lh > INT32_MAX - sm_count()) return cudaErrorInvalidValue;
  CUtensorMap k, v;
  if (!encode_pool_maps(pool, 1u << pool.page_shift, &k, &v)) return cudaErrorNotSupported;
  TilesArgs ta{};
  ta.a = a;
  ta.items = static_cast<int32_t>(items);
  ta.sms = split_among(a.batch.num_seqs, lh);
  // Sequences of N tokens in all see at least their own, so that the plan's T is at least
  // heads * group * (N / 128)^2 / sequences: where even a whole row of the table has less
  // than two pieces then, neither the plan nor the joining kernel is needed (4 prompts
  // of 8192: 1175 us instead of 1193).
  const double n = static_cast<double>(a.batch.n_tokens) / kTile;
  const double row = static_cast<double>(a.table.max_pages) * (1 << pool.page_shift) / kTile + 1;
  if (row * ta.sms < 2 * n * n * a.group / a.batch.num_seqs * static_cast<double>(lh)) ta.sms = 0;
  if (ta.sms > 0) {
    if (a.min_rows > 0) {
      // no more sequences than have so many rows, and a tile of each is not full
      const int64_t rows = a.batch.n_tokens * a.group, most = rows / kRows + rows / a.min_rows;
      ta.items = static_cast<int32_t>(items = items < most ? items : most);
    }
    // a split item has two pieces or more
    const int64_t room = ta.sms / lh / 2;
    ta.room = static_cast<int32_t>(items < room ? items : room);
  }
  ta.count = static_cast<int32_t*>(a.workspace);
  ta.split = static_cast<int4*>(a.workspace) + 1;
  ta.partial = reinterpret_cast<float*>(ta.split + ta.sms);
  switch (pool.head_dim) {
    case 64: return launch<64>(ta, k, v, lh, stream);
    case 128: return launch<128>(ta, k, v, lh, stream);
    default: return launch<256>(ta, k, v, lh, stream);
  }
}

}  // namespace kv8
}  // namespace cmr

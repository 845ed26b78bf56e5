// decode_attn: one query token per sequence attends to the sequence's own pages
// and to the pages of a prefix that it shares with others.
//
//   S_j = scale q.k_j,  m = max S_j,  l = sum e^(S_j - m),  O = sum e^(S_j - m) v_j / l
//
// over any split of the keys: parts (O_k, LSE_k) join as
//   LSE = ln sum e^LSE_k,  O = sum e^(LSE_k - LSE) O_k.
//
// Three kernels, each a dependent launch of the one before:
//   prefix_kernel (with prefix groups of more than a few rows)  256 rows (sequence,
//       head) of a group at once against the prefix's keys: its K and V are read once
//       per 256 rows instead of once per sequence.  tcgen05, bound by the tensor cores
//       for many rows, by memory for few.
//   own_kernel   8 or 16 query heads of one KV head of one sequence against its
//       own keys (and the rows of a small group against its prefix).  Each K and V value
//       is used for these few rows only: bound by memory, its matrix products are small
//       (mma.sync m16n8k16).
//   merge_kernel joins the parts of a row.
// The first two spread their work the same way: the key tiles of all units
// (sequence or row tile, KV head) in a row are cut into equal ranges, one per
// CTA, whatever the lengths are.  A unit that lies inside one range is whole;
// of the others a CTA has at most two, the one it begins in and the one it ends
// in, and writes them as parts into its two slots of the workspace.
//
// Rounding.  P goes to the product with V in bf16, V's type, as in the chunk attention: the
// tensor cores take both operands of one type, and P as two bf16 terms would double the
// products.  It costs the result 0.0017-0.0023 (relative L2 against 64 bits) where P in 32
// bits has 0.0016-0.0017, nearly all of it the rounding of the bf16 output.  Sums take the
// unrounded p; scores, maxima, sums, O and the merge are fp32.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace {

using namespace oomb;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum moves when a tile's exceeds it by more than 2^8: sums and
// products are rescaled rarely, and p <= 256 is as exact in bf16 as p <= 1.
constexpr float kRescaleThreshold = 8.0f;

constexpr int kOwnTile = 64;   // keys per tile of own_kernel
constexpr int kPreTile = 128;  // keys, and rows, per tile of prefix_kernel
constexpr int kPreSplit = 1, kPreOwn = 2;  // see pre_meta
constexpr int kFewRows = 16;   // rows of a group that own_kernel takes in one pass over its keys

struct DecodeParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int64_t q_stride, o_stride;
  const int32_t* page_tables;
  const int32_t* seq_lens;
  const int32_t* prefix_pages;
  const int32_t* prefix_lens;
  const int32_t* group_start;
  uint32_t* status;
  int n_seqs, Hq, Hkv, G, P, max_pages, n_groups, max_prefix_pages, num_pages;
  int own_rows;   // query heads of a unit of own_kernel: 8 or 16
  int row_tiles;  // a sequence's units per KV head there
  int own_group_rows; // groups of up to so many rows per KV head are units of own_kernel
  float scale_log2;
  // Workspace.  Part results are normalised O (fp32) and base-2 LSE.
  // own_meta [unit] {first CTA, CTAs}; slots [2 CTA + (0: begins before, 1: ends
  // after this CTA)][rows]; rows [n_seqs Hq]: whole results that the merge joins
  // with the other kernel's.
  int2* own_meta;
  float* own_slot_o;
  float* own_slot_lse;
  float* own_row_o;
  float* own_row_lse;
  // of a prefix: [n_seqs Hq] {first CTA, 4 CTAs + kPreOwn of own_kernel's + kPreSplit of a
  // split unit}; a slot per softmax lane; the second rows are lane 1's of a whole split unit
  int2* pre_meta;
  float* pre_slot_o;
  float* pre_slot_lse;
  float* pre_row_o[2];
  float* pre_row_lse[2];
};

// A length, clamped to what its page table holds.
__device__ __forceinline__ int checked_len(int len, int max_pages, int P, uint32_t* status) {
  const long long most = static_cast<long long>(max_pages) * P;
  if (len >= 0 && len <= most) return len;
  if (status) atomicOr(status, OOMB_DEV_BAD_COUNT);
  return len < 0 ? 0 : static_cast<int>(most);
}

struct Group {
  int lo, hi;  // its sequences
  int len;     // its prefix
};
__device__ __forceinline__ Group group_of(const DecodeParams& p, int j, uint32_t* status) {
  Group r;
  const int lo = p.group_start[j], hi = p.group_start[j + 1];
  r.lo = min(max(lo, 0), p.n_seqs);
  r.hi = min(max(hi, r.lo), p.n_seqs);
  if ((r.lo != lo || r.hi != hi) && status) atomicOr(status, OOMB_DEV_BAD_COUNT);
  r.len = checked_len(p.prefix_lens[j], p.max_prefix_pages, p.P, status);
  return r;
}

// The LSE of a part as the merge takes it: of parts it takes the maximum, which drops
// NaN, so NaN goes as +inf, and exp(inf - inf) is NaN again.
__device__ __forceinline__ float part_lse(float x) { return x != x ? INFINITY : x; }

// Tiles of a length; an empty sequence of own_kernel has one (all masked) per unit,
// which writes its result.
__device__ __forceinline__ int tiles_of(int len, int tile) { return len > 0 ? (len - 1) / tile + 1 : 0; }
__device__ __forceinline__ int own_tiles(int len) { return max(1, tiles_of(len, kOwnTile)); }

// Quotients of 64-bit numbers that nearly always fit 32 bits, where a division
// takes a fifth of the time.
__device__ __forceinline__ long long fast_div(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The CTA's range [t0, t1) of a row of `total` places cut into equal parts, and the
// item (of n) in which t0 lies.  weight(i) gives an item's key tiles and units; each
// unit takes `cost` places more than its tiles, for what its start and end take: as
// many as a CTA has tiles, less one, but at most COST.  All threads sum the weights of
// n / blockDim consecutive items each.
struct Weight {
  long long tiles, units;
};
struct Range {
  long long total, per, t0, t1;
  long long item_at;  // first place of the item
  int item, cost;
};
template <int NT, int COST, class W>
__device__ __forceinline__ Range find_range(int n, W weight) {
  __shared__ Weight warp_sum[NT / 32];
  __shared__ Range sh;
  const int t = threadIdx.x;
  const int each = (n + NT - 1) / NT, i0 = min(n, t * each), i1 = min(n, i0 + each);
  Weight mine{0, 0};
  for (int i = i0; i < i1; ++i) {
    const Weight w = weight(i, true);
    mine.tiles += w.tiles;
    mine.units += w.units;
  }
  Weight inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long a = __shfl_up_sync(0xffffffffu, inc.tiles, d);
    const long long b = COST ? __shfl_up_sync(0xffffffffu, inc.units, d) : 0;
    if ((t & 31) >= d) {
      inc.tiles += a;
      inc.units += b;
    }
  }
  if ((t & 31) == 31) warp_sum[t / 32] = inc;
  __syncthreads();
  Weight before{inc.tiles - mine.tiles, inc.units - mine.units}, all{0, 0};
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const Weight x = warp_sum[w];
    if (w < t / 32) {
      before.tiles += x.tiles;
      before.units += x.units;
    }
    all.tiles += x.tiles;
    all.units += x.units;
  }
  Range r;
  r.cost = 0;
  r.total = all.tiles;
  r.per = fast_div(r.total + gridDim.x - 1, gridDim.x);
  if (COST) {
    r.cost = static_cast<int>(min(max(r.per - 1, 0ll), static_cast<long long>(COST)));
    r.total += r.cost * all.units;
    r.per = fast_div(r.total + gridDim.x - 1, gridDim.x);
  }
  r.t0 = min(r.total, r.per * blockIdx.x);
  r.t1 = min(r.total, r.t0 + r.per);
  long long at = before.tiles + r.cost * before.units;
  const long long end = at + mine.tiles + r.cost * mine.units;
  if (r.t0 < r.t1 && at <= r.t0 && r.t0 < end) {
    int i = i0;
    for (;; ++i) {
      const Weight w = weight(i, false);
      const long long places = w.tiles + r.cost * w.units;
      if (r.t0 < at + places) break;
      at += places;
    }
    sh.item = i;
    sh.item_at = at;
  }
  __syncthreads();
  r.item = sh.item;
  r.item_at = sh.item_at;
  return r;
}

// ---------------------------------------------------------------- own keys
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Barrier of own_kernel's warps 0-3.
__device__ __forceinline__ void consumer_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NT>
struct OwnCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = 2;
  static constexpr int kCtasPerSm = D == 64 ? 4 : NT == 1 ? 3 : 2;  // what shared memory holds
  static constexpr int kTileBytes = kOwnTile * D * 2 * 2;  // K and V
  static constexpr int kQRow = D * 2 + 16;                 // padded: ldmatrix without bank conflicts
  static constexpr int kQBytes = kRows * kQRow;
  static constexpr int kPRow = kOwnTile * 2 + 16;
  static constexpr int kPBytes = kRows * kPRow;
  static constexpr int kSmem = kStages * (kTileBytes + kQBytes) + 2 * kPBytes + 1024;
};

// What the producer tells the consumers of a tile.
struct TileInfo {
  int lim;    // valid keys of the tile, at most kOwnTile
  int bad;    // bit w: the page of keys [16 w, 16 w + 16) is none
  int flags;  // 1: first tile of the unit in this CTA, 2: last one, 4: whole unit, 8: it begins
              // here, 16: of a prefix
  int b, h0, rows;  // the unit: sequence, first query head, query heads
};

// The products are taken with the keys as the 16 rows of an m16n8k16: S^T = K Q^T
// (16 keys x 8 heads), O^T += V^T P^T (16 of D x 8 heads).  With up to 8 heads per
// KV head no row of an instruction is empty, and half the exponentials, registers
// and instructions go that 16 rows of queries would take; more heads are NT = 2
// such columns on the same K and V fragments.
// Warps 0-3 take 16 keys of each tile for the scores (of one page: pages have 16
// tokens or more), exchange P through shared memory, and take a quarter of D each
// for O += P V over all 64 keys: two barriers a tile, but O needs no joining at the
// end of a unit, which short sequences would pay for most.  Warp 4 fills the ring of
// tiles by TMA (K and V of a page and head are neighbours in the pool: one box of
// both per 64 columns).  The number of barriers does not depend on what is found, so
// a wait that gives up leaves nobody behind.
// Bound by memory where sequences are long: 3 x 100-131 thousand keys (745 MB) take
// 113-116 us, 6.4-6.6 TB/s.  A ragged batch (48 sequences, 103 MB) takes 22.0-22.8 us
// alone, 4.6 TB/s: CTAs have 7 tiles each, and their start, the look at lengths and pages,
// takes as long as three.  Three CTAs of two tiles each keep more loads under way than two
// of three (22.6 and 24.6 us); a separate warp for a unit's end costs the registers that
// the third CTA needs.
// Up to 16 query heads per KV head, that is: of more, every 16 are units of their own, which
// read the keys again.  3 x 100-131 thousand keys of 4 KV heads (709 MB) take 117 us with 16
// query heads each, 200 with 24 and 321 with 40; the ragged batch (125 MB) 36, 57 and 80.
//
// PRE: the keys of prefixes with few rows are units too, of up to kRows rows (sequence,
// query head) of a group; items [0, n_groups) are groups, the others sequences.  A sequence
// is the item of its own G rows.
constexpr int kOwnThreads = 160;
template <bool PRE, int ROWS>
struct OwnItem {
  const int32_t* table;  // its pages
  int len;
  int lo, rows;          // first sequence, rows per KV head
  int nt, row_tiles;     // tiles, units per KV head
  __device__ __forceinline__ void set(const DecodeParams& p, int i, int raw_len, int g0, int g1,
                                      uint32_t* status) {
    if (PRE && i < p.n_groups) {
      lo = min(max(g0, 0), p.n_seqs);
      const int hi = min(max(g1, lo), p.n_seqs);
      if ((lo != g0 || hi != g1) && status) atomicOr(status, OOMB_DEV_BAD_COUNT);
      len = checked_len(raw_len, p.max_prefix_pages, p.P, status);
      table = p.prefix_pages + static_cast<size_t>(i) * p.max_prefix_pages;
      rows = (hi - lo) * p.G;
      nt = tiles_of(len, kOwnTile);
      row_tiles = rows <= p.own_group_rows ? (rows + ROWS - 1) / ROWS : 0;
    } else {
      lo = PRE ? i - p.n_groups : i;
      len = checked_len(raw_len, p.max_pages, p.P, status);
      table = p.page_tables + static_cast<size_t>(lo) * p.max_pages;
      rows = p.G;
      nt = own_tiles(len);
      row_tiles = p.row_tiles;
    }
  }
  __device__ __forceinline__ void load(const DecodeParams& p, int i, uint32_t* status) {
    if (PRE && i < p.n_groups)
      set(p, i, p.prefix_lens[i], p.group_start[i], p.group_start[i + 1], status);
    else
      set(p, i, p.seq_lens[PRE ? i - p.n_groups : i], 0, 0, status);
  }
  __device__ __forceinline__ long long weight(const DecodeParams& p) const {
    return static_cast<long long>(nt) * row_tiles * p.Hkv;
  }
};

template <int D, int NT, bool PRE>
__global__ void __launch_bounds__(kOwnThreads, OwnCfg<D, NT>::kCtasPerSm)
    own_kernel(const DecodeParams p, const __grid_constant__ CUtensorMap kvmap) {
  using Cfg = OwnCfg<D, NT>;
  constexpr int kRows = Cfg::kRows;
  using Item = OwnItem<PRE, kRows>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sq = ring + Cfg::kStages * Cfg::kTileBytes;
  uint8_t* sp = sq + Cfg::kStages * Cfg::kQBytes;
  __shared__ uint64_t full[Cfg::kStages], empty[Cfg::kStages];
  __shared__ TileInfo info[Cfg::kStages];
  // of a tile: maxima per warp and whether they move the running ones; of a unit: sums
  __shared__ __align__(16) float sm[2][4][kRows], sl[2][4][kRows];
  __shared__ __align__(16) int moved[2][4];
  __shared__ int out_rows[PRE ? Cfg::kStages : 1][kRows];  // sequence x Hq + head of a unit's rows
  __shared__ int abort_sh, issued_sh, used_sh;
  const int warp = warp_id(), lane = lane_id();
  volatile int* abort_flag = &abort_sh;
  pdl_launch_dependents();
  if (threadIdx.x == 128) prefetch_tensormap(&kvmap);
  if (threadIdx.x == 0) {
    abort_sh = issued_sh = used_sh = 0;
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    fence_mbar_init();
  }
  const int n_items = (PRE ? p.n_groups : 0) + p.n_seqs;
  const Range rg = find_range<kOwnThreads, 0>(n_items, [&](int i, bool note) {
    Item it;
    it.load(p, i, note && blockIdx.x == 0 ? p.status : nullptr);
    return Weight{it.weight(p), 0};
  });
  const int n_mine = static_cast<int>(rg.t1 - rg.t0);

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int lg_p = __ffs(p.P) - 1, lg_r = min(lg_p, 6);
    const int R = 1 << lg_r;                 // rows of a box
    const int slots = kOwnTile >> lg_r;      // boxes of a tile, per 64 columns
    const uint32_t box_bytes = 2u * R * 128;
    const int s = lane / Cfg::kHalves, hf = lane % Cfg::kHalves;  // this lane's box
    const int per = static_cast<int>(rg.per);
    Item it;
    int item = rg.item, tile = 0, g = 0, rt = 0, first_id = -1, ids = 0, issued = 0;
    // the next item's length (and group) and first page ids, under way while this one's
    // tiles are
    int next_len = 0, next_g0 = 0, next_g1 = 0, next_ids = -1;
    auto look_ahead = [&] {
      const int i = item + 1;
      if (i >= n_items) return;
      const bool group = PRE && i < p.n_groups;
      if (group) {
        next_len = p.prefix_lens[i];
        next_g0 = p.group_start[i];
        next_g1 = p.group_start[i + 1];
        if (lane < p.max_prefix_pages)
          next_ids = p.prefix_pages[static_cast<size_t>(i) * p.max_prefix_pages + lane];
      } else {
        const int b = PRE ? i - p.n_groups : i;
        next_len = p.seq_lens[b];
        if (lane < p.max_pages) next_ids = p.page_tables[static_cast<size_t>(b) * p.max_pages + lane];
      }
    };
    bool ok = true;
    if (n_mine > 0) {
      it.load(p, item, nullptr);
      look_ahead();
      const long long off = rg.t0 - rg.item_at;
      const int u = static_cast<int>(fast_div(off, it.nt));
      tile = static_cast<int>(off - static_cast<long long>(u) * it.nt);
      g = u / it.row_tiles;
      rt = u - g * it.row_tiles;
    }
    for (int i = 0; i < n_mine; ++i) {
      const int st = i % Cfg::kStages;
      const bool first = i == 0 || tile == 0, last = i == n_mine - 1 || tile == it.nt - 1;
      const int key0 = tile * kOwnTile;
      // 32 page ids at a time, one per lane
      const int pg0 = key0 >> lg_p;
      if (first_id < 0 || pg0 < first_id || pg0 + slots > first_id + 32) {
        first_id = pg0;
        const int at = pg0 + lane;
        ids = at * static_cast<long long>(p.P) < it.len ? it.table[at] : -1;
      }
      const int page = __shfl_sync(0xffffffffu, ids, (pg0 - first_id + s) & 31);
      const int row0 = key0 + (s << lg_r);  // first token of the box
      const bool here = s < slots && row0 < it.len;
      const bool good = here && page >= 0 && page < p.num_pages;
      const unsigned goods = __ballot_sync(0xffffffffu, good);
      unsigned bad = 0;
      if (goods != __ballot_sync(0xffffffffu, here)) {
        for (int k = 0; k < 4; ++k)  // keys [16 k, 16 k + 16)
          if (key0 + 16 * k < it.len && !((goods >> (((16 * k) >> lg_r) * Cfg::kHalves)) & 1u))
            bad |= 1u << k;
        if (here && !good && hf == 0 && g == 0 && rt == 0) atomicOr(p.status, OOMB_DEV_BAD_PAGE);
      }
      // the unit's rows: row r of the item is head r % G of sequence lo + r / G
      const int r0 = rt * kRows, rows = min(kRows, it.rows - r0);
      int seq = it.lo, head = g * p.G + r0 + lane;
      if (PRE && item < p.n_groups) {
        const int d = (r0 + lane) / p.G;
        seq += d;
        head -= d * p.G;
      }
      // after a wait that ran out nothing is loaded any more, but the merge, which follows
      // all the same, finds every unit's parts where it may look for them
      if (ok && lane == 0) ok = mbar_wait(&empty[st], ((i / Cfg::kStages) & 1) ^ 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      issued += ok;
      if (PRE && ok) {
        if (last && lane < rows) out_rows[st][lane] = seq * p.Hq + head;
        __syncwarp();
      }
      if (ok && lane == 0) {
        // the unit's first tile is this CTA's if it is not further back than its range
        const bool begins = i >= tile, ends = tile == it.nt - 1;
        TileInfo t;
        t.lim = min(kOwnTile, it.len - key0);
        t.bad = static_cast<int>(bad);
        t.flags = (first ? 1 : 0) | (last ? 2 : 0) | (begins && ends ? 4 : 0) | (begins ? 8 : 0) |
                  (PRE && item < p.n_groups ? 16 : 0);
        t.b = seq;
        t.h0 = head;
        t.rows = rows;
        info[st] = t;
        mbar_arrive_expect_tx(&full[st], __popc(goods) * box_bytes + (first ? rows * D * 2 : 0));
      }
      __syncwarp();
      if (ok && good)
        tma_load_4d(ring + st * Cfg::kTileBytes + (hf * slots + s) * box_bytes, &kvmap, &full[st],
                    hf * 64, row0 & (p.P - 1), 2 * g, page);
      if (ok && first && lane < rows)
        bulk_load(sq + st * Cfg::kQBytes + lane * Cfg::kQRow, p.q + seq * p.q_stride + head * D, D * 2,
                  &full[st]);
      if (tile == 0) {
        const int over = it.nt - (n_mine - i);  // its tiles in later CTAs
        const int n = over <= 0 ? 1 : 1 + (over + per - 1) / per;
        if (PRE && item < p.n_groups) {
          if (lane < rows)
            p.pre_meta[static_cast<size_t>(seq) * p.Hq + head] = make_int2(blockIdx.x, 4 * n + kPreOwn);
        } else if (lane == 0) {
          p.own_meta[(static_cast<size_t>(it.lo) * p.Hkv + g) * p.row_tiles + rt] =
              make_int2(blockIdx.x, n);
        }
      }
      // next tile
      if (++tile == it.nt) {
        tile = 0;
        if (++rt == it.row_tiles) {
          rt = 0;
          ++g;
        }
        if (g == p.Hkv) {
          g = 0;
          do {  // groups without keys or rows, and prefix_kernel's, have no tiles
            if (++item >= n_items) break;
            it.set(p, item, next_len, next_g0, next_g1, nullptr);
            first_id = 0;
            ids = next_ids;
            look_ahead();
          } while (it.weight(p) == 0);
        }
      }
    }
    if (lane == 0) {
      issued_sh = issued;
      if (*abort_flag) atomicOr(p.status, OOMB_DEV_WAIT_LIMIT);
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int lg_r = min(__ffs(p.P) - 1, 6), R = 1 << lg_r, slots = kOwnTile >> lg_r;
    const uint32_t box_bytes = 2u * R * 128;
    const uint32_t ring_at = smem_u32(ring), sq_at = smem_u32(sq), sp_at = smem_u32(sp);
    constexpr int MT = D / 64;  // 16-row tiles of this warp's D / 4 rows of O^T
    // ldmatrix addresses in a tile.  K: this warp's 16 keys (slot and row of a box), two
    // chunks of 8 columns.  V transposed: two chunks of 8 of this warp's columns, keys
    // 0-7 and 8-15 of each 16.
    const int kr = ((warp * 16) & (R - 1)) + (lane & 15), kc = lane >> 4;
    const uint32_t k_at = ((warp * 16) >> lg_r) * box_bytes + kr * 128;
    const int col0 = warp * (D / 4);
    const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (col0 % 64) / 8 + ((lane >> 3) & 1);
    const uint32_t v_at = (col0 / 64) * slots * box_bytes + R * 128 + vr * 128;
    // the scores' thread: keys lane / 4 and + 8, heads (lane % 4) 2 + {0, 1}
    const int hd = (lane & 3) * 2;
    uint32_t qf[NT][D / 16][2];
    float acc[NT][MT][4], m[NT][2], l[NT][2];
    int used = 0, n_units = 0;
    bool ok = true;
    for (int i = 0; i < n_mine; ++i) {
      const int st = i % Cfg::kStages, buf = i & 1;
      if (ok) {
        ok = warp_wait(&full[st], (i / Cfg::kStages) & 1, abort_flag);
        if (!ok) {
          *abort_flag = 1;
          if (lane == 0) atomicOr(p.status, OOMB_DEV_WAIT_LIMIT);
        }
      }
      TileInfo t{};
      if (ok) {
        t = info[st];
        ++used;
      }
      const uint32_t tile_at = ring_at + st * Cfg::kTileBytes;
      if (t.flags & 1) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int kk = 0; kk < D / 16; kk += 2)
            ldsm4(sq_at + st * Cfg::kQBytes + (n * 8 + (lane & 7)) * Cfg::kQRow + kk * 32 +
                      (lane >> 3) * 16,
                  qf[n][kk]);
          // rows past the unit's last hold what an earlier unit left: as zeros they ask for no
          // rescaling of the others
          if (n * 8 + lane / 4 >= t.rows)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) qf[n][kk][0] = qf[n][kk][1] = 0;
#pragma unroll
          for (int c = 0; c < MT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][c][e] = 0.f;
          m[n][0] = m[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.f;
        }
      }
      const int lim = t.lim - warp * 16;  // valid keys of this warp
      const bool here = lim > 0 && !((t.bad >> warp) & 1);
      float s[NT][4];
      bool need = false;
      if (here) {
        float s2[NT][4];  // two chains of products
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t kb[4];
          ldsm4(tile_at + k_at + (kk / 4) * slots * box_bytes + ((((kk % 4) * 2 + kc) ^ (kr & 7)) << 4),
                kb);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(kk & 1 ? s2[n] : s[n], kb, qf[n][kk][0], qf[n][kk][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[n][e] = (s[n][e] + s2[n][e]) * p.scale_log2;
            if (lim < 16 && lane / 4 + (e >> 1) * 8 >= lim) s[n][e] = -INFINITY;
          }
          need |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kRescaleThreshold ||
                  fmaxf(s[n][1], s[n][3]) > m[n][1] + kRescaleThreshold;
        }
        need = __any_sync(0xffffffffu, need);
        if (need) {  // the maximum is only taken when a key is too far above the running one
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mt = fmaxf(s[n][e], s[n][e + 2]);
              mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
              mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
              mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
              if (lane < 4) sm[buf][warp][n * 8 + hd + e] = mt;
            }
        }
      }
      if (lane == 0) moved[buf][warp] = need;
      consumer_barrier();
      const int4 mv = *reinterpret_cast<const int4*>(moved[buf]);
      if (mv.x | mv.y | mv.z | mv.w) {
        const int by[4] = {mv.x, mv.y, mv.z, mv.w};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float2 top = make_float2(m[n][0], m[n][1]);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (by[w]) {
              const float2 x = *reinterpret_cast<const float2*>(&sm[buf][w][n * 8 + hd]);
              top = make_float2(fmaxf(top.x, x.x), fmaxf(top.y, x.y));
            }
          const float a0 = top.x > m[n][0] ? fast_exp2(m[n][0] - top.x) : 1.f;
          const float a1 = top.y > m[n][1] ? fast_exp2(m[n][1] - top.y) : 1.f;
          m[n][0] = top.x;
          m[n][1] = top.y;
          l[n][0] *= a0;
          l[n][1] *= a1;
#pragma unroll
          for (int c = 0; c < MT; ++c) {
            acc[n][c][0] *= a0;
            acc[n][c][1] *= a1;
            acc[n][c][2] *= a0;
            acc[n][c][3] *= a1;
          }
        }
      }
      const uint32_t p_at = sp_at + buf * Cfg::kPBytes;
      if (here) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
          const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
          const float p0 = fast_exp2(s[n][0] - m0), p1 = fast_exp2(s[n][1] - m1);
          const float p2 = fast_exp2(s[n][2] - m0), p3 = fast_exp2(s[n][3] - m1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          // P [head][key]: head lane / 4, keys (lane % 4) 2 + {0, 1} and + 8
          const uint32_t at = p_at + (n * 8 + lane / 4) * Cfg::kPRow + warp * 32 + hd * 2;
          sts32(at, transpose8(pack_bf16(p0, p1)));
          sts32(at + 16, transpose8(pack_bf16(p2, p3)));
        }
      }
      if (t.flags & 2) {  // the unit's sums over this warp's keys
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
            if (lane < 4) sl[n_units & 1][warp][n * 8 + hd + e] = l[n][e];
          }
      }
      consumer_barrier();
      if (!ok) continue;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {  // keys [16 ks, 16 ks + 16)
        const int left = t.lim - 16 * ks;
        if (left <= 0) break;
        if ((t.bad >> ks) & 1) continue;
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          ldsm2(p_at + (n * 8 + (lane & 7)) * Cfg::kPRow + ks * 32 + ((lane >> 3) & 1) * 16, pf[n]);
        const uint32_t at = tile_at + v_at + ((16 * ks) >> lg_r) * box_bytes + ((16 * ks) & (R - 1)) * 128;
#pragma unroll
        for (int c = 0; c < MT; ++c) {
          uint32_t va[4];
          ldsm4t(at + (((vc + 2 * c) ^ (vr & 7)) << 4), va);
          if (left < 16) {
            // values behind the end count 0 times, but 0 times NaN is NaN
            const uint32_t lo = (hd < left ? 0xffffu : 0u) | (hd + 1 < left ? 0xffff0000u : 0u);
            const uint32_t hi = (hd + 8 < left ? 0xffffu : 0u) | (hd + 9 < left ? 0xffff0000u : 0u);
            va[0] &= lo;
            va[1] &= lo;
            va[2] &= hi;
            va[3] &= hi;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(acc[n][c], va, pf[n][0], pf[n][1]);
        }
      }
      __syncwarp();
      if (!(PRE && (t.flags & 2)) && lane == 0) mbar_arrive(&empty[st]);
      if (!(t.flags & 2)) continue;

      // ---------------------------------------------------------- end of a unit
      const bool whole = t.flags & 4, direct = !PRE && whole && p.n_groups == 0;
      const bool pre = t.flags & 16;
      const size_t row0 = static_cast<size_t>(t.b) * p.Hq + t.h0;
      const size_t slot0 = (static_cast<size_t>(blockIdx.x) * 2 + (t.flags & 8 ? 1 : 0)) * kRows;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 total = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 x = *reinterpret_cast<const float2*>(&sl[n_units & 1][w][n * 8 + hd]);
          total = make_float2(total.x + x.x, total.y + x.y);
        }
        // a sum is 0 without keys, and NaN (which stays) with a score of NaN or +inf; others are
        // between 1 (the key of the maximum) and 2^8 times the number of keys, where the quick quotient is good to
        // 2 ulp and the quick logarithm to 2^-21, far below the output's step
        const float i0 = total.x != 0.f ? __fdividef(1.f, total.x) : 0.f;
        const float i1 = total.y != 0.f ? __fdividef(1.f, total.y) : 0.f;
        if (warp == 0 && lane < 4) {
          const float lse[2] = {total.x != 0.f ? m[n][0] + __log2f(total.x) : -INFINITY,
                                total.y != 0.f ? m[n][1] + __log2f(total.y) : -INFINITY};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = n * 8 + hd + e;
            if (row >= t.rows) continue;
            if (direct) {
              if (p.lse) p.lse[row0 + row] = kLn2 * lse[e];
            } else if (!whole) {
              p.own_slot_lse[slot0 + row] = part_lse(lse[e]);
            } else {
              (PRE && pre ? p.pre_row_lse[0] : p.own_row_lse)[PRE ? out_rows[st][row] : row0 + row] =
                  part_lse(lse[e]);
            }
          }
        }
        if (direct) {
          const int row = n * 8 + lane / 4;
          __nv_bfloat16* dst = p.o + t.b * p.o_stride + (t.h0 + row) * D + col0 + hd;
#pragma unroll
          for (int c = 0; c < MT; ++c) {
            const uint32_t x = transpose8(pack_bf16(acc[n][c][0] * i0, acc[n][c][1] * i1));
            const uint32_t y = transpose8(pack_bf16(acc[n][c][2] * i0, acc[n][c][3] * i1));
            if (row < t.rows) {
              *reinterpret_cast<uint32_t*>(dst + 16 * c) = x;
              *reinterpret_cast<uint32_t*>(dst + 16 * c + 8) = y;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = n * 8 + hd + e;
            if (row >= t.rows) continue;
            float* dst = !whole ? p.own_slot_o + (slot0 + row) * D
                                : (PRE && pre ? p.pre_row_o[0] : p.own_row_o) +
                                      (PRE ? static_cast<size_t>(out_rows[st][row]) : row0 + row) * D;
            dst += col0 + lane / 4;
#pragma unroll
            for (int c = 0; c < MT; ++c) {
              dst[16 * c] = acc[n][c][e] * (e ? i1 : i0);
              dst[16 * c + 8] = acc[n][c][e + 2] * (e ? i1 : i0);
            }
          }
        }
      }
      ++n_units;
      if (PRE) {  // out_rows of this stage has been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
    }
    if (threadIdx.x == 0) used_sh = used;
  }
  __syncthreads();
  // after an abort, wait (bounded) for loads still landing in shared memory
  if (abort_sh && threadIdx.x == 0)
    for (int i = used_sh; i < issued_sh; ++i)
      mbar_wait_drain(&full[i % Cfg::kStages], (i / Cfg::kStages) & 1);
  __syncthreads();

  pdl_wait();  // complete only after the kernel before: the merge waits for this one alone
}

// ---------------------------------------------------------------- shared prefixes
template <int D>
struct PreCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kPreTile * D * 2;  // Q, K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 10;     // of the ring that K and V tiles share
  static constexpr int kSmem = kTileBytes * (2 + kSlots) + 1024;
  static constexpr uint32_t kTmemCols = 512;
};
constexpr int kPreThreads = 384;

// Steps through the CTA's share.  A unit is one KV head and up to 256 rows of a
// group, 128 for each of the two softmax lanes; both take the same key tile in a
// step.  Where only 128 rows are left, both lanes have these rows and take two key
// tiles a step (`split`), lane 1 every second one.  A unit takes `cost` places behind
// its steps in the row that is cut among the CTAs: a CTA with the end of one unit and the
// start of the next, which take as long as four steps, gets fewer steps (d = 128: 96
// sequences behind 8191 tokens 46.2 -> 43.5 us, 37 behind 32768 55.7 -> 50.3; for d = 64,
// where less is written at the end, the longer ranges cost as much as they save: 256
// behind 8192 tokens 35.4 us without, 37.1 with).
template <int D>
constexpr int kUnitCost = D == 128 ? 4 : 0;
struct PreWalk {
  Group gr;
  int j, g, pair, step;
  int nt, row_tiles;
  int cost, left;  // places of a unit's end; places left of the CTA's range
  int here;        // steps of the current unit in this CTA
  __device__ __forceinline__ void load(const DecodeParams& p, uint32_t* status = nullptr) {
    gr = group_of(p, j, status);
    nt = tiles_of(gr.len, kPreTile);
    const int rows = (gr.hi - gr.lo) * p.G;
    row_tiles = rows > p.own_group_rows ? (rows - 1) / kPreTile + 1 : 0;
  }
  __device__ __forceinline__ bool none() const { return nt == 0 || row_tiles == 0; }
  // steps and units of one KV head
  __device__ __forceinline__ Weight head() const {
    if (none()) return Weight{0, 0};
    return Weight{static_cast<long long>(row_tiles / 2) * nt + (row_tiles & 1) * ((nt + 1) / 2),
                  (row_tiles + 1) / 2};
  }
  __device__ __forceinline__ bool split() const { return 2 * pair + 1 == row_tiles; }
  __device__ __forceinline__ int steps() const { return split() ? (nt + 1) / 2 : nt; }
  __device__ __forceinline__ bool ends() const { return step + here == steps(); }
  // key tile of a lane i steps on; it has none where this is not below nt
  __device__ __forceinline__ int tile(int i, int ln) const {
    return split() ? 2 * (step + i) + ln : step + i;
  }
  // CTAs with steps of this unit, which begins here
  __device__ __forceinline__ int parts(int per) const {
    const int over = steps() - left;
    return over <= 0 ? 1 : 1 + (over + per - 1) / per;
  }
  __device__ __forceinline__ void start(const DecodeParams& p, const Range& r) {
    j = r.item;
    load(p);
    cost = r.cost;
    left = static_cast<int>(r.t1 - r.t0);
    here = 0;
    const Weight h = head();
    const long long off = r.t0 - r.item_at, hp = h.tiles + cost * h.units;
    g = static_cast<int>(fast_div(off, hp));
    const long long rem = off - g * hp;
    pair = static_cast<int>(min(fast_div(rem, nt + cost), h.units - 1));
    step = static_cast<int>(rem - static_cast<long long>(pair) * (nt + cost));
  }
  // On to the next unit with steps of this CTA, if there is one.
  __device__ __forceinline__ bool next(const DecodeParams& p) {
    step += here;
    left -= here;
    here = 0;
    while (left > 0) {
      if (step < steps()) {
        here = min(steps() - step, left);
        return true;
      }
      left -= steps() + cost - step;
      step = 0;
      if (++pair < (row_tiles + 1) / 2) continue;
      pair = 0;
      if (++g < p.Hkv) continue;
      g = 0;
      if (left <= 0) break;
      do {
        ++j;
        load(p);
      } while (none());
    }
    return false;
  }
};

__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}

// A place in a ring of NS slots and the parity of its barriers' phase.
template <int NS>
struct RingPos {
  int slot;
  uint32_t par;
  __device__ __forceinline__ RingPos at(int n) const {  // n <= NS places on
    RingPos r{slot + n, par};
    if (r.slot >= NS) {
      r.slot -= NS;
      r.par ^= 1;
    }
    return r;
  }
};
// Two fp32 values at once, and the largest of three (sm_100).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 256 rows (sequence, query head of the KV head) of a group against 128 keys a
// step.  Warps 0-3 and 4-7 are two softmax lanes of 128 rows each (thread r owns
// row r, TMEM lane r): scores come from TMEM, p = 2^x goes back in their place, O
// is rescaled when the maximum moves, and normalised at the end.  While one lane
// computes, the tensor core does the other's O += P V and next S = Q K^T: one lane
// alone would leave it idle for the softmax's latency.  Warp 8 loads K and V tiles by
// TMA, warp 9 issues the products, in the order
//   S0 S1 | PV0 S0' PV1 S1' | PV0' S0'' PV1' S1'' ...
// so a lane's scores are complete only after its last O += P V: O stands still while
// the lane looks at them.  TMEM columns: S of lane 0 and 1 [0,128) [128,256) (P in
// their first half), O [256,384) [384,512).  Q is in shared memory, written by its
// lane's threads.
// Bound by the tensor cores' clock and the chain of a step for many rows: 256 sequences
// behind 32773 tokens (1792 rows per KV head, 120 GFLOP) take about 129 us at 1.64 GHz
// (1.9 without this load), 930 TFLOP/s.  No one part holds it up: without the exponentials
// the call takes 127 instead of 135 us, without the loads 129, with an eighth of the PV
// products 131.  Two threads per row (139), exponentials by a polynomial for a part of the
// row (137-164), asking for barriers ahead of time (168) and a product warp per lane (174)
// were slower.
template <int D>
__global__ void __launch_bounds__(kPreThreads, 1)
    prefix_kernel(const DecodeParams p, const __grid_constant__ CUtensorMap kvmap) {
  using Cfg = PreCfg<D>;
  constexpr int NS = Cfg::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = sQ + 2 * Cfg::kTileBytes;
  __shared__ uint64_t full[NS], empty[NS];
  __shared__ uint64_t bar_q[2], bar_s[2], bar_p[2][2], bar_fin[2], bar_drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, issued_sh;
  const int warp = warp_id(), lane = lane_id();
  pdl_launch_dependents();
  if (threadIdx.x == 256) prefetch_tensormap(&kvmap);
  if (threadIdx.x == 0) {
    abort_sh = issued_sh = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q[i], 4);
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_p[i][0], 4);
      mbar_init(&bar_p[i][1], 4);
      mbar_init(&bar_fin[i], 1);
    }
    mbar_init(&bar_drain, 1);
    fence_mbar_init();
  }
  const Range rg = find_range<kPreThreads, kUnitCost<D>>(p.n_groups, [&](int j, bool note) {
    PreWalk w;
    w.j = j;
    w.load(p, note && blockIdx.x == 0 ? p.status : nullptr);
    const Weight h = w.head();
    return Weight{h.tiles * p.Hkv, h.units * p.Hkv};
  });
  if (rg.t0 >= rg.t1) return;  // the same for all threads of the CTA
  const int per = static_cast<int>(rg.per);
  if (warp == 8) {
    tmem_alloc(&tmem_base_sh, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;

  if (warp >= 8) {
    // 208 and 88 registers: with 224 and 56 (216 and 72) these warps spill, to L2, as shared
    // memory leaves no L1: 256 sequences behind 32773 tokens 145 (145) us, now 135; with 200
    // and 104 the softmax does, 138 us.  For d = 64, which has not been measured apart, the
    // kernel spills 164 bytes with this split
    reg_dec<88>();
    if (warp == 8) {
      // ---------------------------------------------------------- loads
      PreWalk w;
      w.start(p, rg);
      const int lg_p = __ffs(p.P) - 1, per_tile = kPreTile >> lg_p;
      const int s = lane / Cfg::kHalves, hf = lane % Cfg::kHalves;  // this lane's box
      int ids = 0, ids_j = -1, first_id = 0, issued = 0;
      bool ok = true;
      // tile `t` of the current group: K (which 0) or V (1)
      auto load = [&](int t, int which) {
        const int pg0 = t * per_tile;
        if (ids_j != w.j || pg0 < first_id || pg0 + per_tile > first_id + 32) {
          ids_j = w.j;
          first_id = pg0;
          const int at = pg0 + lane;
          ids = p.num_pages;  // beyond the pool: filled with zeros
          if (static_cast<long long>(at) * p.P < w.gr.len) {
            ids = p.prefix_pages[static_cast<size_t>(w.j) * p.max_prefix_pages + at];
            if (ids < 0 || ids >= p.num_pages) {
              atomicOr(p.status, OOMB_DEV_BAD_PAGE);
              ids = p.num_pages;
            }
          }
        }
        const int page = __shfl_sync(0xffffffffu, ids, (pg0 - first_id + s) & 31);
        const int st = issued % NS;
        int good = 1;
        if (lane == 0) {
          good = mbar_wait(&empty[st], ((issued / NS) & 1) ^ 1, abort_flag);
          if (good) mbar_arrive_expect_tx(&full[st], Cfg::kTileBytes);
        }
        if (!__shfl_sync(0xffffffffu, good, 0)) return false;
        ++issued;
        if (s < per_tile)
          tma_load_4d(ring + st * Cfg::kTileBytes + hf * kPreTile * 128 + ((s << lg_p) * 128), &kvmap,
                      &full[st], hf * 64, 0, 2 * w.g + which, page);
        return true;
      };
      while (ok && w.next(p)) {
        for (int i = 0; ok && i < w.here; ++i) {
          const int ta = w.tile(i, 0), tb = w.tile(i, 1);
          const bool two = w.split() && tb < w.nt;
          ok = load(ta, 0) && (!two || load(tb, 0)) && load(ta, 1) && (!two || load(tb, 1));
        }
      }
      if (lane == 0) {
        issued_sh = issued;
        if (*abort_flag) atomicOr(p.status, OOMB_DEV_WAIT_LIMIT);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- products
      // The whole warp goes through this code with the same values in every lane (those
      // that come from memory are made so by a shuffle): the descriptors then live in
      // uniform registers.  Issued from a branch of one lane, each product first moves
      // its operands there, and takes longer than the tensor core needs for it (256
      // sequences behind 32773 tokens: 213 us so, 153 us in this form).
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
      // low words of the descriptors (address / 16, leading offset); the high words are constant
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
      constexpr uint32_t kTile16 = Cfg::kTileBytes >> 4;
      const uint32_t q_lo = (smem_u32(sQ) >> 4) | (1u << 16);
      const uint32_t k_lo = (smem_u32(ring) >> 4) | (1u << 16);
      const uint32_t v_lo = (smem_u32(ring) >> 4) | (((kPreTile * 128u) >> 4) << 16);
      PreWalk w;
      w.start(p, rg);
      uint32_t par_p[2] = {1, 1}, par_q[2] = {1, 1};  // of a lane's latest P and queries
      RingPos<NS> pos{0, 0};                          // the step's first tile
      bool ok = true;
      auto qk = [&](int ln, RingPos<NS> k, bool arrived, bool release) {  // S = Q K^T
        if (!arrived) ok = ok && warp_wait(&full[k.slot], k.par, abort_flag);
        tc_fence_after();
        const uint32_t a = q_lo + ln * kTile16, b = k_lo + k.slot * kTile16;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (kPreTile * 128) + (kk % 4) * 32) >> 4;
            umma_ss(tmem + ln * 128, desc64(a + off, kHi), desc64(b + off, kHi), idesc_s, kk > 0);
          }
          umma_commit(&bar_s[ln]);
          if (release) umma_commit(&empty[k.slot]);
        }
        __syncwarp();
        par_p[ln] ^= 1;
      };
      auto pv = [&](int ln, RingPos<NS> v, bool arrived, bool fresh, bool release, bool last) {
        if (!arrived) ok = ok && warp_wait(&full[v.slot], v.par, abort_flag);
        const uint32_t b = v_lo + v.slot * kTile16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // O += P V
          ok = ok && warp_wait(&bar_p[ln][half], par_p[ln], abort_flag);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k2 = 0; k2 < kPreTile / 32; ++k2) {
              const int kk = half * (kPreTile / 32) + k2;
              umma_ts(tmem + 256 + ln * 128, tmem + ln * 128 + kk * 8, desc64(b + kk * 128, kHi),
                      idesc_pv, (!fresh || kk > 0) ? 1u : 0u);
            }
            if (half == 1) {
              if (release) umma_commit(&empty[v.slot]);
              if (last) umma_commit(&bar_fin[ln]);
            }
          }
          __syncwarp();
        }
      };
      while (ok && __shfl_sync(0xffffffffu, w.next(p), 0)) {
        // a unit: its steps here, whether lane 1 has a tile of its own, and in the last step
        const int here = __shfl_sync(0xffffffffu, w.here, 0);
        const bool split = __shfl_sync(0xffffffffu, w.split(), 0);
        const bool odd = __shfl_sync(0xffffffffu, w.split() && w.ends() && (w.nt & 1), 0);
        // the lanes' queries come when the old unit's O has been read
        const bool two0 = !(odd && here == 1);
        for (int ln = 0; ln < 1 + two0; ++ln) {
          par_q[ln] ^= 1;
          ok = ok && warp_wait(&bar_q[ln], par_q[ln], abort_flag);
        }
        if (!ok) break;
        if (!split) {
          // both lanes take the same tiles
          qk(0, pos, false, false);
          qk(1, pos, true, true);
          for (int i = 0; ok && i < here; ++i) {
            const bool last = i + 1 == here;
            const RingPos<NS> v = pos.at(1);
            pos = pos.at(2);
            pv(0, v, false, i == 0, false, last);
            if (!last) qk(0, pos, false, false);
            pv(1, v, true, i == 0, true, last);
            if (!last) qk(1, pos, true, true);
          }
        } else {
          // a tile each, lane 1 perhaps none in the last step
          qk(0, pos, false, true);
          if (two0) qk(1, pos.at(1), false, true);
          for (int i = 0; ok && i < here; ++i) {
            const bool more = i + 1 < here, two = more || !odd, ntwo = more && (i + 2 < here || !odd);
            const RingPos<NS> v = pos.at(1 + two);
            pos = pos.at(2 + 2 * two);
            pv(0, v, false, i == 0, true, !more);
            if (more) qk(0, pos, false, true);
            if (two) pv(1, v.at(1), false, i == 0, true, !ntwo);
            if (ntwo) qk(1, pos.at(1), false, true);
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.status, OOMB_DEV_WAIT_LIMIT);
      }
      // every product of this CTA has completed once bar_drain fires
      if (elect_one()) umma_commit(&bar_drain);
      mbar_wait_drain(&bar_drain, 0);
    }
  } else {
    reg_inc<208>();
    // ------------------------------------------------------------ softmax
    const int ln = warp / 4, r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + ln * 128, to = tmem + lane_off + 256 + ln * 128;
    const int lg_p = __ffs(p.P) - 1, per_tile = kPreTile >> lg_p;
    PreWalk w;
    w.start(p, rg);
    float m_used = -INFINITY, l = 0.f;
    size_t out_row = 0;
    int cnt = 0, n_s = 0, n_units = 0;
    bool ok = true, valid = false, begins = false, any = false;
    int seq = 0, h = 0;
    auto begin = [&] {  // this thread's row of the unit, and where its parts will be
      const unsigned rr = (2u * w.pair + (w.split() ? 0 : ln)) * kPreTile + r;
      const unsigned rs = rr / static_cast<unsigned>(p.G);
      seq = w.gr.lo + static_cast<int>(rs);
      h = w.g * p.G + static_cast<int>(rr - rs * p.G);
      valid = seq < w.gr.hi;
      begins = w.step == 0;
      out_row = static_cast<size_t>(seq) * p.Hq + h;
      if (valid && begins && (ln == 0 || !w.split()))
        p.pre_meta[out_row] = make_int2(blockIdx.x, 4 * w.parts(per) + (w.split() ? kPreSplit : 0));
    };
    while (ok && w.next(p)) for (int i = 0; ok && i < w.here; ++i) {
      const bool split = w.split();
      const bool two = !split || w.tile(i, 1) < w.nt, extra = split && two;
      const int vc = cnt + 1 + extra + (extra ? ln : 0);  // ring index of this lane's V tile
      cnt += 2 + 2 * extra;
      const bool mine = ln == 0 || two;
      if (i == 0) {
        begin();
        if (mine) {
          // its query into shared memory (A operand, K-major, 128-byte swizzle)
          const __nv_bfloat16* qrow = p.q + seq * p.q_stride + h * D;
          uint4 v[D / 8];
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch)
            v[ch] = valid ? *reinterpret_cast<const uint4*>(qrow + ch * 8) : make_uint4(0, 0, 0, 0);
          uint8_t* qs = sQ + ln * Cfg::kTileBytes;
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch)
            *reinterpret_cast<uint4*>(qs + (ch / 8) * kPreTile * 128 + sw128_offset(r, (ch % 8) * 8)) =
                v[ch];
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_q[ln]);
        }
        m_used = -INFINITY;
        l = 0.f;
        any = false;
      }
      if (mine) {
        const int tile = w.tile(i, ln);
        // a listed page that is none: its keys are masked (its tile holds zeros)
        bool bad_page = false;
        {
          const int li = tile * per_tile + lane;
          if (lane < per_tile && static_cast<long long>(li) * p.P < w.gr.len) {
            const int id = p.prefix_pages[static_cast<size_t>(w.j) * p.max_prefix_pages + li];
            bad_page = id < 0 || id >= p.num_pages;
          }
        }
        if (!(ok = warp_wait(&bar_s[ln], n_s & 1, abort_flag))) break;
        ++n_s;
        tc_fence_after();
        float s[kPreTile];
#pragma unroll
        for (int c = 0; c < kPreTile / 32; ++c)
          tmem_ld32(ts + c * 32, reinterpret_cast<uint32_t*>(s + c * 32));
        tmem_ld_wait();
        const int lim = w.gr.len - tile * kPreTile;
        if (lim < kPreTile) {
#pragma unroll
          for (int c = 0; c < kPreTile; ++c) s[c] = c < lim ? s[c] : -INFINITY;
          // values behind the end count 0 times, but 0 times NaN is NaN: zero their rows
          if (!(ok = warp_wait(&full[vc % NS], (vc / NS) & 1, abort_flag))) break;
          if (r >= lim) {
#pragma unroll
            for (int hf = 0; hf < Cfg::kHalves; ++hf) {
              uint4* row = reinterpret_cast<uint4*>(ring + (vc % NS) * Cfg::kTileBytes +
                                                    hf * kPreTile * 128 + r * 128);
#pragma unroll
              for (int e = 0; e < 8; ++e) row[e] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_async_smem();
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, bad_page);
        if (bad) {
          uint32_t drop = 0;
          for (int k = 0; k < kPreTile / 16; ++k)
            if ((bad >> ((16 * k) >> lg_p)) & 1u) drop |= 1u << k;
#pragma unroll
          for (int c = 0; c < kPreTile; ++c) s[c] = ((drop >> (c >> 4)) & 1u) ? -INFINITY : s[c];
        }
        // eight chains of maxima of three
        float m8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) m8[e] = max3(s[e], s[8 + e], s[16 + e]);
#pragma unroll
        for (int c = 24; c < kPreTile; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            m8[e] = c + 8 < kPreTile ? max3(m8[e], s[c + e], s[c + 8 + e]) : fmaxf(m8[e], s[c + e]);
        const float mt = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]),
                              fmaxf(m8[6], m8[7])) * p.scale_log2;
        const bool need = mt > m_used + kRescaleThreshold;
        const float m_new = need ? mt : m_used;
        const float alpha = need ? fast_exp2(m_used - m_new) : 1.f;
        if (any && __any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(to + c * 32, o);
          }
          tmem_st_wait();
        }
        any = true;
        m_used = m_new;
        const float neg_mref = m_used == -INFINITY ? 0.f : -m_used;
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), neg2 = pack2(neg_mref, neg_mref);
        uint64_t l2[4] = {0, 0, 0, 0};
        // P in two halves: the first half's product runs while the second is computed
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int q = 2 * half; q < 2 * half + 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float x0, x1;
              unpack2(fma2(pack2(s[32 * q + 2 * c], s[32 * q + 2 * c + 1]), scale2, neg2), x0, x1);
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              l2[c & 3] = add2(l2[c & 3], pack2(p0, p1));
              pk[c] = pack_bf16(p0, p1);
            }
            tmem_st16(ts + q * 16, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_p[ln][half]);
        }
        float la, lb;
        unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), la, lb);
        l = l * alpha + (la + lb);
      }

      if (i == w.here - 1) {
        // ------------------------------------------------ end of a unit
        const bool whole = begins && w.ends();
        const size_t slot_row =
            ((static_cast<size_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * 2 + ln) * kPreTile + r;
        float* od = whole ? p.pre_row_o[split ? ln : 0] + out_row * D : p.pre_slot_o + slot_row * D;
        if (any) {
          if (!(ok = warp_wait(&bar_fin[ln], n_units & 1, abort_flag))) break;
          ++n_units;
          tc_fence_after();
          const float inv = l != 0.f ? 1.f / l : 0.f;
          // half a row at a time through the place of the warp's own queries, which nothing
          // reads any more (other warps may be writing the next unit's into theirs): D / 8
          // lanes then write a row's half together
          constexpr int LPR = D / 8, RPI = 32 / LPR;
          const unsigned long long addr = valid ? reinterpret_cast<unsigned long long>(od) : 0ull;
          uint8_t* qs = sQ + ln * Cfg::kTileBytes;
          auto stage = [&](int row, int ch) {  // 16-byte chunk of a row of the warp
            return reinterpret_cast<float4*>(qs + (ch / 8) * kPreTile * 128 +
                                             sw128_offset((warp & 3) * 32 + row, (ch % 8) * 8));
          };
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tmem_ld16(to + half * (D / 2) + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *stage(lane, 4 * c + e) = make_float4(
                    __uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                    __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
            }
            __syncwarp();
#pragma unroll 4
            for (int it = 0; it < 32 / RPI; ++it) {
              const int sub = it * RPI + lane / LPR, ch = lane % LPR;
              const unsigned long long a = __shfl_sync(0xffffffffu, addr, sub);
              const float4 x = *stage(sub, ch);
              if (a) *reinterpret_cast<float4*>(a + (half * LPR + ch) * 16) = x;
            }
            __syncwarp();
          }
        }
        if (valid)
          *(whole ? p.pre_row_lse[split ? ln : 0] + out_row : p.pre_slot_lse + slot_row) =
              any && l != 0.f ? part_lse(m_used + log2f(l)) : -INFINITY;
        tc_fence_before();  // these reads come before the next unit's products
      }
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(p.status, OOMB_DEV_WAIT_LIMIT);
      while (w.next(p)) begin();  // the merge looks for these parts all the same
    }
  }

  tc_fence_before();
  __syncthreads();
  // After an abort, wait (bounded) for TMA loads still landing in shared memory.
  if (abort_sh && threadIdx.x == 256)
    for (int i = max(0, issued_sh - NS); i < issued_sh; ++i)
      mbar_wait_drain(&full[i % NS], (i / NS) & 1);
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// ---------------------------------------------------------------- merge
// The group of sequence b: the last j with group_start[j] <= b, looked for by a
// warp in steps of 32 (two round trips for up to 1024 groups); -1: none.
__device__ __forceinline__ int find_group(const DecodeParams& p, int b) {
  const int lane = lane_id();
  int base = -1, n = p.n_groups + 1, from = 0;
  while (n > 0) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool le = at < n && p.group_start[from + at] <= b;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) break;
    base = from + (c - 1) * step;
    if (step == 1) break;
    from = base;
    n = min(step, n - (c - 1) * step);
  }
  return base >= 0 && base < p.n_groups ? base : -1;
}

// W warps per row (sequence, head); a lane takes 4 values of a part, a warp
// 128 / D parts at once.  Bound by latency: its launch (a dependent one), the look for a
// row's parts, then the parts, four at a time.  Alone 5.5-6.9 us with 84 rows of up to 150
// parts (W 16) or 1344 rows (W 4), 14 us with 7168 rows of about 10 parts from DRAM
// (W 1, 27 MB); in a call the parts come from L2.
template <int D, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) merge_kernel(const DecodeParams p) {
  constexpr int TPR = D / 4, PPW = 32 / TPR;
  constexpr int kWarps = W > 4 ? W : 4;
  __shared__ float4 sx[kWarps][TPR];
  __shared__ float sm[kWarps], sl[kWarps];
  const int warp = warp_id(), lane = lane_id();
  const long long n_rows = static_cast<long long>(p.n_seqs) * p.Hq;
  const long long row = static_cast<long long>(blockIdx.x) * (kWarps / W) + warp / W;
  const bool active = row < n_rows;
  const int b = active ? static_cast<int>(row / p.Hq) : 0, h = active ? static_cast<int>(row % p.Hq) : 0;
  int n_pre = 0, pre_row_in = 0;  // row of its 256-row unit
  if (p.n_groups > 0 && active) {
    const int j = find_group(p, b);
    if (j >= 0) {
      const Group gr = group_of(p, j, nullptr);
      if (b >= gr.lo && b < gr.hi && gr.len > 0) {
        n_pre = 1;
        pre_row_in = static_cast<int>(
            (static_cast<long long>(b - gr.lo) * p.G + h % p.G) % (2 * kPreTile));
      }
    }
  }
  pdl_wait();
  int2 own = make_int2(0, 0), pre = make_int2(0, 0);
  if (active) {
    own = p.own_meta[(static_cast<size_t>(b) * p.Hkv + h / p.G) * p.row_tiles + h % p.G / p.own_rows];
    if (n_pre) pre = p.pre_meta[row];
    // own_kernel has written this row already
    if (p.n_groups == 0 && own.y == 1) own.y = -1;
  }
  const bool work = active && own.y >= 0;
  const int split = pre.y & kPreSplit, pre_ctas = pre.y >> 2;
  const bool pre_own = pre.y & kPreOwn;
  const int n = work ? own.y + (pre_ctas << split) : 0;
  const int own_row_in = h % p.G % p.own_rows;
  // where part k is: its row in the arrays of O and LSE
  struct Part {
    const float* o;
    const float* lse;
  };
  auto part = [&](int k) {
    Part r;
    if (k < own.y) {
      const size_t slot = static_cast<size_t>(own.x + k) * 2 + (k == 0);
      const size_t at = own.y == 1 ? row : slot * p.own_rows + own_row_in;
      r.o = (own.y == 1 ? p.own_row_o : p.own_slot_o) + at * D;
      r.lse = (own.y == 1 ? p.own_row_lse : p.own_slot_lse) + at;
    } else {
      k -= own.y;
      const int ln = split ? k & 1 : pre_own ? 0 : pre_row_in / kPreTile;
      const int c = k >> split;
      size_t slot = static_cast<size_t>(pre.x + c) * 2 + (c == 0);
      if (!pre_own) slot = slot * 2 + ln;
      const size_t at = pre_ctas == 1   ? static_cast<size_t>(row)
                        : pre_own ? slot * p.own_rows + pre_row_in % p.own_rows
                                       : slot * kPreTile + pre_row_in % kPreTile;
      r.o = (pre_ctas == 1  ? p.pre_row_o[split ? ln : 0]
             : pre_own ? p.own_slot_o
                            : p.pre_slot_o) + at * D;
      r.lse = (pre_ctas == 1  ? p.pre_row_lse[split ? ln : 0]
               : pre_own ? p.own_slot_lse
                              : p.pre_slot_lse) + at;
    }
    return r;
  };
  const int w = warp % W, sub = lane / TPR, d4 = (lane % TPR) * 4;
  // each warp (or part of one) its share of the parts, four loads of LSE and O at
  // once: a running maximum instead of a pass over the LSEs first, which would be one
  // more round trip
  float top = -INFINITY, total = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 4;
  for (int k0 = w * PPW + sub; k0 < n; k0 += kBatch * W * PPW) {
    float lk[kBatch];
    float4 y[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * W * PPW;
      lk[i] = -INFINITY;
      if (k < n) {
        const Part r = part(k);
        lk[i] = *r.lse;
        y[i] = *reinterpret_cast<const float4*>(r.o + d4);
      }
    }
    const float m = fmaxf(fmaxf(fmaxf(lk[0], lk[1]), fmaxf(lk[2], lk[3])), top);
    if (m == -INFINITY) continue;
    const float c = fast_exp2(top - m);
    top = m;
    total *= c;
    x = make_float4(x.x * c, x.y * c, x.z * c, x.w * c);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (lk[i] == -INFINITY) continue;  // no such part, or one without keys
      const float f = fast_exp2(lk[i] - m);
      total += f;
      x.x = fmaf(f, y[i].x, x.x);
      x.y = fmaf(f, y[i].y, x.y);
      x.z = fmaf(f, y[i].z, x.z);
      x.w = fmaf(f, y[i].w, x.w);
    }
  }
  __syncwarp();
  auto join = [&](float t2, float l2, float4 y) {
    const float m = fmaxf(top, t2);
    if (m == -INFINITY) return;
    const float f = fast_exp2(top - m), f2 = fast_exp2(t2 - m);
    top = m;
    total = total * f + l2 * f2;
    x = make_float4(x.x * f + y.x * f2, x.y * f + y.y * f2, x.z * f + y.z * f2,
                    x.w * f + y.w * f2);
  };
#pragma unroll
  for (int d = TPR; d < 32; d *= 2) {
    float4 y;
    y.x = __shfl_xor_sync(0xffffffffu, x.x, d);
    y.y = __shfl_xor_sync(0xffffffffu, x.y, d);
    y.z = __shfl_xor_sync(0xffffffffu, x.z, d);
    y.w = __shfl_xor_sync(0xffffffffu, x.w, d);
    const float t2 = __shfl_xor_sync(0xffffffffu, top, d);
    const float l2 = __shfl_xor_sync(0xffffffffu, total, d);
    join(t2, l2, y);
  }
  if (W > 1) {
    if (sub == 0) sx[warp][lane] = x;
    if (lane == 0) {
      sm[warp] = top;
      sl[warp] = total;
    }
    __syncthreads();
    if (w != 0) return;
    top = -INFINITY;
#pragma unroll
    for (int v = 0; v < W; ++v) top = fmaxf(top, sm[warp + v]);
    total = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float t2 = sm[warp + v];
      const float f = t2 == -INFINITY ? 0.f : fast_exp2(t2 - top);
      const float4 y = sx[warp + v][lane % TPR];
      total = fmaf(f, sl[warp + v], total);
      x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
    }
  }
  if (!work || sub != 0) return;
  const float inv = total != 0.f ? 1.f / total : 0.f;
  *reinterpret_cast<uint2*>(p.o + b * p.o_stride + h * D + d4) =
      make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
  if (lane == 0 && p.lse) p.lse[row] = total != 0.f ? kLn2 * (top + log2f(total)) : -INFINITY;
}

// ---------------------------------------------------------------- host
bool good_shape(int32_t n_seqs, int32_t Hq, int32_t Hkv, int32_t D, int32_t n_groups) {
  return n_seqs >= 0 && n_seqs <= 65535 && Hkv > 0 && Hq > 0 && Hq % Hkv == 0 &&
         supported_head_dim(D) && n_groups >= 0 && n_groups <= n_seqs &&
         static_cast<int64_t>(n_seqs) * Hq <= INT32_MAX;
}

// Groups of up to how many rows (sequences x query heads per KV head) are units of
// own_kernel: none (0), those of one pass over their keys (kFewRows), all (INT_MAX).  The
// kernels look at each group's own size; the host, which does not know the sizes, decides
// whether prefix_kernel is launched at all, from the rows of a group on average and the
// length that prefix_pages has room for.  prefix_kernel takes 128 rows' time for a few, and
// is one more launch; own_kernel reads the keys again for every 16 rows.
// Both ways for equal groups, own_kernel first, d = 128, 4 KV heads: 64 groups of 7 rows
// behind 500 tokens 27 and 39 us; 6 x 14 rows, 16000 tokens 54 and 60; 12 x 28 rows, 1200
// tokens (12 tiles per SM) 25 and 29; 12 x 28 rows, 4000 tokens (41 per SM) 54 and 51; 30 x
// 35 rows, 2000 tokens 92 and 57.  At 17 to 32 rows the bound on the tiles also bounds what one
// group with all of them would take (48 sequences of 7 rows in one of 12 groups, 1200 tokens,
// 26 and 24).
// Few rows on average: if one group had all of them, its passes would take own_kernel, and
// both kernels with each group where it belongs: 210 rows, 500 tokens (3 tiles per SM) 18
// and 20 us; 210 rows, 1000 tokens (6) 28 and 22; 420 rows, 1000 tokens (12) 55 and 28; 1400
// rows, 32773 tokens 1374 and 124.  With both, equal small groups pay 2-3 us for the launch
// (100 of 7 rows, 8000 tokens 406 and 409; 16 of 14 rows, 1000 tokens, 14 per SM, 18 and 20).
// Many rows on average because most sequences have no prefix: prefix_kernel, 6-8 us
// more (4 groups of 7 rows behind 2000 tokens, 96 sequences without 20 and 26; 64 behind 500,
// 336 without 47 and 54).
int prefix_rows_in_own(int n_seqs, int G, int Hkv, int n_groups, int64_t max_len, int sms) {
  if (n_groups == 0) return 0;
  const int64_t rows = static_cast<int64_t>(n_seqs / n_groups) * G;
  const int64_t tiles = Hkv * ((max_len + kOwnTile - 1) / kOwnTile);  // of one pass, one group
  if (rows > kFewRows) return rows <= 32 && 2 * n_groups * tiles <= 16ll * sms ? INT_MAX : 0;
  const int64_t passes = (static_cast<int64_t>(n_seqs) * G + kFewRows - 1) / kFewRows;
  return passes <= 1 || passes * tiles <= 8ll * sms ? INT_MAX : kFewRows;
}
// Rows of a unit of own_kernel: one column of 8, or two.
int own_unit_rows(int G, bool pre) { return G <= 8 && !pre ? 8 : 16; }
int own_ctas(int sms, int D, int rows) {
  return sms * (D == 128 ? rows == 8 ? OwnCfg<128, 1>::kCtasPerSm : OwnCfg<128, 2>::kCtasPerSm
                         : OwnCfg<64, 1>::kCtasPerSm);
}

// Lays the workspace out from `base` (null: only counts) and returns its bytes.
size_t lay_out(uint8_t* base, int n_seqs, int Hq, int Hkv, int D, int n_groups,
               int own_group_rows, int sms, DecodeParams* p) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t rows = static_cast<size_t>(n_seqs) * Hq;
  const int G = Hq / Hkv;
  p->own_group_rows = own_group_rows;
  p->own_rows = own_unit_rows(G, own_group_rows > 0);
  p->row_tiles = (G + p->own_rows - 1) / p->own_rows;
  const size_t own_rows = 2 * static_cast<size_t>(own_ctas(sms, D, p->own_rows)) * p->own_rows;
  const size_t pre_rows = 4 * static_cast<size_t>(sms) * kPreTile;
  p->own_meta = reinterpret_cast<int2*>(take(static_cast<size_t>(n_seqs) * Hkv * p->row_tiles * 8));
  p->own_slot_o = reinterpret_cast<float*>(take(own_rows * D * 4));
  p->own_slot_lse = reinterpret_cast<float*>(take(own_rows * 4));
  p->own_row_o = p->own_row_lse = p->pre_slot_o = p->pre_slot_lse = nullptr;
  p->pre_row_o[0] = p->pre_row_o[1] = p->pre_row_lse[0] = p->pre_row_lse[1] = nullptr;
  p->pre_meta = nullptr;
  if (n_groups > 0) {
    p->own_row_o = reinterpret_cast<float*>(take(rows * D * 4));
    p->own_row_lse = reinterpret_cast<float*>(take(rows * 4));
    p->pre_meta = reinterpret_cast<int2*>(take(rows * 8));
    const bool prefix = own_group_rows < INT_MAX;
    if (prefix) {
      p->pre_slot_o = reinterpret_cast<float*>(take(pre_rows * D * 4));
      p->pre_slot_lse = reinterpret_cast<float*>(take(pre_rows * 4));
    }
    for (int ln = 0; ln < (prefix ? 2 : 1); ++ln) {
      p->pre_row_o[ln] = reinterpret_cast<float*>(take(rows * D * 4));
      p->pre_row_lse[ln] = reinterpret_cast<float*>(take(rows * 4));
    }
  }
  return at;
}

// Bytes of the workspace: enough for every way with the prefixes, which also goes by
// lengths that are not known here.
size_t workspace_bytes(int n_seqs, int Hq, int Hkv, int D, int n_groups, int sms) {
  DecodeParams p;
  size_t bytes = 0;
  for (int own_group_rows : {0, kFewRows, INT_MAX})
    if (own_group_rows == 0 || n_groups > 0)
      bytes = std::max(bytes, lay_out(nullptr, n_seqs, Hq, Hkv, D, n_groups, own_group_rows, sms, &p));
  return bytes;
}

// K and V boxes of `rows` tokens x 64 columns x `both` (1: K or V, 2: K and V).
bool kv_map(CUtensorMap* map, const oomb_pool* pool, uint32_t rows, uint32_t both) {
  const oomb_pool_desc& d = pool->desc;
  const uint64_t D = d.head_dim, P = d.page_size, H2 = 2 * static_cast<uint64_t>(d.num_kv_heads);
  const uint64_t dims[4] = {D, P, H2, static_cast<uint64_t>(d.num_pages)};
  const uint64_t strides[3] = {D * 2, P * D * 2, H2 * P * D * 2};
  const uint32_t box[4] = {64, rows, both, 1};
  return make_bf16_map(map, pool->kv, 4, dims, strides, box);
}

template <int D, int NT, bool PRE>
bool own_attributes() {
  return cudaFuncSetAttribute(own_kernel<D, NT, PRE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              OwnCfg<D, NT>::kSmem) == cudaSuccess;
}

template <int D>
oomb_status launch(const oomb_pool* pool, const DecodeParams& p, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  if (!once_per_device(attr_done, [] {
        return own_attributes<D, 1, false>() && own_attributes<D, 2, false>() &&
               own_attributes<D, 2, true>() &&
               cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    PreCfg<D>::kSmem) == cudaSuccess;
      }))
    return OOMB_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = attr;
  cudaError_t e = cudaSuccess;
  CUtensorMap map;
  const bool prefix = p.n_groups > 0 && p.own_group_rows < INT_MAX;
  if (prefix) {
    if (!kv_map(&map, pool, p.P, 1)) return OOMB_ERR_CUDA;
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(kPreThreads);
    cfg.dynamicSmemBytes = PreCfg<D>::kSmem;
    cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&cfg, prefix_kernel<D>, p, map);
  }
  if (!kv_map(&map, pool, std::min(p.P, kOwnTile), 2)) return OOMB_ERR_CUDA;
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(own_ctas(sms, D, p.own_rows));
    cfg.blockDim = dim3(kOwnThreads);
    cfg.numAttrs = prefix ? 1 : 0;
    cfg.dynamicSmemBytes = p.own_rows == 8 ? OwnCfg<D, 1>::kSmem : OwnCfg<D, 2>::kSmem;
    e = p.own_group_rows  ? cudaLaunchKernelEx(&cfg, own_kernel<D, 2, true>, p, map)
        : p.own_rows == 8 ? cudaLaunchKernelEx(&cfg, own_kernel<D, 1, false>, p, map)
                          : cudaLaunchKernelEx(&cfg, own_kernel<D, 2, false>, p, map);
  }
  if (e == cudaSuccess) {
    const int64_t rows = static_cast<int64_t>(p.n_seqs) * p.Hq;
    // warps per row: as many as keep about every SM's warp slots filled once
    const int w = rows < 4 * sms ? 16 : rows < 16 * sms ? 4 : 1;
    cfg.gridDim = dim3(static_cast<unsigned>(w == 1 ? (rows + 3) / 4 : rows));
    cfg.blockDim = dim3(w == 16 ? 512 : 128);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = w == 16  ? cudaLaunchKernelEx(&cfg, merge_kernel<D, 16>, p)
        : w == 4 ? cudaLaunchKernelEx(&cfg, merge_kernel<D, 4>, p)
                 : cudaLaunchKernelEx(&cfg, merge_kernel<D, 1>, p);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return OOMB_ERR_CUDA;
  }
  return check_launch();
}

}  // namespace

extern "C" size_t oomb_decode_attn_workspace_size(int32_t n_seqs, int32_t num_q_heads,
                                                  int32_t num_kv_heads, int32_t head_dim,
                                                  int32_t n_groups) {
  if (!good_shape(n_seqs, num_q_heads, num_kv_heads, head_dim, n_groups)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = 0;
  }
  return workspace_bytes(n_seqs, num_q_heads, num_kv_heads, head_dim, n_groups, sm_count(dev));
}

extern "C" oomb_status oomb_decode_attn(oomb_pool* pool, const oomb_decode_args* a, void* stream) {
  if (!pool || !a || pool->desc.location != OOMB_LOC_DEVICE) return OOMB_ERR_INVALID_ARG;
  const oomb_pool_desc& d = pool->desc;
  const int D = d.head_dim, Hq = a->num_q_heads;
  if (a->head_dim != D || a->device != d.device) return OOMB_ERR_INVALID_ARG;
  if (!good_shape(a->n_seqs, Hq, d.num_kv_heads, D, a->n_groups)) return OOMB_ERR_INVALID_ARG;
  // the exponentials are powers of 2: an infinite factor would make scores of 0 NaN
  const float scale_log2 = a->softmax_scale * kLog2e;
  if (!(a->softmax_scale > 0.f && scale_log2 <= FLT_MAX)) return OOMB_ERR_INVALID_ARG;
  if (a->n_seqs == 0) return OOMB_OK;
  const int64_t width = static_cast<int64_t>(Hq) * D;
  if (!a->q || !a->o || !aligned16(a->q) || !aligned16(a->o) || a->q_stride % 8 ||
      a->o_stride % 8 || a->q_stride < width || a->o_stride < width)
    return OOMB_ERR_INVALID_ARG;
  if (a->q == a->o && a->n_seqs > 1 && a->q_stride != a->o_stride) return OOMB_ERR_INVALID_ARG;
  if (a->max_pages <= 0 || !a->page_tables || !a->seq_lens) return OOMB_ERR_INVALID_ARG;
  if (a->n_groups > 0 &&
      (a->max_prefix_pages <= 0 || !a->prefix_pages || !a->prefix_lens || !a->group_start))
    return OOMB_ERR_INVALID_ARG;
  DecodeParams p;
  const int sms = sm_count(d.device);
  const int own_group_rows =
      prefix_rows_in_own(a->n_seqs, Hq / d.num_kv_heads, d.num_kv_heads, a->n_groups,
                         static_cast<int64_t>(a->max_prefix_pages) * d.page_size, sms);
  if (!a->workspace || !aligned16(a->workspace) ||
      a->workspace_bytes < workspace_bytes(a->n_seqs, Hq, d.num_kv_heads, D, a->n_groups, sms))
    return OOMB_ERR_INVALID_ARG;
  lay_out(static_cast<uint8_t*>(a->workspace), a->n_seqs, Hq, d.num_kv_heads, D, a->n_groups,
          own_group_rows, sms, &p);
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.o = static_cast<__nv_bfloat16*>(a->o);
  p.lse = a->lse;
  p.q_stride = a->q_stride;
  p.o_stride = a->o_stride;
  p.page_tables = a->page_tables;
  p.seq_lens = a->seq_lens;
  p.prefix_pages = a->prefix_pages;
  p.prefix_lens = a->prefix_lens;
  p.group_start = a->group_start;
  p.status = pool->d_status;
  p.n_seqs = a->n_seqs;
  p.Hq = Hq;
  p.Hkv = d.num_kv_heads;
  p.G = Hq / d.num_kv_heads;
  p.P = d.page_size;
  p.max_pages = a->max_pages;
  p.n_groups = a->n_groups;
  p.max_prefix_pages = a->max_prefix_pages;
  p.num_pages = d.num_pages;
  p.scale_log2 = scale_log2;
  DeviceGuard guard(d.device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch<128>(pool, p, sms, s) : launch<64>(pool, p, sms, s);
}

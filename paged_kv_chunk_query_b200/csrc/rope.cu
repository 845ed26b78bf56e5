// kv_append_rope: keys and values of a ragged batch of tokens into the pages of
// their sequences, keys and queries rotated by their positions on the way; and
// its backward, which takes the paged fp32 gradients out token-major and
// rotates them back.  Page means: by the same CTAs for few tokens per sequence, else by
// a second, dependent launch (page_mean_kernel).
//
// Rotation of pair i of a token at position p by the angle a = p f_i:
//   y_a = x_a cos a - x_b sin a,   y_b = x_b cos a + x_a sin a,
// the inverse with -sin a.  The kernels move bytes: a value is read and written
// once and takes 3 flops, so they are bound by memory.  Everything else is kept
// off that path: a CTA computes its tokens' angles once, in 64 bits, for all
// heads, and keeps cos and sin in shared memory.
#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace {

using namespace oomb;

constexpr int kThreads = 256;
constexpr int kMeanThreads = 512;
constexpr int kMeanCtas = 3;  // per SM, of one token each, that take page means too
constexpr int kMaxTile = 32; // tokens per CTA
constexpr int kMaxHalf = 64; // pairs of a head
constexpr int kMaxCount = 1 << 30;  // tokens, sequences: their sums with a tile stay in 32 bits
constexpr int kBatch = 3;    // rounds of loads that a warp has under way

struct RopeParams {
  const int32_t* seq_start;
  const int32_t* cached_lens;
  const int32_t* page_tables;
  const int32_t* positions;
  const float* inv_freq;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  __nv_bfloat16* kv;
  float* grad;
  float* summary;
  uint32_t* status;
  int n_tokens, n_seqs, max_pages, Hq, Hkv, P, num_pages;
  int half;         // rotated pairs of a head
  int interleaved;
  int lg_p;         // log2(P)
  int tile;         // tokens per CTA
  int batch;        // rounds of heads per piece, at most kBatch
};

// Where the tokens [t0, t0 + n) of a CTA go.
struct Places {
  int page[32];  // physical page; < 0: the token is not written
  int row[32];
  int last[32];  // it is the last token that this call puts into its page
  int first[32]; // row of the first one
  int used[32];  // the token belongs to a sequence (its queries are rotated)
};

// Finds the sequence of each of the CTA's n <= 32 tokens: its index is the number
// of starts <= t, less one.  count_starts: all threads look through seq_start
// together (one round trip for up to 256 sequences, where a binary search would
// take eight): starts up to t0 are counted, those inside the tile marked.  After
// a barrier, warp 0 looks the places up (find_places).  `note`: report what is
// wrong (one kernel of a call does).
__device__ __forceinline__ void count_starts(const RopeParams& p, int t0, int n, int first,
                                             int* mark) {
  const int t = threadIdx.x;
  if (t < 32) mark[t] = 0;
  __syncthreads();
  int before = 0;
  for (int i = t, s = first; i <= p.n_seqs;) {
    if (s <= t0) ++before;
    else if (s < t0 + n) atomicAdd(&mark[s - t0], 1);
    if ((i += blockDim.x) <= p.n_seqs) s = p.seq_start[i];
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (before && t % 32 == 0) atomicAdd(&mark[0], before);
  __syncthreads();
}
__device__ __forceinline__ void find_places(const RopeParams& p, int t0, int n, Places* out,
                                            const int* mark, bool note) {
  const int t = threadIdx.x;  // < 32
  int seq = mark[t];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, seq, d);
    if (t >= d) seq += v;
  }
  --seq;
  int page = -1, row = 0, last = 0, first = 0, used = 0;
  if (t < n && seq >= 0 && seq < p.n_seqs) {
    const int tok = t0 + t, lo = p.seq_start[seq], hi = p.seq_start[seq + 1];
    const int cached = p.cached_lens[seq];
    uint32_t bad = 0;
    if (lo < 0 || tok < lo || tok >= hi || hi > p.n_tokens) {
      bad = OOMB_DEV_BAD_COUNT;  // starts that decrease or leave the batch
    } else {
      used = 1;
      const long long c = static_cast<long long>(cached) + (tok - lo);
      const long long pi = c >> p.lg_p;
      if (cached < 0 || pi >= p.max_pages) {
        bad = OOMB_DEV_BAD_COUNT;
      } else {
        row = static_cast<int>(c) & (p.P - 1);
        page = p.page_tables[static_cast<size_t>(seq) * p.max_pages + pi];
        last = row == p.P - 1 || tok + 1 == hi;
        first = static_cast<int>(max(cached - (pi << p.lg_p), 0ll));
        if (page < 0 || page >= p.num_pages) {
          bad = OOMB_DEV_BAD_PAGE;
          page = -1;
        }
      }
    }
    if (bad && note) atomicOr(p.status, bad);
  }
  out->page[t] = page;
  out->row[t] = row;
  out->last[t] = last;
  out->first[t] = first;
  out->used[t] = used;
}

// cos and sin of pos * f, each rounded once to fp32.  pos * f has up to 55
// bits and its turns up to 31 bits before the point: the product, its rounding
// error and 1 / 2 pi in two parts keep the fraction of a turn to about 2^-52
// at every position, where fp32 would have no bits of it left at 2^24.
__device__ __forceinline__ void turn(int pos, float f, float* c, float* s) {
  constexpr double kInv2Pi = 0.15915494309189535;        // fl(1 / 2 pi)
  constexpr double kInv2PiLo = -9.839338337591243e-18;   // 1 / 2 pi - fl(1 / 2 pi)
  const double x = pos, y = f;
  const double a = x * y, a_lo = fma(x, y, -a);
  const double t = a * kInv2Pi;
  const double e = fma(a, kInv2Pi, -t) + (a * kInv2PiLo + a_lo * kInv2Pi);
  double ds, dc;
  sincospi(2.0 * ((t - rint(t)) + e), &ds, &dc);
  *c = static_cast<float>(dc);
  *s = static_cast<float>(ds);
}

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// Rotates eight pairs in place, of a lane's two 8-value vectors x and y of a
// head: pair i = (x[i], y[i]), or neighbours in x (i < 4) and in y.  Products and
// sums are rounded one by one (no contraction): what is stored is then the plain
// formula's value in fp32.
template <bool BACK, bool IL>
__device__ __forceinline__ void rotate(float* x, float* y, const float* cs, const float* sn) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 c4 = *reinterpret_cast<const float4*>(cs + 4 * q);
    const float4 s4 = *reinterpret_cast<const float4*>(sn + 4 * q);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * q + e;
      float& pa = IL ? (q == 0 ? x[2 * e] : y[2 * e]) : x[i];
      float& pb = IL ? (q == 0 ? x[2 * e + 1] : y[2 * e + 1]) : y[i];
      const float a = pa, b = pb;
      const float bs = __fmul_rn(b, s[e]), as = __fmul_rn(a, s[e]);
      pa = BACK ? __fadd_rn(__fmul_rn(a, c[e]), bs) : __fsub_rn(__fmul_rn(a, c[e]), bs);
      pb = BACK ? __fsub_rn(__fmul_rn(b, c[e]), as) : __fadd_rn(__fmul_rn(b, c[e]), as);
    }
  }
}

// The representative of the page into which token `tok` goes, row `row`, the last row
// written by this call: the mean of the keys of rows [0, row].  Rows from `first` on are
// this call's, possibly written by other CTAs: their keys are rotated anew from the
// inputs, the others read from the page.  All threads of a CTA: a KV head has `share`
// warps, a row UPH lanes as in rope_kernel.  cs, sn: the token's angles, and place for those
// of kMaxTile tokens.
template <int D, bool IL>
__device__ __forceinline__ void mean_of_page(const RopeParams& p, int tok, int page, int row,
                                             int first, float* cs, float* sn) {
  constexpr int UPH = D / 16, RPW = 32 / UPH, kWarps = kThreads / 32;
  constexpr int kRows = 4;  // rows under way per lane
  __shared__ __align__(16) float red[kWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int u = lane % UPH, sub = lane / UPH;
  const bool turned = u < p.half / 8;
  const int ea = !IL && turned ? 8 * u : 16 * u;
  const int eb = !IL && turned ? ea + p.half : ea + 8;
  int share = 1;
  while (2 * share <= kWarps && 2 * share * p.Hkv <= kWarps) share *= 2;
  const int part = warp % share, step = share * RPW;
  auto add = [](float* acc, const uint4& v) {
    float x[8];
    unpack8(v, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += x[e];
  };
  auto sum_stored = [&](int g, float* ax, float* ay) {  // rows [0, first)
    const __nv_bfloat16* src = p.kv + (static_cast<size_t>(page) * p.Hkv + g) * 2 * p.P * D;
    for (int r0 = part * RPW + sub; r0 < first; r0 += kRows * step) {
      uint4 a[kRows], b[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (r0 + i * step < first) {
          a[i] = *reinterpret_cast<const uint4*>(src + (r0 + i * step) * D + ea);
          b[i] = *reinterpret_cast<const uint4*>(src + (r0 + i * step) * D + eb);
        }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (r0 + i * step >= first) break;
        add(ax, a[i]);
        add(ay, b[i]);
      }
    }
  };
  auto sum_new = [&](int g, int from, int to, float* ax, float* ay) {  // their angles in cs, sn
    for (int r = from + part * RPW + sub; r < to; r += step) {
      const __nv_bfloat16* src = p.k + (static_cast<int64_t>(tok) - row + r) * p.k_stride + g * D;
      uint4 a = *reinterpret_cast<const uint4*>(src + ea), b = *reinterpret_cast<const uint4*>(src + eb);
      if (turned) {
        float x[8], y[8];
        unpack8(a, x);
        unpack8(b, y);
        const int at = (r - from) * p.half + 8 * u;
        rotate<false, IL>(x, y, cs + at, sn + at);
        a = pack8(x);  // as stored
        b = pack8(y);
      }
      add(ax, a);
      add(ay, b);
    }
  };
  const int g = warp / share;  // Hkv <= kWarps
  const bool active = g < p.Hkv;
  float x[8], y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
  if (active) {
    sum_stored(g, x, y);
    if (first == row) sum_new(g, row, row + 1, x, y);
  }
  if (first < row) {  // angles of kMaxTile rows at a time
    for (int r = first; r <= row; r += kMaxTile) {
      const int to = min(row + 1, r + kMaxTile);
      __syncthreads();
      for (int i = threadIdx.x; i < (to - r) * p.half; i += kThreads)
        turn(p.positions[tok - row + r + i / p.half], p.inv_freq[i % p.half], cs + i, sn + i);
      __syncthreads();
      if (active) sum_new(g, r, to, x, y);
    }
  }
#pragma unroll
  for (int m = UPH; m < 32; m *= 2)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] += __shfl_xor_sync(0xffffffffu, x[e], m);
      y[e] += __shfl_xor_sync(0xffffffffu, y[e], m);
    }
  if (sub == 0) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      *reinterpret_cast<float4*>(red[warp] + ea + e) = *reinterpret_cast<const float4*>(x + e);
      *reinterpret_cast<float4*>(red[warp] + eb + e) = *reinterpret_cast<const float4*>(y + e);
    }
  }
  __syncthreads();
  const float n = static_cast<float>(row + 1);
  for (int i = threadIdx.x; i < p.Hkv * D; i += kThreads) {
    const int w = i / D, e = i % D;
    float total = red[w * share][e];
    for (int k = 1; k < share; ++k) total += red[w * share + k][e];
    p.summary[static_cast<size_t>(page) * p.Hkv * D + i] = total / n;
  }
}

// One CTA: `tile` <= 32 tokens.  A warp takes heads of a token (counted K, V, then Q)
// 32 / (D / 16) at a time, `batch` <= kBatch times; these pieces of all the CTA's
// tokens are dealt out to its warps in turn.  A lane has the same two 16-byte vectors
// of each head, values [ea, ea + 8) and [eb, eb + 8), chosen so that eight pairs lie in
// them.  The loads of a warp's first piece are issued before the angles and places are
// known.
// A chunk of 4096 tokens (28 query, 4 KV heads of 128) moves 92 MB in 16.6-17.4 us alone
// and cold (5.3-5.5 TB/s), its backward 84 MB in 16.4-16.5 (5.1 TB/s).  Between the floor and
// this stand the start (places and angles, about 3 us before the first store) and the
// issue slots (57% used).  One wave of CTAs, four per SM: three, or seven warps each so
// that the mean kernel fits beside, were slower (24.6 us with the means, now 20.5).
//
// MEAN (CTAs of one token): the page means too, see mean_of_page.
template <int D, bool BWD, bool IL, bool MEAN>
__global__ void __launch_bounds__(kThreads, MEAN ? kMeanCtas : 4) rope_kernel(const RopeParams p) {
  constexpr int UPH = D / 16;       // lanes per head
  constexpr int HPP = 32 / UPH;     // heads of a warp at once
  __shared__ Places pl;
  __shared__ int mark[32];
  __shared__ __align__(16) float cs[kMaxTile * kMaxHalf], sn[kMaxTile * kMaxHalf];
  if (!BWD && !MEAN) pdl_launch_dependents();
  const int t0 = blockIdx.x * p.tile;
  const int n = min(p.tile, p.n_tokens - t0);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int u = lane % UPH;
  const bool turned = u < p.half / 8;
  const int ea = !IL && turned ? 8 * u : 16 * u;
  const int eb = !IL && turned ? ea + p.half : ea + 8;
  const int kv_heads = 2 * p.Hkv;
  const int h_to = BWD ? p.Hq : kv_heads + p.Hq;  // backward: queries first
  const int pieces = (h_to + HPP * p.batch - 1) / (HPP * p.batch);  // of a token
  uint4 xa[kBatch], xb[kBatch];
  auto load = [&](int j, int h0) {
    const size_t tok = t0 + j;
    const __nv_bfloat16* qrow = p.q + tok * p.q_stride - (BWD ? 0 : kv_heads * D);
    const __nv_bfloat16* krow = p.k + tok * p.k_stride;
    const __nv_bfloat16* vrow = p.v + tok * p.v_stride - p.Hkv * D;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * HPP;
      if (i < p.batch && h < h_to) {
        const __nv_bfloat16* src =
            (BWD || h >= kv_heads ? qrow : h >= p.Hkv ? vrow : krow) + h * D;
        xa[i] = *reinterpret_cast<const uint4*>(src + ea);
        xb[i] = *reinterpret_cast<const uint4*>(src + eb);
      }
    }
  };
  int j = pieces > 0 ? warp / pieces : n, piece = warp - j * pieces;
  if (j < n) load(j, piece * p.batch * HPP + lane / UPH);

  count_starts(p, t0, n, threadIdx.x <= p.n_seqs ? p.seq_start[threadIdx.x] : 0, mark);
  if (warp == 0) find_places(p, t0, n, &pl, mark, true);
  else
    for (int i = threadIdx.x - 32; i < n * p.half; i += kThreads - 32)
      turn(p.positions[t0 + i / p.half], p.inv_freq[i % p.half], cs + i, sn + i);
  __syncthreads();

  const size_t head_elems = static_cast<size_t>(p.P) * D;
  for (bool first = true; j < n; first = false) {
    const int h0 = piece * p.batch * HPP + lane / UPH;
    if (!first) load(j, h0);
    const size_t tok = t0 + j;
    const bool used = pl.used[j];
    const float* cj = cs + j * p.half + 8 * u;
    const float* sj = sn + j * p.half + 8 * u;
    // forward: the token's row of KV head 0's keys in the pool
    const int page = BWD ? 0 : pl.page[j];
    const size_t pool_row = BWD || page < 0 ? 0
                                            : static_cast<size_t>(page) * kv_heads * head_elems +
                                                  static_cast<size_t>(pl.row[j]) * D;
    __nv_bfloat16* orow = p.q_out + tok * p.q_out_stride - (BWD ? 0 : kv_heads * D);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * HPP;
      if (i >= p.batch || h >= h_to) break;
      const bool is_q = BWD || h >= kv_heads, is_v = !is_q && h >= p.Hkv;
      if (is_q ? !used : page < 0) continue;
      // blocks of a page: K and V of KV head 0, of KV head 1, ...
      const int block = is_v ? 2 * (h - p.Hkv) + 1 : 2 * h;
      const size_t at = pool_row + block * head_elems;
      __nv_bfloat16* dst = is_q ? orow + h * D : p.kv + at;
      if (turned && !is_v) {
        float x[8], y[8];
        unpack8(xa[i], x);
        unpack8(xb[i], y);
        rotate<BWD, IL>(x, y, cj, sj);
        xa[i] = pack8(x);
        xb[i] = pack8(y);
      }
      *reinterpret_cast<uint4*>(dst + ea) = xa[i];
      *reinterpret_cast<uint4*>(dst + eb) = xb[i];
      if (!BWD && !is_q && p.grad) {
        float4* gz = reinterpret_cast<float4*>(p.grad + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) gz[u + e * UPH] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    for (piece += kThreads / 32; piece >= pieces; piece -= pieces) ++j;
  }
  if (MEAN && pl.last[0] && pl.page[0] >= 0)
    mean_of_page<D, IL>(p, t0, pl.page[0], pl.row[0], pl.first[0], cs, sn);
  if (!BWD) return;
  // the fp32 gradients of the tokens' keys and values
  const int rounds = (kv_heads + HPP - 1) / HPP;  // of a token
#pragma unroll 2
  for (int i = warp; i < n * rounds; i += kThreads / 32) {
    j = i / rounds;
    const int h = (i - j * rounds) * HPP + lane / UPH, page = pl.page[j];
    if (h >= kv_heads || page < 0) continue;
    const size_t tok = t0 + j;
    const bool is_v = h >= p.Hkv;
    const float* src = p.grad + static_cast<size_t>(page) * kv_heads * head_elems +
                       (is_v ? 2 * (h - p.Hkv) + 1 : 2 * h) * head_elems +
                       static_cast<size_t>(pl.row[j]) * D;
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      *reinterpret_cast<float4*>(x + e) = *reinterpret_cast<const float4*>(src + ea + e);
      *reinterpret_cast<float4*>(y + e) = *reinterpret_cast<const float4*>(src + eb + e);
    }
    if (turned && !is_v) rotate<BWD, IL>(x, y, cs + j * p.half + 8 * u, sn + j * p.half + 8 * u);
    __nv_bfloat16* dst = is_v ? p.v + tok * p.v_stride + (h - p.Hkv) * D
                              : p.k + tok * p.k_stride + h * D;
    *reinterpret_cast<uint4*>(dst + ea) = pack8(x);
    *reinterpret_cast<uint4*>(dst + eb) = pack8(y);
  }
}

// Representatives of the pages that received tokens: the mean of the stored
// keys of rows [0, r], r the last row written; the CTA that finds a page's last new
// token in its tile takes it.  Keys are summed anew rather than added to the old mean:
// a sequence that was cut back to fewer tokens and went on gets the right mean, and
// the call can be repeated.  One warp per (page, head), or up to 16 where a CTA has
// few of them: the load latency of 64 rows is then paid once.  Bound by latency: 7.3-7.8 us
// alone for a chunk of 4096 tokens, about 5 behind rope_kernel.  A single launch in which a
// CTA owns a page's keys and values needs none of this, but is uneven: the chunk took
// 28-30 us.  A ticket per page, by which the last of its CTAs takes the mean, is no faster
// (the chunk 18.5 us both ways, with 16 KV heads of 128-token pages 40 instead of 30).
template <int D>
__global__ void __launch_bounds__(kMeanThreads, 2) page_mean_kernel(const RopeParams p) {
  constexpr int VPR = D / 8;      // 16-byte vectors per row
  constexpr int RPW = 32 / VPR;   // rows that a warp reads at once
  constexpr int kWarps = kMeanThreads / 32;
  constexpr int kBatch = 8;       // loads in flight per lane
  __shared__ Places pl;
  __shared__ int mark[32], tok[32], n_pages;
  __shared__ __align__(16) float red[kWarps][D];
  const int t0 = blockIdx.x * p.tile;
  const int n = min(p.tile, p.n_tokens - t0);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  count_starts(p, t0, n, threadIdx.x <= p.n_seqs ? p.seq_start[threadIdx.x] : 0, mark);
  if (warp == 0) {
    find_places(p, t0, n, &pl, mark, false);
    const bool last = pl.last[lane] && pl.page[lane] >= 0;
    const unsigned all = __ballot_sync(0xffffffffu, last);
    if (last) tok[__popc(all & ((1u << lane) - 1))] = lane;
    if (lane == 0) n_pages = __popc(all);
  }
  __syncthreads();
  pdl_wait();  // the keys of this call are in the pages
  const int items = n_pages * p.Hkv;
  int share = 1;  // warps per (page, head)
  while (2 * share <= kWarps && 2 * share * items <= kWarps) share *= 2;
  const int vec = lane % VPR, sub = lane / VPR, part = warp % share;
  for (int i = warp / share; i < items; i += kWarps / share) {
    const int j = tok[i / p.Hkv], g = i % p.Hkv;
    const size_t head = static_cast<size_t>(pl.page[j]) * p.Hkv + g;
    const __nv_bfloat16* src = p.kv + head * 2 * p.P * D + vec * 8;
    const int rows = pl.row[j] + 1, step = share * RPW;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int r0 = part * RPW + sub; r0 < rows; r0 += kBatch * step) {
      uint4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (r0 + b * step < rows) v[b] = *reinterpret_cast<const uint4*>(src + (r0 + b * step) * D);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (r0 + b * step >= rows) break;
        float x[8];
        unpack8(v[b], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += x[e];
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int m = VPR; m < 32; m *= 2) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], m);
    if (share > 1) {  // one round: the (page, head)s are no more than the warps
      if (sub == 0) {
        float4* mine = reinterpret_cast<float4*>(red[warp] + vec * 8);
        mine[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        mine[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / share), "r"(32 * share) : "memory");
      if (part != 0) continue;
      for (int w = 1; w < share; ++w) {
        const float4* other = reinterpret_cast<const float4*>(red[warp + w] + vec * 8);
        const float4 a = other[0], b = other[1];
        acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w;
        acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
      }
    }
    if (sub == 0) {
      const float k = static_cast<float>(rows);
      float4* dst = reinterpret_cast<float4*>(p.summary + head * D + vec * 8);
      dst[0] = make_float4(acc[0] / k, acc[1] / k, acc[2] / k, acc[3] / k);
      dst[1] = make_float4(acc[4] / k, acc[5] / k, acc[6] / k, acc[7] / k);
    }
  }
}

bool good_rows(const void* p, int64_t stride, int64_t heads, int D) {
  return p && aligned16(p) && stride % 8 == 0 && stride >= heads * D;
}

oomb_status make_params(const oomb_pool* pool, const oomb_rope_args* a, bool bwd, RopeParams* p) {
  if (!pool || !a || pool->desc.location != OOMB_LOC_DEVICE) return OOMB_ERR_INVALID_ARG;
  const oomb_pool_desc& d = pool->desc;
  if (a->num_kv_heads != d.num_kv_heads || a->head_dim != d.head_dim || a->device != d.device)
    return OOMB_ERR_INVALID_ARG;
  if (a->n_tokens < 0 || a->n_seqs < 0 || a->n_tokens > kMaxCount || a->n_seqs > kMaxCount)
    return OOMB_ERR_INVALID_ARG;
  if (bwd && !pool->grad) return OOMB_ERR_INVALID_ARG;
  if (a->rotary_dim < 0 || a->rotary_dim > d.head_dim || a->rotary_dim % 16)
    return OOMB_ERR_UNSUPPORTED;
  if (a->interleaved != 0 && a->interleaved != 1) return OOMB_ERR_INVALID_ARG;
  const bool with_q = a->q || a->q_out;
  p->Hq = with_q ? a->num_q_heads : 0;
  if (a->n_tokens > 0 && a->n_seqs > 0) {
    if (a->max_pages <= 0 || !a->seq_start || !a->cached_lens || !a->page_tables ||
        !a->positions || (a->rotary_dim > 0 && !a->inv_freq))
      return OOMB_ERR_INVALID_ARG;
    if (!good_rows(a->k, a->k_stride, d.num_kv_heads, d.head_dim) ||
        !good_rows(a->v, a->v_stride, d.num_kv_heads, d.head_dim))
      return OOMB_ERR_INVALID_ARG;
    if (with_q) {
      if (a->num_q_heads <= 0 || a->num_q_heads % d.num_kv_heads ||
          !good_rows(a->q, a->q_stride, a->num_q_heads, d.head_dim) ||
          !good_rows(a->q_out, a->q_out_stride, a->num_q_heads, d.head_dim))
        return OOMB_ERR_INVALID_ARG;
      if (a->q == a->q_out && a->q_stride != a->q_out_stride) return OOMB_ERR_INVALID_ARG;
    }
  }
  p->seq_start = a->seq_start;
  p->cached_lens = a->cached_lens;
  p->page_tables = a->page_tables;
  p->positions = a->positions;
  p->inv_freq = a->inv_freq;
  p->k = static_cast<__nv_bfloat16*>(a->k);
  p->v = static_cast<__nv_bfloat16*>(a->v);
  p->q = static_cast<const __nv_bfloat16*>(a->q);
  p->q_out = static_cast<__nv_bfloat16*>(a->q_out);
  p->k_stride = a->k_stride;
  p->v_stride = a->v_stride;
  p->q_stride = a->q_stride;
  p->q_out_stride = a->q_out_stride;
  p->kv = static_cast<__nv_bfloat16*>(pool->kv);
  p->grad = pool->grad;
  p->summary = pool->summary;
  p->status = pool->d_status;
  p->n_tokens = a->n_tokens;
  p->n_seqs = a->n_seqs;
  p->max_pages = a->max_pages;
  p->Hkv = d.num_kv_heads;
  p->P = d.page_size;
  p->num_pages = d.num_pages;
  p->half = a->rotary_dim / 2;
  p->interleaved = a->interleaved;
  p->lg_p = __builtin_ctz(static_cast<unsigned>(d.page_size));
  // one wave of the four CTAs that an SM holds
  const int slots = 4 * sm_count(d.device);
  p->tile = std::min(kMaxTile, (a->n_tokens + slots - 1) / slots);
  // as many rounds of loads under way as leave each of a CTA's warps a piece
  const int heads = p->Hq + (bwd ? 0 : 2 * d.num_kv_heads), at_once = 512 / d.head_dim;
  const int rounds = p->tile * ((heads + at_once - 1) / at_once);
  p->batch = std::min(kBatch, std::max(1, rounds / (kThreads / 32)));
  return OOMB_OK;
}

template <bool BWD, bool MEAN>
void launch_rope(const RopeParams& p, int D, cudaStream_t s) {
  const int grid = (p.n_tokens + p.tile - 1) / p.tile;
  if (D == 128) {
    if (p.interleaved) rope_kernel<128, BWD, true, MEAN><<<grid, kThreads, 0, s>>>(p);
    else rope_kernel<128, BWD, false, MEAN><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.interleaved) rope_kernel<64, BWD, true, MEAN><<<grid, kThreads, 0, s>>>(p);
    else rope_kernel<64, BWD, false, MEAN><<<grid, kThreads, 0, s>>>(p);
  }
}

}  // namespace

extern "C" oomb_status oomb_kv_append_rope(oomb_pool* pool, const oomb_rope_args* args,
                                           void* stream) {
  RopeParams p;
  oomb_status st = make_params(pool, args, false, &p);
  if (st != OOMB_OK || args->n_tokens == 0 || args->n_seqs == 0) return st;
  const oomb_pool_desc& d = pool->desc;
  DeviceGuard guard(d.device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Few tokens per sequence, one CTA each, take the page means in the same launch: a page
  // then has few new rows to be rotated a second time.  One launch and two, with the time of
  // a call from Python (device alone in brackets): 64 x 1 token, 28 and 4 heads of 128, 10.2
  // (6.2) and 11.9 us (8.2); 50 x 8 tokens 9.9 (8.7) and 12.7 (10.3); 300 x 1, 8 KV heads,
  // 128-token pages 14.4 (14.4) and 16.2 (16.1).  One prompt of 440 tokens 14.8 and 12.1;
  // with 16 KV heads a CTA has two per warp: 200 x 2 tokens 25.5 and 20.0.
  if (p.n_tokens <= kMeanCtas * sm_count(d.device) && p.n_tokens / 8 <= p.n_seqs &&
      p.Hkv <= kThreads / 32) {
    launch_rope<false, true>(p, d.head_dim, s);
    return check_launch();
  }
  launch_rope<false, false>(p, d.head_dim, s);
  // page means: a dependent launch, its search for the pages runs beside the rotation
  const int slots = 2 * sm_count(d.device);
  p.tile = std::min(32, (p.n_tokens + slots - 1) / slots);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.n_tokens + p.tile - 1) / p.tile);
  cfg.blockDim = dim3(kMeanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = d.head_dim == 128 ? cudaLaunchKernelEx(&cfg, page_mean_kernel<128>, p)
                                          : cudaLaunchKernelEx(&cfg, page_mean_kernel<64>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return OOMB_ERR_CUDA;
  }
  return check_launch();
}

extern "C" oomb_status oomb_kv_append_rope_bwd(oomb_pool* pool, const oomb_rope_args* args,
                                               void* stream) {
  RopeParams p;
  oomb_status st = make_params(pool, args, true, &p);
  if (st != OOMB_OK || args->n_tokens == 0 || args->n_seqs == 0) return st;
  DeviceGuard guard(pool->desc.device);
  launch_rope<true, false>(p, pool->desc.head_dim, static_cast<cudaStream_t>(stream));
  return check_launch();
}

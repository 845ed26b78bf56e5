// kv_append_rope: keys and values of a ragged batch of tokens into the pages of
// their sequences, keys and queries rotated by their positions on the way; and
// its backward, which takes the paged fp32 gradients out token-major and
// rotates them back.
//
// Rotation of pair i of a token at position p by the angle a = p f_i:
//   y_a = x_a cos a - x_b sin a,   y_b = x_b cos a + x_a sin a,
// the inverse with -sin a.  The kernels move bytes: a value is read and written
// once and takes 3 flops, so they are bound by memory.  Everything else is kept
// off that path: a CTA computes its tokens' angles once, in 64 bits, for all
// heads, and keeps cos and sin in shared memory.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace {

using namespace oomb;

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;  // tokens per CTA
constexpr int kMaxHalf = 64; // pairs of a head

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
  int tile;         // tokens per CTA
};

__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Where the tokens [t0, t0 + n) of a CTA go.
struct Places {
  int page[32];  // physical page; < 0: the token is not written
  int row[32];
  int last[32];  // it is the last token that this call puts into its page
  int used[32];  // the token belongs to a sequence (its queries are rotated)
};

// Finds the sequence of each of the CTA's n <= 32 tokens: its index is the number
// of starts <= t, less one.  All threads look through seq_start together (one
// round trip for up to 256 sequences, where a binary search would take eight):
// starts up to t0 are counted, those inside the tile marked.  `note`: report
// what is wrong (one kernel of a call does).
__device__ __forceinline__ void find_places(const RopeParams& p, int t0, int n, Places* out,
                                            int* mark, bool note) {
  const int t = threadIdx.x;
  if (t < 32) mark[t] = 0;
  __syncthreads();
  int before = 0;
  for (int i = t; i <= p.n_seqs; i += blockDim.x) {
    const int s = p.seq_start[i];
    if (s <= t0) ++before;
    else if (s < t0 + n) atomicAdd(&mark[s - t0], 1);
  }
  if (before) atomicAdd(&mark[0], before);
  __syncthreads();
  if (t < n) {
    int seq = -1;
    for (int j = 0; j <= t; ++j) seq += mark[j];
    int page = -1, row = 0, last = 0, used = 0;
    if (seq >= 0 && seq < p.n_seqs) {
      const int tok = t0 + t, lo = p.seq_start[seq], hi = p.seq_start[seq + 1];
      uint32_t bad = 0;
      if (lo < 0 || tok < lo || tok >= hi || hi > p.n_tokens) {
        bad = OOMB_DEV_BAD_COUNT;  // starts that decrease or leave the batch
      } else {
        used = 1;
        const int cached = p.cached_lens[seq];
        const long long c = static_cast<long long>(cached) + (tok - lo);
        const long long pi = c / p.P;
        if (cached < 0 || pi >= p.max_pages) {
          bad = OOMB_DEV_BAD_COUNT;
        } else {
          row = static_cast<int>(c % p.P);
          page = p.page_tables[static_cast<size_t>(seq) * p.max_pages + pi];
          last = row == p.P - 1 || tok + 1 == hi;
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
    out->used[t] = used;
  }
  __syncthreads();
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

// Unit u of a head: two 8-value vectors that are rotated (or copied) together.
struct Unit {
  int a, b;  // their first elements in the head
  int f;     // first of their pairs, -1: not rotated
};
template <bool IL>
__device__ __forceinline__ Unit unit_of(int u, int half, bool rotated) {
  const bool turned = rotated && u < half / 8;
  Unit r;
  r.a = 16 * u;
  r.b = r.a + 8;
  r.f = turned ? 8 * u : -1;
  if (!IL && turned) {
    r.a = 8 * u;
    r.b = r.a + half;
  }
  return r;
}

// Rotates the unit's values in place.  Products and sums are rounded one by
// one (no contraction): what is stored is then the plain formula's value in
// fp32, whichever of these kernels computes it.
template <bool BACK, bool IL>
__device__ __forceinline__ void rotate(float* x, float* y, const float* cs, const float* sn) {
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
    *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(sn + i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (BACK) s[i] = -s[i];
    // pair i of the unit: (x[i], y[i]), or neighbours in x (i < 4) and in y
    float& pa = IL ? (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]) : x[i];
    float& pb = IL ? (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]) : y[i];
    const float a = pa, b = pb;
    pa = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
    pb = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
  }
}

// One CTA: `tile` tokens, all their heads.  Heads are counted K, V, then Q; a
// thread takes one unit (two 16-byte vectors) of one head of one token at a time.
template <int D, bool BWD, bool IL>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int UPH = D / 16;  // units per head
  __shared__ Places pl;
  __shared__ int mark[32];
  __shared__ __align__(16) float cs[kMaxTile * kMaxHalf], sn[kMaxTile * kMaxHalf];
  if (!BWD) pdl_launch_dependents();
  const int t0 = blockIdx.x * p.tile;
  const int n = min(p.tile, p.n_tokens - t0);
  for (int i = threadIdx.x; i < n * p.half; i += kThreads)
    turn(p.positions[t0 + i / p.half], p.inv_freq[i % p.half], cs + i, sn + i);
  find_places(p, t0, n, &pl, mark, true);

  const int heads = 2 * p.Hkv + p.Hq;
  const int total = n * heads * UPH;
  const size_t head_elems = static_cast<size_t>(p.P) * D;
#pragma unroll 4
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const int u = i % UPH, h = (i / UPH) % heads, j = i / (UPH * heads);
    const size_t tok = t0 + j;
    const bool is_q = h >= 2 * p.Hkv, is_v = !is_q && h >= p.Hkv;
    const int page = pl.page[j];
    if (is_q ? !pl.used[j] : page < 0) continue;
    const Unit un = unit_of<IL>(u, p.half, !is_v);
    const int g = is_q ? h - 2 * p.Hkv : is_v ? h - p.Hkv : h;
    // this head's row in the pool (K and V only)
    const size_t at = is_q ? 0
                           : ((static_cast<size_t>(page) * p.Hkv + g) * 2 + is_v) * head_elems +
                                 static_cast<size_t>(pl.row[j]) * D;
    __nv_bfloat16* tok_row = is_q ? nullptr
                                  : (is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + g * D;
    float x[8], y[8];
    if (BWD && !is_q) {
      const float* src = p.grad + at;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4*>(x + e) = *reinterpret_cast<const float4*>(src + un.a + e);
        *reinterpret_cast<float4*>(y + e) = *reinterpret_cast<const float4*>(src + un.b + e);
      }
    } else {
      const __nv_bfloat16* src = is_q ? p.q + tok * p.q_stride + g * D : tok_row;
      unpack8(*reinterpret_cast<const uint4*>(src + un.a), x);
      unpack8(*reinterpret_cast<const uint4*>(src + un.b), y);
    }
    if (un.f >= 0) rotate<BWD, IL>(x, y, cs + j * p.half + un.f, sn + j * p.half + un.f);
    __nv_bfloat16* dst = is_q ? p.q_out + tok * p.q_out_stride + g * D : BWD ? tok_row : p.kv + at;
    *reinterpret_cast<uint4*>(dst + un.a) = pack8(x);
    *reinterpret_cast<uint4*>(dst + un.b) = pack8(y);
    if (!BWD && !is_q && p.grad) {
      float4* gz = reinterpret_cast<float4*>(p.grad + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) gz[u + e * UPH] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// Representatives of the pages that received tokens: the mean of the stored
// keys of rows [0, r], r the last row written.  One warp per (page, head), the
// one that finds the page's last new token in its CTA's tile.  Keys are summed
// anew rather than added to the old mean: a sequence that was cut back to
// fewer tokens and went on gets the right mean, and the call can be repeated.
template <int D>
__global__ void __launch_bounds__(kThreads) page_mean_kernel(const RopeParams p) {
  constexpr int VPR = D / 8;      // 16-byte vectors per row
  constexpr int RPW = 32 / VPR;   // rows that a warp reads at once
  __shared__ Places pl;
  __shared__ int mark[32];
  const int t0 = blockIdx.x * p.tile;
  const int n = min(p.tile, p.n_tokens - t0);
  find_places(p, t0, n, &pl, mark, false);
  pdl_wait();  // the keys of this call are in the pages
  const int lane = threadIdx.x % 32, vec = lane % VPR, sub = lane / VPR;
  const int g = blockIdx.y;
  for (int j = threadIdx.x / 32; j < n; j += kThreads / 32) {
    if (!pl.last[j] || pl.page[j] < 0) continue;
    const size_t head = static_cast<size_t>(pl.page[j]) * p.Hkv + g;
    const __nv_bfloat16* src = p.kv + head * 2 * p.P * D + vec * 8;
    const int rows = pl.row[j] + 1;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 8
    for (int r = sub; r < rows; r += RPW) {
      float x[8];
      unpack8(*reinterpret_cast<const uint4*>(src + static_cast<size_t>(r) * D), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int m = VPR; m < 32; m *= 2) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], m);
      acc[e] /= static_cast<float>(rows);
    }
    if (sub == 0) {
      float4* dst = reinterpret_cast<float4*>(p.summary + head * D + vec * 8);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
  }
}

int sm_count(int device) {
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0)
    n = 148;
  return n;
}

bool good_rows(const void* p, int64_t stride, int64_t heads, int D) {
  return p && aligned16(p) && stride % 8 == 0 && stride >= heads * D;
}

oomb_status make_params(const oomb_pool* pool, const oomb_rope_args* a, bool bwd, RopeParams* p) {
  if (!pool || !a || pool->desc.location != OOMB_LOC_DEVICE) return OOMB_ERR_INVALID_ARG;
  const oomb_pool_desc& d = pool->desc;
  if (a->n_tokens < 0 || a->n_seqs < 0) return OOMB_ERR_INVALID_ARG;
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
  // about four CTAs per SM before a CTA takes more than one token
  p->tile = std::min(kMaxTile, std::max(1, a->n_tokens / (4 * sm_count(d.device))));
  return OOMB_OK;
}

template <bool BWD>
void launch_rope(const RopeParams& p, int D, cudaStream_t s) {
  const int grid = (p.n_tokens + p.tile - 1) / p.tile;
  if (D == 128) {
    if (p.interleaved) rope_kernel<128, BWD, true><<<grid, kThreads, 0, s>>>(p);
    else rope_kernel<128, BWD, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.interleaved) rope_kernel<64, BWD, true><<<grid, kThreads, 0, s>>>(p);
    else rope_kernel<64, BWD, false><<<grid, kThreads, 0, s>>>(p);
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
  launch_rope<false>(p, d.head_dim, s);
  // page means: a dependent launch, its search for the pages runs beside the rotation
  p.tile = std::min(32, std::max(1, p.n_tokens / (4 * sm_count(d.device))));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.n_tokens + p.tile - 1) / p.tile, d.num_kv_heads);
  cfg.blockDim = dim3(kThreads);
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
  launch_rope<true>(p, pool->desc.head_dim, static_cast<cudaStream_t>(stream));
  return check_launch();
}

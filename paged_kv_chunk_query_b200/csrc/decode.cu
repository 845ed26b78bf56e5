// decode_attn: one query token per sequence attends to the sequence's own pages
// and to the pages of a prefix that it shares with others.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace {

using namespace oomb;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  const __nv_bfloat16* kv;
  uint32_t* status;
  int n_seqs, Hq, Hkv, G, P, max_pages, n_groups, max_prefix_pages, num_pages;
  float scale_log2;
};

// One CTA per (head, sequence): a warp takes a key at a time, a lane D / 32 of its values.
template <int D>
__global__ void __launch_bounds__(128) decode_kernel(const DecodeParams p) {
  constexpr int E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const int h = blockIdx.x, b = blockIdx.y, g = h / p.G;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[b * p.q_stride + h * D + lane * E + e]);
    acc[e] = 0.f;
  }
  int group = -1, at = 0;
  for (int j = 0; j < p.n_groups; ++j) {
    int lo = p.group_start[j], hi = p.group_start[j + 1];
    if (lo < at || hi < lo || hi > p.n_seqs) {
      if (threadIdx.x == 0) atomicOr(p.status, OOMB_DEV_BAD_COUNT);
      lo = min(max(lo, at), p.n_seqs);
      hi = min(max(hi, lo), p.n_seqs);
    }
    if (b >= lo && b < hi) group = j;
    at = hi;
  }
  for (int part = 0; part < 2; ++part) {
    if (part && group < 0) break;
    const int cap = part ? p.max_prefix_pages : p.max_pages;
    const int32_t* table =
        part ? p.prefix_pages + static_cast<size_t>(group) * cap : p.page_tables + static_cast<size_t>(b) * cap;
    int len = part ? p.prefix_lens[group] : p.seq_lens[b];
    const long long most = static_cast<long long>(cap) * p.P;
    if (len < 0 || len > most) {
      if (threadIdx.x == 0) atomicOr(p.status, OOMB_DEV_BAD_COUNT);
      len = len < 0 ? 0 : static_cast<int>(most);
    }
    for (int t = warp; t < len; t += 4) {
      const int page = table[t / p.P];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.status, OOMB_DEV_BAD_PAGE);
        continue;
      }
      const __nv_bfloat16* kr =
          p.kv + ((static_cast<size_t>(page) * p.Hkv + g) * 2 * p.P + t % p.P) * D + lane * E;
      const __nv_bfloat16* vr = kr + static_cast<size_t>(p.P) * D;
      float s = 0.f;
      for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(kr[e]), s);
      for (int o = 16; o; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= p.scale_log2;
      const float m_new = fmaxf(m, s);
      const float w = m_new == -INFINITY ? 0.f : fast_exp2(s - m_new);
      const float c = m == -INFINITY ? 0.f : fast_exp2(m - m_new);
      l = l * c + w;
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + w * __bfloat162float(vr[e]);
      m = m_new;
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, sm[w]);
  float f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.f : fast_exp2(sm[w] - top);
    total += f[w] * sl[w];
  }
  if (threadIdx.x < D) {
    float o = 0.f;
    for (int w = 0; w < 4; ++w) o += f[w] * so[w][threadIdx.x];
    p.o[b * p.o_stride + h * D + threadIdx.x] =
        __float2bfloat16(total > 0.f ? o / total : 0.f);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[static_cast<size_t>(b) * p.Hq + h] = total > 0.f ? kLn2 * (top + log2f(total)) : -INFINITY;
}

bool good_shape(int32_t n_seqs, int32_t Hq, int32_t Hkv, int32_t D, int32_t n_groups) {
  return n_seqs >= 0 && n_seqs <= 65535 && Hkv > 0 && Hq > 0 && Hq % Hkv == 0 &&
         supported_head_dim(D) && n_groups >= 0 && n_groups <= n_seqs;
}

}  // namespace

extern "C" size_t oomb_decode_attn_workspace_size(int32_t n_seqs, int32_t num_q_heads,
                                                  int32_t num_kv_heads, int32_t head_dim,
                                                  int32_t n_groups) {
  if (!good_shape(n_seqs, num_q_heads, num_kv_heads, head_dim, n_groups)) return 0;
  return 256;
}

extern "C" oomb_status oomb_decode_attn(oomb_pool* pool, const oomb_decode_args* a, void* stream) {
  if (!pool || !a || pool->desc.location != OOMB_LOC_DEVICE) return OOMB_ERR_INVALID_ARG;
  const oomb_pool_desc& d = pool->desc;
  const int D = d.head_dim, Hq = a->num_q_heads;
  if (!good_shape(a->n_seqs, Hq, d.num_kv_heads, D, a->n_groups)) return OOMB_ERR_INVALID_ARG;
  if (!(a->softmax_scale > 0.f)) return OOMB_ERR_INVALID_ARG;
  if (a->n_seqs == 0) return OOMB_OK;
  const int64_t width = static_cast<int64_t>(Hq) * D;
  if (!a->q || !a->o || !aligned16(a->q) || !aligned16(a->o) || a->q_stride % 8 ||
      a->o_stride % 8 || a->q_stride < width || a->o_stride < width)
    return OOMB_ERR_INVALID_ARG;
  if (a->max_pages <= 0 || !a->page_tables || !a->seq_lens) return OOMB_ERR_INVALID_ARG;
  if (a->n_groups > 0 &&
      (a->max_prefix_pages <= 0 || !a->prefix_pages || !a->prefix_lens || !a->group_start))
    return OOMB_ERR_INVALID_ARG;
  if (!a->workspace || !aligned16(a->workspace) ||
      a->workspace_bytes <
          oomb_decode_attn_workspace_size(a->n_seqs, Hq, d.num_kv_heads, D, a->n_groups))
    return OOMB_ERR_INVALID_ARG;
  DecodeParams p;
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
  p.kv = static_cast<const __nv_bfloat16*>(pool->kv);
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
  p.scale_log2 = a->softmax_scale * kLog2e;
  DeviceGuard guard(d.device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(Hq, a->n_seqs);
  if (D == 128) decode_kernel<128><<<grid, 128, 0, s>>>(p);
  else decode_kernel<64><<<grid, 128, 0, s>>>(p);
  return check_launch();
}

// Attention over the paged cache, one warp per query row and head: the
// scores, the running maximum and sum of the softmax and the weighted sum of
// the values in one pass over the keys,
//   m' = max(m, s_j),  l' = l 2^(m - m') + 2^(s_j - m'),  o' = o 2^(m - m') + 2^(s_j - m') v_j,
// with s_j = scale log2(e) q . k_j.  fp32 throughout, one rounding at the end.
#pragma once

#include "rope.cuh"

namespace serq {
namespace attn {

struct Args {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  long long ldq, ldo;
  float scale_log2;
  int T, n_heads, prefix;  // positions below prefix are sequence 0's
  BatchArgs b;
  CacheArgs c;
};

template <int D>
__global__ void __launch_bounds__(128) k_attn_rows(const Args a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  grid_dep_wait();
  if (w >= (long long)a.T * a.n_heads) return;
  const int t = (int)(w / a.n_heads), h = (int)(w % a.n_heads);
  const int b = warp_find_seq(a.b, t, lane);
  if (b >= a.b.batch) return;
  const int n_keys_all = a.b.kv_len[b];
  int keys = a.b.cu_q ? n_keys_all - (a.b.cu_q[b + 1] - t) + 1 : n_keys_all;
  const int cap = a.b.max_pages << a.c.page_shift;
  if (keys > cap) {
    if (lane == 0) note_bad_page();
    keys = cap;
  }
  const int kvh = h / (a.n_heads / a.c.n_kv_heads);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[t * a.ldq + h * D + e * 32 + lane]) * a.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int32_t* table = a.b.table + (long long)b * a.b.ldt;
  for (int j = 0; j < keys; ++j) {
    const int page = (j < a.prefix ? a.b.table : table)[j >> a.c.page_shift];
    const bool good = page >= 0 && page < a.c.n_pages;
    if (!good && lane == 0) note_bad_page();
    const long long at = good ? page * a.c.page_stride +
                                    (((long long)kvh << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1))) * D
                              : 0;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += good ? q[e] * __bfloat162float(a.c.K[at + e * 32 + lane]) : 0.f;
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float r = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * r + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * r + (good ? p * __bfloat162float(a.c.V[at + e * 32 + lane]) : 0.f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.o[t * a.ldo + h * D + e * 32 + lane] = __float2bfloat16_rn(o[e] * inv);
}

template <int D>
inline cudaError_t launch_rows(const Args& a, cudaStream_t st) {
  const long long warps = (long long)a.T * a.n_heads;
  k_attn_rows<D><<<(unsigned)((warps + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace serq

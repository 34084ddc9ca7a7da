// Position rotation of a decoder layer's queries and keys, with the optional
// RMS norm of each head in front of it, and the append of keys and values to
// a paged cache: one pass over the rows that the q/k/v linears wrote.
//
//   x' = x * w / sqrt(mean(x^2) + eps)                       (per head; optional)
//   (x1, x2) -> A (x1 cos a - x2 sin a, x1 sin a + x2 cos a),  a = position * f_i
//
// Angles: a position times a frequency has to keep its fraction of a turn, so
// the product is taken in fp64 turns (f_i / 2 pi, made once at creation), its
// nearest integer is subtracted, and only the remainder (|r| <= 1/2) is
// rounded to fp32 for sincospi.  fp32 angles would be off by 2^-24 of 120000
// radians, 0.007, at position 120000.
//
// The pass is bound by memory: 4 bytes per element read and written, 15.6 us
// of HBM time for 2048 tokens of 96 heads of 128.
#pragma once

#include "attn_common.cuh"

namespace serq {

// The batch that rope_append and the attention calls share: queries of
// sequence b are rows [cu_q[b], cu_q[b + 1]), at positions kv_len[b] - n_b ...
// kv_len[b] - 1; position p of the sequence lives in page
// table[b * ldt + p / page_size].
struct BatchArgs {
  const int32_t* cu_q;    // batch + 1; nullptr in decode, whose row b is sequence b's
  const int32_t* kv_len;  // batch
  const int32_t* table;   // batch rows of max_pages entries
  int batch, max_pages, ldt;
};

// The paged cache as kernels see it.
struct CacheArgs {
  __nv_bfloat16 *K, *V;  // pages of n_kv_heads x page_size x head_dim
  long long page_stride;  // elements
  int n_pages, page_shift, n_kv_heads;
};

__device__ __forceinline__ void note_bad_page() { atomicCAS(&g_device_status, 0, kDevBadPage); }

// Sequence of query row t: the number of sequences that end at or before t
// (the whole warp calls).  batch when t lies in front of the first or behind
// the last one.
__device__ __forceinline__ int warp_find_seq(const BatchArgs& b, int t, int lane) {
  int n = 0;
  for (int i = lane; i < b.batch; i += 32) n += b.cu_q[i + 1] <= t;
  n = __reduce_add_sync(0xffffffffu, n);
  return t < b.cu_q[0] ? b.batch : n;
}

namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 2;  // tokens per CTA

struct Args {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* q_out;
  long long ldq, ldk, ldv, ldqo;
  const __nv_bfloat16 *qw, *kw;  // both null: no norm
  float eps, amp;
  const double* turns;  // rot / 2: frequencies in turns per position
  int T, n_heads, rot, tokens;  // tokens per CTA
  BatchArgs b;
  CacheArgs c;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t&>(p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// D / 16 threads per head, 16 elements each: two 16-byte chunks that hold
// whole pairs.  HALF: chunks e0 and e0 + rot / 2 of the rotated part (chunk
// pairs of the rest lie side by side); interleaved: neighbouring chunks.
template <int D, bool HALF, bool NORM>
__global__ void __launch_bounds__(kThreads) k_rope_append(const Args a) {
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ int s_pos[kMaxTokens];            // position, or -1: a row that is left alone
  __shared__ long long s_slot[kMaxTokens];     // cache offset of (page, head 0, slot), or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, a.T - t0);
  grid_dep_wait();
  if (warp < nt) {
    const int t = t0 + warp;
    const int b = warp_find_seq(a.b, t, lane);
    int pos = -1;
    long long slot = -1;
    if (b < a.b.batch) {
      const int kv = a.b.kv_len[b];
      pos = max(-1, kv - (a.b.cu_q[b + 1] - t));
      if (pos >= 0) {
        const int pg = pos >> a.c.page_shift;
        const int page = pg < a.b.max_pages ? a.b.table[(long long)b * a.b.ldt + pg] : -1;
        if (page >= 0 && page < a.c.n_pages)
          slot = page * a.c.page_stride + (long long)(pos & ((1 << a.c.page_shift) - 1)) * D;
        else if (lane == 0)
          note_bad_page();
      }
    }
    if (lane == 0) {
      s_pos[warp] = pos;
      s_slot[warp] = slot;
    }
  }
  __syncthreads();
  const int half = a.rot >> 1;
  for (int i = tid; i < nt * half; i += kThreads) {
    const int ti = i / half, p = i - ti * half;
    double r = (double)s_pos[ti] * a.turns[p];
    r -= rint(r);
    float s, c;
    sincospif((float)(2.0 * r), &s, &c);
    cs[ti][p] = make_float2(c * a.amp, s * a.amp);
  }
  __syncthreads();

  constexpr int TPH = D / 16;
  const int heads = a.n_heads + 2 * a.c.n_kv_heads;
  const int items = nt * heads * TPH;
  for (int i = blockIdx.y * kThreads + tid; i < items; i += kThreads * gridDim.y) {
    const int c = i % TPH, hh = i / TPH;
    const int ti = hh / heads;
    int h = hh - ti * heads;
    if (s_pos[ti] < 0) continue;  // whole heads: the threads of a head agree
    const long long t = t0 + ti;
    const __nv_bfloat16 *src, *w = nullptr;
    __nv_bfloat16* dst;
    bool turn = true;
    if (h < a.n_heads) {
      src = a.q + t * a.ldq + h * D;
      dst = a.q_out + t * a.ldqo + h * D;
      w = a.qw;
    } else {
      h -= a.n_heads;
      const bool is_v = h >= a.c.n_kv_heads;
      if (is_v) h -= a.c.n_kv_heads;
      src = (is_v ? a.v + t * a.ldv : a.k + t * a.ldk) + h * D;
      const long long slot = s_slot[ti];
      dst = slot < 0 ? nullptr : (is_v ? a.c.V : a.c.K) + slot + ((long long)h << a.c.page_shift) * D;
      w = a.kw;
      turn = !is_v;
    }
    // element offsets of this thread's two chunks, and its first pair
    int e0, e1, p0;
    bool rotated;
    if (HALF) {
      rotated = c * 16 < a.rot;
      e0 = rotated ? c * 8 : c * 16;
      e1 = rotated ? e0 + half : e0 + 8;
      p0 = e0;
    } else {
      rotated = c * 16 < a.rot;
      e0 = c * 16;
      e1 = e0 + 8;
      p0 = c * 8;
    }
    const uint4 u0 = *reinterpret_cast<const uint4*>(src + e0);
    const uint4 u1 = *reinterpret_cast<const uint4*>(src + e1);
    uint4 o0 = u0, o1 = u1;
    if (turn && (NORM || rotated)) {
      float x0[8], x1[8];
      unpack8(u0, x0);
      unpack8(u1, x1);
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += x0[j] * x0[j] + x1[j] * x1[j];
        const uint32_t mask = ((1u << TPH) - 1u) << (lane & ~(TPH - 1));
#pragma unroll
        for (int m = TPH / 2; m; m >>= 1) ss += __shfl_xor_sync(mask, ss, m);
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
        float w0[8], w1[8];
        unpack8(*reinterpret_cast<const uint4*>(w + e0), w0);
        unpack8(*reinterpret_cast<const uint4*>(w + e1), w1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x0[j] *= inv * w0[j];
          x1[j] *= inv * w1[j];
        }
      }
      if (rotated) {
        const float2* f = &cs[ti][p0];
        if (HALF) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float p = x0[j], r = x1[j];
            x0[j] = p * f[j].x - r * f[j].y;
            x1[j] = p * f[j].y + r * f[j].x;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float p = x0[2 * j], r = x0[2 * j + 1];
            x0[2 * j] = p * f[j].x - r * f[j].y;
            x0[2 * j + 1] = p * f[j].y + r * f[j].x;
            p = x1[2 * j], r = x1[2 * j + 1];
            x1[2 * j] = p * f[4 + j].x - r * f[4 + j].y;
            x1[2 * j + 1] = p * f[4 + j].y + r * f[4 + j].x;
          }
        }
      }
      o0 = pack8(x0);
      o1 = pack8(x1);
    }
    if (dst != nullptr) {
      *reinterpret_cast<uint4*>(dst + e0) = o0;
      *reinterpret_cast<uint4*>(dst + e1) = o1;
    }
  }
}

template <int D>
inline cudaError_t launch(Args a, bool half, int sms, cudaStream_t st) {
  // Two tokens per CTA share the look-up and still leave CTAs enough for an even
  // load (2048 tokens of 96 heads of 128: 16.9 us, 5.96 TB/s; with one 18.6, with
  // four 20.0); few tokens are spread over the SMs.
  a.tokens = a.T >= 8 * sms ? kMaxTokens : 1;
  const int items = a.tokens * (a.n_heads + 2 * a.c.n_kv_heads) * (D / 16);
  const int gx = (a.T + a.tokens - 1) / a.tokens;
  int gy = 1;
  while (gx * gy < 2 * sms && gy * kThreads < items) ++gy;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool norm = a.qw != nullptr;
  if (half) return norm ? cudaLaunchKernelEx(&cfg, k_rope_append<D, true, true>, a)
                        : cudaLaunchKernelEx(&cfg, k_rope_append<D, true, false>, a);
  return norm ? cudaLaunchKernelEx(&cfg, k_rope_append<D, false, true>, a)
              : cudaLaunchKernelEx(&cfg, k_rope_append<D, false, false>, a);
}

}  // namespace rope
}  // namespace serq

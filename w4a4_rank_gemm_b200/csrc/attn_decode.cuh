// Decode attention: one query token per sequence over the paged cache, bound
// by the bytes of K and V.
//
// Work is counted in units, laid end to end over the batch: a (sequence, kv
// head, 16 query heads) pair's blocks of 64 keys and two more for its end, which
// takes as long as one to two blocks; share c of G is the c-th equal part,
// whatever the lengths are, as the streaming GEMV shares the weights.  (64
// sequences of 1 ... 700 keys, 32 MHA heads: 84.0 us with none for the end, 65.9
// with one, 66.9 with two, 66.2 with three; 200 of 1 ... 500, 8 heads of 64: 38.3,
// 31.0, 28.5, 28.6; one of 8191, 8 kv heads: 12.3, 12.3, 11.7 with two.)  A share
// is a run of segments: the end of one pair's keys, whole pairs, the beginning
// of another's.  Whole pairs are finished here; the first and last segment of
// a share may be partial and go to the workspace (slots 2c and 2c + 1), to be
// joined in share order by k_join.
//
// A CTA works on two shares at once, so that one's joining of warps at a
// segment's end (about 1400 cycles) overlaps the other's blocks.  Each has four
// warps, 16 keys of a block each, and a warp that streams K and V blocks by TMA
// into its ring (192 KB in flight per SM), across segment boundaries.  Scores
// and output by mma.sync m16n8k16 with the group's query heads as the 16 rows.
// Their use of the tensor core is far below its rate (16 flop per byte read), so
// nothing is gained by tcgen05 here; its 128-row tiles would be 1/32 to 1/8 full.
#pragma once

#include "attn_tc.cuh"

namespace serq {
namespace attn {

constexpr int kDecThreads = 320;  // warps 0-3 and 4-7: two shares' blocks; 8 and 9: their loads
constexpr int kBlockKeys = 64;
constexpr int kEndUnits = 2;

struct DecArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  long long ldq, ldo;
  float c;      // |scale| log2 e
  float sign;   // of scale
  int n_heads, group, row_blocks;  // row_blocks: 16-head blocks per kv head
  int rows;     // rows per workspace slot, min(group, 16)
  int prefix;   // keys in front that the shared-prefix pass has done
  int common;   // keys in front whose pages are sequence 0's
  int shares;   // G, two per CTA
  float* so;    // slots [2 G (+ batch x blocks of heads when prefix)][rows][D], normalised
  float* slse;  // [slot][rows]
  const float* po;    // the prefix pass's slots [slot][256][D] and their log-sums
  const float* plse;
  int ptokens, pshares;  // its tokens per tile and shares
  BatchArgs b;
  CacheArgs c_;
};

template <int D>
struct DecLayout {
  static constexpr int kHalves = D / 64;
  static constexpr int kOperand = kBlockKeys * D * 2;  // bytes of a block's K or V
  static constexpr int kSlots = D == 128 ? 3 : 6;      // of a share
  static constexpr int oRing = 0;
  static constexpr int kRing = kSlots * 2 * kOperand;
  static constexpr int oMerge = 2 * kRing;               // 32 D floats per share
  static constexpr int oStat = oMerge + 64 * D * 4;      // per share m and l: [2][4][16] floats
  static constexpr int oBar = oStat + 2 * 8 * 16 * 4;
  static constexpr int oMisc = oBar + 4 * kSlots * 8;
  static constexpr int kAlloc = oMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory of a CTA");
};

// Blocks of sequence b behind the prefix.
__device__ __forceinline__ int dec_blocks(const DecArgs& a, int b) {
  const int cap = a.b.max_pages << a.c_.page_shift;
  return ceil_div(max(0, min(a.b.kv_len[b], cap) - a.prefix), kBlockKeys);
}

// Units of a pair of nb blocks.
__device__ __forceinline__ int dec_units(int nb) { return nb > 0 ? nb + kEndUnits : 0; }

// Warp sum of non-negative counts; `small`: it stays below 2^31.
__device__ __forceinline__ long long warp_sum(long long v, bool small) {
  if (small) return __reduce_add_sync(0xffffffffu, (uint32_t)v);
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Position in the batch's run of pairs.
struct DecPos {
  int b, h, blk, nb;  // sequence, head block, next block, blocks of the sequence
};

// Finds a share's beginning.  Lane i counts the units of sequences
// [i q, (i + 1) q), q = ceil(batch / 32), in one round of loads.
struct DecFind {
  int q;
  long long mine, upto, total;  // of the lane's sequences, of them and those before, of all
  __device__ DecFind(const DecArgs& a, int lane) {
    q = ceil_div(a.b.batch, 32);
    mine = 0;
#pragma unroll 4
    for (int i = 0; i < q; ++i) {
      const int b = lane * q + i;
      if (b < a.b.batch) mine += dec_units(dec_blocks(a, b));
    }
    upto = mine;
    if (a.b.batch <= 32) {  // fewer than 2^26 units each
      int v = (int)mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      upto = v;
      total = __shfl_sync(0xffffffffu, v, 31);
    } else {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      total = __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  // The place of unit w < total * heads (the warp calls); blk >= nb: a pair's end.
  __device__ DecPos find(const DecArgs& a, long long w, int heads) const {
    const int src = __ffs(__ballot_sync(0xffffffffu, w < upto * heads)) - 1;
    long long rest = w - __shfl_sync(0xffffffffu, upto - mine, src) * heads;
    DecPos p;
    p.b = src * q;
    for (;; ++p.b) {
      p.nb = dec_blocks(a, p.b);
      if (rest < (long long)dec_units(p.nb) * heads) break;
      rest -= (long long)dec_units(p.nb) * heads;
    }
    p.h = (int)quotient(rest, dec_units(p.nb));
    p.blk = (int)(rest - (long long)p.h * dec_units(p.nb));
    return p;
  }
};

__device__ __forceinline__ void dec_next_pair(const DecArgs& a, DecPos& p, int heads) {
  p.blk = 0;
  if (++p.h == heads) {
    p.h = 0;
    do {
      ++p.b;
      p.nb = p.b < a.b.batch ? dec_blocks(a, p.b) : 1;
    } while (p.nb == 0);
  }
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return reinterpret_cast<const uint32_t&>(h);
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 1)
    k_decode_attn(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecArgs a) {
  using L = DecLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool loads = warp >= 8;
  const int wg = loads ? warp - 8 : warp >> 2;       // which of the CTA's two shares
  const int share = 2 * blockIdx.x + wg;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::oBar) + wg * 2 * L::kSlots;
  uint64_t* empty = full + L::kSlots;
  uint8_t* ring = smem + L::oRing + wg * L::kRing;
  if (loads && lane == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
  }
  __syncthreads();
  // Behind the shared-prefix pass of the same call (which has waited for
  // whatever came before it) there is nothing to wait for until the end.
  if (a.prefix == 0) grid_dep_wait();
  grid_dep_launch();

  const int heads = a.c_.n_kv_heads * a.row_blocks;
  const DecFind batch(a, lane);
  const Shares shares(batch.total * heads, a.shares);
  long long w0 = share < a.shares ? shares.start(share) : 0;
  const long long w1 = share < a.shares ? shares.start(share + 1) : 0;
  const int cap = a.b.max_pages << a.c_.page_shift;
  // keys of a copy: a block's K or V lie in shared memory as box rows of its
  // first 64 columns, the same rows of the next 64, then the next box
  const int box = min(1 << a.c_.page_shift, kBlockKeys);
  DecPos p = {};
  if (w0 < w1) {
    p = batch.find(a, w0, heads);
    if (p.blk >= p.nb) {  // another share has done the pair
      w0 += dec_units(p.nb) - p.blk;
      dec_next_pair(a, p, heads);
    }
  }

  if (loads) {
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    // The pages of up to 32 copies (8 to 32 blocks of one pair) are looked up
    // at once, one such batch ahead of the copies: a lookup costs a trip to L2,
    // about as long as a block takes.
    const int page = 1 << a.c_.page_shift;
    const int per_block = kBlockKeys / box, max_n = 32 / per_block;
    auto lookup = [&](const DecPos& at, int n) {
      const int key = a.prefix + at.blk * kBlockKeys + lane * box;
      int pg = a.c_.n_pages;  // outside the map: filled with zeros
      if (lane < n * per_block && key < min(a.b.kv_len[at.b], cap)) {
        const int e = a.b.table[(key < a.common ? 0 : (long long)at.b * a.b.ldt) + (key >> a.c_.page_shift)];
        if (e >= 0 && e < a.c_.n_pages) pg = e;
        else note_bad_page();
      }
      return pg;
    };
    uint32_t slot = 0, ph = 0;
    bool ok = true;
    long long w = w0;
    int n = (int)min(min((long long)(p.nb - p.blk), w1 - w), (long long)max_n);
    int pg = w < w1 ? lookup(p, n) : 0;
    while (w < w1 && ok) {
      const DecPos cur = p;
      const int cur_n = n, cur_pg = pg;
      w += n;
      p.blk += n;
      if (p.blk == p.nb) {
        dec_next_pair(a, p, heads);
        w += kEndUnits;
      }
      n = (int)min(min((long long)(p.nb - p.blk), w1 - w), (long long)max_n);
      if (w < w1) pg = lookup(p, n);
      const int y0 = ((cur.h / a.row_blocks) << a.c_.page_shift);
      for (int i = 0; i < cur_n; ++i) {
        const int at_pg = __shfl_sync(0xffffffffu, cur_pg, (i * per_block + lane) & 31);  // lane: copy within the block
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ph ^ 1, abort_flag, kDevTimeoutProducer));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2 * L::kOperand);
        __syncwarp();
        if (lane < per_block) {
          const int key = a.prefix + (cur.blk + i) * kBlockKeys + lane * box;
          const int y = y0 + (key & (page - 1));
          uint8_t* dst = ring + slot * 2 * L::kOperand + lane * box * (2 * D);
          tma_load_4d(dst, &tmK, &full[slot], 0, y, 0, at_pg);
          tma_load_4d(dst + L::kOperand, &tmV, &full[slot], 0, y, 0, at_pg);
        }
        __syncwarp();
        if (++slot == L::kSlots) slot = 0, ph ^= 1;
      }
    }
  } else {
    const int wv = warp & 3, kq = wv * 16;  // this warp's keys of a block
    const int quad = lane >> 2, qc = (lane & 3) * 2;
    const int in_box = kq & (box - 1), box_at = (kq - in_box) * (2 * D), half_at = box * 128;
    bool ok = true;
    float* merge = reinterpret_cast<float*>(smem + L::oMerge) + wg * 32 * D;
    float* st_m = reinterpret_cast<float*>(smem + L::oStat) + wg * 8 * 16;
    float* st_l = st_m + 4 * 16;
    uint32_t slot_at = 0, ph = 0;
    // the query fragments of the pair at position `at`
    auto load_q = [&](const DecPos& at, uint32_t(&f)[D / 16][4]) {
      const int kvh = at.h / a.row_blocks, rb = at.h - kvh * a.row_blocks, nrows = a.group - 16 * rb;
      const __nv_bfloat16* q0 = a.q + at.b * a.ldq + (long long)(kvh * a.group + 16 * rb + quad) * D + qc;
      const __nv_bfloat16* q1 = q0 + 8 * D;
      const bool v0 = quad < nrows, v1 = quad + 8 < nrows;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        f[k][0] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + 16 * k) : 0u;
        f[k][1] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + 16 * k) : 0u;
        f[k][2] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + 16 * k + 8) : 0u;
        f[k][3] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + 16 * k + 8) : 0u;
      }
    };
    uint32_t qf[D / 16][4];
    if (w0 < w1) load_q(p, qf);
    for (long long w = w0; w < w1;) {
      const int n = (int)min((long long)(p.nb - p.blk), w1 - w);
      const int kvh = p.h / a.row_blocks, rb = p.h - kvh * a.row_blocks;
      const int nrows = min(16, a.group - 16 * rb);
      const int head0 = kvh * a.group + 16 * rb;
      const int kv = min(a.b.kv_len[p.b], cap);
      if ((threadIdx.x & 127) == 0 && a.b.kv_len[p.b] > cap) note_bad_page();
      float o[D / 8][4] = {};
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows quad and quad + 8
      for (int i = 0; i < n; ++i) {
        const uint32_t slot = slot_at;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[slot], ph, abort_flag, kDevTimeoutEpilogue));
        if (!ok) continue;
        const uint32_t kb = smem_u32(ring + slot * 2 * L::kOperand), vb = kb + L::kOperand;
        const int key0 = a.prefix + (p.blk + i) * kBlockKeys + kq;  // first key of this warp
        if (key0 < kv) {
          // even and odd 16-column steps apart: two chains of products per 8 keys
          float s[2][4] = {}, s2[2][4] = {};
          {
            const int r = in_box + ((lane >> 4) << 3) + (lane & 7), cb = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t f[4];
              const int ch = (k & 3) * 2 + cb;
              ldsm_x4(kb + box_at + (k >> 2) * half_at + r * 128 + ((ch ^ (r & 7)) << 4), f);
              mma_bf16(k & 1 ? s2[0] : s[0], qf[k], f[0], f[1]);
              mma_bf16(k & 1 ? s2[1] : s[1], qf[k], f[2], f[3]);
            }
          }
          const bool partial = key0 + 16 > kv;
          uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;  // which of this thread's values exist
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = (s[t][e] + s2[t][e]) * a.sign;
          if (partial) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 8 * t + qc + (e & 1) >= kv) s[t][e] = -INFINITY;
            vm0 = (key0 + qc < kv ? 0xffffu : 0u) | (key0 + qc + 1 < kv ? 0xffff0000u : 0u);
            vm1 = (key0 + 8 + qc < kv ? 0xffffu : 0u) | (key0 + 8 + qc + 1 < kv ? 0xffff0000u : 0u);
          }
          float c0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
          float c1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, d));
            c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, d));
          }
          c0 *= a.c;
          c1 *= a.c;
          const bool g0 = c0 > m0 + kLazyMax, g1 = c1 > m1 + kLazyMax;
          if (__any_sync(0xffffffffu, g0 || g1)) {
            const float f0 = g0 ? ex2(m0 - c0) : 1.f, f1 = g1 ? ex2(m1 - c1) : 1.f;
            if (g0) m0 = c0;
            if (g1) m1 = c1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
              o[t][0] *= f0;
              o[t][1] *= f0;
              o[t][2] *= f1;
              o[t][3] *= f1;
            }
          }
          const float b0 = m0 == -INFINITY ? 0.f : -m0, b1 = m1 == -INFINITY ? 0.f : -m1;
          float e[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            e[t][0] = ex2(fmaf(s[t][0], a.c, b0));
            e[t][1] = ex2(fmaf(s[t][1], a.c, b0));
            e[t][2] = ex2(fmaf(s[t][2], a.c, b1));
            e[t][3] = ex2(fmaf(s[t][3], a.c, b1));
          }
          l0 += (e[0][0] + e[0][1]) + (e[1][0] + e[1][1]);
          l1 += (e[0][2] + e[0][3]) + (e[1][2] + e[1][3]);
          // The weights are rounded to bf16, the type of V that the product wants:
          // an error of at most 2^-8 in each, so that the result's, rounded to
          // bf16 anyway, is 2.2e-3 where it would be 1.66e-3 (root mean square,
          // 8191 keys).  A second product with what the rounding leaves over brings
          // that back for 0 to 1% where memory bounds the call, and 3 to 9% in
          // the others: one sequence of 8191 12.3 us for 11.7, 200 of 1 ... 500
          // 29.4 for 26.8.
          const uint32_t pf[4] = {pack_bf16(e[0][0], e[0][1]), pack_bf16(e[0][2], e[0][3]),
                                  pack_bf16(e[1][0], e[1][1]), pack_bf16(e[1][2], e[1][3])};
          const int r = in_box + (((lane >> 3) & 1) << 3) + (lane & 7), cb = lane >> 4;
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            uint32_t f[4];
            const int ch = (t & 3) * 2 + cb;
            ldsm_x4_t(vb + box_at + (t >> 2) * half_at + r * 128 + ((ch ^ (r & 7)) << 4), f);
            if (partial) {  // values that do not exist may be NaN
              f[0] &= vm0;
              f[1] &= vm1;
              f[2] &= vm0;
              f[3] &= vm1;
            }
            mma_bf16(o[2 * t], pf, f[0], f[1]);
            mma_bf16(o[2 * t + 1], pf, f[2], f[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot_at == L::kSlots) slot_at = 0, ph ^= 1;
      }
      DecPos nx = p;  // the next segment, whose queries load during the join
      nx.blk = p.blk + n;
      w += n;
      if (nx.blk == nx.nb) {
        dec_next_pair(a, nx, heads);
        w += kEndUnits;
      }
      if (w < w1) load_q(nx, qf);
      // ------------------------------------------------- join the four warps
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      if ((lane & 3) == 0) {
        st_m[wv * 16 + quad] = m0;
        st_m[wv * 16 + quad + 8] = m1;
      }
      auto sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
      sync();
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        M0 = fmaxf(M0, st_m[v * 16 + quad]);
        M1 = fmaxf(M1, st_m[v * 16 + quad + 8]);
      }
      const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M1);
      if ((lane & 3) == 0) {
        st_l[wv * 16 + quad] = l0 * f0;
        st_l[wv * 16 + quad + 8] = l1 * f1;
      }
      // where the segment goes: whole pairs to O, or (with a prefix to join) to
      // the pair's slot; a partial first segment to slot 2c, a partial last one
      // to 2c + 1
      const bool starts = p.blk == 0, ends = p.blk + n == p.nb;
      const long long slot = !starts ? 2 * (long long)share
                             : !ends ? 2 * (long long)share + 1
                                     : 2 * (long long)a.shares + (long long)p.b * heads + p.h;
      const bool final = starts && ends && a.prefix == 0;
      // each warp's share of O goes through shared memory, all columns of up to
      // 8 rows at once or half of them for up to 16: [warp][row][column], rows
      // turned by 8 columns each
      auto join = [&](auto rows_tag) {
        constexpr int NR = decltype(rows_tag)::value, NC = 8 * D / NR;
        auto place = [&](int v, int row, int col) { return merge + (v * NR + row) * NC + ((col + 8 * row) & (NC - 1)); };
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += NC) {
#pragma unroll
          for (int t = 0; t < NC / 8; ++t) {
            const float(&x)[4] = o[c0 / 8 + t];
            if (quad < nrows) *reinterpret_cast<float2*>(place(wv, quad, 8 * t + qc)) = make_float2(x[0] * f0, x[1] * f0);
            if (NR == 16 && quad + 8 < nrows)
              *reinterpret_cast<float2*>(place(wv, quad + 8, 8 * t + qc)) = make_float2(x[2] * f1, x[3] * f1);
          }
          sync();
          for (int e = threadIdx.x & 127; e < nrows * (NC / 4); e += 128) {
            const int row = e / (NC / 4), c4 = (e % (NC / 4)) * 4;
            float z = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float4 y = *reinterpret_cast<const float4*>(place(v, row, c4));
              z += st_l[v * 16 + row];
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            const float inv = z != 0.f ? 1.f / z : 0.f;  // a NaN stays one
            x.x *= inv;
            x.y *= inv;
            x.z *= inv;
            x.w *= inv;
            if (!ok) continue;
            if (final) {
              *reinterpret_cast<uint2*>(a.o + p.b * a.ldo + (long long)(head0 + row) * D + c0 + c4) =
                  make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
            } else {
              *reinterpret_cast<float4*>(a.so + (slot * a.rows + row) * D + c0 + c4) = x;
              if (c0 + c4 == 0) {
                float mm = -INFINITY;
#pragma unroll
                for (int v = 0; v < 4; ++v) mm = fmaxf(mm, st_m[v * 16 + row]);
                a.slse[slot * a.rows + row] = z != 0.f ? mm + log2f(z) : -INFINITY;
              }
            }
          }
          sync();  // the buffer may be written again
        }
      };
      if (nrows <= 8) join(std::integral_constant<int, 8>{});
      else join(std::integral_constant<int, 16>{});
      p = nx;
    }
  }
  if (a.prefix != 0) grid_dep_wait();  // k_join waits for this grid only
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      // let copies already issued land before the shared memory is released
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < 100000ull) {
      }
    }
    __syncthreads();
  }
}

// Joins what k_decode_attn left in slots, and the shared prefix's partials:
// O = sum_s 2^(lse_s - M) O_s / sum_s 2^(lse_s - M).  W warps per sequence and
// head, each with every W-th part, four warps per CTA; lanes look up 32 parts
// at a time, whose rows are then read together and added in order.  A sequence
// without keys gets zeros.
template <int D, int W>
__global__ void __launch_bounds__(128) k_join(const DecArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
  const int h = min((int)blockIdx.y * (4 / W) + warp / W, a.n_heads - 1), mine = warp % W;
  // The lengths are inputs of the call: k_decode_attn lets this grid start
  // only after its own wait (or starts behind a prefix pass that has waited), so
  // they were complete before this grid was launched.  (Read past L1 they would
  // not depend on a launch finding L1 clean, at 100 sequences of 1 ... 60 keys
  // 43.2 us for 33.8, one of 8191 13.9 for 11.7.)
  const int heads = a.c_.n_kv_heads * a.row_blocks;
  long long before = 0, total = 0;
  for (int i = lane; i < a.b.batch; i += 32) {
    const int n = dec_units(dec_blocks(a, i));
    total += n;
    if (i < b) before += n;
  }
  before = warp_sum(before, a.b.batch <= 32);
  total = warp_sum(total, a.b.batch <= 32) * heads;
  const int kvh = h / a.group, hr = h - kvh * a.group;
  const int hb = kvh * a.row_blocks + hr / 16, row = hr & 15;
  const int nb = dec_blocks(a, b);
  const long long s0 = before * heads + (long long)hb * dec_units(nb), s1 = s0 + nb;
  // shares that hold the pair's first and last block
  const Shares shares(total, a.shares);
  int c0 = 0, c1 = -1;
  if (nb > 0) {
    c0 = shares.of(s0);
    c1 = shares.of(s1 - 1);
  }
  // the prefix's parts, as ShareWalk lays them out: pairs of `keys` keys each
  int p0 = 0, np = 0, item = 0, prow = 0;
  long long pstart = 0, keys = 0, ptotal = 0;
  if (a.prefix) {
    int k = 0;
    for (int i = lane; i < a.b.batch; i += 32) k = max(k, min(a.b.kv_len[i], a.prefix));
    keys = __reduce_max_sync(0xffffffffu, k);
    const int pair = 2 * a.ptokens, pairs = ceil_div(a.b.batch, pair), tile = b / pair;
    const int in = b - tile * pair, x = in >= a.ptokens;
    prow = 128 * x + (in - x * a.ptokens) * a.group + hr;
    item = kvh * pairs + tile;
    pstart = item * keys;
    ptotal = keys * pairs * a.c_.n_kv_heads;
  }
  const Shares pshares(ptotal, max(a.pshares, 1));
  if (keys > 0) {
    p0 = pshares.of(pstart);
    np = pshares.of(pstart + keys - 1) - p0 + 1;
  }
  const int n = np + c1 - c0 + 1;
  // Place of part i: its row (in rows of D floats) and log-sum, null when it
  // has none.
  auto place = [&](int i, const float*& src, const float*& lse) {
    src = a.so;
    lse = nullptr;
    if (i < np) {
      const long long c = p0 + i;
      const long long lo = max(0ll, pshares.start(c) - pstart), hi = min(keys, pshares.start(c + 1) - pstart);
      const int steps = ceil_div((int)keys, kTileKeys);
      const int shi = hi == keys ? steps : (int)(hi / kTileKeys);
      if (lo < hi && lo / kTileKeys < shi) {  // else: no step of its own
        const long long slot = lo > 0 ? 2 * c : hi < keys ? 2 * c + 1 : 2ll * a.pshares + item;
        lse = a.plse + slot * 256 + prow;
        src = a.po + (slot * 256 + prow) * D;
      }
    } else if (i < n) {
      const long long c = c0 + i - np, slot = shares.start(c) > s0       ? 2 * c
                                              : shares.start(c + 1) < s1 ? 2 * c + 1
                                                                         : 2ll * a.shares + (long long)b * heads + hb;
      lse = a.slse + slot * a.rows + row;
      src = a.so + (slot * a.rows + row) * D;
    }
  };
  const float *src, *at_lse;
  place(lane * W + mine, src, at_lse);
  grid_dep_wait();
  if (nb > 0 && c0 == c1 && a.prefix == 0) return;  // finished by its CTA
  constexpr int E = D / 32;
  if ((int)blockIdx.y * (4 / W) + warp / W >= a.n_heads) return;
  float acc[E] = {}, z = 0.f, top = -INFINITY;
  for (int i0 = 0; i0 * W < n; i0 += 32) {
    if (i0) place((i0 + lane) * W + mine, src, at_lse);
    const float lse = at_lse ? *at_lse : -INFINITY;
    float mx = lse;
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if (mx == -INFINITY && __all_sync(0xffffffffu, lse == -INFINITY)) continue;  // mx passes over a NaN
    const float mn = fmaxf(top, mx), f = ex2(top - mn);
    top = mn;
    const float w = lse == -INFINITY ? 0.f : ex2(lse - mn);
    float zz = w;
#pragma unroll
    for (int d = 16; d; d >>= 1) zz += __shfl_xor_sync(0xffffffffu, zz, d);
    z = z * f + zz;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
    const int cnt = min(32, (n - mine + W - 1) / W - i0);
    for (int i1 = 0; i1 < cnt; i1 += 8) {
      // eight rows in flight; an empty part's row is not written, nor read
      float x[8][E], wi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wi[i] = __shfl_sync(0xffffffffu, w, (i1 + i) & 31);
        const float* from = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), (i1 + i) & 31));
        if (i1 + i >= cnt) wi[i] = 0.f;
        load_part<E>(from + lane * E, wi[i] != 0.f, x[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wi[i] * x[i][e];
    }
  }
  if (W > 1) {
    __shared__ float all[W][D + 2];
#pragma unroll
    for (int e = 0; e < E; ++e) all[mine][lane * E + e] = acc[e];
    if (lane == 0) {
      all[mine][D] = z;
      all[mine][D + 1] = top;
    }
    __syncthreads();
    if (mine) return;
    top = -INFINITY;
#pragma unroll
    for (int v = 0; v < W; ++v) top = fmaxf(top, all[v][D + 1]);
    z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float f = all[v][D + 1] == -INFINITY ? 0.f : ex2(all[v][D + 1] - top);
      z += f * all[v][D];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * all[v][lane * E + e];
    }
  }
  const float inv = z != 0.f ? 1.f / z : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + b * a.ldo + (long long)h * D + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
}

template <int D>
inline cudaError_t launch_decode(const CUtensorMap& tmK, const CUtensorMap& tmV, const DecArgs& a, cudaStream_t st) {
  auto kern = k_decode_attn<D>;
  cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), DecLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.shares + 1) / 2);
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = DecLayout<D>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tmK, tmV, a);
  if (e != cudaSuccess) return e;
  // Four warps share a head's parts when there are few heads, and so many parts
  // of each (one sequence of 8191 keys, 32 heads in 37 parts: 11.7 us with four,
  // 15.4 with one; 64 sequences over a prefix: 60.8 with four, 51.7 with one).
  const bool few = (long long)a.b.batch * a.n_heads <= 512;
  cfg.gridDim = dim3(a.b.batch, few ? a.n_heads : (a.n_heads + 3) / 4);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return few ? cudaLaunchKernelEx(&cfg, k_join<D, 4>, a) : cudaLaunchKernelEx(&cfg, k_join<D, 1>, a);
}

}  // namespace attn
}  // namespace serq

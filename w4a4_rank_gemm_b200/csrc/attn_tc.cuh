// Attention of many rows on the tensor cores: prompts (causal), and the
// shared prefix of a decode batch.
//
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  l += sum P,  c = scale log2 e
//
// One pass over the keys per 128-row tile with the running maximum m and sum
// l of each row; O and S never leave tensor memory and registers.
//
// P is rounded to bf16, the type of V that a tensor-core product wants (m and l
// are not): the result's error, 1.63e-3 from its own rounding, becomes 2.07e-3
// (root mean square, 2048 tokens).  Bringing it back takes a second product with
// what the rounding leaves over, half as many MMAs again in a step whose MMAs
// are 2048 of 3400 cycles.
//
// Rows of a tile are (token, query head of the kv head's group): all heads of
// a group read the same keys, so 128 / g tokens x g heads share one tile, and
// one token of a whole group fills g rows.  A CTA works on a pair of tiles (A:
// the earlier tokens, B: the next) that share the K and V tiles it streams:
// while the tensor core computes one tile's products the other's softmax runs.
//
// TMEM (512 columns): S_A, S_B (128 fp32 columns each; P_X in bf16 takes the
// first 64 columns of S_X as its scores have been read), O_A, O_B (D each).
//
// Warps: 0-3 softmax of A (one row per thread), 4-7 of B, 8 loads, 9 MMAs, 10
// zeroes values behind the last key, 11 decodes work items ahead.
// Every role waits for the grid in front before its first bounded wait, whose
// limit then never counts that grid's time.
// Persistent: a CTA takes work items (tile pair, kv head, range of key steps)
// and the next item's Q, K and first scores overlap the epilogue of the last.
#pragma once

#include <algorithm>
#include <type_traits>

#include "rope.cuh"

namespace serq {
namespace attn {

constexpr int kTileRows = 128;  // rows of a tile
constexpr int kTileKeys = 128;  // keys of a step
// Three warpgroups.  Launched with 168 registers a thread (384 x 168 = 64512);
// loads and MMAs keep 88, the softmax threads take 208, each holding a row of
// 128 scores: 128 x 88 + 256 x 208 = 64512.
constexpr int kTcThreads = 384;
constexpr int kRegsIssue = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= kTcThreads * 168, "register split");
constexpr int kFmaPairs = 4;  // of 16 pairs of exponentials, how many go to the FMA pipe
constexpr float kSumLimit = 1.0995116e12f;  // 2^40: see LONG below
constexpr float kLazyMax = 8.0f;            // log2: how far a row's scores may exceed the maximum in use
// Limit of the waits that may last as long as an item or the kernel: for a work
// item, and a tile's for its scores while the other tile's item goes on (an item
// of 80 million keys lasts a second).
constexpr unsigned long long kItemWaitNs = 100 * kWaitLimitNs;

struct TcArgs {
  __nv_bfloat16* o;
  long long ldo;
  float* po;    // partial outputs [slot][row of the pair][D], normalised
  float* plse;  // and log2 of their sums [slot][row of the pair], -inf: nothing
  float c;           // |scale| log2 e, never 0
  int neg;           // scale < 0: the product is taken with -Q
  int T, group, tokens;  // tokens: per tile, 128 / group
  int pair_shift;    // log2 of a pair's tokens, or -1
  int shares;        // > 0: equal shares of the work for that many CTAs; 0: whole items
  int prefix;        // > 0: decode rows; every row is at sequence 0's first `prefix` keys, up to its own kv_len
  BatchArgs b;
  CacheArgs c_;
};

struct Item {
  int done;
  int j0, endA, endB;  // steps [j0, end) of 128 keys; end <= j0: none
  int row0, n_tok;     // first token row, tokens of the pair
  int lim0;            // keys that the first token sees (causal: one more for each next)
  int kv_end;          // keys that exist
  int kvh, seq;
  int slot;            // of the partial output; -1: the item's rows are finished here
};

template <int D>
struct TcLayout {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = 128 * D * 2;  // bytes of a Q tile, and of a K or V step
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * kTile;
  static constexpr int oStage = oKV + kSlots * kTile;  // 4 KB per softmax warp
  static constexpr int oItem = oStage + 8 * 4096;
  static constexpr int oBar = oItem + 2 * 64;
  static constexpr int kBars = 2 * kSlots + 2 * 8 + 3;
  static constexpr int oMisc = oBar + kBars * 8;
  static constexpr int kAlloc = oMisc + 32 + 1024;
  static_assert(kAlloc <= 232448, "shared memory of a CTA");
  static_assert(oMisc % 8 == 0, "alignment");
};
static_assert(sizeof(Item) <= 64, "item slot");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger one, or NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 2^y on the FMA pipe: n = round(y), r = y - n in [-1/2, 1/2], a
// degree-4 polynomial for 2^r (least maximum relative error with constant term
// 1, found by reweighted least squares: 2.9e-6, a 1400th of the bf16 rounding that
// follows), n added to its exponent.  -127 and below give 0; CAP: above 127 as
// 127, else y stays below that.  A NaN gives what is not finite as a bf16 (CAP:
// 2^127, which is never used).
template <bool CAP>
__device__ __forceinline__ float2 ex2_fma(float2 y) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: the sum's low bits are n
  y.x = max_nan(y.x, -127.0f);
  y.y = max_nan(y.y, -127.0f);
  if (CAP) {
    y.x = fminf(y.x, 127.0f);
    y.y = fminf(y.y, 127.0f);
  }
  const float2 t = add2(y, make_float2(kRound, kRound));
  const float2 r = add2(y, add2(make_float2(kRound, kRound), make_float2(-t.x, -t.y)));
  float2 p = make_float2(0.009582852944731712f, 0.009582852944731712f);
  p = fma2(p, r, make_float2(0.055906426161527634f, 0.055906426161527634f));
  p = fma2(p, r, make_float2(0.24024099111557007f, 0.24024099111557007f));
  p = fma2(p, r, make_float2(0.6931241750717163f, 0.6931241750717163f));
  p = fma2(p, r, make_float2(1.0f, 1.0f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A sequence's tile pairs: pair i holds tokens [i pair, (i + 1) pair) and sees
// the keys up to its last token.
struct Pairs {
  int n, first, kv;  // query rows, first row, cached tokens
  int np;            // tile pairs
  int keys;          // of kv, those that the page table holds
};

// n / (2 tokens), n >= 0; by a shift where it can be (the scheduler's counting
// divides often, and a work item waits for it).
__device__ __forceinline__ int div_pair(const TcArgs& a, int n) {
  return a.pair_shift >= 0 ? n >> a.pair_shift : n / (2 * a.tokens);
}

__device__ __forceinline__ Pairs load_pairs(const TcArgs& a, int b) {
  const int pair = 2 * a.tokens;
  Pairs s = {0, 0, 0, 0, 0};
  if (a.prefix == 0 && b < a.b.batch) {
    s.first = a.b.cu_q[b];
    s.n = max(0, a.b.cu_q[b + 1] - s.first);
    s.kv = a.b.kv_len[b];
    s.np = div_pair(a, s.n + pair - 1);
    s.keys = max(0, min(s.kv, a.b.max_pages << a.c_.page_shift));
  }
  return s;
}

// Keys and steps of pair i.
__device__ __forceinline__ int pair_steps(const Pairs& s, int i, int pair) {
  return ceil_div(max(0, min(s.keys, s.kv - s.n + min(s.n, (i + 1) * pair))), kTileKeys);
}

// The item of pair `tile` of sequence `seq` and kv head, steps [lo, hi).
__device__ __forceinline__ void fill_item(const TcArgs& a, const Pairs& s, int seq, int tile, int kvh, int lo, int hi,
                                          Item& it) {
  const int pair = 2 * a.tokens;
  it.done = 0;
  it.seq = seq;
  it.kvh = kvh;
  it.row0 = s.first + tile * pair;
  it.n_tok = min(pair, s.n - tile * pair);
  it.kv_end = s.keys;
  int limA, limB;  // most keys that a row of the tile sees
  if (a.prefix) {
    it.lim0 = 0;
    limA = limB = s.keys;
  } else {
    it.lim0 = s.kv - s.n + tile * pair + 1;
    limA = min(s.keys, it.lim0 + min(a.tokens, it.n_tok) - 1);
    limB = min(s.keys, it.lim0 + it.n_tok - 1);
    if (s.kv > s.keys && s.kv > 0) note_bad_page();
  }
  it.j0 = lo;
  it.endA = min(hi, ceil_div(max(limA, 0), kTileKeys));
  it.endB = it.n_tok > a.tokens ? min(hi, ceil_div(max(limB, 0), kTileKeys)) : 0;
}

// Whole items in falling cost.  `mine` is lane's sequence (batch <= 32), so
// that an item is found without touching memory: the r-th costliest pair has
// the largest number of steps X with more than r pairs of at least X, counted
// per sequence in closed form.  Batches above 32 take pairs from the back.
__device__ __forceinline__ void ranked_item(const TcArgs& a, const Pairs& mine, int w, int lane, Item& it) {
  const int pair = 2 * a.tokens, heads = a.c_.n_kv_heads;
  const int r = w / heads, kvh = w - r * heads;
  it.slot = -1;
  it.done = 1;
  if (a.b.batch <= 32) {
    const int total = __reduce_add_sync(0xffffffffu, mine.np);
    if (r >= total) return;
    auto at_least = [&](int x) {  // this lane's pairs of at least x steps
      if (x <= 0) return mine.np;
      const int v = (x - 1) * kTileKeys;
      if (mine.np == 0 || min(mine.keys, mine.kv) <= v) return 0;
      return mine.np - min(mine.np, div_pair(a, max(0, v - (mine.kv - mine.n))));
    };
    int x = 0;
    if (total * heads > (int)gridDim.x) {
      int hi = __reduce_max_sync(0xffffffffu, ceil_div(mine.keys, kTileKeys)) + 1;
      while (hi - x > 1) {
        const int mid = (x + hi) >> 1;
        if ((int)__reduce_add_sync(0xffffffffu, at_least(mid)) > r) x = mid;
        else hi = mid;
      }
    } else {
      x = -1;  // one round: any order
    }
    const int ge = x < 0 ? mine.np : at_least(x), gt = x < 0 ? 0 : at_least(x + 1);
    const int left = r - (int)__reduce_add_sync(0xffffffffu, gt), eq = ge - gt;
    int incl = eq;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, left < incl)) - 1;
    const int tile = __shfl_sync(0xffffffffu, mine.np - ge + left - (incl - eq), src);
    Pairs s;
    s.n = __shfl_sync(0xffffffffu, mine.n, src);
    s.first = __shfl_sync(0xffffffffu, mine.first, src);
    s.kv = __shfl_sync(0xffffffffu, mine.kv, src);
    s.np = 0;
    s.keys = __shfl_sync(0xffffffffu, mine.keys, src);
    fill_item(a, s, src, tile, kvh, 0, 0x7fffffff, it);
    return;
  }
  int total = 0;
  for (int b0 = 0; b0 < a.b.batch; b0 += 32)
    total += __reduce_add_sync(0xffffffffu, load_pairs(a, b0 + lane).np);
  if (r >= total) return;
  int left = total - 1 - r;
  for (int b0 = 0;; b0 += 32) {
    const Pairs p = load_pairs(a, b0 + lane);
    int incl = p.np;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, left < incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int tile = __shfl_sync(0xffffffffu, left - (incl - p.np), src);
      fill_item(a, load_pairs(a, b0 + src), b0 + src, tile, kvh, 0, 0x7fffffff, it);
      return;
    }
    left -= __shfl_sync(0xffffffffu, incl, 31);
  }
}

__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Equal shares of `total` units of work: the first total % G have one more.
struct Shares {
  long long base, more;  // of a share, shares with one more
  __device__ Shares(long long total, int g) {
    base = quotient(total, g);
    more = total - base * g;
  }
  __device__ long long start(long long c) const { return c * base + min(c, more); }
  __device__ int of(long long w) const {  // the share that holds unit w
    const long long m = more * (base + 1);
    return (int)(w < m ? quotient(w, base + 1) : more + quotient(w - m, base));
  }
};

// Equal shares.  Work is laid out by sequence, kv head and tile pair and
// measured in keys, m_i = E + past + (i + 1) pair for pair i (every pair of the
// shared prefix: its keys), whose sums have a closed form; E stands for an
// item's beginning and end.  An item cut at key x is cut at step x / 128, if it
// has that many.  (E = 0, 128, 256, 384, 512: 6 chunks of up to 700 tokens over
// up to 5000, 14/2 heads of 64, 94.1, 77.0, 65.7, 66.1, 68.1 us; 16 of 50 tokens
// over 0 ... 7500, 32/8 heads of 128, 141.8, 109.0, 95.0, 94.6, 95.4.)
constexpr int kItemKeys = 2 * kTileKeys;
struct Measure {
  long long past, inc;  // m_i = past + (i + 1) inc
  __device__ long long of(int i) const { return past + (i + 1) * inc; }
  __device__ long long before(long long i) const { return i * past + inc * (i * (i + 1) / 2); }
};
__device__ __forceinline__ Measure measure(const TcArgs& a, const Pairs& s) {
  Measure m;
  m.past = a.prefix ? s.keys : max(kItemKeys, s.kv - s.n + kItemKeys);
  m.inc = a.prefix ? 0 : 2 * a.tokens;
  return m;
}

// The one pseudo-sequence of a decode batch's shared prefix (the warp calls).
// Where the table holds nothing but the prefix no other kernel sees a sequence
// that is longer than it.
__device__ __forceinline__ Pairs prefix_pairs(const TcArgs& a, int lane) {
  const int cap = a.b.max_pages << a.c_.page_shift;
  int m = 0;
  for (int b = lane; b < a.b.batch; b += 32) {
    const int kv = a.b.kv_len[b];
    m = max(m, min(kv, a.prefix));
    if (kv > cap) note_bad_page();
  }
  Pairs s;
  s.n = a.T;
  s.first = 0;
  s.kv = s.keys = __reduce_max_sync(0xffffffffu, m);
  s.np = s.keys ? ceil_div(a.T, 2 * a.tokens) : 0;
  return s;
}

// Work of one kv head over the sequences before b, and over all (the warp calls).
__device__ __forceinline__ void share_sums(const TcArgs& a, int b, int lane, long long& before, long long& total) {
  long long lo = 0, all = 0;
  for (int i = lane; i < a.b.batch; i += 32) {
    const Pairs s = load_pairs(a, i);
    const long long m = measure(a, s).before(s.np);
    all += m;
    if (i < b) lo += m;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    lo += __shfl_xor_sync(0xffffffffu, lo, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
  before = lo;
  total = all;
}

// The next segment of a share; state is the same in every lane.
struct ShareWalk {
  long long x, x1;  // position, end
  long long start;  // of the current item
  int seq, kvh, tile;
  Pairs s;

  // All work there is (the warp calls, and locate).
  __device__ long long total(const TcArgs& a, int lane) {
    if (a.prefix == 0) {
      long long before, all;
      share_sums(a, 0, lane, before, all);
      return all * a.c_.n_kv_heads;
    }
    s = prefix_pairs(a, lane);
    return measure(a, s).before(s.np) * a.c_.n_kv_heads;
  }

  // The item that holds unit `at` of the work.
  __device__ void locate(const TcArgs& a, long long at, int lane) {
    const int heads = a.c_.n_kv_heads;
    seq = 0;
    long long base = 0, per_head = 0;
    if (a.prefix) {
      per_head = measure(a, s).before(s.np);
    } else {
      for (int b0 = 0;; b0 += 32) {
        const Pairs p = load_pairs(a, b0 + lane);
        const long long m = measure(a, p).before(p.np);
        long long incl = m;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, at < (base + incl) * heads);
        if (hit) {
          const int src = __ffs(hit) - 1;
          seq = b0 + src;
          per_head = __shfl_sync(0xffffffffu, m, src);
          base += __shfl_sync(0xffffffffu, incl, src) - per_head;
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      s = load_pairs(a, seq);
    }
    const long long rest = at - base * heads;
    kvh = (int)quotient(rest, per_head);
    const long long in = rest - kvh * per_head;
    const Measure m = measure(a, s);
    int lo = 0, hi = s.np;  // the tile with before(lo) <= in < before(lo + 1)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (m.before(mid) <= in) lo = mid;
      else hi = mid;
    }
    tile = lo;
    start = base * heads + kvh * per_head + m.before(lo);
  }

  __device__ void init(const TcArgs& a, int lane) {
    const Shares shares(total(a, lane), a.shares);
    x = shares.start(blockIdx.x);
    x1 = shares.start(blockIdx.x + 1);
    if (x < x1) locate(a, x, lane);
  }

  // False: the share is finished.  Segments without a step are passed over.
  __device__ bool next(const TcArgs& a, Item& it) {
    const int heads = a.c_.n_kv_heads;
    while (x < x1) {
      const long long size = measure(a, s).of(tile);
      const int steps = a.prefix ? ceil_div(s.keys, kTileKeys) : pair_steps(s, tile, 2 * a.tokens);
      const long long lo = x - start, hi = min(x1 - start, size);
      const int slo = (int)min((long long)steps, lo / kTileKeys);
      const int shi = hi == size ? steps : (int)min((long long)steps, hi / kTileKeys);
      const bool emit = shi > slo || (steps == 0 && lo == 0);
      if (emit) {
        fill_item(a, s, seq, tile, kvh, slo, shi, it);
        it.slot = a.prefix == 0 && slo == 0 && shi == steps ? -1
                  : lo > 0                                  ? 2 * (int)blockIdx.x
                  : hi < size                               ? 2 * (int)blockIdx.x + 1
                                                            : 2 * a.shares + kvh * s.np + tile;
      }
      x = start + hi;
      if (hi == size) {
        start += size;
        if (++tile == s.np) {
          tile = 0;
          if (++kvh == heads) {
            kvh = 0;
            if (x < x1) {  // then another sequence with rows follows
              do s = load_pairs(a, ++seq);
              while (s.np == 0);
            }
          }
        }
      }
      if (emit) return true;
    }
    return false;
  }
};

template <int D, bool LONG>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_attn(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
           const __grid_constant__ CUtensorMap tmV, const TcArgs a) {
  using L = TcLayout<D>;
  constexpr uint32_t kS = 0, kO = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Item* items = reinterpret_cast<Item*>(smem + L::oItem);  // two, 64 bytes apart
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::oBar);
  uint64_t* kv_full = bar;
  uint64_t* kv_empty = kv_full + L::kSlots;
  uint64_t* q_full = kv_empty + L::kSlots;  // [2] tile X's rows landed
  uint64_t* q_empty = q_full + 2;           // [2] the item's last scores of X are computed
  uint64_t* s_full = q_empty + 2;           // [2] scores ready (and every MMA before them)
  uint64_t* p_full = s_full + 2;            // [2] weights written (and O rescaled)
  uint64_t* p_half = p_full + 2;            // [2] the first 64 keys' weights
  uint64_t* o_full = p_half + 2;            // [2] the item's last product of X is done
  uint64_t* it_full = o_full + 2;           // [2]
  uint64_t* it_empty = it_full + 2;         // [2]
  uint64_t* drain = it_empty + 2;
  uint64_t* clean_ask = drain + 1;          // values to zero: slot and first row in clean_req
  uint64_t* clean_done = drain + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oMisc + 4);
  volatile int* clean_req = reinterpret_cast<volatile int*>(smem + L::oMisc + 8);
  auto item_at = [&](int i) -> Item& {
    return *reinterpret_cast<Item*>(reinterpret_cast<uint8_t*>(items) + (i & 1) * 64);
  };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&p_half[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&it_full[x], 1);
      mbar_init(&it_empty[x], 10);
    }
    mbar_init(drain, 1);
    mbar_init(clean_ask, 1);
    mbar_init(clean_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc<1>(tmem_slot, 512);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 8) {
      // --------------------------------------------------------------- loads
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      grid_dep_wait();
      const int page = 1 << a.c_.page_shift;
      const int box = min(page, kTileKeys);         // rows per copy
      const int copies = kTileKeys / box * L::kHalves;  // per step and operand
      uint32_t slot = 0, slot_ph = 0, qn[2] = {0, 0};
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&it_full[i & 1], (i >> 1) & 1, abort_flag, kDevTimeoutProducer))) break;
        const Item it = item_at(i);
        __syncwarp();
        if (lane == 0) mbar_arrive(&it_empty[i & 1]);
        if (it.done) break;
        const int32_t* table = a.b.table + (long long)it.seq * a.b.ldt;
        const int end = max(it.endA, it.endB);
        // this lane's copy of a step: its page is looked up one step ahead
        const int half = lane & (L::kHalves - 1), r = lane / L::kHalves * box;
        auto lookup = [&](int j) {
          const int key = j * kTileKeys + r;
          int pg = a.c_.n_pages;  // past the keys that exist: zeros, from outside the map
          if (lane < copies && key < it.kv_end) {
            const int e = table[key >> a.c_.page_shift];
            if (e >= 0 && e < a.c_.n_pages) pg = e;
            else note_bad_page();
          }
          return pg;
        };
        auto load = [&](const CUtensorMap* tm, int j, int pg) {
          ok = __all_sync(0xffffffffu,
                          mbar_wait_idle(&kv_empty[slot], slot_ph ^ 1, abort_flag, kDevTimeoutProducer, kWaitLimitNs));
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], L::kTile);
          __syncwarp();
          if (lane < copies)
            tma_load_3d(smem + L::oKV + slot * L::kTile + half * (L::kTile / L::kHalves) + r * 128, tm, &kv_full[slot],
                        64 * half, (it.kvh << a.c_.page_shift) + ((j * kTileKeys + r) & (page - 1)), pg);
          __syncwarp();
          if (++slot == L::kSlots) slot = 0, slot_ph ^= 1;
        };
        int pg = it.j0 < end ? lookup(it.j0) : 0;
#pragma unroll 1
        for (int j = it.j0; j < end && ok; ++j) {
          const int pg_next = j + 1 < end ? lookup(j + 1) : 0;
          load(&tmK, j, pg);
          if (j == it.j0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || (x ? it.endB : it.endA) <= it.j0) continue;
              ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[x], (qn[x] & 1) ^ 1, abort_flag, kDevTimeoutProducer));
              if (!ok) continue;
              ++qn[x];
              if (lane == 0) {
                mbar_arrive_expect_tx(&q_full[x], a.tokens * a.group * D * 2);
                for (int h = 0; h < L::kHalves; ++h)
                  tma_load_3d(smem + L::oQ + x * L::kTile + h * (L::kTile / L::kHalves), &tmQ, &q_full[x], 64 * h,
                              it.kvh * a.group, it.row0 + x * a.tokens);
              }
              __syncwarp();
            }
          }
          if (ok) load(&tmV, j, pg);
          pg = pg_next;
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMAs
      // One thread runs the whole loop: the tensor core takes a step's 32 MMAs
      // about as fast as they are issued, so what the issuing thread spends
      // between them on waits and votes leaves the tensor core idle (with the
      // whole warp waiting and electing a lane each time, a step of two tiles
      // took 3400 cycles, 2048 of them MMAs).
      grid_dep_wait();
      if (elect_one()) {
        const uint32_t idesc_qk = umma_idesc_bf16(128, kTileKeys, false, a.neg);
        constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D, true, false);
        constexpr int kHalfBytes = L::kTile / L::kHalves;
        const uint64_t desc_q = umma_desc_k_sw128(smem_u32(smem + L::oQ));
        const uint64_t desc_k = umma_desc_k_sw128(smem_u32(smem + L::oKV));
        const uint64_t desc_v = umma_desc_mn_sw128(smem_u32(smem + L::oKV), kHalfBytes);
        uint32_t slot = 0, slot_ph = 0, qn[2] = {0, 0}, pn[2] = {0, 0}, cn = 0;
        bool ok = true;
        auto wait = [&](uint64_t* b, uint32_t ph) { return ok = ok && mbar_wait(b, ph, abort_flag, kDevTimeoutMma); };
        auto next_slot = [&] {
          if (++slot == L::kSlots) slot = 0, slot_ph ^= 1;
        };
        auto scores = [&](int x, uint32_t ks) {
          const uint64_t dq = desc_q + (uint64_t)(x * (L::kTile >> 4)), dk = desc_k + (uint64_t)(ks * (L::kTile >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (uint64_t)((k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2);
            umma_bf16_ss(tmem + kS + 128u * x, dq + off, dk + off, idesc_qk, k > 0);
          }
        };
        auto values = [&](int x, uint32_t vs, bool acc, int half) {
          const uint64_t dv = desc_v + (uint64_t)(vs * (L::kTile >> 4));
#pragma unroll
          for (int k = half * 4; k < half * 4 + 4; ++k)
            umma_bf16_ts(tmem + kO + (uint32_t)(D * x), tmem + kS + 128u * x + 8u * k, dv + (uint64_t)(128 * k), idesc_pv,
                         acc || k > 0);
        };
        // An item's first scores are issued as soon as the previous item leaves
        // room, in front of its other tile's last products where they can be.
        struct Steps {
          int done, j0, endA, endB, kv_end;
          __device__ int last(int x) const { return x ? endB : endA; }
          __device__ int end() const { return max(endA, endB); }
        };
        int n_read = 0;
        auto read_item = [&](Steps& t) {
          const Item& it = item_at(n_read);
          t.done = it.done, t.j0 = it.j0, t.endA = it.endA, t.endB = it.endB, t.kv_end = it.kv_end;
          mbar_arrive(&it_empty[n_read & 1]);
          ++n_read;
        };
        auto first_scores = [&](const Steps& t, int x) {
          ++qn[x];
          tc_fence_after();
          scores(x, slot);
          umma_commit<1>(&s_full[x]);
          if (t.j0 + 1 == t.last(x)) umma_commit<1>(&q_empty[x]);
        };
        Steps cur, nxt;
        bool have = false;              // nxt holds the next item
        bool given[2] = {false, false};  // its first scores are issued
        while (ok) {
          if (have) {
            cur = nxt;
            have = false;
          } else {
            if (!wait(&it_full[n_read & 1], (n_read >> 1) & 1)) break;
            read_item(cur);
          }
          if (cur.done) break;
          const int end = cur.end();
          if (end <= cur.j0) continue;
          if (!wait(&kv_full[slot], slot_ph)) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!given[x] && cur.j0 < cur.last(x) && wait(&q_full[x], qn[x] & 1)) first_scores(cur, x);
            given[x] = false;
          }
          if (!ok) break;
          umma_commit<1>(&kv_empty[slot]);
          next_slot();
          for (int j = cur.j0; j < end; ++j) {
            const uint32_t vs = slot;
            if (!wait(&kv_full[slot], slot_ph)) break;
            next_slot();
            const uint32_t ks = slot;
            bool ahead = false;  // the next item's first keys have landed
            if (j + 1 < end) {
              if (!wait(&kv_full[slot], slot_ph)) break;
              next_slot();
            } else if (mbar_try_wait(&it_full[n_read & 1], (n_read >> 1) & 1)) {
              read_item(nxt);
              have = true;
              ahead = !nxt.done && nxt.j0 < nxt.end() && mbar_try_wait(&kv_full[slot], slot_ph);
            }
            if (cur.kv_end - j * kTileKeys < kTileKeys) {  // values that do not exist: see the helper warp
              clean_req[0] = (int)vs;
              clean_req[1] = cur.kv_end - j * kTileKeys;
              mbar_arrive(clean_ask);
              if (!wait(clean_done, cn++ & 1)) break;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int last = cur.last(x);
              if (j < last) {
                if (!wait(&p_half[x], pn[x] & 1)) continue;
                tc_fence_after();
                values(x, vs, j > cur.j0, 0);
                if (!wait(&p_full[x], pn[x] & 1)) continue;
                ++pn[x];
                tc_fence_after();
                values(x, vs, true, 1);
                if (j + 1 < last) {
                  scores(x, ks);
                  umma_commit<1>(&s_full[x]);
                  if (j + 2 == last) umma_commit<1>(&q_empty[x]);
                } else {
                  umma_commit<1>(&o_full[x]);
                }
              }
              if (ahead && nxt.j0 < nxt.last(x) && mbar_try_wait(&q_full[x], qn[x] & 1)) {
                first_scores(nxt, x);
                given[x] = true;
              }
            }
            if (!ok) break;
            umma_commit<1>(&kv_empty[vs]);
            if (j + 1 < end) umma_commit<1>(&kv_empty[ks]);
          }
        }
        // every MMA issued has completed before TMEM and shared memory are freed
        umma_commit<1>(drain);
        mbar_wait(drain, 0, nullptr, kDevTimeoutMma);
        clean_req[0] = -1;
        mbar_arrive(clean_ask);
      }
      __syncwarp();
    } else if (warp == 10) {
      // -------------------------------------------------------------- helper
      // Rows of V behind the last key, up to the end of its page, may hold
      // anything, and a zero weight times a NaN is one: on the MMA thread's
      // request they are zeroed once they have landed.
      constexpr int kHalfBytes = L::kTile / L::kHalves;
      grid_dep_wait();
      for (uint32_t n = 0;; ++n) {
        // lasts as long as the kernel does: the MMA thread, whose own waits are
        // bounded, always ends it
        if (!__all_sync(0xffffffffu, mbar_wait_idle(clean_ask, n & 1, abort_flag, kDevTimeoutMma, kItemWaitNs))) break;
        const int vs = clean_req[0], have = clean_req[1];
        __syncwarp();
        if (vs < 0) break;
        const int upto = min(kTileKeys, (have + (1 << a.c_.page_shift) - 1) >> a.c_.page_shift << a.c_.page_shift);
        const int chunks = (upto - have) * (D / 8);
        for (int e = lane; e < chunks; e += 32) {
          const int r = have + e / (D / 8), c = e % (D / 8);
          *reinterpret_cast<uint4*>(smem + L::oKV + vs * L::kTile + (c >> 3) * kHalfBytes + r * 128 + (c & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(clean_done);
      }
    } else {
      // ----------------------------------------------------------- scheduling
      // Decodes the CTA's work items ahead of their use.
      grid_dep_wait();
      grid_dep_launch();
      ShareWalk walk;
      Pairs mine = {0, 0, 0, 0, 0};
      if (a.shares) walk.init(a, lane);
      else if (a.b.batch <= 32) mine = load_pairs(a, lane);
      for (int i = 0;; ++i) {
        Item it;
        it.done = 1;
        if (a.shares) {
          if (!walk.next(a, it)) it.done = 1;
        } else {
          // every other round backwards: the items come in falling cost, so that
          // each CTA's sum stays near the mean
          ranked_item(a, mine, i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x), lane, it);
        }
        if (!__all_sync(0xffffffffu, mbar_wait_idle(&it_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag,
                                                    kDevTimeoutProducer, kItemWaitNs)))
          break;
        if (lane == 0) {
          item_at(i) = it;
          mbar_arrive(&it_full[i & 1]);
        }
        if (it.done) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------- softmax
    grid_dep_wait();
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + kS + 128u * x, tO = tmem + lanes + kO + (uint32_t)(D * x);
    const int tok = row / a.group, head = row - tok * a.group;
    uint32_t sn = 0, on = 0;
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&it_full[i & 1], (i >> 1) & 1, abort_flag, kDevTimeoutEpilogue, kItemWaitNs)))
        break;
      const Item it = item_at(i);
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[i & 1]);
      if (it.done) break;
      const int end = x ? it.endB : it.endA;
      const int ti = x * a.tokens + tok;  // token within the pair
      const int t = it.row0 + ti;
      const bool valid = tok < a.tokens && ti < it.n_tok && t >= 0 && t < a.T;
      // keys this row sees; a row that is no row masks nothing
      int lim = 0x7fffffff;
      if (valid) lim = a.prefix ? min(a.b.kv_len[t], it.kv_end) : min(it.lim0 + ti, it.kv_end);
      const int warp_lim = __reduce_min_sync(0xffffffffu, lim);
      float mc = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = it.j0; j < end; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x], sn++ & 1, abort_flag, kDevTimeoutEpilogue, kItemWaitNs));
        if (!ok) break;
        tc_fence_after();
        // The scores are read from TMEM twice, for the maximum and for the
        // weights: held in registers in between, they left too few for the
        // exponentials' temporaries (spills; 750 cycles per 64 keys, not 560).
        const int base = j * kTileKeys;
        // LONG: past an item's first step the maximum in use mostly still serves,
        // and then need not be known: weights are formed with it, kept in
        // registers, and used as long as their sum stays below 2^40 (bf16 and fp32
        // are as exact there); only a larger sum, a first step and an edge look
        // for the maximum.  This saves a step's first reading of the scores, at
        // the price of more code, which short items do not pay back: 300 new
        // tokens over 300, ten times, 44.7 us with it and 41.5 without, prompts of
        // 2048 tokens 42.5 and 42.1, of 4096 141 and 147, of 8192 513 and 553.
        if (LONG && j > it.j0 && base + kTileKeys <= warp_lim) {
          const float sub = mc == -INFINITY ? 0.f : -mc;
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
          uint32_t w[4][16];
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(tS, s[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_ld_wait_regs(s[q & 1]);
            if (q < 3) tmem_ld_32x32b_x32(tS + 32u * (q + 1), s[(q + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 s2 = make_float2(__uint_as_float(s[q & 1][2 * e]), __uint_as_float(s[q & 1][2 * e + 1]));
              const float2 y = fma2(s2, make_float2(a.c, a.c), make_float2(sub, sub));
              const float2 p = (e * kFmaPairs) % 16 < kFmaPairs ? ex2_fma<true>(y) : make_float2(ex2(y.x), ex2(y.y));
              if (e & 1) sum1 = add2(sum1, p);
              else sum0 = add2(sum0, p);
              const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
              w[q][e] = reinterpret_cast<const uint32_t&>(h);
            }
          }
          const float sum = (sum0.x + sum0.y) + (sum1.x + sum1.y);
          if (!__any_sync(0xffffffffu, valid && !(sum < kSumLimit))) {
            l += sum;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tmem_st_32x32b_x16(tS + 16u * q, w[q]);
              if (q & 1) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q == 1 ? &p_half[x] : &p_full[x]);
              }
            }
            continue;
          }
        }
        auto mask = [&](uint32_t(&r)[32], int c0) {  // scores of columns c0 ... c0 + 31
          if (base + c0 + 32 > warp_lim) {
            const int left = lim - base - c0;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) r[e] = 0xff800000u;  // -inf
          }
        };
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 64) {
          uint32_t r[2][32];
          tmem_ld_32x32b_x32(tS + c0, r[0]);
          tmem_ld_32x32b_x32(tS + c0 + 32, r[1]);
          tmem_ld_wait_regs(r[0]);
          tmem_ld_wait_regs(r[1]);
          mask(r[0], c0);
          mask(r[1], c0 + 32);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            mx0 = max3_nan(mx0, __uint_as_float(r[0][e]), __uint_as_float(r[0][e + 1]));
            mx1 = max3_nan(mx1, __uint_as_float(r[1][e]), __uint_as_float(r[1][e + 1]));
          }
        }
        const float cand = max_nan(mx0, mx1) * a.c;
        // A NaN score makes the row's sum one, and so its result and its log-sum,
        // whatever weight its part has in the end; exponentials on the FMA pipe
        // turn it into 2^127 at most, which a larger score would outweigh.
        if (cand != cand) l = cand;
        // the maximum in use follows only when it falls behind by 2^8: weights
        // up to 2^8 cost nothing in bf16 or fp32, and most steps leave O alone
        const bool grow = valid && cand > mc + kLazyMax;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(mc - cand) : 1.0f;
          if (grow) {
            mc = cand;
            l *= f;
          }
          if (j > it.j0) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(tO + 16u * q, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(tO + 16u * q, o);
            }
          }
        }
        const float sub = mc == -INFINITY ? 0.f : -mc;
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 64) {
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(tS + c0, s[0]);
          tmem_ld_32x32b_x32(tS + c0 + 32, s[1]);
          tmem_ld_wait_regs(s[0]);
          tmem_ld_wait_regs(s[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            mask(s[q], c0 + 32 * q);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 s2 = make_float2(__uint_as_float(s[q][2 * e]), __uint_as_float(s[q][2 * e + 1]));
              const float2 y = fma2(s2, make_float2(a.c, a.c), make_float2(sub, sub));
              // the XU pipe's 16 exponentials a cycle would bound the kernel: part
              // of them is computed on the FMA pipe
              const float2 p = (e * kFmaPairs) % 16 < kFmaPairs ? ex2_fma<false>(y) : make_float2(ex2(y.x), ex2(y.y));
              if (e & 1) sum1 = add2(sum1, p);
              else sum0 = add2(sum0, p);
              const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
              w[e] = reinterpret_cast<const uint32_t&>(h);
            }
            // weights of columns c take columns c / 2, whose scores have been read
            tmem_st_32x32b_x16(tS + (c0 >> 1) + 16u * q, w);
          }
          // half of the keys: their product may start
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(c0 == 0 ? &p_half[x] : &p_full[x]);
        }
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
      }
      if (!ok) break;
      // -------------------------------------------------------- epilogue
      const bool any = end > it.j0;
      if (any) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], on++ & 1, abort_flag, kDevTimeoutEpilogue));
        if (!ok) break;
        tc_fence_after();
      }
      const float inv = l != 0.f ? 1.0f / l : 0.f;  // a NaN stays one
      const int h = it.kvh * a.group + head;
      uint8_t* stage = smem + L::oStage + warp * 4096;
      if (it.slot >= 0) {
        const long long at = (long long)it.slot * 256 + 128 * x + row;
        if (valid) a.plse[at] = l != 0.f ? mc + log2f(l) : -INFINITY;
        const bool write = valid && l != 0.f;
        const uint32_t writes = __ballot_sync(0xffffffffu, write);
        if (any) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + 32u * q, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                  make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                              __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
            __syncwarp();
            float* dst = a.po + (at - lane) * D + 32 * q + 4 * (lane & 7);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int rr = 4 * e + (lane >> 3);
              if (writes >> rr & 1)
                *reinterpret_cast<float4*>(dst + rr * D) =
                    *reinterpret_cast<const float4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            }
            __syncwarp();
          }
        }
      } else {
        // 64 columns at a time through the warp's 4 KB of shared memory, so that
        // rows leave as whole 128-byte lines (16-byte chunks swizzled by the row)
        __nv_bfloat16* dst = valid ? a.o + (long long)t * a.ldo + (long long)h * D : nullptr;
        __nv_bfloat16* to[8];  // the rows that this lane stores 16 bytes of
#pragma unroll
        for (int e = 0; e < 8; ++e)
          to[e] = reinterpret_cast<__nv_bfloat16*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), 4 * e + (lane >> 3)));
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {
          uint32_t o[2][32];
          if (any) {
            tmem_ld_32x32b_x32(tO + 64u * q, o[0]);
            tmem_ld_32x32b_x32(tO + 64u * q + 32u, o[1]);
            tmem_ld_wait_regs(o[0]);
            tmem_ld_wait_regs(o[1]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // a row that saw no key has inv = 0 and is written as zeros
              const float v0 = l != 0.f ? __uint_as_float(o[e >> 2][(8 * e + 2 * k) & 31]) * inv : 0.f;
              const float v1 = l != 0.f ? __uint_as_float(o[e >> 2][(8 * e + 2 * k + 1) & 31]) * inv : 0.f;
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v0, v1);
              w[k] = reinterpret_cast<const uint32_t&>(b2);
            }
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int rr = 4 * e + (lane >> 3), ch = lane & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
            if (to[e] != nullptr) *reinterpret_cast<uint4*>(to[e] + 64 * q + 8 * ch) = v;
          }
          __syncwarp();
        }
      }
      // the next item's first product overwrites O: its weights are only
      // signalled after these loads
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // let copies already issued land before the shared memory is released
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 100000ull) {
    }
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 512);
  }
}

// E = 2 or 4 consecutive floats, or zeros without a read.  (A branch around
// the read would make each of a row's parts wait for the one before it.)
template <int E>
__device__ __forceinline__ void load_part(const float* p, bool take, float (&x)[E]) {
  if constexpr (E == 4)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\tmov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
        "mov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t@q ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
        : "l"(p), "r"((int)take));
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\tmov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
        "@q ld.global.v2.f32 {%0, %1}, [%2];\n\t}"
        : "=f"(x[0]), "=f"(x[1])
        : "l"(p), "r"((int)take));
}

// Joins the parts of items that shares cut:
//   O = sum_s 2^(lse_s - M) O_s / sum_s 2^(lse_s - M),  s in share order.
// CTAs run over tile pairs, kv heads and (z) parts of a pair's rows; items that
// are not cut leave at once.  Four rows of a warp are joined together, KP parts
// at a time, all in flight together.
template <int D, int KP>
__global__ void __launch_bounds__(256, KP == 2 ? 2 : 1) k_merge(const TcArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Lengths and offsets are inputs of the call: k_attn lets this grid start
  // only after its own wait, so they are complete here.  (Every CTA waits
  // before it leaves: what follows in the stream may rely on this grid's end
  // for k_attn's.)
  const int pair = 2 * a.tokens, heads = a.c_.n_kv_heads, kvh = blockIdx.y;
  int seq = -1, tile = blockIdx.x;
  for (int b0 = 0; b0 < a.b.batch; b0 += 32) {
    const Pairs p = load_pairs(a, b0 + lane);
    int incl = p.np;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, tile < incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      seq = b0 + src;
      tile -= __shfl_sync(0xffffffffu, incl - p.np, src);
      break;
    }
    tile -= __shfl_sync(0xffffffffu, incl, 31);
  }
  if (seq < 0) {
    grid_dep_wait();
    return;
  }
  const Pairs s = load_pairs(a, seq);
  long long before, total;
  share_sums(a, seq, lane, before, total);
  const Measure m = measure(a, s);
  const long long s0 = before * heads + kvh * m.before(s.np) + m.before(tile), size = m.of(tile);
  total *= heads;
  const int steps = pair_steps(s, tile, pair);
  const Shares shares(total, a.shares);
  const int c0 = shares.of(s0), c1 = shares.of(s0 + size - 1);
  // slot of share c's part; -1: no step of the item, -2: all of them
  auto part = [&](int c) {
    if (c > c1) return -1;
    const long long lo = max(0ll, shares.start(c) - s0), hi = min(size, shares.start(c + 1) - s0);
    if (lo >= hi) return -1;
    const int slo = (int)min((long long)steps, lo / kTileKeys);
    const int shi = hi == size ? steps : (int)min((long long)steps, hi / kTileKeys);
    return slo >= shi ? -1 : slo == 0 && shi == steps ? -2 : lo > 0 ? 2 * c : 2 * c + 1;
  };
  bool whole = steps == 0;
  for (int c = c0 + lane; c <= c1; c += 32) whole |= part(c) == -2;
  grid_dep_wait();
  if (__any_sync(0xffffffffu, whole)) return;  // finished by its CTA
  constexpr int E = D / 32;
#pragma unroll 1
  for (int g = blockIdx.z; g < 8; g += gridDim.z) {
    long long at[4];  // output offset, -1: no row
    float acc[4][E] = {}, z[4] = {}, top[4];
    const int r0 = g * 32 + warp * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i, x = r >> 7, tok = (r & 127) / a.group, ti = x * a.tokens + tok;
      const int t = s.first + tile * pair + ti;
      const bool row = tok < a.tokens && ti < min(pair, s.n - tile * pair) && t >= 0 && t < a.T;
      at[i] = row ? t * a.ldo + (long long)(kvh * a.group + (r & 127) - tok * a.group) * D : -1;
      top[i] = -INFINITY;
    }
    if (at[0] < 0 && at[1] < 0 && at[2] < 0 && at[3] < 0) continue;
    for (int b0 = c0; b0 <= c1; b0 += 32) {
      const int slot = part(b0 + lane);
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lse = slot >= 0 && at[i] >= 0 ? a.plse[(long long)slot * 256 + r0 + i] : -INFINITY;
        float mx = lse;
#pragma unroll
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        mx = fmaxf(mx, top[i]);
        const float f = mx == -INFINITY ? 1.f : ex2(top[i] - mx);
        top[i] = mx;
        w[i] = lse == -INFINITY ? 0.f : ex2(lse - mx);
        float zz = w[i];
#pragma unroll
        for (int d = 16; d; d >>= 1) zz += __shfl_xor_sync(0xffffffffu, zz, d);
        z[i] = z[i] * f + zz;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] *= f;
      }
      const int cnt = min(32, c1 - b0 + 1);
      for (int k1 = 0; k1 < cnt; k1 += KP) {
        float v[KP][4][E], wk[KP][4];
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          const int sk = __shfl_sync(0xffffffffu, slot, (k1 + k) & 31);
          const float* src = a.po + ((long long)sk * 256 + r0) * D + lane * E;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            wk[k][i] = __shfl_sync(0xffffffffu, w[i], (k1 + k) & 31);
            if (k1 + k >= cnt) wk[k][i] = 0.f;
            // an empty part's row is not written, nor read
            load_part<E>(src + i * D, wk[k][i] != 0.f, v[k][i]);
          }
        }
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] += wk[k][i] * v[k][i][e];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at[i] < 0) continue;
      const float inv = z[i] != 0.f ? 1.f / z[i] : 0.f;
      __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.o + at[i] + lane * E);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) dst[e] = __floats2bfloat162_rn(acc[i][2 * e] * inv, acc[i][2 * e + 1] * inv);
    }
  }
}

// Shares of a call whose work is at most `items` tile pairs times kv heads of
// `keys` keys: none for less than 256 keys, and of few items an equal number of
// shares each, so that equal items are cut alike and no CTA starts twice (100
// tokens over 1000, 2 kv heads: 19.3 us, 21.2 with shares of 512 keys; 1 token
// over 8000, one kv head: 24.2, 22.8 and, with 128 keys, 30.2).
inline int tc_shares(long long items, long long keys, int sms) {
  const long long cuts = (keys + 255) / 256;
  if (items * 3 <= sms) return (int)std::max(1ll, items * std::min<long long>(sms / std::max(1ll, items), cuts));
  return (int)std::max(1ll, std::min<long long>(sms, items * cuts));
}

template <int D>
inline cudaError_t launch_tc(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const TcArgs& a,
                             int ctas, bool longer, cudaStream_t st) {
  auto kern = longer ? k_attn<D, true> : k_attn<D, false>;
  const cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), TcLayout<D>::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = TcLayout<D>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tmQ, tmK, tmV, a);
}

template <int D>
inline cudaError_t launch_merge(const TcArgs& a, int pairs, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // a CTA's look-ups cost about as much as joining 64 rows: more CTAs per item,
  // with more parts in flight, only where items are few (and have many parts)
  const bool few = (long long)pairs * a.c_.n_kv_heads * 3 <= sms;
  cfg.gridDim = dim3(pairs, a.c_.n_kv_heads, few ? 8 : 2);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, k_merge<D, 4>, a) : cudaLaunchKernelEx(&cfg, k_merge<D, 2>, a);
}

}  // namespace attn
}  // namespace serq

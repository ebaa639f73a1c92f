// Attention of whole prompts whose queries, keys and values are at hand in 16 bits
// (kvq_prompt_attention): packed sequences, causal, heads in groups.
//
// out = sum_t p_t v_t / sum_t p_t, p_t = 2^(z_t - m), z_t = sm_scale log2(e) <q, k_t>,
// with a running maximum m over tiles of 128 keys and float32 sums: one pass over
// the keys, no score leaves the SM.
//
// Split: an item of work is two halves of up to 128 rows (token, query head) of one
// sequence and kv-head; row R of a half is query head R % G of its token R / G, so the G
// heads that share keys fill a half together.  Per 128 keys and half it takes two
// tcgen05 products, S = Q K^T (operands in shared memory) and O += P V (P in tensor
// memory, over S's own columns); one half's products run while the other half's
// softmax does.  Q, K and V come by TMA from the caller's own rows, whatever their stride.
//
// One CTA per SM goes through a list of items that it makes itself: all items by falling
// number of keys, dealt out to and fro (0 1 2 .. 2 1 0), which evens the sums out.  Every
// role runs ahead as far as its buffers reach, across items too: an item's loads and first
// scores are made while the one before is finished and stored.
//
// Warps: one warpgroup per half for the softmax (a thread a row), one warp that issues
// the products, one that loads, two that look at the values of tiles that some row sees
// only in part (a probability of 0 times a value that is not finite would not be 0), the
// second of which makes the list.
//
// The maximum: bf16 keeps float32's range, so p need not be near 1, and a maximum that is
// far from the true one does as well.  Each row takes its first keys' and keeps it until a
// step of 64 keys sums to more than 2^20, which the sum itself says: no pass over the
// scores looks for maxima, only a step that has gone wrong is made again.
//
// Bound by the tensor cores for long prompts of 128-wide heads: 16,384 tokens, 64 / 8 heads
// 2,730 to 2,970 us, 1,480 to 1,610 TFLOP/s, as the power limit allows (2,895 in most
// runs), against 2,620 with the softmax left out (its best run); a pass for maxima and two
// warps a row took 2,910 where this took 2,730.  Heads of 64 have half the products per exponential and
// are bound by the softmax, whose two warps per scheduler do not hide all of their
// latency: 0.63 us per half and 128 keys, where the products take 0.35.
#include <algorithm>
#include <atomic>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "mbarrier.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_prompt)

namespace {

constexpr int kKeys = 128;       // keys per tile
constexpr int kDrain = 1 << 18;  // polls for what is in flight at a CTA's end (a second)
constexpr int kQuick = 1 << 9;   // the issuing warp's looks before it waits as the others do (some 10 us)
constexpr int kStep = 64;        // keys whose probabilities are handed over together
constexpr float kMost = 0x1p20f; // largest sum of a step before the maximum is raised

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int SOFT = 2;                     // softmax warpgroups: one per half
  static constexpr int THREADS = 128 * (SOFT + 1);
  static constexpr int GROUPS = D / 64;              // 64-element column groups of an operand row
  static constexpr int GROUP_BYTES = 128 * 128;      // 128 rows of 128 bytes
  static constexpr int TILE = GROUPS * GROUP_BYTES;  // a 128-row operand
  // score buffers (in turn for all halves and tiles), what tensor memory holds beside the
  // accumulators; stages of K and of V
  static constexpr int NB = (512 - 2 * D) / 128, ST = D == 128 ? 2 : 4;
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * TILE;
  static constexpr int V = K + ST * TILE;
  static constexpr int ORDER = V + ST * TILE;  // the sequences by falling length
  static constexpr int CTRL = ORDER + 128 * 20;
  static constexpr int SMEM = CTRL + 1024 + 1024;
  static constexpr uint32_t S(int b) { return b * 128; }
  static constexpr uint32_t O(int w) { return NB * 128 + w * D; }
  static constexpr uint32_t TMEM = 512;
  // registers per thread: together no more than the 168 each that the block is launched with
  static constexpr int R_SOFTMAX = 184, R_REST = 136;
  static_assert(SOFT * R_SOFTMAX + R_REST <= (SOFT + 1) * 168, "registers");
};

// An item of work, and where it stands in the CTA's sequences of products, tiles and halves.
struct Item {
  int q0, tok0, tok1, h;  // first packed token of the sequence, the item's positions, kv-head (-1: no more items)
  int kept, skip, tiles;  // key tiles: `kept` leading ones, then those from `skip` tiles later on
  int of0, of1;           // key tiles of each half (0: none)
  int n0;                 // score products before it
  int t0;                 // key tiles before it
  int c0, c1, o0, o1;     // key tiles and items of each half before it
  int bad_lo, bad_hi;     // its key tiles with values that are not finite
  __device__ __forceinline__ int of(int w) const { return w ? of1 : of0; }
};
constexpr int kItems = 4;  // items in view

// Control words in shared memory.  A wait sees a phase's parity only, so whoever waits has
// to know that the phase before it is over.  A half's warps know that of their own last
// tiles but not of what the products do meanwhile: what they wait for goes round kTurns
// barriers by the half's own count, more than the products are ever ahead or behind.
constexpr int kTurns = 4;
struct Ctrl {
  unsigned long long q_full, q_empty, k_full[4], k_empty[4], v_full[4], v_empty[4], v_ok[4], p_half[3], p_full[3],
      s_full[2][kTurns], half_done[2][kTurns], pv_done[2][kTurns], o_full[2][kTurns], item_full[kItems], item_empty[kItems], drained;
  uint32_t tmem;
  int abort;
  Item items[kItems];
};
static_assert(sizeof(Ctrl) <= 1024, "control words");

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

// The rows of sequence s: first packed token and length, cut to fit.
__device__ __forceinline__ int2 seq_rows(const PromptArgs& a, int s, bool& bad) {
  const int c0 = a.cu_seqlens[s], c1 = a.cu_seqlens[s + 1];
  const int total = static_cast<int>(a.total);
  const int q0 = clamp_int(c0, 0, total), q1 = clamp_int(c1, q0, total);
  const int q = min(q1 - q0, a.max_len);
  bad = c0 != q0 || c1 != q1 || q != q1 - q0;
  return make_int2(q0, q);
}

// The list of items.  Up to kOrdered sequences: all row tiles by falling tile number, so by
// falling number of keys (without a window).  With the sequences by falling count of tiles
// t_0 >= t_1 >= .., the tiles numbered t_(i+1) .. t_i - 1 are those of the first i + 1
// sequences, and ends[i] = sum_(k <= i) t_k - (i + 1) t_(i+1) tiles come up to there.
// More sequences: in their order, found by walking along them.
constexpr int kOrdered = 128;
struct Sequence {
  int tiles, q0, len;
};
template <class C>
struct List {
  Sequence* by_len;
  int* ends;
  int base, before;  // the walk: sequences base .. base + 31, tiles before them

  __device__ __forceinline__ explicit List(uint8_t* smem)
      : by_len(reinterpret_cast<Sequence*>(smem + C::ORDER)), ends(reinterpret_cast<int*>(by_len + kOrdered)), base(0), before(0) {}

  // By the whole block, once; raises what is wrong with the offsets (CTA 0).
  __device__ void make(const PromptArgs& a, int2* scratch) {
    unsigned err = 0;
    const int tid = threadIdx.x, n = a.num_seqs;
    if (n <= kOrdered) {
      int2 r = make_int2(0, 0);
      bool bad = false;
      if (tid < n) {
        r = seq_rows(a, tid, bad);
        scratch[tid] = r;
      }
      if (bad) err = 256u;  // KVQ_DEVERR_TOKENS
      __syncthreads();
      if (tid < n) {
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += scratch[j].y > r.y || (scratch[j].y == r.y && j < tid);
        by_len[rank] = {(r.y + a.tokens_per_tile - 1) / a.tokens_per_tile, r.x, r.y};
      }
      __syncthreads();
      if (tid < n) {
        int sum = 0;
#pragma unroll 4
        for (int j = 0; j <= tid; ++j) sum += by_len[j].tiles;
        ends[tid] = sum - (tid + 1) * (tid + 1 < n ? by_len[tid + 1].tiles : 0);
      }
    } else if (blockIdx.x == 0) {
      for (int s = tid; s < n; s += blockDim.x) {
        bool bad;
        seq_rows(a, s, bad);
        if (bad) err = 256u;
      }
    }
    if (err && blockIdx.x == 0) raise_error(err);
  }

  // Row tile number x by a warp: its sequence and tile; false behind the last.  With more
  // than kOrdered sequences x must not fall from call to call.
  __device__ __forceinline__ bool find(const PromptArgs& a, int x, int lane, Sequence& s, int& tile) {
    if (a.num_seqs <= kOrdered) {
      for (int i0 = 0; i0 < a.num_seqs; i0 += 32) {
        const int i = i0 + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, i < a.num_seqs && x < ends[i]);
        if (hit == 0) continue;
        const int k = i0 + __ffs(hit) - 1;
        const int y = x - (k > 0 ? ends[k - 1] : 0);
        tile = by_len[k].tiles - 1 - y / (k + 1);
        s = by_len[y % (k + 1)];
        return true;
      }
      return false;
    }
    for (; base < a.num_seqs; base += 32) {
      bool bad;
      const int2 r = base + lane < a.num_seqs ? seq_rows(a, base + lane, bad) : make_int2(0, 0);
      const int v = (r.y + a.tokens_per_tile - 1) / a.tokens_per_tile;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x < before + incl);
      if (hit != 0) {
        const int k = __ffs(hit) - 1;
        s = {__shfl_sync(0xffffffffu, v, k), __shfl_sync(0xffffffffu, r.x, k), __shfl_sync(0xffffffffu, r.y, k)};
        tile = before + __shfl_sync(0xffffffffu, incl, k) - 1 - x;
        return true;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
};

// The key tiles that rows at positions p_lo..p_hi see.
__device__ __forceinline__ void key_span(const PromptArgs& a, int p_lo, int p_hi, Item& x) {
  x.kept = x.skip = 0;
  x.tiles = p_hi / kKeys + 1;
  if (a.window > 0) {
    const int win = max(p_lo - a.window + 1, 0);
    x.kept = (min(a.sinks, win) + kKeys - 1) / kKeys;
    x.skip = max(win / kKeys - x.kept, 0);
    x.tiles -= x.skip;
  }
}
__device__ __forceinline__ int tile_key(const Item& s, int i) { return kKeys * (i < s.kept ? i : i + s.skip); }
// Positions of half w, `half` tokens each.
__device__ __forceinline__ int first_of(const Item& x, int w, int half) { return x.tok0 + w * half; }
__device__ __forceinline__ int last_of(const Item& x, int w, int half) { return min(x.tok0 + (w + 1) * half, x.tok1) - 1; }
// Every row of the half sees every key of the tile at t0.
__device__ __forceinline__ bool sees_all(const PromptArgs& a, const Item& x, int w, int half, int t0) {
  return t0 + kKeys - 1 <= first_of(x, w, half) &&
         (a.window == 0 || t0 > last_of(x, w, half) - a.window || t0 + kKeys <= a.sinks);
}
// The number of the score product of half w and tile i within the item: tile by tile, the
// halves that have it in order.
__device__ __forceinline__ int product(const Item& x, int w, int i) {
  const int both = min(x.of0, x.of1);
  return i < both ? 2 * i + w : both + i;
}

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  return (finite_bf16(w) ? w & 0xFFFFu : 0u) | (finite_bf16(w >> 16) ? w & 0xFFFF0000u : 0u);
}
// Bit 15 (31) set where the lower (upper) of two bf16 values is not finite: one more in an
// exponent of all ones carries into the sign's place.
__device__ __forceinline__ uint32_t not_finite_bits(uint32_t w) { return (w & 0x7FFF7FFFu) + 0x00800080u; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Which of the 64 columns from c0 on a row sees: those <= last that are >= first or < kept.
__device__ __forceinline__ uint64_t columns_below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; }
__device__ __forceinline__ uint64_t seen_columns(int c0, int last, int first, int kept) {
  return columns_below(last + 1 - c0) & (~columns_below(first - c0) | columns_below(kept - c0));
}
// The largest logit: score times scale, which may be negative.
__device__ __forceinline__ float top_logit(const uint32_t (&s)[kStep], float scale) {
  const uint32_t turn = scale < 0.f ? 0x80000000u : 0u;
  float x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = -INFINITY;
#pragma unroll
  for (int e = 0; e < kStep; e += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = max3f(x[k], __uint_as_float(s[e + 2 * k] ^ turn), __uint_as_float(s[e + 2 * k + 1] ^ turn));
  return fmaxf(max3f(x[0], x[1], x[2]), x[3]) * fabsf(scale);
}

// Every row of the item sees every key of the tile at t0, so that its values are as they were.
__device__ __forceinline__ bool untouched(const PromptArgs& a, const Item& x, int half, int t0) {
  return sees_all(a, x, 0, half, t0) && (x.of1 == 0 || sees_all(a, x, 1, half, t0));
}
// Of two bf16 values, those that are +inf or NaN (bits 15 and 31 of up), and -inf or NaN (of down).
__device__ __forceinline__ void add_not_finite(uint32_t w, uint32_t& up, uint32_t& down) {
  const uint32_t bad = not_finite_bits(w) & 0x80008000u, nan = ((w & 0x007F007Fu) + 0x007F007Fu) << 8;
  up |= bad & (nan | ~w);
  down |= bad & (nan | w);
}
// Values that are not finite among those 32 from `value` on (of the sequence's first token)
// that the row at position p sees in the key tiles i_lo..i_hi that were touched.  Only called
// when the checking warps met one; by a whole warp, whose rows have the same keys (each 64
// bytes of it one address), until all of its rows have met a NaN or both infinities everywhere.
// 2 prompts of 9,000, 16 / 4 heads of 128, window 8,192: 0.53 ms; one of them all NaN 0.57, all
// +inf 1.83.
__device__ __noinline__ void find_not_finite(const PromptArgs& a, const Item* x, const uint16_t* value, bool mine, int p, int i_lo,
                                             int i_hi, uint32_t (&up_out)[16], uint32_t (&down_out)[16]) {
  const int half_tokens = 128 / a.gqa;
  uint32_t up[16], down[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) up[e] = down[e] = mine ? 0u : 0x80008000u;
  bool full = false;
  for (int i = i_lo; i <= i_hi && !full; ++i) {
    const int t0 = tile_key(*x, i);
    if (untouched(a, *x, half_tokens, t0)) continue;
    const int t1 = min(t0 + kKeys, x->tok1);
#pragma unroll 2
    for (int t = t0; t < t1 && !full; ++t) {
      const bool seen = mine && t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
      if (!__any_sync(0xffffffffu, seen)) continue;
      const uint4* const row = reinterpret_cast<const uint4*>(value + t * a.value_stride);
      uint32_t w[16], bad = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 y = __ldg(row + k);
        w[4 * k] = y.x;
        w[4 * k + 1] = y.y;
        w[4 * k + 2] = y.z;
        w[4 * k + 3] = y.w;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) bad |= not_finite_bits(w[e]);
      if ((bad & 0x80008000u) == 0) continue;  // the same in every lane
      uint32_t all = 0x80008000u;
      if (seen) {
#pragma unroll
        for (int e = 0; e < 16; ++e) add_not_finite(w[e], up[e], down[e]);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) all &= up[e] & down[e];
      full = __all_sync(0xffffffffu, all == 0x80008000u);
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    up_out[e] = up[e];
    down_out[e] = down[e];
  }
}

// 2^x, and two values as bf16, in the order in which they are written down.
__device__ __forceinline__ float ordered_exp2(float x) {
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ uint32_t ordered_pack_bf162(float lo, float hi) {
  uint32_t r;
  asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 bf16 values, 16-byte aligned; by whole sectors where 32-byte aligned (a warp's store
// touches 32 rows, a cycle each: half as many stores hold the SM up half as long).
__device__ __forceinline__ void store64(uint16_t* to, const uint32_t (&w)[16], bool sectors) {
  if (sectors) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 16 * k), "r"(w[8 * k]), "r"(w[8 * k + 1]),
                   "r"(w[8 * k + 2]), "r"(w[8 * k + 3]), "r"(w[8 * k + 4]), "r"(w[8 * k + 5]), "r"(w[8 * k + 6]), "r"(w[8 * k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(to)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}
// 32 columns of a row's accumulators times mul, as bf16.
__device__ __forceinline__ void scale_result(uint32_t (&w)[16], const uint32_t* o, float mul) {
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = pack_bf162(__uint_as_float(o[2 * e]) * mul, __uint_as_float(o[2 * e + 1]) * mul);
}
// A row's result where values that are not finite were met: what they make of theirs.
template <int D>
__device__ __noinline__ void store_not_finite(const PromptArgs& a, const volatile Item* live, uint32_t o_addr, float mul, bool mine,
                                              int pos, uint16_t* to) {
  Item x;
  x.tok0 = live->tok0;
  x.tok1 = live->tok1;
  x.kept = live->kept;
  x.skip = live->skip;
  x.of1 = live->of1;
  const int bad_lo = live->bad_lo, bad_hi = live->bad_hi;
  const uint16_t* const value = a.value + static_cast<int64_t>(live->q0) * a.value_stride + static_cast<int64_t>(live->h) * D;
#pragma unroll 1
  for (int k = 0; k < D / 32; ++k) {
    uint32_t o[32], w[16], up[16], down[16];
    find_not_finite(a, &x, value + 32 * k, mine, pos, bad_lo, bad_hi, up, down);
    __syncwarp();
    tmem_ld32(o, o_addr + 32 * k);
    tmem_wait_ld32(o);
    scale_result(w, o, mul);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      add_not_finite(w[e], up[e], down[e]);  // with what came from the tiles left as they were
      const uint32_t met = ((up[e] | down[e]) >> 15 & 0x00010001u) * 0xFFFFu;
      w[e] = (w[e] & ~met) | ((0x7F807F80u | (down[e] & ~up[e]) | (up[e] & down[e]) >> 9) & met);
    }
    if (mine) store64(to + 32 * k, w, false);
  }
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
    prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // swizzled tiles: 1024-byte aligned
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + C::CTRL);
  volatile int* abort = &ctrl->abort;
  const int spin = a.spin_limit;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7;
  constexpr int kIssuer = 4 * C::SOFT;
  const int G = a.gqa, half_tokens = 128 / G;
  auto bar = [&](const void* p) { return base + static_cast<uint32_t>(static_cast<const uint8_t*>(p) - smem); };

  List<C> list(smem);
  list.make(a, reinterpret_cast<int2*>(smem));  // the stages are not in use yet
  if (tid == 0) {
    mbar_init(bar(&ctrl->q_full), 1);
    mbar_init(bar(&ctrl->q_empty), 1);
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(bar(&ctrl->k_full[i]), 1);
      mbar_init(bar(&ctrl->v_full[i]), 1);
      mbar_init(bar(&ctrl->k_empty[i]), 1);
      mbar_init(bar(&ctrl->v_empty[i]), 1);
      mbar_init(bar(&ctrl->v_ok[i]), 2);
    }
    for (int i = 0; i < C::NB; ++i) {
      mbar_init(bar(&ctrl->p_half[i]), 4);
      mbar_init(bar(&ctrl->p_full[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < kTurns; ++j) {
        mbar_init(bar(&ctrl->s_full[i][j]), 1);
        mbar_init(bar(&ctrl->half_done[i][j]), 1);
        mbar_init(bar(&ctrl->pv_done[i][j]), 1);
        mbar_init(bar(&ctrl->o_full[i][j]), 1);
      }
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(&ctrl->item_full[i]), 1);
      mbar_init(bar(&ctrl->item_empty[i]), 4 * C::SOFT + 4);  // a warp each
    }
    mbar_init(bar(&ctrl->drained), 1);
    ctrl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) tmem_alloc(bar(&ctrl->tmem), C::TMEM);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the list's scratch, before loads over it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;
  auto give_up = [&]() {
    raise_error(16u);  // KVQ_DEVERR_TIMEOUT: the results of this launch are invalid
    *abort = 1;
  };
  // Waits of a converged warp: all lanes go on or none does.
  auto wait = [&](const void* b, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_wait_or_abort(bar(b), parity, spin, abort))) return true;
    give_up();
    return false;
  };
  // The same of the count-th of what goes round kTurns barriers.
  auto wait_turn = [&](const unsigned long long (&b)[kTurns], int count) {
    return wait(&b[count % kTurns], (count / kTurns) & 1);
  };
  // Item k: false when there is none.
  auto get_item = [&](int k, Item& x) {
    const int slot = k % kItems;
    if (!wait(&ctrl->item_full[slot], (k / kItems) & 1)) return false;
    x = ctrl->items[slot];
    return x.h >= 0;
  };
  auto done_with = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(&ctrl->item_empty[k % kItems]));
  };

  if (wg < C::SOFT) {
    // ================= softmax: thread = row =================
    reg_take<C::R_SOFTMAX>();
    const int half = wg, row = tid & 127, row_token = row / G, row_head = row - row_token * G;
    const float scale = a.sm_scale_log2;
    const bool sectors = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride % 16 == 0;
    const uint32_t never = scale < 0.f ? 0x7F800000u : 0xFF800000u;  // times scale: -inf
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t o_addr = tmem + C::O(half) + lane_base;
    Item x;
    bool ok = true;
    for (int item = 0; ok && get_item(item, x); ++item) {
      const int tiles = x.of(half);
      const int tok = first_of(x, half, half_tokens) + row_token, last_tok = last_of(x, half, half_tokens);
      const bool mine = tiles > 0 && row < half_tokens * G && tok <= last_tok;
      const bool has_rows = __any_sync(0xffffffffu, mine);
      const int pos = mine ? tok : last_tok;
      float m = mine ? -INFINITY : 0.f, l = 0.f;  // rows that are not there take no part in what the warp decides
      for (int i = 0; ok && i < tiles; ++i) {
        const int n = x.n0 + product(x, half, i), buf = n % C::NB, c = (half ? x.c1 : x.c0) + i;
        const uint32_t s_addr = tmem + C::S(0) + buf * 128 + lane_base;
        const int t0 = tile_key(x, i);
        const bool all = sees_all(a, x, half, half_tokens, t0);
        ok = wait_turn(ctrl->s_full[half], c);
        if (!ok) break;
        if (!has_rows) {
          if (lane == 0) {
            mbar_arrive(bar(&ctrl->p_half[buf]));
            mbar_arrive(bar(&ctrl->p_full[buf]));
          }
          continue;
        }
        tc_fence_after();
        uint32_t s[kStep];
        auto load = [&](int c0) {  // scores of 64 keys, on their way
          tmem_ld32(s, s_addr + c0);
          tmem_ld32(s + 32, s_addr + c0 + 32);
        };
#pragma unroll 1
        for (int c0 = 0; c0 < kKeys; c0 += kStep) {
          // with nothing seen yet, or a step made again, the row takes a (new) maximum first
          bool seek = m == -INFINITY, again = false;
          load(c0);
          float sum;
          uint32_t p[kStep / 2];
#pragma unroll 1
          while (true) {
            tmem_wait_ld32(s);
            tmem_waited32(s + 32);
            if (!all) {
              const int last = pos - t0;
              const uint64_t seen = seen_columns(c0, last, a.window > 0 ? last - a.window + 1 : -1, a.sinks - t0);
              if (!__any_sync(0xffffffffu, seen != 0)) {  // a step that no row of the warp sees
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < kStep / 2; ++e) p[e] = 0;
                break;
              }
              if (__any_sync(0xffffffffu, ~seen != 0)) {
                const uint32_t lo = static_cast<uint32_t>(seen), hi = static_cast<uint32_t>(seen >> 32);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  s[e] = lo >> e & 1 ? s[e] : never;
                  s[e + 32] = hi >> e & 1 ? s[e + 32] : never;
                }
              }
            }
            if (__any_sync(0xffffffffu, seek)) {
              const float up = seek ? fmaxf(m, top_logit(s, scale)) : m;
              const float f = up == m ? 1.f : fast_exp2(m - up);
              m = up;
              l *= f;
              if (again && i + c0 > 0) {  // once the products so far are done
                ok = c0 > 0 ? wait_turn(ctrl->half_done[half], c) : wait_turn(ctrl->pv_done[half], c - 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                  uint32_t o[16];
                  tmem_ld16(o, o_addr + d);
                  tmem_wait_ld16(o);
#pragma unroll
                  for (int e = 0; e < 16; e += 2) {
                    float u, v;
                    mul2(u, v, __uint_as_float(o[e]), __uint_as_float(o[e + 1]), f, f);
                    o[e] = __float_as_uint(u);
                    o[e + 1] = __float_as_uint(v);
                  }
                  tmem_st16(o_addr + d, o);
                }
              }
            }
            // Probabilities as bf16 pairs (rounded to nearest: their errors do not add up in
            // one direction; the sum takes them before it), four at a time: the next four's
            // exponentials are on their way while these are added and packed.  One warp has to
            // keep its scheduler busy here, so the order matters: as the compiler lays it
            // out, a long prompt takes 3 % more.
            const float off = m == -INFINITY ? 0.f : -m;
            float part[4] = {0.f, 0.f, 0.f, 0.f}, e2[kStep];
#pragma unroll
            for (int b = 0; b <= kStep; b += 4) {
              if (b < kStep) {
#pragma unroll
                for (int e = b; e < b + 4; e += 2)
                  fma2(e2[e], e2[e + 1], __uint_as_float(s[e]), __uint_as_float(s[e + 1]), scale, scale, off, off);
#pragma unroll
                for (int e = b; e < b + 4; ++e) e2[e] = ordered_exp2(e2[e]);
              }
              if (b > 0) {
#pragma unroll
                for (int e = b - 4; e < b; e += 2) {
                  add2(part[e & 2], part[(e & 2) + 1], part[e & 2], part[(e & 2) + 1], e2[e], e2[e + 1]);
                  p[e / 2] = ordered_pack_bf162(e2[e], e2[e + 1]);
                }
              }
            }
            sum = (part[0] + part[1]) + (part[2] + part[3]);
            if (again) break;
            seek = mine && !(sum <= kMost);
            if (!__any_sync(0xffffffffu, seek)) break;
            again = true;
            load(c0);
          }
          if (!ok) break;
          l += sum;
          tmem_st32(s_addr + c0 / 2, p);  // over scores that have been read
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(c0 == 0 ? &ctrl->p_half[buf] : &ctrl->p_full[buf]));
        }
      }
      // ---- the row's result
      if (ok && has_rows && (ok = wait_turn(ctrl->o_full[half], half ? x.o1 : x.o0))) {
        tc_fence_after();
        const float mul = 1.f / l;
        const volatile Item* live = &ctrl->items[item % kItems];
        uint16_t* const to = a.out + (static_cast<int64_t>(x.q0) + tok) * a.out_stride + (static_cast<int64_t>(x.h) * G + row_head) * D;
        if (live->bad_hi >= 0) {
          store_not_finite<D>(a, live, o_addr, mul, mine, pos, to);
        } else {
#pragma unroll 1
          for (int k = 0; k < D; k += 64) {
            uint32_t o[64], w[16];
            tmem_ld32(o, o_addr + k);
            tmem_ld32(o + 32, o_addr + k + 32);
            tmem_wait_ld32(o);
            tmem_waited32(o + 32);
            scale_result(w, o, mul);
            if (mine) store64(to + k, w, sectors);
            scale_result(w, o + 32, mul);
            if (mine) store64(to + k + 32, w, sectors);
          }
        }
      }
      done_with(item);
    }
  } else {
    reg_give<C::R_REST>();
    if (warp == kIssuer + 1) {
      // ================= loads =================
      Item x;
      int last_k = 0, last_items = 0;  // key tiles and items whose loads were issued
      bool ok = true, v_too = true;
      for (int item = 0; ok && get_item(item, x); ++item) {
        const int halves = x.of1 > 0 ? 2 : 1;
        if (item > 0) ok = wait(&ctrl->q_empty, (item - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect(bar(&ctrl->q_full), halves * C::GROUPS * half_tokens * G * 128);
          for (int w = 0; w < halves; ++w)
#pragma unroll
            for (int g = 0; g < C::GROUPS; ++g)
              tma_load_3d(base + C::Q + w * C::TILE + g * C::GROUP_BYTES, &map_q, 64 * g, x.h * G,
                          x.q0 + first_of(x, w, half_tokens), bar(&ctrl->q_full));
        }
        last_items = item + 1;
        for (int i = 0; ok && i < x.tiles; ++i) {
          const int t = x.t0 + i, st = t % C::ST, y = x.q0 + tile_key(x, i);
          const uint32_t parity = (t / C::ST + 1) & 1;
          auto load = [&](const CUtensorMap* map, const void* full, int stages) {
            if (lane != 0) return;
            mbar_arrive_expect(bar(full), C::TILE);
#pragma unroll
            for (int g = 0; g < C::GROUPS; ++g)
              tma_load_3d(base + stages + st * C::TILE + g * C::GROUP_BYTES, map, 64 * g, x.h, y, bar(full));
          };
          if (t >= C::ST) ok = wait(&ctrl->k_empty[st], parity);
          if (!ok) break;
          load(&map_k, &ctrl->k_full[st], C::K);
          last_k = t + 1;
          v_too = false;
          if (t >= C::ST) ok = wait(&ctrl->v_empty[st], parity);
          if (!ok) break;
          load(&map_v, &ctrl->v_full[st], C::V);
          v_too = true;
        }
        done_with(item);
      }
      // Leave with no copy in flight, whoever gave up: the last queries and the last of each stage are there.
      if (last_items > 0) mbar_wait(bar(&ctrl->q_full), (last_items - 1) & 1, kDrain);
      for (int t = max(last_k - C::ST, 0); t < last_k; ++t) {
        mbar_wait(bar(&ctrl->k_full[t % C::ST]), (t / C::ST) & 1, kDrain);
        if (v_too || t + 1 < last_k) mbar_wait(bar(&ctrl->v_full[t % C::ST]), (t / C::ST) & 1, kDrain);
      }
      __syncwarp();
    } else if (warp == kIssuer) {
      // ================= products =================
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t leader = elect_lane();
      const uint32_t qk_desc = mma_desc(128, kKeys, true, false), pv_desc = mma_desc(128, D, true, true);
      const uint64_t q_op = smem_desc(base + C::Q, 16), k_op = smem_desc(base + C::K, 16);
      const uint64_t v_op = smem_desc(base + C::V, C::GROUP_BYTES);
      // test hook: in place of this K tile (-1: none) the products wait for what nothing signals
      const int withheld = static_cast<int>(blockIdx.x) == a.withhold_cta ? a.withhold_tile : -1;
      // Score products run ahead of value products by the score buffers; products run in the
      // order of their issue, so one that overwrites probabilities only needs to be issued
      // behind those that read them.
      struct Cursor {
        int item, i, w;                               // item, tile and half
        int tiles, of0, of1, t0, c0, c1, o0, o1;      // as in Item
      };
      auto step = [&](Cursor& u) {  // on to the next (tile, half) of the item; false behind its last
        if (u.w == 0 && u.i < u.of1) {
          u.w = 1;
          return true;
        }
        ++u.i;
        u.w = u.i < u.of0 ? 0 : 1;
        return u.i < u.tiles;
      };
      auto open = [&](Cursor& u, int item) {  // an item's first (half 0 has a tile); false behind the last item
        Item x;
        const bool any = get_item(item, x);
        auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };  // in every lane, and known as such
        u = {same(item), 0, 0, same(x.tiles), same(x.of0), same(x.of1), same(x.t0), same(x.c0), same(x.c1), same(x.o0), same(x.o1)};
        return any;
      };
      Cursor sc, pv;
      bool more_s = open(sc, 0), more_v = more_s, ok = true;
      pv = sc;
      int ns = 0, nv = 0;  // products of each kind issued
      // The tensor cores take some four products ahead, 256 cycles' worth, and stall the issuing
      // warp behind that: between the last of one group and the first of the next, everything
      // has to be done in that time.  So barriers are looked at together, in one loop.  A look
      // takes no time of its own, so those are not counted: what takes longer is waited for,
      // `spin` times, by waits that sleep, as everywhere else.
      auto look = [](uint32_t b, uint32_t parity) { return mbar_test(b, parity); };
      auto sleep = [](uint32_t b, uint32_t parity) { return mbar_try_wait(b, parity); };
      auto poll = [&](auto ready) {  // until all that ready(look) looks at is there
        for (int n = 0; n < kQuick; ++n) {
          if (__all_sync(0xffffffffu, ready(look))) return true;
          if ((n & 15) == 15 && __any_sync(0xffffffffu, *abort)) break;
        }
        for (int n = 0; n < spin; ++n) {
          if (__all_sync(0xffffffffu, ready(sleep))) return true;
          if (__any_sync(0xffffffffu, *abort)) break;
        }
        give_up();
        return false;
      };
      bool s_ready = false;  // the next score product's operands are there
      auto scores_ready = [&](auto test) {
        const int t = sc.t0 + sc.i;
        return test(bar(&ctrl->q_full), sc.item & 1) & test(bar(&ctrl->k_full[t % C::ST]), (t / C::ST) & 1);
      };
      auto scores = [&]() {  // the next score product
        const int t = sc.t0 + sc.i, st = t % C::ST, w = sc.w, buf = ns % C::NB;
        const uint64_t qa = q_op + w * (C::TILE >> 4), ka = k_op + st * (C::TILE >> 4);
        if (t == withheld) {
          ok = wait(&ctrl->drained, 0);
          return;
        }
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int at = ((k >> 2) * C::GROUP_BYTES + (k & 3) * 32) >> 4;
          mma_ss(leader, tm + C::S(0) + buf * 128, qa + at, ka + at, qk_desc, k > 0);
        }
        tc_commit(leader, bar(&ctrl->s_full[w][((w ? sc.c1 : sc.c0) + sc.i) % kTurns]));
        ++ns;
        s_ready = false;
        const int i = sc.i;
        const bool more = step(sc);
        if (!more || sc.i != i) tc_commit(leader, bar(&ctrl->k_empty[st]));
        if (!more) {
          tc_commit(leader, bar(&ctrl->q_empty));
          more_s = open(sc, sc.item + 1);
          if (!more_s && *abort) ok = false;
        }
      };
      while (ok && more_v) {
        while (ok && more_s && ns < nv + C::NB) {
          // where there are no scores to go on with, the next ones' operands are waited for
          if (!s_ready && ns == nv) ok = poll(scores_ready);
          else if (!s_ready && !__all_sync(0xffffffffu, scores_ready(look))) break;
          if (ok) scores();
        }
        if (!ok) break;
        const int t = pv.t0 + pv.i, st = t % C::ST, buf = nv % C::NB, w = pv.w, turn = ((w ? pv.c1 : pv.c0) + pv.i) % kTurns;
        const uint64_t va = v_op + st * (C::TILE >> 4);
        auto values = [&](int k0) {  // O_w += P V, keys 16 k0 .. 16 k0 + 63
#pragma unroll
          for (int k = k0; k < k0 + kStep / 16; ++k)
            mma_ts(leader, tm + C::O(0) + w * D, tm + C::S(0) + buf * 128 + 8 * k, va + k * (2048 >> 4), pv_desc, pv.i > 0 || k > 0);
        };
        const uint32_t p_parity = (nv / C::NB) & 1, v_parity = (t / C::ST) & 1;
        const uint32_t p_half = bar(&ctrl->p_half[buf]), p_full = bar(&ctrl->p_full[buf]), v_full = bar(&ctrl->v_full[st]),
                       v_ok = bar(&ctrl->v_ok[st]);
        ok = poll([&](auto test) { return test(p_half, p_parity) & test(v_full, v_parity) & test(v_ok, v_parity); });
        if (!ok) break;
        tc_fence_after();
        values(0);
        tc_commit(leader, bar(&ctrl->half_done[w][turn]));
        const bool last = pv.i + 1 == (w ? pv.of1 : pv.of0);
        ok = poll([&](auto test) {
          s_ready = more_s && scores_ready(look);
          return test(p_full, p_parity);
        });
        if (!ok) break;
        s_ready = __all_sync(0xffffffffu, s_ready);
        tc_fence_after();
        values(kStep / 16);
        tc_commit(leader, bar(&ctrl->pv_done[w][turn]));
        if (last) tc_commit(leader, bar(&ctrl->o_full[w][(w ? pv.o1 : pv.o0) % kTurns]));
        ++nv;
        const int i = pv.i;
        const bool more = step(pv);
        if (!more || pv.i != i) tc_commit(leader, bar(&ctrl->v_empty[st]));
        if (!more) {
          done_with(pv.item);
          more_v = open(pv, pv.item + 1);
        }
      }
      // Leave with no product in flight, whoever gave up.
      tc_commit(leader, bar(&ctrl->drained));
      mbar_wait(bar(&ctrl->drained), 0, kDrain);
      __syncwarp();
    } else {
      // ================= the list, and values of tiles that a row sees only in part =================
      const int w = warp - kIssuer - 2;
      const bool lists = w == 1;
      int n0 = 0, t0 = 0, c0 = 0, c1 = 0, o0 = 0, o1 = 0;
      bool ended = false;
      auto publish = [&](int k) {  // item k; false if a wait ran out
        const int slot = k % kItems;
        if (k >= kItems && !wait(&ctrl->item_empty[slot], (k / kItems - 1) & 1)) return false;
        // dealt to and fro; walked along many sequences, straight on
        const int g = gridDim.x, at = (k & 1) && a.num_seqs <= kOrdered ? g - 1 - blockIdx.x : blockIdx.x;
        const int64_t u = static_cast<int64_t>(k) * g + at;
        Sequence s;
        int tile = 0;
        Item x;
        x.h = -1;
        if (u < static_cast<int64_t>(a.tiles) * a.num_kv_heads && list.find(a, static_cast<int>(u / a.num_kv_heads), lane, s, tile)) {
          x.h = static_cast<int>(u % a.num_kv_heads);
          x.q0 = s.q0;
          x.tok0 = tile * a.tokens_per_tile;
          x.tok1 = min(x.tok0 + a.tokens_per_tile, s.len);
          key_span(a, x.tok0, x.tok1 - 1, x);
          x.of0 = last_of(x, 0, half_tokens) / kKeys + 1 - x.skip;  // the first half may end before the second
          x.of1 = x.tok1 - x.tok0 > half_tokens ? x.tiles : 0;
          x.n0 = n0;
          x.t0 = t0;
          n0 += x.of0 + x.of1;
          t0 += x.tiles;
          x.c0 = c0;
          x.c1 = c1;
          x.o0 = o0;
          x.o1 = o1;
          c0 += x.of0;
          c1 += x.of1;
          ++o0;
          o1 += x.of1 > 0;
          x.bad_lo = 0x7fffffff;
          x.bad_hi = -1;
        }
        ended = x.h < 0;
        if (lane == 0) {
          ctrl->items[slot] = x;
          mbar_arrive(bar(&ctrl->item_full[slot]));
        }
        __syncwarp();
        return true;
      };
      bool ok = !lists || (publish(0) && (ended || publish(1)));
      Item x;
      for (int item = 0; ok; ++item) {
        if (lists && !ended) ok = publish(item + 2);
        if (!ok || !get_item(item, x)) break;
        for (int i = 0; i < x.tiles; ++i) {
          const int t = x.t0 + i, st = t % C::ST, key = tile_key(x, i);
          ok = wait(&ctrl->v_full[st], (t / C::ST) & 1);
          if (!ok) break;
          if (!untouched(a, x, half_tokens, key)) {
            uint4* const v = reinterpret_cast<uint4*>(smem + C::V + st * C::TILE) + 32 * w + lane;
            uint32_t bad = 0;
#pragma unroll 8
            for (int k = 0; k < C::TILE / 16; k += 64) {
              const uint4 y = v[k];
              bad |= not_finite_bits(y.x) | not_finite_bits(y.y) | not_finite_bits(y.z) | not_finite_bits(y.w);
            }
            bad &= 0x80008000u;
            if (bad) {
#pragma unroll 1
              for (int k = 0; k < C::TILE / 16; k += 64) {
                const uint4 y = v[k];
                v[k] = make_uint4(finite_or_zero(y.x), finite_or_zero(y.y), finite_or_zero(y.z), finite_or_zero(y.w));
              }
              atomicMin(&ctrl->items[item % kItems].bad_lo, i);
              atomicMax(&ctrl->items[item % kItems].bad_hi, i);
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&ctrl->v_ok[st]));
        }
        if (!ok) break;
        done_with(item);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, C::TMEM);
}

// Rows [tokens, heads, D] of 16 bits, tokens `stride` elements apart, boxes of 64 columns.
bool encode_rows(CUtensorMap* m, const uint16_t* p, int d, int heads, int64_t tokens, int64_t stride, int box_heads,
                 int box_tokens) {
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)}, estr[3] = {1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(p), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_t(const PromptArgs& a, cudaStream_t st, int num_sms) {
  using C = Cfg<D>;
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  CUtensorMap q, k, v;
  if (tensor_map_encoder() == nullptr ||
      !encode_rows(&q, a.query, D, a.num_q_heads, a.total, a.query_stride, a.gqa, 128 / a.gqa) ||
      !encode_rows(&k, a.key, D, a.num_kv_heads, a.total, a.key_stride, 1, kKeys) ||
      !encode_rows(&v, a.value, D, a.num_kv_heads, a.total, a.value_stride, 1, kKeys))
    return cudaErrorInvalidValue;
  const int64_t items = static_cast<int64_t>(a.tiles) * a.num_kv_heads;
  prompt_kernel<D><<<static_cast<unsigned>(std::min<int64_t>(items, num_sms)), C::THREADS, C::SMEM, st>>>(a, q, k, v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& args, int head_dim, cudaStream_t st, int num_sms) {
  PromptArgs a = args;
  // with scale 0 every logit is 0: as good as 0, and a masked score times it is still -inf
  if (a.sm_scale_log2 == 0.f) a.sm_scale_log2 = 1.17549435e-38f;
  // two halves a tile, or one where tiles of two would leave half of the SMs idle
  const int64_t half = 128 / a.gqa;
  auto tiles_of = [&](int64_t tokens) {
    return std::min(a.num_seqs * ((a.max_len + tokens - 1) / tokens), a.total / tokens + a.num_seqs);
  };
  a.tokens_per_tile = static_cast<int>(2 * tiles_of(2 * half) * a.num_kv_heads <= num_sms ? half : 2 * half);
  const int64_t tiles = tiles_of(a.tokens_per_tile);
  if (tiles > INT32_MAX) return cudaErrorNotSupported;
  a.tiles = static_cast<int>(tiles);
  if (head_dim == 64) return launch_t<64>(a, st, num_sms);
  if (head_dim == 128) return launch_t<128>(a, st, num_sms);
  return cudaErrorNotSupported;
}

}  // namespace kvq

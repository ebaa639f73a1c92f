// Attention of whole prompts whose queries, keys and values are at hand in 16 bits
// (kvq_prompt_attention): packed sequences, causal, heads in groups.
//
// out = sum_t p_t v_t / sum_t p_t, p_t = 2^(z_t - m), z_t = sm_scale log2(e) <q, k_t>,
// with a running maximum m over tiles of 128 keys and float32 sums: one pass over
// the keys, no score leaves the SM.
//
// Split: a CTA owns two halves of up to 128 rows (token, query head) of one sequence
// and kv-head; row R of a half is query head R % G of its token R / G, so the G heads
// that share keys fill a half together.  Per 128 keys and half it runs two
// tcgen05 products, S = Q K^T (operands in shared memory) and O += P V (P in tensor
// memory, over S's own columns); one half's products run while the other half's
// softmax does.  Q, K and V come by TMA from the caller's own rows, whatever their stride.
//
// Warps: two warpgroups per half for the softmax, each thread half of a row's 64 + 64
// scores (all in registers; the two threads of a row agree on a new maximum through a
// barrier of their two warps, which also tells both that none is needed), one warp that issues
// the products, one that loads, two that look at the values of tiles that some row sees
// only in part: a probability of 0 times a value that is not finite would not be 0.
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
constexpr int kDrain = 1 << 18;  // polls for what is in flight at a CTA's end (some seconds)
constexpr float kLazy = 8.0f;    // a maximum that grows by less (log2) is not raised: p <= 2^8

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int SOFT = 4;                     // softmax warpgroups: two per half
  static constexpr int THREADS = 128 * (SOFT + 1);
  static constexpr int GROUPS = D / 64;              // 64-element column groups of an operand row
  static constexpr int GROUP_BYTES = 128 * 128;      // 128 rows of 128 bytes
  static constexpr int TILE = GROUPS * GROUP_BYTES;  // a 128-row operand
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * TILE;
  static constexpr int V = K + 2 * TILE;
  static constexpr int SWAP = V + 2 * TILE;  // [half][column half][row] floats, twice (maxima, sums)
  static constexpr int CTRL = SWAP + 2 * 2 * 2 * 128 * 4;
  static constexpr int SMEM = CTRL + 512 + 1024;
  static constexpr uint32_t S(int w) { return w * 128; }
  static constexpr uint32_t O(int w) { return 256 + w * 128; }
  static constexpr uint32_t TMEM = 512;
  // registers per thread: together no more than the 96 each that the block is launched with
  static constexpr int R_SOFTMAX = 104, R_REST = 64;
  static_assert(SOFT * R_SOFTMAX + R_REST <= (SOFT + 1) * 96, "registers");
};

// Control words in shared memory.
struct Ctrl {
  unsigned long long q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], v_ok[2], s_full[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  int abort;
  int failed[8];              // per pair of softmax warps
  int seq, tile, q0, len;     // this CTA's rows
  int bad_lo, bad_hi;         // key tiles with values that are not finite
  int scan[32];
};
static_assert(sizeof(Ctrl) <= 512, "control words");

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

// The sequence and tile that tile number `want` of all sequences is, found by the whole
// block.  Up to kOrdered sequences count by rising length (the launch starts from the
// last tile, so the longest come first), more in their order.
constexpr int kOrdered = 128;
__device__ void find_tile(const PromptArgs& a, Ctrl* c, int2* lens, int want) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  if (tid == 0) c->seq = -1;
  int before = 0;  // tiles of the sequences before the chunk
  unsigned err = 0;
  for (int base = 0; base < a.num_seqs; base += blockDim.x) {
    const int s = base + tid;
    int2 r = make_int2(0, 0);
    int v = 0;
    if (s < a.num_seqs) {
      bool bad;
      r = seq_rows(a, s, bad);
      if (bad) err |= 256u;  // KVQ_DEVERR_TOKENS
      v = (r.y + a.tokens_per_tile - 1) / a.tokens_per_tile;
    }
    int first = before, total = 0;
    if (a.num_seqs <= kOrdered) {
      if (s < a.num_seqs) lens[s] = make_int2(r.y, v);
      __syncthreads();
      if (s < a.num_seqs) {
#pragma unroll 8
        for (int j = 0; j < a.num_seqs; ++j) {
          const int2 t = lens[j];
          if (t.x < r.y || (t.x == r.y && j < s)) first += t.y;
        }
      }
    } else {
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) c->scan[warp] = incl;
      __syncthreads();
      for (int w = 0; w < warps; ++w) {
        if (w < warp) first += c->scan[w];
        total += c->scan[w];
      }
      first += incl - v;
    }
    if (first <= want && want < first + v) {
      c->seq = s;
      c->tile = want - first;
      c->q0 = r.x;
      c->len = r.y;
    }
    before += total;
    __syncthreads();
    if (before > want && blockIdx.x != 0) break;  // block 0 checks every sequence
  }
  if (err && blockIdx.x == 0) raise_error(err);
}

// The key tiles that rows at positions p_lo..p_hi see: `kept` leading ones, then those from
// `skip` tiles later on.
struct Span {
  int kept, skip, tiles;
};
__device__ __forceinline__ Span key_span(const PromptArgs& a, int p_lo, int p_hi) {
  Span s{0, 0, p_hi / kKeys + 1};
  if (a.window > 0) {
    const int win = max(p_lo - a.window + 1, 0);
    s.kept = (min(a.sinks, win) + kKeys - 1) / kKeys;
    s.skip = max(win / kKeys - s.kept, 0);
    s.tiles -= s.skip;
  }
  return s;
}
__device__ __forceinline__ int tile_key(const Span& s, int i) { return kKeys * (i < s.kept ? i : i + s.skip); }

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  return (finite_bf16(w) ? w & 0xFFFFu : 0u) | (finite_bf16(w >> 16) ? w & 0xFFFF0000u : 0u);
}
// Whether one of two bf16 values is not finite: their exponents all ones.
__device__ __forceinline__ bool any_not_finite(uint32_t w) {
  return !finite_bf16(w) || !finite_bf16(w >> 16);
}

// Barrier of the two warps that share rows; whether one of their 64 threads came with `p`.
__device__ __forceinline__ bool pair_any(int id, bool p) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 64, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(p)), "r"(id)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Scores that the row does not see become `never`: columns c > last, and those < first that
// are not < kept.  s holds columns c0 .. c0 + 63.
__device__ __forceinline__ void mask_scores(uint32_t (&s)[64], int c0, int last, int first, int kept, uint32_t never) {
  last -= c0;
  first -= c0;
  kept -= c0;
#pragma unroll
  for (int e = 0; e < 64; ++e)
    if (e > last || (e < first && e >= kept)) s[e] = never;
}
// The score that makes the largest logit times scale, over one thread's 64.
__device__ __forceinline__ float top_logit(const uint32_t (&s)[64], float scale) {
  float x[4];
  if (scale >= 0.f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = -INFINITY;
#pragma unroll
    for (int e = 0; e < 64; e += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = max3f(x[k], __uint_as_float(s[e + 2 * k]), __uint_as_float(s[e + 2 * k + 1]));
    return fmaxf(max3f(x[0], x[1], x[2]), x[3]) * scale;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = INFINITY;
#pragma unroll
  for (int e = 0; e < 64; e += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = min3f(x[k], __uint_as_float(s[e + 2 * k]), __uint_as_float(s[e + 2 * k + 1]));
  return fminf(min3f(x[0], x[1], x[2]), x[3]) * scale;
}

// Values that are not finite among those that the row at position p sees in key tiles
// i_lo..i_hi, of dimensions d0 .. d0 + 32 W - 1: bit d of hi for +inf, of lo for -inf, of both for
// NaN.  Only called when the checking warps met one.
template <int W>
__device__ __noinline__ void find_not_finite(const PromptArgs& a, const Span& span, int q0, int h, int d, int p, int i_lo,
                                             int i_hi, int d0, uint32_t (&hi)[W], uint32_t (&lo)[W]) {
  for (int i = i_lo; i <= i_hi; ++i) {
    const int t0 = tile_key(span, i);
    for (int t = t0; t < t0 + kKeys && t <= p; ++t) {
      if (a.window > 0 && t <= p - a.window && t >= a.sinks) continue;
      const uint16_t* row = a.value + (static_cast<int64_t>(q0) + t) * a.value_stride + static_cast<int64_t>(h) * d + d0;
      for (int e = 0; e < 32 * W; ++e) {
        const uint32_t v = row[e];
        if (finite_bf16(v)) continue;
        const bool nan = (v & 0x7Fu) != 0;
        if (nan || !(v & 0x8000u)) hi[e >> 5] |= 1u << (e & 31);
        if (nan || (v & 0x8000u)) lo[e >> 5] |= 1u << (e & 31);
      }
    }
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
  const int h = blockIdx.x % a.num_kv_heads;
  const int tile_id = a.tiles - 1 - blockIdx.x / a.num_kv_heads;  // later rows see more keys: first
  auto bar = [&](const void* p) { return base + static_cast<uint32_t>(static_cast<const uint8_t*>(p) - smem); };

  find_tile(a, ctrl, reinterpret_cast<int2*>(smem + C::SWAP), tile_id);
  __syncthreads();
  if (ctrl->seq < 0) return;  // the launch has room for more tiles than the batch has
  const int len = ctrl->len, q0 = ctrl->q0, G = a.gqa;
  const int half_tokens = 128 / G;
  const int tok0 = ctrl->tile * a.tokens_per_tile, tok1 = min(tok0 + a.tokens_per_tile, len);
  const int halves = tok1 - tok0 > half_tokens ? 2 : 1;
  // positions and rows of a half
  auto first_of = [&](int w) { return tok0 + w * half_tokens; };
  auto last_of = [&](int w) { return min(tok0 + (w + 1) * half_tokens, tok1) - 1; };
  auto warps_of = [&](int w) { return w < halves ? ((last_of(w) - first_of(w) + 1) * G + 31) / 32 : 0; };
  const Span span = key_span(a, tok0, tok1 - 1);
  const int nk = span.tiles;
  // key tiles of a half: the first may end before the second
  auto tiles_of = [&](int w) { return last_of(w) / kKeys + 1 - span.skip; };
  // every row of the half sees every key of the tile at t0
  auto whole = [&](int w, int t0) {
    return t0 + kKeys - 1 <= first_of(w) && (a.window == 0 || t0 > last_of(w) - a.window || t0 + kKeys <= a.sinks);
  };

  if (tid == 0) {
    mbar_init(bar(&ctrl->q_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&ctrl->k_full[i]), 1);
      mbar_init(bar(&ctrl->v_full[i]), 1);
      mbar_init(bar(&ctrl->k_empty[i]), 1);
      mbar_init(bar(&ctrl->v_empty[i]), 1);
      mbar_init(bar(&ctrl->v_ok[i]), 2);
      mbar_init(bar(&ctrl->s_full[i]), 1);
      mbar_init(bar(&ctrl->p_full[i]), max(2 * warps_of(i), 1));
      mbar_init(bar(&ctrl->o_full[i]), 1);
    }
    mbar_init(bar(&ctrl->drained), 1);
    ctrl->abort = 0;
    for (int i = 0; i < 8; ++i) ctrl->failed[i] = 0;
    ctrl->bad_lo = 0x7fffffff;
    ctrl->bad_hi = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) tmem_alloc(bar(&ctrl->tmem), C::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;
  auto give_up = [&]() {
    raise_error(16u);  // KVQ_DEVERR_TIMEOUT: the results of this launch are invalid
    *abort = 1;
  };

  if (wg < C::SOFT) {
    // ================= softmax: two threads a row, 64 of 128 columns each =================
    reg_take<C::R_SOFTMAX>();
    const int half = wg >> 1, ch = wg & 1, row = tid & 127, quarter = warp & 3;
    if (quarter < warps_of(half)) {
      const int tok = first_of(half) + row / G;
      const bool mine = row < half_tokens * G && tok <= last_of(half);
      const int pos = mine ? tok : last_of(half);
      const float scale = a.sm_scale_log2;
      const uint32_t never = scale < 0.f ? 0x7F800000u : 0xFF800000u;  // times scale: -inf
      const int tiles = tiles_of(half), pair = half * 4 + quarter;
      const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
      const uint32_t s_addr = tmem + C::S(half) + lane_base + 64 * ch;
      const uint32_t o_addr = tmem + C::O(half) + lane_base + (D / 2) * ch;
      float* const swap = reinterpret_cast<float*>(smem + C::SWAP) + half * 256;
      float* const sums = swap + 512;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = 0; i < tiles; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(bar(&ctrl->s_full[half]), i & 1, spin, abort));
        float top = -INFINITY;
        uint32_t s[64];
        if (ok) {
          tc_fence_after();
          tmem_ld32(s, s_addr);
          tmem_ld32(s + 32, s_addr + 32);
          tmem_wait_ld32(s);
          tmem_waited32(s + 32);
          const int t0 = tile_key(span, i);
          if (!whole(half, t0)) {
            const int last = pos - t0;
            mask_scores(s, 64 * ch, last, a.window > 0 ? last - a.window + 1 : -1, a.sinks - t0, never);
          }
          top = top_logit(s, scale);
        }
        // Both warps of the pair come here every tile, also the one that gave up.
        if (pair_any(1 + pair, !ok || top > m + kLazy)) {
          swap[128 * ch + row] = top;
          if (!ok && lane == 0) {
            give_up();
            ctrl->failed[pair] = 1;
          }
          pair_any(1 + pair, false);
          if (*reinterpret_cast<volatile int*>(&ctrl->failed[pair])) {
            ok = false;
            break;
          }
          const float up = max3f(m, top, swap[128 * (1 - ch) + row]);
          const float f = up == -INFINITY ? 1.f : fast_exp2(m - up);
          m = up;
          l *= f;
          if (i > 0) {  // the products so far are done: S of this tile was issued behind them
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t o[16];
              tmem_ld16(o, o_addr + c);
              tmem_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float x, y;
                mul2(x, y, __uint_as_float(o[e]), __uint_as_float(o[e + 1]), f, f);
                o[e] = __float_as_uint(x);
                o[e + 1] = __float_as_uint(y);
              }
              tmem_st16(o_addr + c, o);
            }
          }
        }
        // probabilities over this thread's own scores, as bf16 pairs (rounded to nearest: their
        // errors do not add up in one direction; the sum takes them before it)
        const float off = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x, y;
            fma2(x, y, __uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1]), scale, scale, off, off);
            x = fast_exp2(x);
            y = fast_exp2(y);
            add2(sum[e & 2], sum[(e & 2) + 1], sum[e & 2], sum[(e & 2) + 1], x, y);
            p[e / 2] = pack_bf162(x, y);
          }
          tmem_st16(s_addr + c / 2, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&ctrl->p_full[half]));
      }
      // ---- the row's result, half of its columns
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_or_abort(bar(&ctrl->o_full[half]), 0, spin, abort));
      if (!ok && lane == 0) {
        give_up();
        ctrl->failed[pair] = 1;
      }
      sums[128 * ch + row] = l;
      pair_any(1 + pair, false);
      if (ok) {
        tc_fence_after();
        const float mul = 1.f / (l + sums[128 * (1 - ch) + row]);
        constexpr int W = D / 64;  // 32-column pieces of this thread
        uint32_t hi[W], lo[W];
#pragma unroll
        for (int k = 0; k < W; ++k) hi[k] = lo[k] = 0;
        const int bad_hi = *reinterpret_cast<volatile int*>(&ctrl->bad_hi);
        if (bad_hi >= 0 && mine)
          find_not_finite<W>(a, span, q0, h, D, pos, *reinterpret_cast<volatile int*>(&ctrl->bad_lo), bad_hi,
                             ch * (D / 2), hi, lo);
        __syncwarp();
        uint16_t* const to = a.out + (static_cast<int64_t>(q0) + tok) * a.out_stride +
                             (static_cast<int64_t>(h) * G + row % G) * D + ch * (D / 2);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          uint32_t o[32];
          tmem_ld32(o, o_addr + 32 * k);
          tmem_wait_ld32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * mul);
          if (hi[k] | lo[k]) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t up = hi[k] >> e & 1, down = lo[k] >> e & 1;
              o[e] = up && down ? 0x7FC00000u : up ? 0x7F800000u : down ? 0xFF800000u : o[e];
            }
          }
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack_bf162(__uint_as_float(o[e + 2 * j]), __uint_as_float(o[e + 2 * j + 1]));
              *reinterpret_cast<uint4*>(to + 32 * k + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  } else {
    reg_give<C::R_REST>();
    if (warp == kIssuer + 1) {
      // ================= loads =================
      if (lane == 0) {
        mbar_arrive_expect(bar(&ctrl->q_full), halves * C::GROUPS * half_tokens * G * 128);
        for (int w = 0; w < halves; ++w)
#pragma unroll
          for (int g = 0; g < C::GROUPS; ++g)
            tma_load_3d(base + C::Q + w * C::TILE + g * C::GROUP_BYTES, &map_q, 64 * g, h * G, q0 + first_of(w), bar(&ctrl->q_full));
        int issued = 0;  // K and V tiles
        bool ok = true;
        for (; ok && issued < 2 * nk; ++issued) {
          const int i = issued >> 1, st = i & 1;
          const bool is_v = issued & 1;
          if (i >= 2) ok = mbar_wait_or_abort(bar(is_v ? &ctrl->v_empty[st] : &ctrl->k_empty[st]), ((i >> 1) + 1) & 1, spin, abort);
          if (!ok) break;
          const uint32_t full = bar(is_v ? &ctrl->v_full[st] : &ctrl->k_full[st]);
          const uint32_t dst = base + (is_v ? C::V : C::K) + st * C::TILE;
          mbar_arrive_expect(full, C::TILE);
#pragma unroll
          for (int g = 0; g < C::GROUPS; ++g)
            tma_load_3d(dst + g * C::GROUP_BYTES, is_v ? &map_v : &map_k, 64 * g, h, q0 + tile_key(span, i), full);
        }
        if (!ok) give_up();
        // Leave with no copy in flight, whoever gave up: the queries and the last of each stage are there.
        mbar_wait(bar(&ctrl->q_full), 0, kDrain);
        for (int t = max(issued - 4, 0); t < issued; ++t)
          mbar_wait(bar((t & 1) ? &ctrl->v_full[t >> 1 & 1] : &ctrl->k_full[t >> 1 & 1]), (t >> 2) & 1, kDrain);
      }
      __syncwarp();
    } else if (warp == kIssuer) {
      // ================= products =================
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int tiles = __shfl_sync(0xffffffffu, nk, 0), used = __shfl_sync(0xffffffffu, halves, 0);
      const int first_tiles = __shfl_sync(0xffffffffu, tiles_of(0), 0);
      const uint32_t leader = elect_lane();
      const uint32_t qk_desc = mma_desc(128, kKeys, true, false), pv_desc = mma_desc(128, D, true, true);
      const uint64_t q_op = smem_desc(base + C::Q, 16), k_op = smem_desc(base + C::K, 16);
      const uint64_t v_op = smem_desc(base + C::V, C::GROUP_BYTES);
      auto wait = [&](const void* b, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_wait_or_abort(bar(b), parity, spin, abort))) return true;
        give_up();
        return false;
      };
      // test hook: in place of this K tile (-1: none) the products wait for what nothing signals
      const int withheld = static_cast<int>(blockIdx.x) == a.withhold_cta ? a.withhold_tile : -1;
      auto k_there = [&](int i) {
        return i == withheld ? wait(&ctrl->drained, 0) : wait(&ctrl->k_full[i & 1], (i >> 1) & 1);
      };
      auto scores = [&](int w, int stage) {  // S_w = Q_w K^T
        const uint64_t qa = q_op + w * (C::TILE >> 4), ka = k_op + stage * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int at = ((k >> 2) * C::GROUP_BYTES + (k & 3) * 32) >> 4;
          mma_ss(leader, tm + C::S(0) + w * 128, qa + at, ka + at, qk_desc, k > 0);
        }
        tc_commit(leader, bar(&ctrl->s_full[w]));
      };
      auto values = [&](int w, int stage, bool add) {  // O_w += P_w V; each column half's pairs lie in its own columns
        const uint64_t va = v_op + stage * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(leader, tm + C::O(0) + w * 128, tm + C::S(0) + w * 128 + (k & 4) * 16 + (k & 3) * 8, va + k * (2048 >> 4),
                 pv_desc, add || k > 0);
      };
      // Products run in the order of their issue, so scores that overwrite probabilities
      // only need to be issued behind the products that read them.
      bool ok = wait(&ctrl->q_full, 0) && k_there(0);
      if (ok) {
        tc_fence_after();
        for (int w = 0; w < used; ++w) scores(w, 0);
        tc_commit(leader, bar(&ctrl->k_empty[0]));
      }
      for (int i = 0; ok && i < tiles; ++i) {
        const int st = i & 1, ns = (i + 1) & 1;
        ok = wait(&ctrl->v_full[st], (i >> 1) & 1) && wait(&ctrl->v_ok[st], (i >> 1) & 1) && (i + 1 == tiles || k_there(i + 1));
        for (int w = 0; ok && w < used; ++w) {
          const int mine = w == 0 ? first_tiles : tiles;
          if (i >= mine) continue;
          ok = wait(&ctrl->p_full[w], i & 1);
          if (!ok) break;
          tc_fence_after();
          values(w, st, i > 0);
          if (i + 1 < mine) scores(w, ns);
          else tc_commit(leader, bar(&ctrl->o_full[w]));
        }
        tc_commit(leader, bar(&ctrl->v_empty[st]));
        if (i + 1 < tiles) tc_commit(leader, bar(&ctrl->k_empty[ns]));
      }
      // Leave with no product in flight, whoever gave up.
      tc_commit(leader, bar(&ctrl->drained));
      mbar_wait(bar(&ctrl->drained), 0, kDrain);
      __syncwarp();
    } else {
      // ================= values of tiles that a row sees only in part =================
      const int w = warp - kIssuer - 2;
      for (int i = 0; i < nk; ++i) {
        const int st = i & 1, t0 = tile_key(span, i);
        if (!__all_sync(0xffffffffu, mbar_wait_or_abort(bar(&ctrl->v_full[st]), (i >> 1) & 1, spin, abort))) {
          give_up();
          break;
        }
        if (!whole(0, t0) || (halves > 1 && !whole(1, t0))) {
          uint4* const v = reinterpret_cast<uint4*>(smem + C::V + st * C::TILE) + 32 * w + lane;
          bool bad = false;
#pragma unroll 4
          for (int k = 0; k < C::TILE / 16; k += 64) {
            const uint4 x = v[k];
            if (any_not_finite(x.x) || any_not_finite(x.y) || any_not_finite(x.z) || any_not_finite(x.w)) {
              bad = true;
              v[k] = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
            }
          }
          if (bad) {
            atomicMin(&ctrl->bad_lo, i);
            atomicMax(&ctrl->bad_hi, i);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&ctrl->v_ok[st]));
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
cudaError_t launch_t(const PromptArgs& a, cudaStream_t st) {
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
  prompt_kernel<D><<<static_cast<unsigned>(a.tiles) * a.num_kv_heads, C::THREADS, C::SMEM, st>>>(a, q, k, v);
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
  if (tiles * a.num_kv_heads > INT32_MAX) return cudaErrorNotSupported;
  a.tiles = static_cast<int>(tiles);
  if (head_dim == 64) return launch_t<64>(a, st);
  if (head_dim == 128) return launch_t<128>(a, st);
  return cudaErrorNotSupported;
}

}  // namespace kvq

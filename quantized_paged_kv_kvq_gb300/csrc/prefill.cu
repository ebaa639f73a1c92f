// Attention of each sequence's new tokens to its paged, quantized context
// (kvq_paged_prefill).
//
// out = sum_t p_t v_t / sum_t p_t, p_t = 2^(z_t - m), z_t = sm_scale log2(e) <q, k_t>,
// with a running maximum m over tiles of 128 keys and float32 sums: one pass over
// the context, no score leaves the SM.
//
// Split: a CTA owns 64, 128 or 256 rows (token, query head) of one sequence and
// kv-head (the fewest that hold the longest chunk: 64 leave room for one more tile of
// V on its way, and warps without rows sit out: 68 -> 57 us in the case below); row R of the sequence is query head R % G of new token R / G, so the
// G heads that share keys fill a tile together.  Per 128 keys and 128 rows it
// runs two tcgen05 products, S = Q K^T (operands in shared memory) and
// O += P V (P in tensor memory, over S's own columns), S and O in tensor memory.
// With 256 rows one half's products run while the other half's softmax does,
// started when half of its probabilities are there; with 128 the next tile's
// scores go to a second buffer meanwhile.
//
// Warps: one warpgroup per 128 rows for the softmax (a thread a row: no
// shuffles), one that loads and dequantizes K, one for V, and one warp that
// issues the products.  A producer thread copies 16-byte pieces (cp.async) into a
// queue of its own and turns them into 16-bit operands in the 128-byte swizzle
// that the products read: codes become exact fp16 values with byte permutes onto
// 1024.0 or the native fp8 conversion, asymmetric rows one or two operations more.
// The 16-bit cache is copied straight into place.
//
// Where many row tiles read the same keys, dequantizing them in every CTA costs
// more than the products hide (the schedulers issue 0.6 instructions a cycle, a third
// of them for it).  Then stage_kernel writes the operands to memory once, by whole
// tiles, and one thread per CTA loads them by TMA: 2 x 4,096 tokens on 10,000 keys of
// int8, 32 / 8 heads of 128, 1.18 TFLOP: 0.79 to 0.80 ms, 1,490 TFLOP/s, 78 % of the measured
// matrix rate, against 1.01 ms (30 us of it the staging; the tensor pipe is 69 % busy).
// What is left is the chain of a row's tile: scores, softmax (1,500 cycles), products.
//
// Few rows over long contexts: the keys are cut into num_splits parts, whose
// (m, sum, accumulators) a second kernel joins.  32 x 1..8 tokens on 256..4,096 keys:
// 57 us, 2.4 TB/s (int8; bf16 73, int4 78, uint8 84, KVarN 96: rows made in float32).  A tile takes 2,650 cycles, the softmax of the one warp with rows
// 2,050 of them and the producers as much (a third converting, half issuing copies);
// a CTA's start and end 14,000 (7 us).
//
// Measured and not kept: score buffers of 64 keys, two ahead (1.13 ms for 1.01); an
// issuing warp per half (1.21); codes through registers instead of the queue (1.04);
// scores held in 128 registers (0.85 ms for 0.85, 0.48 for 0.35 with masks and KVarN);
// fully unrolled softmax and conversions (2.1 ms: instruction fetch).  With few rows:
// up to 32 rows in four copies, each warp a quarter of a tile's keys (63 us for 57: the
// producers bound it, and the copies have to be joined); keys cut into parts for two or
// four waves of CTAs (with 128 rows a tile: 91 us for 68 with 32 sequences, 47 and 51 for
// 32 with 2, 45 and 59 for 43 with 8; 52 and 65 for 61 with 12, whose 96 CTAs leave a
// third of the SMs idle).
#include <atomic>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "mbarrier.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_prefill)

namespace {

constexpr int kKeys = 128;            // keys per tile
constexpr int kProducers = 128;       // threads that load and dequantize K; as many for V
constexpr int kDrain = 1 << 18;       // polls for what is in flight at a CTA's end (a second)
constexpr float kLazy = 8.0f;         // a maximum that grows by less (log2) is not raised: p <= 2^8
// Probabilities are made 2^7 times as large, sums and accumulators with them, so that
// as 16-bit operands they end at 2^15 and reach down to 2^-32 of the maximum's: fp16
// alone would drop what is below 2^-25, and 131,072 such keys weigh 0.4 % of one that
// dominates (often a first token whose own value is next to nothing).
constexpr float kLift = 7.0f;

// Block formats: codes are exact operands, as those of the other 8-bit formats, and a page's
// scales, which may lie anywhere in float32's range, stay out of them: K's multiplies the
// score, V's the probability.  p times V's scale is the 16-bit operand, so the row's m is the
// largest z + log2(scale) less kBlockLift, and raised when one passes 2^15.  That log2 counts as
// kBlockLeast at least, so that m is never lower than the largest z less 100 and the sum stays in
// range where all values are zeros.  (Folded into the operands, rows past 65,504 were infinite
// and those below 2^-14 lost bits.)  int8, 8 x 4,096 keys, 4 row tiles a sequence: 142 us, where
// rows made in float32 took 156; dequantized ahead, 8 tiles 270, where such rows took 261.
constexpr float kBlockLift = 9.0f, kBlockRaise = 15.0f;
constexpr float kBlockLeast = -91.0f;
// Scales of a tile, one of each for 8 keys: of the scores (sm_scale and log2(e) with it), of the
// values, and those' log2.  A ring of kScaleSlots tiles: a slot is written up to four tiles
// ahead of the score products that are done and read until the tile's softmax is, at most two
// behind them, so that six are in use.
constexpr int kGroups = kKeys / 8, kScaleBytes = 3 * kGroups * 4, kScaleSlots = 8;

// head_dim, rows, keys dequantized ahead, block formats
template <int D_, int ROWS_, bool STAGED = false, bool BLOCK_ = false>
struct Cfg {
  static constexpr bool BLOCK = BLOCK_;
  static constexpr int D = D_, ROWS = ROWS_;
  static constexpr int NW = ROWS == 256 ? 2 : 1;  // softmax warpgroups
  static constexpr int THREADS = 128 * NW + (STAGED ? 0 : 2 * kProducers) + 128;
  static constexpr int GROUPS = D / 64;              // 64-element column groups of an operand row
  static constexpr int GROUP_BYTES = 128 * 128;      // 128 rows of 128 bytes
  static constexpr int TILE = GROUPS * GROUP_BYTES;  // a 128-row operand
  static constexpr int RAW = 128 * D;                // largest code tile that is dequantized
  // tiles that the producers' loads run ahead (slots of their queues); what shared
  // memory leaves room for
  static constexpr int AHEAD_K = NW == 2 ? 1 : 2, AHEAD_V = ROWS == 64 ? 2 : 1;
  // shared memory: queries, K and V stages, raw queue, raw metadata, control.  With 64
  // rows the products read 64 more of a group, which are what lies behind: rows of
  // scores that no one reads.
  static constexpr int Q = 0;
  static constexpr int Q_GROUP = ROWS == 64 ? 64 * 128 : GROUP_BYTES;
  static constexpr int K = Q + NW * GROUPS * Q_GROUP;
  static constexpr int V = K + 2 * TILE;
  static constexpr int RAWQ = V + 2 * TILE;
  static constexpr int META = RAWQ + (STAGED ? 0 : (AHEAD_K + AHEAD_V) * RAW);  // slots of K, then of V
  static constexpr int CTRL = META + (AHEAD_K + AHEAD_V) * 3 * kKeys * 2;
  static_assert(kScaleSlots * kScaleBytes <= CTRL - META, "the ring of tiles' scales lies where other formats' metadata does");
  static constexpr int SIGNS = CTRL + 256;  // the rotation's diagonal as masks of pairs of sign bits
  static constexpr int SMEM = SIGNS + 2 * D + 1024;
  // tensor memory columns: two score buffers (one per warpgroup, or the two that one
  // warpgroup's tiles take in turn), then the accumulators
  static constexpr uint32_t S(int b) { return b * 128; }
  static constexpr uint32_t O(int w) { return 256 + w * 128; }
  static constexpr uint32_t TMEM = 512;
  // registers per thread of the softmax, producer and issuing warpgroups: together
  // no more than the block is launched with (96, 128 or, staged, 168 each)
  static constexpr int R_SOFTMAX = STAGED ? 216 : NW == 2 ? 128 : 192;
  static constexpr int R_PRODUCE = NW == 2 ? 88 : 104;
  static constexpr int R_ISSUE = STAGED ? 72 : NW == 2 ? 48 : 64;
};

// Control words in shared memory.
struct Ctrl {
  unsigned long long q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2], pv_done, o_full[2], drained,
      scales[kScaleSlots];
  uint32_t tmem;
  int abort;
  int seq, tile, q0, q, n;  // this CTA's rows
  int bad_lo, bad_hi;  // tiles with values that are not finite
};

static_assert(sizeof(Ctrl) <= 256, "control words");

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

// The rows of sequence s: first packed row and count, cut to fit.
__device__ __forceinline__ int2 seq_rows(const PrefillArgs& a, int s, bool& bad) {
  const int c0 = a.cu_query[s], c1 = a.cu_query[s + 1];
  const int total = static_cast<int>(a.total_q);
  const int q0 = clamp_int(c0, 0, total), q1 = clamp_int(c1, q0, total);
  const int q = min(q1 - q0, a.max_query_len);
  bad = c0 != q0 || c1 != q1 || q != q1 - q0;
  return make_int2(q0, q);
}

// The sequence and row tile that tile number `want` (of all sequences, ROWS
// rows each) is, found by the whole block.  Up to kOrdered sequences count by rising
// length (the launch starts from the last tile, so the longest come first; scan: two
// words a sequence, which is what the metadata slots hold), more in their order (a scan;
// a word a warp): 32 x 1..8 tokens on 256..4,096 keys, 256 CTAs on 152 SMs: 93 us in
// their order, 68 so (of 128 rows each).  Of many sequences the order matters less: 128
// such take 206 us, 129 in their order 227.
constexpr int kOrdered = 128;
static_assert(kOrdered * 8 <= 2 * 3 * kKeys * 2, "fits the metadata slots, which are not in use yet");
template <int ROWS>
__device__ void find_tile(const PrefillArgs& a, Ctrl* c, int* scan, int want) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  if (tid == 0) c->seq = -1;
  int before = 0;  // tiles of the sequences before the chunk
  unsigned err = 0;
  for (int base = 0; base < a.num_seqs; base += blockDim.x) {
    const int s = base + tid;
    int2 r = make_int2(0, 0);
    int v = 0, len = 0;
    if (s < a.num_seqs) {
      bool bad;
      r = seq_rows(a, s, bad);
      if (bad) err |= 256u;  // KVQ_DEVERR_TOKENS
      const long long rows = static_cast<long long>(r.y) * a.gqa;
      v = static_cast<int>((rows + ROWS - 1) / ROWS);
      const int n = a.context_lens[s];
      len = clamp_int(n, 0, a.max_context_len);
      if (n != len || len < r.y) err |= 4u;
    }
    int first = before, total = 0;
    if (a.num_seqs <= kOrdered) {
      int2* tiles = reinterpret_cast<int2*>(scan);
      if (s < a.num_seqs) tiles[s] = make_int2(len, v);
      __syncthreads();
      if (s < a.num_seqs) {
#pragma unroll 8
        for (int j = 0; j < a.num_seqs; ++j) {
          const int2 t = tiles[j];
          if (t.x < len || (t.x == len && j < s)) first += t.y;
        }
      }
    } else {
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      for (int w = 0; w < warps; ++w) {
        if (w < warp) first += scan[w];
        total += scan[w];
      }
      first += incl - v;
    }
    if (first <= want && want < first + v) {
      c->seq = s;
      c->tile = want - first;
      c->q0 = r.x;
      c->q = r.y;
      c->n = len;
    }
    before += total;
    __syncthreads();
    if (before > want && blockIdx.x != 0) break;  // block 0 checks every sequence
  }
  if (err && blockIdx.x == 0) raise_error(err);
}

// What the rows [R0, R1) of a sequence see: positions p_lo..p_hi of their
// tokens, and the key tiles, `kept` leading ones and then those from `skip`
// tiles later on.
struct Span {
  int p_lo, p_hi;
  int win;  // first position in the window of the first row (0 without a window)
  int kept, skip, tiles;
};
__device__ __forceinline__ Span row_span(const PrefillArgs& a, int n, int q, int R0, int R1) {
  Span s{0, -1, 0, 0, 0, 0};
  s.p_lo = max(n - q + R0 / a.gqa, 0);
  s.p_hi = n - q + (R1 - 1) / a.gqa;
  if (s.p_hi < 0) return s;
  s.tiles = s.p_hi / kKeys + 1;
  if (a.window > 0) {
    s.win = max(s.p_lo - a.window + 1, 0);
    s.kept = (min(a.sinks, s.win) + kKeys - 1) / kKeys;
    s.skip = max(s.win / kKeys - s.kept, 0);
    s.tiles -= s.skip;
  }
  return s;
}
__device__ __forceinline__ int tile_key(const Span& s, int i) { return kKeys * (i < s.kept ? i : i + s.skip); }

// A row's fields, each an fp16 value twice, as dequantize16 takes them.  Rotated rows:
// scale and zero point times the deviation, in float32 (products of 11 bits each: exact).
template <bool KVARN>
struct RowFields {
  uint32_t s, z;
  __device__ __forceinline__ RowFields(uint32_t scale, uint32_t zero, uint32_t) : s(scale), z(zero) {}
};
template <>
struct RowFields<true> {
  float s, z;
  __device__ __forceinline__ RowFields(uint32_t scale, uint32_t zero, uint32_t deviation) {
    const float g = __half2float(__ushort_as_half(static_cast<uint16_t>(deviation)));
    s = __half2float(__ushort_as_half(static_cast<uint16_t>(scale))) * g;
    z = __half2float(__ushort_as_half(static_cast<uint16_t>(zero))) * g;
  }
};

// 16 bytes of codes as 16-bit operands: 16 (8-bit codes) or 32 (int4) fp16
// values, in order.  Asymmetric rows are rounded once, to fp16: code * scale + zero
// point by a fused fp16 operation, rotated rows (code * (scale * deviation) + zero point *
// deviation) in float32, where code * scale may pass fp16's range on the way.
template <int F, bool KVARN>
__device__ __forceinline__ void dequantize16(const uint4& raw, const RowFields<KVARN>& row,
                                             uint32_t (&o)[F == INT4A ? 16 : 8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  constexpr uint32_t K64 = 0x64646464u;
  auto affine2 = [&](uint32_t c, uint32_t* p) {  // four codes, a byte each
    if constexpr (KVARN) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(prmt(c, 0x4B000000u, 0x7440u + e));  // 2^23 + code
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float u, v;
        add2(u, v, x[e], x[e + 1], -8388608.f, -8388608.f);
        fma2(u, v, u, v, row.s, row.s, row.z, row.z);
        p[e / 2] = pack_half2(u, v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t h = hsub2_u32(prmt(c, K64, e ? 0x4342u : 0x4140u), 0x64006400u);
        const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&row.s),
                                  *reinterpret_cast<const __half2*>(&row.z));
        p[e] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F == INT8) {
      const uint32_t b = w[i] ^ 0x80808080u;
      o[2 * i] = hsub2_u32(prmt(b, K64, 0x4140), 0x64806480u);
      o[2 * i + 1] = hsub2_u32(prmt(b, K64, 0x4342), 0x64806480u);
    } else if constexpr (F == E4M3) {
      o[2 * i] = e4m3x2_to_f16x2(w[i] & 0xFFFFu);
      o[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
    } else if constexpr (F == E5M2) {
      o[2 * i] = prmt(w[i], 0u, 0x1404);
      o[2 * i + 1] = prmt(w[i], 0u, 0x3424);
    } else if constexpr (F == UINT8A) {
      affine2(w[i], o + 2 * i);
    } else {  // INT4A: element 2i in the low nibble of byte i
      const uint32_t lo = w[i] & 0x0F0F0F0Fu, hi = (w[i] >> 4) & 0x0F0F0F0Fu;
      affine2(prmt(lo, hi, 0x5140), o + 4 * i);
      affine2(prmt(lo, hi, 0x7362), o + 4 * i + 2);
    }
  }
}

// acc + 0 * each of N pairs of 16-bit values: stays 0 (or -0) while they are finite.
template <bool BF, int N>
__device__ __forceinline__ uint32_t track_not_finite(uint32_t acc, const uint32_t (&o)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (BF) {
      const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&o[i]), __nv_bfloat162(),
                                       *reinterpret_cast<const __nv_bfloat162*>(&acc));
      acc = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 zero = __half2half2(__ushort_as_half(0));
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&o[i]), zero,
                                *reinterpret_cast<const __half2*>(&acc));
      acc = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  return acc;
}
__device__ __forceinline__ float half_of_pair(uint32_t p) {
  return fabsf(__half2float(__ushort_as_half(static_cast<uint16_t>(p))));
}
template <bool BF>
__device__ __forceinline__ bool finite16(uint32_t h) {
  return BF ? (h & 0x7F80u) != 0x7F80u : (h & 0x7C00u) != 0x7C00u;
}
template <bool BF>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  return (finite16<BF>(w) ? w & 0xFFFFu : 0u) | (finite16<BF>(w >> 16) ? w & 0xFFFF0000u : 0u);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ldsv4(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds_pair(uint32_t a) {  // a 16-bit value, twice
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r | (static_cast<uint32_t>(r) << 16);
}
template <int BYTES>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, bool read) {
  const int n = read ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// Address of 16-byte chunk q of row `row` in an operand tile.
__device__ __forceinline__ uint32_t chunk_addr(uint32_t tile, int row, int q, int group_bytes = 128 * 128) {
  return tile + (q >> 3) * group_bytes + row * 128 + (((q & 7) ^ (row & 7)) << 4);
}

// One of the two caches, as the producers read it.
struct Source {
  const uint8_t* codes;  // of the kv-head
  const __half* meta;    // of the kv-head, or nullptr (block formats: its float32 scales)
  uint32_t page_bytes, meta_page;  // codes of a block in bytes; metadata of a block in halves (floats)
  int token_bytes;
  int fmt, fields;
};
__device__ __forceinline__ Source make_source(const uint8_t* cache, const __half* meta, int fmt, int kvarn, int d,
                                              int hkv, int h, int bs, bool block) {
  Source s;
  const int rb = row_bytes(fmt, d);
  s.codes = cache + static_cast<size_t>(h) * rb;
  s.token_bytes = hkv * rb;
  s.page_bytes = static_cast<uint32_t>(bs) * s.token_bytes;  // below 2^31: checked on the host
  s.fmt = fmt;
  s.fields = is_asym(fmt) ? (kvarn ? 3 : 2) : 0;
  s.meta = is_asym(fmt) ? meta + static_cast<size_t>(h) * s.fields * bs : block ? meta + 2 * h : nullptr;
  s.meta_page = block ? scale_pitch(hkv) : static_cast<uint32_t>(hkv) * s.fields * bs;
  return s;
}

// Barrier of a producer warpgroup (K's or V's); whether every warp came with `ok`
// (so that all leave together, and none waits here for one that gave up).
__device__ __forceinline__ bool producers_all(bool is_v, bool ok) {
  uint32_t all;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.red.and.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "r"(is_v ? 2 : 1)
      : "memory");
  return all != 0;
}

// The 16-byte pieces of a 128-row code tile that a producer thread owns: piece
// `chunk` of rows row0 + i * STEP, i < PASSES.  The lanes of a quarter-warp take 8 / CL
// neighbouring rows and CL pieces of each, which makes the 16-byte stores of
// their j-th operand chunks (OUT per piece) meet distinct banks under the
// swizzle; a warp's loads still cover whole rows.
template <int F, int D>
struct Pieces {
  static constexpr int CHUNKS = row_bytes(F, D) / 16;  // pieces of a row
  static constexpr int OUT = F == BF16 ? 1 : F == INT4A ? 4 : 2;
  static constexpr int STEP = kProducers / CHUNKS;  // a multiple of 8: the swizzle is the same in every pass
  static constexpr int PASSES = kKeys / STEP;
  static constexpr int CL = CHUNKS < 8 / OUT ? CHUNKS : 8 / OUT;
  int chunk, row0;
  __device__ __forceinline__ explicit Pieces(int tid) {
    constexpr int RL = 8 / CL, CH = CHUNKS / CL;
    chunk = tid % CL + CL * (tid / 8 % CH);
    row0 = tid / CL % RL + RL * (tid / (8 * CH));
  }
};

// Whether some row sees one of the 8 keys from t on.
__device__ __forceinline__ bool group_needed(const PrefillArgs& a, const Span& span, int t) {
  return t <= span.p_hi && (t + 7 >= span.win || t < a.sinks);
}
// What the softmax takes of a group's scale of K: times sm_scale log2(e) (scale > 0), and never
// 0, so that a masked score stays -inf.  Not a number: the rows that see the group get NaN at
// the end (bad), the others' scores are not touched.
__device__ __forceinline__ float key_scale(float scale, float of_page, bool& bad) {
  const float f = scale * of_page;
  bad = of_page != of_page;
  return f >= 1.17549435e-38f ? f : 1.17549435e-38f;
}
// Of V: 0 where it is not finite, as such values are zeroed, too; and what counts as its log2.
__device__ __forceinline__ float value_scale(float of_page, bool& bad) {
  bad = !isfinite(of_page);
  return bad ? 0.f : of_page;
}
__device__ __forceinline__ float log2_scale(float v) { return fmaxf(__log2f(fabsf(v)), kBlockLeast); }

// The producer warpgroup's view of one key tile.
struct KeyTile {
  int t0;     // first key
  int block;  // lane l: block id of the tile's l-th page
};

template <class C>
struct Producer {
  const PrefillArgs& a;
  const Span& span;
  uint32_t smem;
  int tid;  // 0 .. kProducers - 1
  int seq;

  __device__ __forceinline__ bool needed(int t) const {
    return t <= span.p_hi && (t >= span.win || t < a.sinks);
  }
  __device__ __forceinline__ bool all_needed(int t0) const {
    return t0 + kKeys - 1 <= span.p_hi && (t0 >= span.win || t0 + kKeys <= a.sinks);
  }
  // Block ids of tile i's pages, one per lane; pages that no row sees are not looked up.
  __device__ __forceinline__ KeyTile look_up(int i) const {
    KeyTile k;
    k.t0 = tile_key(span, i);
    k.block = 0;
    const int lane = tid & 31, bs = 1 << a.block_shift;
    const int t = k.t0 + lane * bs;
    if (lane < (kKeys >> a.block_shift) && t <= span.p_hi && (t + bs > span.win || t < a.sinks))
      k.block = a.block_table[static_cast<size_t>(seq) * a.max_blocks_per_seq + (t >> a.block_shift)];
    return k;
  }
  // Checked when they are first used, a tile after the look-up, so that nothing waits for it.
  __device__ __forceinline__ void check(KeyTile& k) const {
    if (k.block < 0 || k.block >= a.num_blocks) {
      raise_error(2u);  // KVQ_DEVERR_BLOCK_RANGE: block 0 is read instead
      k.block = 0;
    }
  }
  // Start copying the tile's codes: 8-bit and 4-bit ones into slot `slot` of this
  // thread's queue, 16-bit ones into the operand tile `dst`.
  template <int F>
  __device__ __forceinline__ void copy_codes(const Source& s, const KeyTile& k, int slot, uint32_t dst) const {
    using P = Pieces<F, C::D>;
    const P p(tid);
    const int mask = (1 << a.block_shift) - 1;
    const uint8_t* src0 = s.codes + p.chunk * 16;
    const uint32_t to = F == BF16 ? chunk_addr(dst, p.row0, p.chunk) : smem + C::RAWQ + slot * C::RAW + tid * 16;
    constexpr int TO_STEP = F == BF16 ? P::STEP * 128 : kProducers * 16;
    if (all_needed(k.t0)) {
#pragma unroll 4
      for (int i = 0; i < P::PASSES; ++i) {
        const int row = p.row0 + i * P::STEP;
        const int blk = __shfl_sync(0xffffffffu, k.block, row >> a.block_shift);
        cp_async<16>(to + i * TO_STEP, src0 + static_cast<unsigned long long>(static_cast<uint32_t>(blk)) * s.page_bytes + (row & mask) * s.token_bytes);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < P::PASSES; ++i) {
        const int row = p.row0 + i * P::STEP;
        const int blk = __shfl_sync(0xffffffffu, k.block, row >> a.block_shift);
        cp_async_or_zero<16>(to + i * TO_STEP, src0 + static_cast<unsigned long long>(static_cast<uint32_t>(blk)) * s.page_bytes + (row & mask) * s.token_bytes,
                             needed(k.t0 + row));
      }
    }
  }
  __device__ __forceinline__ void copy(const Source& s, const KeyTile& k, int slot, uint32_t dst) const {
    if (!C::BLOCK && s.fmt == BF16) copy_codes<BF16>(s, k, slot, dst);
    else if (!C::BLOCK && s.fmt == INT4A) copy_codes<INT4A>(s, k, slot, dst);
    else copy_codes<INT8>(s, k, slot, dst);  // any 8-bit code
    if (s.fields > 0) {  // a pair of tokens per thread and field
      const int row = 2 * (tid & 63), t = k.t0 + row;
      const int blk = __shfl_sync(0xffffffffu, k.block, row >> a.block_shift);
      const __half* src = s.meta + static_cast<unsigned long long>(static_cast<uint32_t>(blk)) * s.meta_page +
                          (row & ((1 << a.block_shift) - 1));
      const bool read = needed(t) || needed(t + 1);
      for (int f = tid >> 6; f < s.fields; f += 2)
        cp_async_or_zero<4>(smem + C::META + (slot * 3 + f) * kKeys * 2 + row * 2, src + (f << a.block_shift), read);
    }
  }
  // Block formats, by the first warp: start copying the scales of the tile's groups of 8 keys
  // (lanes 0-15 K's, 16-31 V's; 0 for groups that no row sees) into their slot.
  __device__ __forceinline__ void copy_scales(const Source& ks, const Source& vs, const KeyTile& k, uint32_t to) const {
    const int g = tid % kGroups;
    const int blk = __shfl_sync(0xffffffffu, k.block, (8 * g) >> a.block_shift);
    const Source& s = tid < kGroups ? ks : vs;
    cp_async_or_zero<4>(to + tid * 4, reinterpret_cast<const float*>(s.meta) + static_cast<unsigned long long>(static_cast<uint32_t>(blk)) * s.meta_page,
                        group_needed(a, span, k.t0 + 8 * g));
  }
  // The pieces in slot `slot` as operands; whether one may not be finite (of V,
  // and of formats that can hold such a value; large asymmetric rows count too).
  template <int F, bool KVARN, bool IS_V>
  __device__ __forceinline__ bool convert(const KeyTile& k, int slot, uint32_t dst) const {
    using P = Pieces<F, C::D>;
    const P p(tid);
    const uint32_t raw = smem + C::RAWQ + slot * C::RAW + tid * 16;
    const uint32_t meta = smem + C::META + slot * 3 * kKeys * 2 + p.row0 * 2;
    const bool all = !is_asym(F) || all_needed(k.t0);
    uint32_t to[P::OUT];
#pragma unroll
    for (int j = 0; j < P::OUT; ++j) to[j] = chunk_addr(dst, p.row0, p.chunk * P::OUT + j);
    uint32_t nf[2] = {0u, 0u};
    float largest = 0.f;
    constexpr int U = P::PASSES < 4 || F == INT4A ? 2 : 4;  // pieces in flight
#pragma unroll 1
    for (int i0 = 0; i0 < P::PASSES; i0 += U) {
      uint4 w[U];
      uint32_t sc[U], zp[U], sg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        w[u] = ldsv4(raw + i * (kProducers * 16));
        sc[u] = zp[u] = sg[u] = 0;
        if constexpr (is_asym(F)) {
          if (all || needed(k.t0 + p.row0 + i * P::STEP)) {
            sc[u] = lds_pair(meta + i * P::STEP * 2);
            zp[u] = lds_pair(meta + (kKeys + i * P::STEP) * 2);
            if (KVARN) sg[u] = lds_pair(meta + (2 * kKeys + i * P::STEP) * 2);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t o[4 * P::OUT];
        dequantize16<F, KVARN>(w[u], {sc[u], zp[u], sg[u]}, o);
        if constexpr (IS_V && is_asym(F)) {  // |code * s + z| g is at most this
          float top = fmaf(half_of_pair(sc[u]), static_cast<float>(asym_levels(F)), half_of_pair(zp[u]));
          if (KVARN) top *= half_of_pair(sg[u]);
          largest = top < 65504.f ? largest : 65504.f;  // NaN counts
        } else if constexpr (IS_V && F != INT8) {
          nf[u & 1] = track_not_finite<false>(nf[u & 1], o);
        }
#pragma unroll
        for (int j = 0; j < P::OUT; ++j)
          sts128(to[j] + (i0 + u) * P::STEP * 128, o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      }
    }
    return largest != 0.f || ((nf[0] | nf[1]) & 0x7FFF7FFFu) != 0;
  }
  // 16-bit values are in place already: whether one of them is not finite.
  __device__ __forceinline__ bool check_bf16(uint32_t dst) const {
    using P = Pieces<BF16, C::D>;
    const P p(tid);
    const uint32_t at = chunk_addr(dst, p.row0, p.chunk);
    uint32_t nf[2] = {0u, 0u};
#pragma unroll 4
    for (int i = 0; i < P::PASSES; ++i) {
      const uint4 w = ldsv4(at + i * P::STEP * 128);
      const uint32_t o[4] = {w.x, w.y, w.z, w.w};
      nf[i & 1] = track_not_finite<true>(nf[i & 1], o);
    }
    return ((nf[0] | nf[1]) & 0x7FFF7FFFu) != 0;
  }
  // This thread's values of the operand tile that are not finite become 0 (a
  // probability of 0 times one of them would not be 0).
  template <int F>
  __device__ __forceinline__ void make_finite(uint32_t dst) const {
    using P = Pieces<F, C::D>;
    constexpr bool BF = F == BF16;
    const P p(tid);
#pragma unroll 1
    for (int i = 0; i < P::PASSES * P::OUT; ++i) {
      const uint32_t at = chunk_addr(dst, p.row0 + i / P::OUT * P::STEP, p.chunk * P::OUT + i % P::OUT);
      const uint4 w = ldsv4(at);
      sts128(at, finite_or_zero<BF>(w.x), finite_or_zero<BF>(w.y), finite_or_zero<BF>(w.z), finite_or_zero<BF>(w.w));
    }
  }
  template <bool IS_V>
  __device__ __forceinline__ bool finish(const Source& s, const KeyTile& k, int slot, uint32_t dst) const {
    if constexpr (C::BLOCK) {
      return s.fmt == INT8B ? convert<INT8, false, IS_V>(k, slot, dst) : convert<E4M3, false, IS_V>(k, slot, dst);
    } else {
      switch (s.fmt) {
        case INT8: return convert<INT8, false, IS_V>(k, slot, dst);
        case E4M3: return convert<E4M3, false, IS_V>(k, slot, dst);
        case E5M2: return convert<E5M2, false, IS_V>(k, slot, dst);
        case INT4A:
          return s.fields == 3 ? convert<INT4A, true, IS_V>(k, slot, dst) : convert<INT4A, false, IS_V>(k, slot, dst);
        case UINT8A:
          return s.fields == 3 ? convert<UINT8A, true, IS_V>(k, slot, dst) : convert<UINT8A, false, IS_V>(k, slot, dst);
        default: return IS_V ? check_bf16(dst) : false;
      }
    }
  }
};

__device__ __forceinline__ uint32_t pack16(bool bf, float lo, float hi) {
  return bf ? pack_bf162(lo, hi) : pack_half2(lo, hi);
}

// Scores that the row does not see become -inf: columns c > last, and those
// < first that are not < kept.
__device__ __forceinline__ void mask_scores(uint32_t s_addr, int last, int first, int kept) {
#pragma unroll 1
  for (int c0 = 0; c0 < kKeys; c0 += 32) {
    uint32_t s[32];
    tmem_ld32(s, s_addr + c0);
    tmem_wait_ld32(s);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (c0 + e > last || (c0 + e < first && c0 + e >= kept)) s[e] = 0xFF800000u;
    tmem_st32(s_addr + c0, s);
  }
  tmem_wait_st();
}
__device__ __forceinline__ float largest_score(uint32_t s_addr) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int c0 = 0; c0 < kKeys; c0 += 64) {
    uint32_t s[64];
    tmem_ld32(s, s_addr + c0);
    tmem_ld32(s + 32, s_addr + c0 + 32);
    tmem_wait_ld32(s);
    tmem_waited32(s + 32);
#pragma unroll
    for (int e = 0; e < 64; e += 8)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mx[i] = max3f(mx[i], __uint_as_float(s[e + 2 * i]), __uint_as_float(s[e + 2 * i + 1]));
  }
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}
// p = 2^(s * scale + off) over the scores, as 16-bit pairs in their first half (what
// the product takes); returns the sum, in float32 and before that rounding, whose errors
// (2^-11 of each p, or 2^-8 in bf16) do not add up in one direction.  The first 64 are handed over (half_bar,
// if not 0) when they are there, so that their products run while the others are made.
template <bool BF>
__device__ __forceinline__ float probabilities(uint32_t s_addr, float scale, float off, uint32_t half_bar, int lane) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int c0 = 0; c0 < kKeys; c0 += 64) {
    uint32_t s[64], p[32];
    tmem_ld32(s, s_addr + c0);
    tmem_ld32(s + 32, s_addr + c0 + 32);
    tmem_wait_ld32(s);
    tmem_waited32(s + 32);
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
      float x, y;
      fma2(x, y, __uint_as_float(s[e]), __uint_as_float(s[e + 1]), scale, scale, off, off);
      x = fast_exp2(x);
      y = fast_exp2(y);
      add2(sum[e & 2], sum[(e & 2) + 1], sum[e & 2], sum[(e & 2) + 1], x, y);
      p[e / 2] = BF ? pack_bf162(x, y) : pack_half2(x, y);
    }
    tmem_st32(s_addr + c0 / 2, p);  // over scores that have been read
    if (c0 == 0 && half_bar != 0) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(half_bar);
    }
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}
__device__ __forceinline__ void lds_floats8(float (&x)[8], uint32_t a) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = ldsv4(a + 16 * i);
    x[4 * i] = __uint_as_float(w.x);
    x[4 * i + 1] = __uint_as_float(w.y);
    x[4 * i + 2] = __uint_as_float(w.z);
    x[4 * i + 3] = __uint_as_float(w.w);
  }
}
// Block formats, with a tile's scales at `scales`: the largest logit plus the log2 of its value's
// scale.
__device__ __forceinline__ float largest_weighted(uint32_t s_addr, uint32_t scales) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c0 = 0; c0 < kKeys; c0 += 64) {
    uint32_t s[64];
    tmem_ld32(s, s_addr + c0);
    tmem_ld32(s + 32, s_addr + c0 + 32);
    float f[8], lv[8];
    lds_floats8(f, scales + c0 / 8 * 4);
    lds_floats8(lv, scales + (2 * kGroups + c0 / 8) * 4);
    tmem_wait_ld32(s);
    tmem_waited32(s + 32);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const uint32_t* x = s + 8 * g;
      float mx = max3f(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
      mx = max3f(mx, __uint_as_float(x[3]), __uint_as_float(x[4]));
      mx = max3f(mx, __uint_as_float(x[5]), __uint_as_float(x[6]));
      top = fmaxf(top, fmaf(fmaxf(mx, __uint_as_float(x[7])), f[g], lv[g]));
    }
  }
  return top;
}
// probabilities of block formats: p = 2^(s * its scale + off), handed over times the value's.
__device__ __forceinline__ float probabilities_scaled(uint32_t s_addr, uint32_t scales, float off, uint32_t half_bar, int lane) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int c0 = 0; c0 < kKeys; c0 += 64) {
    uint32_t s[64], p[32];
    tmem_ld32(s, s_addr + c0);
    tmem_ld32(s + 32, s_addr + c0 + 32);
    float f[8], v[8];
    lds_floats8(f, scales + c0 / 8 * 4);
    lds_floats8(v, scales + (kGroups + c0 / 8) * 4);
    tmem_wait_ld32(s);
    tmem_waited32(s + 32);
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
      float x, y;
      fma2(x, y, __uint_as_float(s[e]), __uint_as_float(s[e + 1]), f[e / 8], f[e / 8], off, off);
      x = fast_exp2(x);
      y = fast_exp2(y);
      add2(sum[e & 2], sum[(e & 2) + 1], sum[e & 2], sum[(e & 2) + 1], x, y);
      mul2(x, y, x, y, v[e / 8], v[e / 8]);
      p[e / 2] = pack_half2(x, y);
    }
    tmem_st32(s_addr + c0 / 2, p);  // over scores that have been read
    if (c0 == 0 && half_bar != 0) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(half_bar);
    }
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}
__device__ __forceinline__ void scale_columns(uint32_t addr, int columns, float f) {
#pragma unroll 1
  for (int c = 0; c < columns; c += 32) {
    uint32_t o[32];
    tmem_ld32(o, addr + c);
    tmem_wait_ld32(o);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float x, y;
      mul2(x, y, __uint_as_float(o[e]), __uint_as_float(o[e + 1]), f, f);
      o[e] = __float_as_uint(x);
      o[e + 1] = __float_as_uint(y);
    }
    tmem_st32(addr + c, o);
  }
}

// H x of a row held by one thread, on packed pairs from the second stage on.
template <int D>
__device__ __forceinline__ void fwht_row(float (&x)[D]) {
#pragma unroll
  for (int i = 0; i < D; i += 2) {
    const float u = x[i], v = x[i + 1];
    x[i] = u + v;
    x[i + 1] = u - v;
  }
#pragma unroll
  for (int h = 2; h < D; h <<= 1) {
#pragma unroll
    for (int i = 0; i < D; i += 2) {
      if ((i & h) == 0) {
        const float u0 = x[i], u1 = x[i + 1], v0 = x[i + h], v1 = x[i + h + 1];
        add2(x[i], x[i + 1], u0, u1, v0, v1);
        sub2(x[i + h], x[i + h + 1], u0, u1, v0, v1);
      }
    }
  }
}

// The packed rows that consecutive rows R0 + d (d < 32) of a sequence are: row r
// is head r % G of token r / G.  G <= 8, so d + R0 % G < 39 and a product with
// ceil(1024 / G) divides exactly.
struct RowMap {
  size_t token0;
  int first, recip, g, heads;
  __device__ __forceinline__ RowMap(const PrefillArgs& a, int q0, int h, int R0)
      : token0(static_cast<size_t>(q0) + R0 / a.gqa), first(R0 % a.gqa), recip((1023 + a.gqa) / a.gqa), g(a.gqa),
        heads(a.num_q_heads) {
    token0 = token0 * heads + static_cast<size_t>(h) * g;
  }
  __device__ __forceinline__ size_t operator()(int d) const {  // row of [tokens * heads, D]
    const int x = first + d, t = (x * recip) >> 10;
    return token0 + static_cast<size_t>(t) * heads + (x - t * g);
  }
};

// Rows R .. R+31 (those below R1; zeros behind) of the queries into rows row0 on
// of an operand tile, by a warp: copied as they are, a row being D/8 lanes of 16
// bytes, then turned (sign), rotated for KVarN and rounded to fp16 a row per
// thread.
template <int D, int GROUP>
__device__ __forceinline__ void load_queries(const PrefillArgs& a, uint32_t tile, uint32_t signs, int row0, int R,
                                             int R1, const RowMap& map, float turn, bool bf, int lane) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  const int sub = lane % LPR, grp = lane / LPR;
#pragma unroll 4
  for (int d = grp; d < 32; d += RPI)
    cp_async_or_zero<16>(chunk_addr(tile, row0 + d, sub, GROUP), a.query + map(R + d < R1 ? d : 0) * D + sub * 8, R + d < R1);
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  uint32_t nf = 0;
  if (a.kvarn) {
    float x[D];
#pragma unroll
    for (int q = 0; q < D / 8; ++q) {
      const uint4 w = ldsv4(chunk_addr(tile, row0 + lane, q, GROUP)), m = ldsv4(signs + 16 * q);
      const uint32_t o[4] = {w.x ^ m.x, w.y ^ m.y, w.z ^ m.z, w.w ^ m.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * q + 2 * e] = bf16_lo(o[e]);
        x[8 * q + 2 * e + 1] = bf16_hi(o[e]);
      }
    }
    fwht_row<D>(x);
    const float f = a.cR * turn;
#pragma unroll
    for (int q = 0; q < D / 8; ++q) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack_half2(x[8 * q + 2 * e] * f, x[8 * q + 2 * e + 1] * f);
      nf = track_not_finite<false>(nf, o);
      sts128(chunk_addr(tile, row0 + lane, q, GROUP), o[0], o[1], o[2], o[3]);
    }
  } else {
#pragma unroll 2
    for (int q = 0; q < D / 8; ++q) {
      const uint32_t at = chunk_addr(tile, row0 + lane, q, GROUP);
      const uint4 w = ldsv4(at);
      uint32_t o[4] = {w.x, w.y, w.z, w.w};
      if (!bf || turn != 1.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack16(bf, bf16_lo(o[e]) * turn, bf16_hi(o[e]) * turn);
        sts128(at, o[0], o[1], o[2], o[3]);
      }
      nf = bf ? track_not_finite<true>(nf, o) : track_not_finite<false>(nf, o);
    }
  }
  if (nf & 0x7FFF7FFFu) raise_error(64u);  // KVQ_DEVERR_QUERY_RANGE
}

// Values that are not finite among those that the row at position p sees, per
// dimension: bit d of hi for +inf, of lo for -inf, of both for NaN.  Only called
// when the producers met one; reads the codes of tiles t_lo..t_hi again.
template <class C>
__device__ __noinline__ void find_not_finite(const PrefillArgs& a, const Span& span, int seq, int h, int p, int i_lo,
                                             int i_hi, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  const int bs = 1 << a.block_shift;
  const Source s = make_source(a.v_cache, a.v_meta, a.v_fmt, a.kvarn, C::D, a.num_kv_heads, h, bs, C::BLOCK);
  for (int i = i_lo; i <= i_hi; ++i) {
    const int t0 = tile_key(span, i);
    for (int t = t0; t < t0 + kKeys && t <= p; ++t) {
      if (a.window > 0 && t <= p - a.window && t >= a.sinks) continue;
      int blk = a.block_table[static_cast<size_t>(seq) * a.max_blocks_per_seq + (t >> a.block_shift)];
      if (blk < 0 || blk >= a.num_blocks) blk = 0;
      const int off = t & (bs - 1);
      const uint8_t* row = s.codes + static_cast<size_t>(blk) * s.page_bytes + static_cast<size_t>(off) * s.token_bytes;
      __half sc{}, zp{}, sg{};
      float ps = 0.f;
      if (C::BLOCK) {
        const size_t at = static_cast<size_t>(blk) * s.meta_page + h;
        const float ks = reinterpret_cast<const float*>(a.k_meta)[at];
        ps = ks != ks ? ks : reinterpret_cast<const float*>(a.v_meta)[at];
      } else if (s.fields > 0) {
        const __half* m = s.meta + static_cast<size_t>(blk) * s.meta_page + off;
        sc = m[0];
        zp = m[bs];
        if (s.fields == 3) sg = m[2 * bs];
      }
      for (int d = 0; d < C::D; ++d) {
        uint32_t v;
        if (s.fmt == BF16) {
          v = reinterpret_cast<const uint16_t*>(row)[d];
          if (finite16<true>(v)) continue;
          v = (v & 0x7F) ? 0x7FFFu : (v & 0x8000u) | 0x7C00u;
        } else if (s.fmt == E5M2) {
          v = static_cast<uint32_t>(row[d]) << 8;
        } else if (s.fmt == E4M3) {
          v = e4m3x2_to_f16x2(row[d]) & 0xFFFFu;
        } else if (C::BLOCK) {
          const float c = s.fmt == INT8B ? static_cast<float>(static_cast<int8_t>(row[d]))
                                         : __half2float(__ushort_as_half(static_cast<uint16_t>(e4m3x2_to_f16x2(row[d]))));
          if (isfinite(ps) && isfinite(c)) continue;
          const float x = c * ps;
          v = x != x ? 0x7FFFu : x < 0.f ? 0xFC00u : 0x7C00u;
        } else if (s.fields > 0) {
          const int c = s.fmt == INT4A ? (row[d / 2] >> (4 * (d & 1))) & 15 : row[d];
          __half x = __hfma(__int2half_rn(c), sc, zp);  // as dequantize16
          if (s.fields == 3) {
            const float g = __half2float(sg);
            x = __float2half_rn(fmaf(static_cast<float>(c), __half2float(sc) * g, __half2float(zp) * g));
          }
          v = __half_as_ushort(x);
        } else {
          return;
        }
        if (finite16<false>(v)) continue;
        const bool nan = (v & 0x3FFu) != 0;
        if (s.fields == 3) {  // the inverse rotation spreads it over the whole row
          for (int w = 0; w < 4; ++w) hi[w] = lo[w] = 0xFFFFFFFFu;
          return;
        }
        if (nan || !(v & 0x8000u)) hi[d >> 5] |= 1u << (d & 31);
        if (nan || (v & 0x8000u)) lo[d >> 5] |= 1u << (d & 31);
      }
    }
  }
}

// 32 columns of a row's accumulators times mul; 0 for a row that saw nothing (its
// accumulators are 0 times whatever was there), NaN with a sum that is NaN, and
// what the marked values make of theirs (bits: hi +inf, lo -inf, both NaN).
__device__ __forceinline__ void result_columns(uint32_t (&o)[32], uint32_t addr, int c, float l, float mul, uint32_t hi,
                                               uint32_t lo) {
  tmem_ld32(o, addr + c);
  tmem_wait_ld32(o);
  const float f = l != l ? l : mul;
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * f);
  if (hi | lo) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t up = hi >> e & 1, down = lo >> e & 1;
      o[e] = up && down ? 0x7FC00000u : up ? 0x7F800000u : down ? 0xFF800000u : o[e];
    }
  }
}

template <int D, int ROWS, bool STAGED, bool BLOCK>
__global__ void __launch_bounds__(Cfg<D, ROWS, STAGED, BLOCK>::THREADS, 1)
    prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap map_staged) {
  using C = Cfg<D, ROWS, STAGED, BLOCK>;
  constexpr int NW = C::NW;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // swizzled tiles: 1024-byte aligned
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + C::CTRL);
  volatile int* abort = &ctrl->abort;
  const int spin = a.spin_limit;  // polls of an mbarrier before giving up
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7;
  constexpr int kIssuer = C::THREADS / 32 - 4;  // the warp that issues the products
  const int h = blockIdx.x % a.num_kv_heads;
  const int tile_id = a.tiles - 1 - blockIdx.x / a.num_kv_heads;  // later rows see more keys: first
  auto bar = [&](const void* p) { return base + static_cast<uint32_t>(static_cast<const uint8_t*>(p) - smem); };

  find_tile<C::ROWS>(a, ctrl, reinterpret_cast<int*>(smem + C::META), tile_id);  // not in use yet
  __syncthreads();
  const int seq = ctrl->seq;
  if (seq < 0) return;  // the launch has room for more tiles than the batch has
  const int n = ctrl->n, q = ctrl->q;
  const int R0 = ctrl->tile * C::ROWS, R1 = min(q * a.gqa, R0 + C::ROWS);
  const Span span = row_span(a, n, q, R0, R1);
  // this split's part of the key tiles
  const int split = blockIdx.y;
  const int i0 = static_cast<int>(static_cast<long long>(span.tiles) * split / a.num_splits);
  const int i1 = static_cast<int>(static_cast<long long>(span.tiles) * (split + 1) / a.num_splits);
  const int nk = i1 - i0;
  const int nw = (NW == 2 && R1 - R0 > 128) ? 2 : 1;  // row halves in use
  // warps with rows, of all and of each half (the others of a half only wait for the end)
  const int row_warps = (R1 - R0 + 31) / 32;
  auto half_warps = [&](int w) { return max(min(row_warps - 4 * w, 4), 1); };
  const bool bf = !C::BLOCK && a.k_fmt == BF16;

  if (tid == 0) {
    mbar_init(bar(&ctrl->q_full), row_warps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&ctrl->k_full[i]), STAGED ? 1 : kProducers / 32);
      mbar_init(bar(&ctrl->v_full[i]), STAGED ? 1 : kProducers / 32);
      mbar_init(bar(&ctrl->k_empty[i]), 1);
      mbar_init(bar(&ctrl->v_empty[i]), 1);
      mbar_init(bar(&ctrl->s_full[i]), 1);
      const int arrivals = half_warps(NW == 2 ? i : 0);  // one warpgroup has both buffers
      mbar_init(bar(&ctrl->p_half[i]), arrivals);
      mbar_init(bar(&ctrl->p_full[i]), arrivals);
      mbar_init(bar(&ctrl->o_full[i]), 1);
    }
    mbar_init(bar(&ctrl->pv_done), 1);
    mbar_init(bar(&ctrl->drained), 1);
    if (C::BLOCK)
      for (int i = 0; i < kScaleSlots; ++i) mbar_init(bar(&ctrl->scales[i]), 1);
    ctrl->abort = 0;
    ctrl->bad_lo = 0x7fffffff;
    ctrl->bad_hi = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (a.kvarn && tid < D / 2)
    reinterpret_cast<uint32_t*>(smem + C::SIGNS)[tid] =
        a.signs == nullptr ? 0u : (a.signs[2 * tid] < 0 ? 0x8000u : 0u) | (a.signs[2 * tid + 1] < 0 ? 0x80000000u : 0u);
  if (STAGED && BLOCK) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // find_tile's words, before copies over them
  __syncthreads();
  const size_t seq_head = static_cast<size_t>(seq) * a.num_kv_heads + h;
  if constexpr (STAGED) {  // tiles whose values were not all finite
    for (int i = tid; i < nk; i += C::THREADS) {
      if (a.staged_bad[seq_head * (a.staged_len / kKeys) + tile_key(span, i0 + i) / kKeys]) {
        atomicMin(&ctrl->bad_lo, i0 + i);
        atomicMax(&ctrl->bad_hi, i0 + i);
      }
    }
  }
  if (nk > 0) {
    if (warp == kIssuer) tmem_alloc(bar(&ctrl->tmem), C::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = ctrl->tmem;
  auto scale_slot = [&](int i) { return base + C::META + (i % kScaleSlots) * kScaleBytes; };
  const float abs_scale = a.sm_scale_log2 == 0.f ? 1.f : fabsf(a.sm_scale_log2);  // of block formats' scores
  auto give_up = [&]() {
    raise_error(16u);  // KVQ_DEVERR_TIMEOUT: the results of this launch are invalid
    *abort = 1;
  };

  if (wg < NW) {
    // ================= softmax: thread = row =================
    reg_take<C::R_SOFTMAX>();
    const int r = R0 + tid;  // row of the sequence (warpgroup w: rows 128 w on)
    const bool mine = r < R1;
    const int pos = mine ? n - q + r / a.gqa : span.p_hi;
    float scale = a.sm_scale_log2 * (a.k_head_scale != nullptr ? a.k_head_scale[h] : a.k_scale);
    // a negative scale turns the queries round, so that the largest logit is the
    // largest product; with scale 0 every logit is 0
    const float turn = scale < 0.f ? -1.f : scale > 0.f ? 1.f : 0.f;
    scale = scale == 0.f ? 1.f : fabsf(scale);
    float m = -INFINITY, l = 0.f;
    const bool has_rows = warp < row_warps, active = has_rows && nk > 0;
    const RowMap map(a, ctrl->q0, h, min(R0 + 32 * warp, R1 - 1));
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_first = tmem + C::S(wg) + lane_base, o_addr = tmem + C::O(wg) + lane_base;
    if (active) {
      load_queries<D, C::Q_GROUP>(a, base + C::Q + wg * C::TILE, base + C::SIGNS, 32 * (warp & 3), R0 + 32 * warp, R1, map, turn, bf,
                      lane);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&ctrl->q_full));
      const int p_last = n - q + (min(R0 + 128 * (wg + 1), R1) - 1) / a.gqa;  // this warpgroup's last position
      const int p_first = n - q + (R0 + 128 * wg) / a.gqa;
      for (int i = 0; i < nk; ++i) {
        // Two warpgroups have a score buffer each, one has both in turn, with a barrier
        // each way for either: its warps may be a tile apart.
        const int buf = NW == 2 ? wg : i & 1;
        const uint32_t s_addr = NW == 2 ? s_first : s_first + buf * 128;
        if (BLOCK && !__all_sync(0xffffffffu, mbar_wait_or_abort(bar(&ctrl->scales[i % kScaleSlots]), (i / kScaleSlots) & 1, spin, abort))) {
          give_up();
          break;
        }
        if (!__all_sync(0xffffffffu, mbar_wait_or_abort(bar(&ctrl->s_full[buf]), (NW == 2 ? i : i >> 1) & 1, spin, abort))) {
          give_up();
          break;
        }
        tc_fence_after();
        const int t0 = tile_key(span, i0 + i);
        // every row sees every key of the tile, or each row's own part
        const bool whole = t0 + kKeys - 1 <= p_first &&
                           (a.window == 0 || t0 > p_last - a.window || t0 + kKeys <= a.sinks);
        if (!whole) {
          const int last = pos - t0;
          mask_scores(s_addr, last, a.window > 0 ? last - a.window + 1 : -1, a.sinks - t0);
        }
        const float top = BLOCK ? largest_weighted(s_addr, scale_slot(i)) : largest_score(s_addr) * scale;
        if (__any_sync(0xffffffffu, top > m + (BLOCK ? kBlockRaise : kLazy))) {
          const float up = fmaxf(m, BLOCK ? top - kBlockLift : top);
          const float f = up == -INFINITY ? 1.f : fast_exp2(m - up);
          m = up;
          l *= f;
          if (i > 0) {
            // The products so far are done: with two warpgroups S of this tile was issued
            // behind them; else the next tile's was, whose barrier this warp follows phase by
            // phase (a wait sees no more than a phase's parity), and behind the last but
            // one tile's a commit of their own.
            const bool last = i + 1 == nk;
            if (NW == 1 && !__all_sync(0xffffffffu, mbar_wait_or_abort(bar(last ? &ctrl->pv_done : &ctrl->s_full[(i + 1) & 1]),
                                                                       last ? 0 : ((i + 1) >> 1) & 1, spin, abort))) {
              give_up();
              break;
            }
            tc_fence_after();
            scale_columns(o_addr, D, f);
          }
        }
        const float off = m == -INFINITY ? 0.f : (BLOCK ? 0.f : kLift) - m;  // a row that has seen nothing: every p is 0
        const uint32_t half_bar = NW == 2 ? bar(&ctrl->p_half[wg]) : 0u;
        if constexpr (BLOCK) l = fmaf(probabilities_scaled(s_addr, scale_slot(i), off, half_bar, lane), kSumUnit, l);
        else l += bf ? probabilities<true>(s_addr, scale, off, half_bar, lane)
                     : probabilities<false>(s_addr, scale, off, half_bar, lane);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&ctrl->p_full[buf]));
      }
    }
    // ---- the row's result.  The lanes of a warp decide together whether to go on: the
    // flag may be set between two lanes' looks at it.
    auto aborted = [&]() { return __any_sync(0xffffffffu, *abort != 0); };
    bool done = !aborted();
    if (active && done) {
      done = __all_sync(0xffffffffu, mbar_wait_or_abort(bar(&ctrl->o_full[wg]), 0, spin, abort));
      if (!done) give_up();
    }
    const bool partial = a.num_splits > 1;
    if (has_rows && done) {
      tc_fence_after();
      const float vs = a.v_head_scale != nullptr ? a.v_head_scale[h] : a.v_scale;
      const float mul = partial || l != l ? 1.f : l > 0.f ? vs / l : 0.f;
      uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
      const bool bad = nk > 0 && ctrl->bad_hi >= 0;
      if (bad && mine) find_not_finite<C>(a, span, seq, h, pos, ctrl->bad_lo, ctrl->bad_hi, hi, lo);
      __syncwarp();
      const size_t ws_row = ((static_cast<size_t>(split) * a.tiles + tile_id) * a.num_kv_heads + h) * C::ROWS + tid;
      if (partial && mine) *reinterpret_cast<float2*>(a.ws_ml + 2 * ws_row) = make_float2(m, l);
      // The rows, a thread each, pass through the operand stages, which no product
      // reads any more (16-byte chunks permuted by the row), to be stored whole.
      const uint32_t mine_s = base + C::K + wg * (128 * D * 4) + (warp & 3) * (32 * D * 4);
      const int rows = min(R1 - (R0 + 32 * warp), 32);
      if (partial) {  // float32, a warp a row
#pragma unroll 1
        for (int c = 0; nk > 0 && c < D; c += 32) {
          uint32_t o[32];
          result_columns(o, o_addr, c, l, 1.f, hi[c / 32], lo[c / 32]);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sts128(mine_s + lane * (D * 4) + (((c / 4 + k) ^ (lane & 7)) << 4), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        __syncwarp();
        constexpr int LPR = D / 4, RPI = 32 / LPR;
        const int sub = lane % LPR;
#pragma unroll 4
        for (int d = lane / LPR; nk > 0 && d < rows; d += RPI)
          *reinterpret_cast<uint4*>(a.ws_out + (ws_row - lane + d) * D + 4 * sub) =
              ldsv4(mine_s + d * (D * 4) + ((sub ^ (d & 7)) << 4));
      } else {  // bf16, D/8 lanes a row
        const uint32_t row_s = mine_s + lane * (D * 2);
        if (nk == 0) {
#pragma unroll 1
          for (int q = 0; q < D / 8; ++q) sts128(row_s + (q << 4), 0u, 0u, 0u, 0u);
        } else if (a.kvarn) {
          uint32_t w[D];
#pragma unroll
          for (int c = 0; c < D; c += 32) tmem_ld32(w + c, o_addr + c);
          tmem_wait_ld32(w);
#pragma unroll
          for (int c = 32; c < D; c += 32) tmem_waited32(w + c);
          float x[D];
#pragma unroll
          for (int e = 0; e < D; ++e) x[e] = __uint_as_float(w[e]);
          fwht_row<D>(x);
          const float f = hi[0] ? NAN : l == 0.f ? 0.f : a.cR * (l != l ? l : mul);
#pragma unroll
          for (int q = 0; q < D / 8; ++q) {
            const uint4 m = ldsv4(base + C::SIGNS + 16 * q);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u = x[8 * q + 2 * e] * f, v = x[8 * q + 2 * e + 1] * f;
              o[e] = pack_bf162(u, v);
            }
            if (l == 0.f) o[0] = o[1] = o[2] = o[3] = 0u;
            sts128(row_s + ((q ^ (lane & 7)) << 4), o[0] ^ m.x, o[1] ^ m.y, o[2] ^ m.z, o[3] ^ m.w);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            result_columns(o, o_addr, c, l, mul, hi[c / 32], lo[c / 32]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[e] = pack_bf162(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1]));
              sts128(row_s + (((c / 8 + k) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
            }
          }
        }
        __syncwarp();
        constexpr int LPR = D / 8, RPI = 32 / LPR;
        const int sub = lane % LPR;
#pragma unroll 4
        for (int d = lane / LPR; d < rows; d += RPI)
          *reinterpret_cast<uint4*>(a.out + map(d) * D + 8 * sub) = ldsv4(mine_s + d * (D * 2) + ((sub ^ (d & 7)) << 4));
      }
    }
  } else if (!STAGED && wg < NW + 2) {
    // ================= producers =================
    reg_give<C::R_PRODUCE>();
    if (nk > 0) {
      const int bs = 1 << a.block_shift;
      const bool is_v = wg == NW + 1;
      const Source src = is_v ? make_source(a.v_cache, a.v_meta, a.v_fmt, a.kvarn, D, a.num_kv_heads, h, bs, C::BLOCK)
                              : make_source(a.k_cache, a.k_meta, a.k_fmt, a.kvarn, D, a.num_kv_heads, h, bs, C::BLOCK);
      const Source v_src = BLOCK && !is_v ? make_source(a.v_cache, a.v_meta, a.v_fmt, a.kvarn, D, a.num_kv_heads, h, bs, true) : src;
      const Producer<C> pr{a, span, base, tid & 127, seq};
      const uint32_t operand = base + (is_v ? C::V : C::K);
      unsigned long long* full = is_v ? ctrl->v_full : ctrl->k_full;
      unsigned long long* empty = is_v ? ctrl->v_empty : ctrl->k_empty;
      // 16-bit tiles are copied straight into the operand stages, one ahead
      const int ahead = bf ? 1 : is_v ? C::AHEAD_V : C::AHEAD_K;
      const int slot0 = is_v ? C::AHEAD_K : 0;
      auto wait_empty = [&](int i) {  // the operand stage of tile i: its last reader is done
        if (i < 2) return true;
        const bool ok = mbar_wait_or_abort(bar(empty + (i & 1)), ((i >> 1) + 1) & 1, spin, abort);
        if (__all_sync(0xffffffffu, ok)) return true;
        give_up();
        return false;
      };
      KeyTile next = pr.look_up(i0);
      auto copy_next = [&](int i) {  // tile i's codes, if there is a tile i
        if (i < nk) {
          KeyTile cur = next;
          pr.check(cur);
          if (i + 1 < nk) next = pr.look_up(i0 + i + 1);
          pr.copy(src, cur, slot0 + (ahead == 2 ? i & 1 : 0), operand + (i & 1) * C::TILE);
          if (BLOCK && warp == 4 * NW) pr.copy_scales(src, v_src, cur, scale_slot(i));
        }
        cp_async_commit();
      };
      for (int i = 0; i < ahead; ++i) copy_next(i);
      for (int i = 0; i < nk; ++i) {
        if (ahead == 2) cp_async_wait<1>(); else cp_async_wait<0>();
        bool ok = bf || wait_empty(i);
        if (src.fields > 0) ok = producers_all(is_v, ok);  // and the metadata that other threads copied is there
        if (!ok) break;
        if (BLOCK && warp == 4 * NW) {  // the tile's scales, which this warp's lanes copied
          const uint32_t at = scale_slot(i) + lane * 4;
          bool bad;
          uint32_t x;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
          const float f = lane < kGroups ? key_scale(abs_scale, __uint_as_float(x), bad) : value_scale(__uint_as_float(x), bad);
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(f) : "memory");
          if (lane >= kGroups) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + kGroups * 4), "f"(log2_scale(f)) : "memory");
          if (bad) {
            atomicMin(&ctrl->bad_lo, i0 + i);
            atomicMax(&ctrl->bad_hi, i0 + i);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&ctrl->scales[i % kScaleSlots]));
        }
        const int slot = slot0 + (ahead == 2 ? i & 1 : 0);
        const uint32_t dst = operand + (i & 1) * C::TILE;
        const KeyTile ready{tile_key(span, i0 + i), 0};
        if (is_v) {
          if (pr.template finish<true>(src, ready, slot, dst)) {  // rare
            if (bf) pr.template make_finite<BF16>(dst);
            else if (src.fmt == INT4A) pr.template make_finite<INT4A>(dst);
            else pr.template make_finite<INT8>(dst);
            atomicMin(&ctrl->bad_lo, i0 + i);
            atomicMax(&ctrl->bad_hi, i0 + i);
          }
        } else {
          pr.template finish<false>(src, ready, slot, dst);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(full + (i & 1)));
        if (src.fields > 0) producers_all(is_v, true);  // the slot's metadata is read before its next copy
        if (bf && i + 1 < nk && !wait_empty(i + 1)) break;
        copy_next(i + ahead);
      }
      cp_async_wait<0>();
    }
  } else {
    // ================= products =================
    reg_give<C::R_ISSUE>();
    if constexpr (STAGED) {
      if (warp == kIssuer + 1 && lane == 0 && nk > 0) {
        // K and V tiles from the staged context, a TMA box per 64 columns
        const int rows = a.num_seqs * a.num_kv_heads * a.staged_len;  // of K; V's lie behind
        const int row0 = static_cast<int>(seq_head) * a.staged_len;
        int issued = 0;  // K and V tiles
        bool ok = true;
        for (; ok && issued < 2 * nk; ++issued) {
          const int i = issued >> 1, st = i & 1;
          const bool is_v = issued & 1;
          if (i >= 2) ok = mbar_wait_or_abort(bar(is_v ? &ctrl->v_empty[st] : &ctrl->k_empty[st]), ((i >> 1) + 1) & 1, spin, abort);
          if (!ok) break;
          const uint32_t full = bar(is_v ? &ctrl->v_full[st] : &ctrl->k_full[st]);
          const uint32_t dst = base + (is_v ? C::V : C::K) + st * C::TILE;
          const int y = row0 + tile_key(span, i0 + i) + (is_v ? rows : 0);
          if (BLOCK && !is_v) {
            const uint32_t there = bar(&ctrl->scales[i % kScaleSlots]);
            mbar_arrive_expect(there, kScaleBytes);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(scale_slot(i)),
                         "l"(a.staged_scales + (row0 + tile_key(span, i0 + i)) / kKeys * static_cast<size_t>(3 * kGroups)),
                         "r"(kScaleBytes), "r"(there)
                         : "memory");
          }
          mbar_arrive_expect(full, C::TILE);
#pragma unroll
          for (int g = 0; g < C::GROUPS; ++g)
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                    dst + g * C::GROUP_BYTES),
                "l"(reinterpret_cast<uint64_t>(&map_staged)), "r"(64 * g), "r"(y), "r"(full)
                : "memory");
        }
        if (!ok) give_up();
        // Leave with no copy in flight, whoever gave up: the last of each stage is there.
        for (int t = max(issued - 4, 0); t < issued; ++t)
          mbar_wait(bar((t & 1) ? &ctrl->v_full[t >> 1 & 1] : &ctrl->k_full[t >> 1 & 1]), (t >> 2) & 1, kDrain);
        const int scaled = BLOCK ? (issued + 1) / 2 : 0;
        for (int t = max(scaled - kScaleSlots, 0); t < scaled; ++t)
          mbar_wait(bar(&ctrl->scales[t % kScaleSlots]), (t / kScaleSlots) & 1, kDrain);
      }
      __syncwarp();
    }
    if (warp == kIssuer && nk > 0) {
      // the same in every lane, and known as such
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int tiles = __shfl_sync(0xffffffffu, nk, 0), halves = __shfl_sync(0xffffffffu, nw, 0);
      const uint32_t leader = elect_lane();
      const uint32_t qk_desc = mma_desc(128, kKeys, bf, false), pv_desc = mma_desc(128, D, bf, true);
      const uint64_t q_op = smem_desc(base + C::Q, 16), k_op = smem_desc(base + C::K, 16);
      const uint64_t v_op = smem_desc(base + C::V, C::GROUP_BYTES);
      auto wait = [&](const void* b, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_wait_or_abort(bar(b), parity, spin, abort))) return true;
        give_up();
        return false;
      };
      // test hook: in place of this K tile (-1: none) the products wait for what nothing signals
      const int withheld = static_cast<int>(blockIdx.x) == a.withhold_cta && blockIdx.y == 0 ? a.withhold_tile : -1;
      auto k_there = [&](int i) {
        return i == withheld ? wait(&ctrl->drained, 0) : wait(&ctrl->k_full[i & 1], (i >> 1) & 1);
      };
      auto scores = [&](int w, int buf, int stage) {  // S = Q_w K^T
        const uint64_t qa = q_op + w * (C::TILE >> 4), ka = k_op + stage * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int in_row = (k & 3) * 32;
          mma_ss(leader, tm + C::S(0) + buf * 128, qa + (((k >> 2) * C::Q_GROUP + in_row) >> 4),
                 ka + (((k >> 2) * C::GROUP_BYTES + in_row) >> 4), qk_desc, k > 0);
        }
        tc_commit(leader, bar(&ctrl->s_full[buf]));
      };
      auto values = [&](int w, int buf, int stage, bool add, int k0, int k1) {  // O_w += P V, keys 16 k0 .. 16 k1 - 1
        const uint64_t va = v_op + stage * (C::TILE >> 4);
#pragma unroll
        for (int k = k0; k < k1; ++k)
          mma_ts(leader, tm + C::O(0) + w * 128, tm + C::S(0) + buf * 128 + 8 * k, va + k * (2048 >> 4), pv_desc,
                 add || k > 0);
      };
      // Products run in the order of their issue, so scores that overwrite
      // probabilities only need to be issued behind the products that read them.
      bool ok = wait(&ctrl->q_full, 0) && k_there(0);
      if (ok) {
        tc_fence_after();
        for (int w = 0; w < halves; ++w) scores(w, w, 0);
        tc_commit(leader, bar(&ctrl->k_empty[0]));
        if (NW == 2) ok = wait(&ctrl->v_full[0], 0) && (tiles == 1 || k_there(1));
      }
      for (int i = 0; ok && i < tiles; ++i) {
        const int st = i & 1, ns = (i + 1) & 1;
        if (NW == 1) {  // the next tile's scores, into the other buffer, ahead of this one's probabilities
          if (i + 1 < tiles) {
            ok = k_there(i + 1);
            if (!ok) break;
            tc_fence_after();
            scores(0, ns, ns);
            tc_commit(leader, bar(&ctrl->k_empty[ns]));
          }
          ok = wait(&ctrl->v_full[st], (i >> 1) & 1) && wait(&ctrl->p_full[st], (i >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          values(0, st, st, i > 0, 0, kKeys / 16);
          tc_commit(leader, bar(&ctrl->v_empty[st]));
          if (i + 2 >= tiles) tc_commit(leader, bar(i + 1 < tiles ? &ctrl->pv_done : &ctrl->o_full[0]));
          continue;
        }
        // this tile's V and the next one's K were waited for at the end of the last turn
        for (int w = 0; ok && w < halves; ++w) {
          ok = wait(&ctrl->p_half[w], i & 1);
          if (!ok) break;
          tc_fence_after();
          values(w, w, st, i > 0, 0, kKeys / 32);
          ok = wait(&ctrl->p_full[w], i & 1);
          if (!ok) break;
          tc_fence_after();
          values(w, w, st, true, kKeys / 32, kKeys / 16);
          if (w == halves - 1) tc_commit(leader, bar(&ctrl->v_empty[st]));
          if (i + 1 < tiles) {
            scores(w, w, ns);
            if (w == halves - 1) tc_commit(leader, bar(&ctrl->k_empty[ns]));
          } else {
            tc_commit(leader, bar(&ctrl->o_full[w]));
          }
        }
        if (ok && i + 1 < tiles) ok = wait(&ctrl->v_full[ns], ((i + 1) >> 1) & 1);
        if (ok && i + 2 < tiles) ok = k_there(i + 2);
      }
      // Leave with no product in flight, whoever gave up.
      tc_commit(leader, bar(&ctrl->drained));
      mbar_wait(bar(&ctrl->drained), 0, kDrain);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (nk > 0 && warp == kIssuer) tmem_dealloc(tmem, C::TMEM);
}

// The contexts' rows that some row of the batch sees as 16-bit operands in memory,
// [S, Hkv, staged_len, D] of K and then of V, by whole tiles of 128 keys (rows that
// no one sees are 0; block formats: codes, and their scales apart).  A CTA per (sequence, tile) and kv-head: half its threads K, half V.
// Worth its writes where many row tiles read the same keys.
template <int D, int F, bool KVARN, bool IS_V>
__device__ __forceinline__ bool stage_tile(const PrefillArgs& a, const Source& s, const Span& span, const int* pages,
                                           int t0, uint16_t* dst, int tid) {
  using P = Pieces<F, D>;
  const P p(tid);
  const int mask = (1 << a.block_shift) - 1;
  uint32_t nf = 0;
  bool bad = false;
#pragma unroll 2
  for (int i = 0; i < P::PASSES; ++i) {
    const int row = p.row0 + i * P::STEP, t = t0 + row;
    const bool need = t <= span.p_hi && (t >= span.win || t < a.sinks);
    const unsigned long long blk = static_cast<uint32_t>(pages[row >> a.block_shift]);
    uint32_t o[4 * P::OUT];
    const uint4 w = need ? ldg_stream16(s.codes + blk * s.page_bytes + (row & mask) * s.token_bytes + p.chunk * 16)
                         : make_uint4(0, 0, 0, 0);
    if constexpr (F == BF16) {
      o[0] = w.x;
      o[1] = w.y;
      o[2] = w.z;
      o[3] = w.w;
    } else {
      uint32_t f[3] = {0, 0, 0};
      if (is_asym(F) && need) {
        const __half* m = s.meta + blk * s.meta_page + (row & mask);
#pragma unroll
        for (int k = 0; k < (KVARN ? 3 : 2); ++k) {
          const uint32_t x = __half_as_ushort(m[k << a.block_shift]);
          f[k] = x | x << 16;
        }
      }
      dequantize16<F, KVARN>(w, {f[0], f[1], f[2]}, o);
    }
    if constexpr (IS_V && F != INT8) {
      nf = track_not_finite<F == BF16>(0u, o);
      if (nf & 0x7FFF7FFFu) {
        bad = true;
#pragma unroll
        for (int e = 0; e < 4 * P::OUT; ++e) o[e] = finite_or_zero<F == BF16>(o[e]);
      }
    }
    uint4* to = reinterpret_cast<uint4*>(dst + static_cast<size_t>(row) * D) + p.chunk * P::OUT;
#pragma unroll
    for (int j = 0; j < P::OUT; ++j) to[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  }
  return bad;
}
template <int D, bool IS_V>
__device__ __forceinline__ bool stage_any(const PrefillArgs& a, const Source& s, const Span& span, const int* pages,
                                          int t0, uint16_t* dst, int tid) {
  switch (s.fmt) {
    case INT8:
    case INT8B: return stage_tile<D, INT8, false, IS_V>(a, s, span, pages, t0, dst, tid);
    case E4M3:
    case E4M3B: return stage_tile<D, E4M3, false, IS_V>(a, s, span, pages, t0, dst, tid);
    case E5M2: return stage_tile<D, E5M2, false, IS_V>(a, s, span, pages, t0, dst, tid);
    case INT4A:
      return s.fields == 3 ? stage_tile<D, INT4A, true, IS_V>(a, s, span, pages, t0, dst, tid)
                           : stage_tile<D, INT4A, false, IS_V>(a, s, span, pages, t0, dst, tid);
    case UINT8A:
      return s.fields == 3 ? stage_tile<D, UINT8A, true, IS_V>(a, s, span, pages, t0, dst, tid)
                           : stage_tile<D, UINT8A, false, IS_V>(a, s, span, pages, t0, dst, tid);
    default: return stage_tile<D, BF16, false, IS_V>(a, s, span, pages, t0, dst, tid);
  }
}
template <int D>
__global__ void __launch_bounds__(2 * kProducers) stage_kernel(const __grid_constant__ PrefillArgs a) {
  __shared__ int pages[kKeys / 8];
  const int tiles = a.staged_len / kKeys, tid = threadIdx.x;
  const int seq = blockIdx.x / tiles, tile = blockIdx.x - seq * tiles, h = blockIdx.y, t0 = tile * kKeys;
  bool cut;
  const int q = seq_rows(a, seq, cut).y, n = clamp_int(a.context_lens[seq], 0, a.max_context_len);
  if (q == 0) return;
  const Span span = row_span(a, n, q, 0, q * a.gqa);
  if (t0 > span.p_hi || (t0 + kKeys <= span.win && t0 >= a.sinks)) return;  // no one reads it
  const int bs = 1 << a.block_shift;
  if (tid < (kKeys >> a.block_shift)) {
    const int t = t0 + tid * bs;
    int blk = 0;
    if (t <= span.p_hi && (t + bs > span.win || t < a.sinks)) {
      blk = a.block_table[static_cast<size_t>(seq) * a.max_blocks_per_seq + (t >> a.block_shift)];
      if (blk < 0 || blk >= a.num_blocks) {
        raise_error(2u);  // KVQ_DEVERR_BLOCK_RANGE: block 0 is read instead
        blk = 0;
      }
    }
    pages[tid] = blk;
  }
  __syncthreads();
  const size_t seq_head = static_cast<size_t>(seq) * a.num_kv_heads + h;
  const bool is_v = tid >= kProducers;
  const size_t row = (is_v ? static_cast<size_t>(a.num_seqs) * a.num_kv_heads * a.staged_len : 0) + seq_head * a.staged_len + t0;
  const Source s = is_v ? make_source(a.v_cache, a.v_meta, a.v_fmt, a.kvarn, D, a.num_kv_heads, h, bs, is_block(a.v_fmt))
                        : make_source(a.k_cache, a.k_meta, a.k_fmt, a.kvarn, D, a.num_kv_heads, h, bs, is_block(a.k_fmt));
  uint16_t* dst = a.staged + row * D;
  bool bad = is_v ? stage_any<D, true>(a, s, span, pages, t0, dst, tid & 127)
                  : stage_any<D, false>(a, s, span, pages, t0, dst, tid & 127);
  if (is_block(s.fmt) && (tid & 127) < kGroups) {  // the tile's scales, as the softmax takes them
    const int g = tid & 127;
    const float x = group_needed(a, span, t0 + 8 * g)
                        ? reinterpret_cast<const float*>(s.meta)[static_cast<size_t>(pages[(8 * g) >> a.block_shift]) * s.meta_page]
                        : 0.f;
    float* const to = a.staged_scales + (seq_head * tiles + tile) * (3 * kGroups) + g;
    bool odd;
    if (is_v) {
      const float v = value_scale(x, odd);
      to[kGroups] = v;
      to[2 * kGroups] = log2_scale(v);
    } else {
      to[0] = key_scale(a.sm_scale_log2 == 0.f ? 1.f : fabsf(a.sm_scale_log2), x, odd);
    }
    bad |= odd;
  }
  const int any = __syncthreads_or(bad);
  if (tid == 0) a.staged_bad[seq_head * tiles + tile] = any != 0;
}

// Joins the splits' partial results: out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
// A warp per row, D/32 consecutive elements per lane.
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillArgs a, int rows_per_tile) {
  __shared__ Ctrl ctrl;
  __shared__ __align__(8) int scan[2 * kOrdered];
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, h = blockIdx.x % a.num_kv_heads, tile_id = blockIdx.x / a.num_kv_heads;
  if (rows_per_tile == 64) find_tile<64>(a, &ctrl, scan, tile_id);
  else if (rows_per_tile == 128) find_tile<128>(a, &ctrl, scan, tile_id);
  else find_tile<256>(a, &ctrl, scan, tile_id);
  __syncthreads();
  if (ctrl.seq < 0) return;
  const int R0 = ctrl.tile * rows_per_tile, R1 = min(ctrl.q * a.gqa, R0 + rows_per_tile);
  const float vs = a.v_head_scale != nullptr ? a.v_head_scale[h] : a.v_scale;
  for (int r = R0 + (threadIdx.x >> 5); r < R1; r += blockDim.x >> 5) {
    const size_t step = static_cast<size_t>(a.tiles) * a.num_kv_heads * rows_per_tile;
    const size_t row0 = (static_cast<size_t>(tile_id) * a.num_kv_heads + h) * rows_per_tile + (r - R0);
    float M = -INFINITY;
    for (int i = 0; i < a.num_splits; ++i) M = fmaxf(M, a.ws_ml[2 * (row0 + i * step)]);
    float L = 0.f, x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    for (int i = 0; i < a.num_splits; ++i) {
      const float2 ml = *reinterpret_cast<const float2*>(a.ws_ml + 2 * (row0 + i * step));
      if (ml.y == 0.f) continue;  // saw nothing
      const float w = fast_exp2(ml.x - M);
      L += w * ml.y;
      const float* src = a.ws_out + (row0 + i * step) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] += w * src[e];
    }
    const float mul = L == 0.f ? 0.f : vs / L;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = L == 0.f ? 0.f : x[e] * mul;
    if (a.kvarn) {
      fwht_lanes<E, 32>(x, lane);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] *= a.cR;
        if (a.signs != nullptr && a.signs[lane * E + e] < 0) x[e] = -x[e];
      }
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(
        a.out + ((static_cast<size_t>(ctrl.q0) + r / a.gqa) * a.num_q_heads + static_cast<size_t>(h) * a.gqa + r % a.gqa) * D +
        lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf162(x[e], x[e + 1]);
  }
}

template <int D, int ROWS, bool STAGED, bool BLOCK>
cudaError_t launch_t(const PrefillArgs& a, cudaStream_t st) {
  using C = Cfg<D, ROWS, STAGED, BLOCK>;
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(prefill_kernel<D, ROWS, STAGED, BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  if constexpr (STAGED) {
    const size_t rows = 2 * static_cast<size_t>(a.num_seqs) * a.num_kv_heads * a.staged_len;
    const cuuint64_t dims[2] = {cuuint64_t(D), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(D) * 2};
    const cuuint32_t box[2] = {64, kKeys}, estr[2] = {1, 1};
    if (tensor_map_encoder() == nullptr ||
        tensor_map_encoder()(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.staged, dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    stage_kernel<D><<<dim3(static_cast<unsigned>(a.num_seqs) * (a.staged_len / kKeys), a.num_kv_heads, 1),
                      2 * kProducers, 0, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(a.tiles) * a.num_kv_heads, a.num_splits, 1);
  prefill_kernel<D, ROWS, STAGED, BLOCK><<<grid, C::THREADS, C::SMEM, st>>>(a, map);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.num_splits == 1) return e;
  prefill_join_kernel<D><<<grid.x, 256, 0, st>>>(a, C::ROWS);
  return cudaGetLastError();
}

template <int D, bool BLOCK>
cudaError_t launch_rows(const PrefillArgs& a, cudaStream_t st) {
  if (a.rows_per_tile == 64) return launch_t<D, 64, false, BLOCK>(a, st);
  if (a.rows_per_tile == 128) return launch_t<D, 128, false, BLOCK>(a, st);
  return launch_t<D, 256, false, BLOCK>(a, st);
}
template <int D>
cudaError_t launch_d(const PrefillArgs& a, cudaStream_t st) {
  const bool block = is_block(a.v_fmt);
  if (a.staged != nullptr) return block ? launch_t<D, 256, true, true>(a, st) : launch_t<D, 256, true, false>(a, st);
  return block ? launch_rows<D, true>(a, st) : launch_rows<D, false>(a, st);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, int head_dim, cudaStream_t st) {
  if (head_dim == 64) return launch_d<64>(a, st);
  if (head_dim == 128) return launch_d<128>(a, st);
  return cudaErrorNotSupported;
}

}  // namespace kvq

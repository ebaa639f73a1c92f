// Norm and rotation of queries and keys, each head a row, with or without the
// keys' and values' store into the paged cache (kvq_norm_rope, kvq_norm_rope_write).
//
// A row x of D values becomes
//   y = x / sqrt(mean(x^2) + eps) * (w + offset)      (where weights are given)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)
// over the pairs (a, b) of its first r elements: (i, i + r/2) or (2i, 2i + 1),
// with cos and sin of the token's position from a table; computed in float32
// and rounded once, to bf16.  The store quantizes that bf16 row, so its codes
// are those kvq_write_cache makes of the same row.
//
// Work split: a row is held by D/8 lanes.  With split pairs a lane below r/8 holds
// elements 4i..4i+3 and their partners r/2 + 4i.., so both of a pair meet in a
// lane without a shuffle; with interleaved ones, and behind the rotated part, it
// holds 8 consecutive elements.  The weights are multiplied into the pair's cos
// and sin once per warp (they are the same for every head), which leaves, per row,
//   y_a = (x_a (w_a cos) - x_b (w_b sin)) / rms,  y_b = (x_b (w_b cos) + x_a (w_a sin)) / rms
// on packed float32 pairs.  A warp takes kRopeRows row groups of one kind (queries,
// keys or values) of one token, all loaded before any is worked on.  HBM-bound on
// large batches: every row is read and written once, the table's 4r bytes per
// token come from L2 after the first warp.  16,384 tokens of 32 / 8 heads of 128
// into an FP8 cache, 378 MB: 77 us, 72 % of the copy rate (99 us with a shuffle per
// element for the partner and 8 elements a lane in a row; rows in two to eight
// batches per warp, which spares loads of turns and weights: 74 to 82).  64 tokens
// without a cache: 2.4 us.
#pragma once

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "quant_row.cuh"

namespace kvq {

constexpr int kRopeWarps = 4;  // warps per CTA, of neighbouring tokens
constexpr int kRopeRows = 4;   // row groups (256 / D rows each) per warp

// Bytes that another lane of this kernel may overwrite once they are read
// (outputs in place of inputs): plain loads, not the read-only path.
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Where a lane's elements lie in a row, and which of them are a pair: pair m is
// (a[m], b[m]).  Split: a is the first four elements, b the second four.
// Otherwise a and b are the even and odd ones of 8 consecutive elements.
struct LaneRow {
  int first, second;  // offsets of its two runs of four elements
  bool split;         // its pairs are (run 0, run 1)
  bool turned;        // it lies in the rotated part
};
__device__ __forceinline__ LaneRow lane_row(int sub, int rot, bool interleaved) {
  LaneRow r;
  r.turned = 8 * sub < rot;
  r.split = r.turned && !interleaved;
  r.first = r.split ? 4 * sub : 8 * sub;
  r.second = r.split ? rot / 2 + 4 * sub : 8 * sub + 4;
  return r;
}
__device__ __forceinline__ void to_pairs(const uint2& u, const uint2& v, bool split, float (&a)[4], float (&b)[4]) {
  const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float sa = (m & 1) ? bf16_hi(w[m / 2]) : bf16_lo(w[m / 2]);
    const float sb = (m & 1) ? bf16_hi(w[2 + m / 2]) : bf16_lo(w[2 + m / 2]);
    a[m] = split ? sa : bf16_lo(w[m]);
    b[m] = split ? sb : bf16_hi(w[m]);
  }
}

// What a warp multiplies its rows' pairs with.
struct Turns {
  float ca[4], sa[4], cb[4], sb[4];  // w_a cos, w_a sin, w_b cos, w_b sin
};

// One row's pairs, normalised and turned.  Lanes behind the rotated part (only with
// partly) keep their elements apart from their neighbours': 0 times an infinity
// would not be 0.
template <int D>
__device__ __forceinline__ void norm_rope_row(float (&a)[4], float (&b)[4], const Turns& t, bool norm, float eps,
                                              bool partly, bool turned) {
  constexpr int LPR = D / 8;
  float inv = 1.0f;
  if (norm) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int m = 0; m < 4; m += 2) {
      fma2(s0, s1, a[m], a[m + 1], a[m], a[m + 1], s0, s1);
      fma2(s0, s1, b[m], b[m + 1], b[m], b[m + 1], s0, s1);
    }
    float sq = s0 + s1;
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    inv = rsqrtf(fmaf(sq, 1.0f / D, eps));
  }
#pragma unroll
  for (int m = 0; m < 4; m += 2) {
    float a0 = a[m], a1 = a[m + 1], b0 = b[m], b1 = b[m + 1];  // what the partners get
    if (partly && !turned) a0 = a1 = b0 = b1 = 0.f;
    float p0, p1, q0, q1;
    mul2(p0, p1, b0, b1, -t.sb[m], -t.sb[m + 1]);
    mul2(q0, q1, a0, a1, t.sa[m], t.sa[m + 1]);
    fma2(p0, p1, a[m], a[m + 1], t.ca[m], t.ca[m + 1], p0, p1);
    fma2(q0, q1, b[m], b[m + 1], t.cb[m], t.cb[m + 1], q0, q1);
    mul2(a[m], a[m + 1], p0, p1, inv, inv);
    mul2(b[m], b[m + 1], q0, q1, inv, inv);
  }
}

// The pairs as bf16 words of the lane's two runs.
__device__ __forceinline__ uint4 from_pairs(const float (&a)[4], const float (&b)[4], bool split) {
  return split ? make_uint4(pack2_bf16(a[0], a[1]), pack2_bf16(a[2], a[3]), pack2_bf16(b[0], b[1]), pack2_bf16(b[2], b[3]))
               : make_uint4(pack2_bf16(a[0], b[0]), pack2_bf16(a[1], b[1]), pack2_bf16(a[2], b[2]), pack2_bf16(a[3], b[3]));
}

// Rows of split lanes back to 8 consecutive elements a lane (the order of the
// cache write): elements 8i.. of the first half are the first runs of lanes 2i
// and 2i + 1, those of the second half their second runs.
__device__ __forceinline__ uint4 consecutive(const uint4& w, int sub, int rot, int lane) {
  const int lanes = rot / 8;              // that hold split pairs
  const bool upper = 8 * sub >= rot / 2;  // wants second runs
  const int from = sub < lanes ? lane - sub + 2 * (sub - (upper ? lanes / 2 : 0)) : lane;
  uint4 r;
  const uint32_t x0 = __shfl_sync(0xffffffffu, w.x, from), x1 = __shfl_sync(0xffffffffu, w.y, from);
  const uint32_t z0 = __shfl_sync(0xffffffffu, w.z, from), z1 = __shfl_sync(0xffffffffu, w.w, from);
  const int next = sub < lanes ? from + 1 : lane;
  const uint32_t y0 = __shfl_sync(0xffffffffu, w.x, next), y1 = __shfl_sync(0xffffffffu, w.y, next);
  const uint32_t u0 = __shfl_sync(0xffffffffu, w.z, next), u1 = __shfl_sync(0xffffffffu, w.w, next);
  r.x = upper ? z0 : x0;
  r.y = upper ? z1 : x1;
  r.z = upper ? u0 : y0;
  r.w = upper ? u1 : y1;
  return sub < lanes ? r : w;
}

// WRITE: keys and values are quantized into the cache (formats KF, VF); else
// the keys go to key_out and there are no values.  Grid: (tokens / warps, warps
// per token).
template <int D, bool WRITE, int KF, int VF, bool KVARN>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, ROWS = RPI * kRopeRows;
  const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  if (t >= a.num_tokens) return;
  int piece = blockIdx.y;
  // queries first, then keys, then values
  const int kind = piece < a.q_items ? 0 : piece < a.q_items + a.kv_items ? 1 : 2;
  piece -= kind == 0 ? 0 : kind == 1 ? a.q_items : a.q_items + a.kv_items;
  const int heads = kind == 0 ? a.num_q_heads : a.num_kv_heads;
  const int h0 = piece * ROWS;

  const int rot = a.rot_dim;
  const bool interleaved = a.interleaved != 0;
  LaneRow at = lane_row(sub, rot, interleaved);
  if (kind == 2) at = lane_row(sub, 0, true);
  const uint16_t* src = kind == 0 ? a.query + t * a.query_stride
                        : kind == 1 ? a.key + t * a.key_stride : a.value + t * a.value_stride;
  uint2 r0[kRopeRows], r1[kRopeRows];
#pragma unroll
  for (int u = 0; u < kRopeRows; ++u) {
    const int h = h0 + u * RPI + grp;
    const uint16_t* p = src + static_cast<int64_t>(h) * D;
    r0[u] = h < heads ? ld_stream8(p + at.first) : make_uint2(0, 0);
    r1[u] = h < heads ? ld_stream8(p + at.second) : make_uint2(0, 0);
  }
  int pos = 0;
  if (rot > 0) {
    pos = a.positions[t];
    if (pos < 0 || pos >= a.num_positions) {
      if (lane == 0) raise_error(512u);  // KVQ_DEVERR_POSITION: nothing of the token is written
      return;
    }
  }
  Turns turns;
  bool norm = false;
  if (kind != 2) {
    float c[4], s[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      c[m] = 1.f;
      s[m] = 0.f;
    }
    if (at.turned) {  // four pairs: 4 sub on, in either layout
      const float4* p = reinterpret_cast<const float4*>(a.table + static_cast<int64_t>(pos) * rot + 8 * sub);
      const float4 x = __ldg(p), y = __ldg(p + 1);
      c[0] = x.x; s[0] = x.y; c[1] = x.z; s[1] = x.w;
      c[2] = y.x; s[2] = y.y; c[3] = y.z; s[3] = y.w;
    }
    const uint16_t* weight = kind == 0 ? a.q_weight : a.k_weight;
    norm = weight != nullptr;
    float wa[4], wb[4];
    if (norm) {
      to_pairs(__ldg(reinterpret_cast<const uint2*>(weight + at.first)),
               __ldg(reinterpret_cast<const uint2*>(weight + at.second)), at.split, wa, wb);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        wa[m] += a.weight_offset;
        wb[m] += a.weight_offset;
      }
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) wa[m] = wb[m] = 1.f;
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      turns.ca[m] = wa[m] * c[m];
      turns.sa[m] = wa[m] * s[m];
      turns.cb[m] = wb[m] * c[m];
      turns.sb[m] = wb[m] * s[m];
    }
  }
  const bool partly = rot < D;

  if (!WRITE || kind == 0) {
    uint16_t* dst = kind == 0 ? a.query_out + t * a.query_out_stride : a.key_out + t * a.key_out_stride;
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      if (h0 + u * RPI >= heads) break;
      const int h = h0 + u * RPI + grp;
      float x[4], y[4];
      to_pairs(r0[u], r1[u], at.split, x, y);
      norm_rope_row<D>(x, y, turns, norm, a.eps, partly, at.turned);
      const uint4 w = from_pairs(x, y, at.split);
      if (h < heads) {
        uint16_t* p = dst + static_cast<int64_t>(h) * D;
        *reinterpret_cast<uint2*>(p + at.first) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2*>(p + at.second) = make_uint2(w.z, w.w);
      }
    }
    return;
  }
  if constexpr (WRITE) {
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0) return;
    if (slot >= static_cast<int64_t>(a.num_blocks) * a.block_size) {
      if (lane == 0) raise_error(1u);  // KVQ_DEVERR_SLOT_RANGE
      return;
    }
    const int64_t blk = slot >> a.block_shift;
    const int off = static_cast<int>(slot & (a.block_size - 1));
    const size_t row0 = (static_cast<size_t>(blk) * a.block_size + off) * a.num_kv_heads;
    uint32_t sign_bits = 0;
    if constexpr (KVARN) {
      if (a.signs != nullptr) {
        const uint2 sg = *reinterpret_cast<const uint2*>(a.signs + sub * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t byte = ((i < 4 ? sg.x : sg.y) >> (8 * (i & 3))) & 0xFFu;
          sign_bits |= (byte & 0x80u) ? (1u << i) : 0u;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      if (h0 + u * RPI >= heads) break;
      const int h = h0 + u * RPI + grp;
      const bool act = h < heads;
      float x[8];
      if (kind == 1) {
        float p[4], q[4];
        to_pairs(r0[u], r1[u], at.split, p, q);
        norm_rope_row<D>(p, q, turns, norm, a.eps, partly, at.turned);
        uint4 w = from_pairs(p, q, at.split);  // the key's one rounding
        if (!interleaved && rot > 0) w = consecutive(w, sub, rot, lane);
        unpack8(w, x);
        const float inv = a.k_head_scale != nullptr && act ? __frcp_rn(a.k_head_scale[h]) : a.k_inv;
        quantize_store<D, KF, KVARN>(x, act, h, sub, row0 + h, a.k_cache, a.k_meta, inv, blk, off,
                                     a.num_kv_heads, a.block_size, sign_bits, a.cR);
      } else {
        unpack8(make_uint4(r0[u].x, r0[u].y, r1[u].x, r1[u].y), x);
        const float inv = a.v_head_scale != nullptr && act ? __frcp_rn(a.v_head_scale[h]) : a.v_inv;
        quantize_store<D, VF, KVARN>(x, act, h, sub, row0 + h, a.v_cache, a.v_meta, inv, blk, off,
                                     a.num_kv_heads, a.block_size, sign_bits, a.cR);
      }
    }
  }
}

template <int D, bool WRITE, int KF, int VF, bool KVARN>
cudaError_t launch_norm_rope_t(NormRopeArgs a, cudaStream_t st) {
  constexpr int ROWS = 256 / D * kRopeRows;
  a.q_items = (a.num_q_heads + ROWS - 1) / ROWS;
  a.kv_items = (a.num_kv_heads + ROWS - 1) / ROWS;
  const int pieces = a.q_items + (WRITE ? 2 : 1) * a.kv_items;
  const int64_t blocks = (a.num_tokens + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7fffffffll || pieces > 65535) return cudaErrorNotSupported;
  norm_rope_kernel<D, WRITE, KF, VF, KVARN>
      <<<dim3(static_cast<unsigned>(blocks), pieces, 1), kRopeWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq

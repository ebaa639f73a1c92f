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
// Work split: a row is held by D/8 lanes, 8 consecutive elements (16 bytes)
// each; a warp takes kRows row groups of one kind (queries, keys or values) of
// one token, all loaded before any is worked on.  The pairs' table entries are
// the same for every head, so a warp loads them once.  In the split layout the
// partner of a lane's elements sits r/16 lanes away at the same place in that
// lane, one shuffle per element; interleaved pairs are a lane's own.  HBM-bound
// on large batches: every row is read and written once, the table's 4r bytes
// per token come from L2 after the first warp.
#pragma once

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "quant_row.cuh"

namespace kvq {

constexpr int kRopeWarps = 4;  // warps per CTA
constexpr int kRopeRows = 4;   // row groups (256 / D rows each) per warp

// 16 bytes that another lane of this kernel may overwrite once they are read
// (outputs in place of inputs): a plain load, not the read-only path.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of the pairs that this lane's 8 elements belong to: with split
// pairs element e turns by (c[e], s[e]), with interleaved ones elements 2m and
// 2m + 1 by (c[m], s[m]).
struct LaneTurns {
  float c[8], s[8];
};

__device__ __forceinline__ void load_turns(LaneTurns& t, const float* row, int first, int n) {
  const float4* p = reinterpret_cast<const float4*>(row + 2 * first);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (2 * i < n) {
      const float4 v = __ldg(p + i);
      t.c[2 * i] = v.x;
      t.s[2 * i] = v.y;
      t.c[2 * i + 1] = v.z;
      t.s[2 * i + 1] = v.w;
    }
  }
}

template <int D>
__device__ __forceinline__ void norm_rope_row(float (&x)[8], int sub, const float (&w)[8], bool norm,
                                              float eps, const LaneTurns& t, int rot, bool interleaved) {
  constexpr int LPR = D / 8;
  if (norm) {
    float sq = x[0] * x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float inv = rsqrtf(fmaf(sq, 1.0f / D, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
  }
  if (rot == 0) return;
  const bool turned = 8 * sub < rot;
  if (interleaved) {
    if (turned) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float a = x[2 * m], b = x[2 * m + 1];
        x[2 * m] = a * t.c[m] - b * t.s[m];
        x[2 * m + 1] = b * t.c[m] + a * t.s[m];
      }
    }
  } else {
    const int half = rot >> 4;  // lanes of each half
    const bool upper = sub >= half;
    const int partner = (threadIdx.x & 31) + (turned ? (upper ? -half : half) : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, x[i], partner);
      if (turned) x[i] = x[i] * t.c[i] + (upper ? other : -other) * t.s[i];
    }
  }
}

// WRITE: keys and values are quantized into the cache (formats KF, VF); else
// the keys go to key_out and there are no values.
template <int D, bool WRITE, int KF, int VF, bool KVARN>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, ROWS = RPI * kRopeRows;
  const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t t = item / a.items_per_token;
  if (t >= a.num_tokens) return;
  int piece = static_cast<int>(item - t * a.items_per_token);
  // queries first, then keys, then values
  const int kind = piece < a.q_items ? 0 : piece < a.q_items + a.kv_items ? 1 : 2;
  piece -= kind == 0 ? 0 : kind == 1 ? a.q_items : a.q_items + a.kv_items;
  const int heads = kind == 0 ? a.num_q_heads : a.num_kv_heads;
  const int h0 = piece * ROWS;

  const int rot = a.rot_dim;
  const bool interleaved = a.interleaved != 0;
  int pos = 0;
  if (rot > 0) {
    pos = a.positions[t];
    if (pos < 0 || pos >= a.num_positions) {
      if (lane == 0) raise_error(512u);  // KVQ_DEVERR_POSITION: nothing of the token is written
      return;
    }
  }
  const uint16_t* src = kind == 0 ? a.query + t * a.query_stride
                        : kind == 1 ? a.key + t * a.key_stride : a.value + t * a.value_stride;
  uint4 raw[kRopeRows];
#pragma unroll
  for (int u = 0; u < kRopeRows; ++u) {
    const int h = h0 + u * RPI + grp;
    raw[u] = h < heads ? ld_stream16(src + static_cast<int64_t>(h) * D + sub * 8) : make_uint4(0, 0, 0, 0);
  }
  LaneTurns turns;
#pragma unroll
  for (int i = 0; i < 8; ++i) turns.c[i] = turns.s[i] = 0.f;
  float w[8];
  bool norm = false;
  if (kind != 2) {
    if (rot > 0 && 8 * sub < rot) {
      const float* row = a.table + static_cast<int64_t>(pos) * rot;
      if (interleaved) load_turns(turns, row, 4 * sub, 4);
      else load_turns(turns, row, (8 * sub) % (rot / 2), 8);
    }
    const uint16_t* weight = kind == 0 ? a.q_weight : a.k_weight;
    norm = weight != nullptr;
    if (norm) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(weight + sub * 8)), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] += a.weight_offset;
    }
  }
  if (!norm) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  }

  if (!WRITE || kind == 0) {
    uint16_t* dst = kind == 0 ? a.query_out + t * a.query_out_stride : a.key_out + t * a.key_out_stride;
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      if (h0 + u * RPI >= heads) break;
      const int h = h0 + u * RPI + grp;
      float x[8];
      unpack8(raw[u], x);
      norm_rope_row<D>(x, sub, w, norm, a.eps, turns, rot, interleaved);
      if (h < heads) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(h) * D + sub * 8) = pack8_bf16(x);
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
      unpack8(raw[u], x);
      if (kind == 1) {
        norm_rope_row<D>(x, sub, w, norm, a.eps, turns, rot, interleaved);
        unpack8(pack8_bf16(x), x);  // the key's one rounding
        const float inv = a.k_head_scale != nullptr && act ? __frcp_rn(a.k_head_scale[h]) : a.k_inv;
        quantize_store<D, KF, KVARN>(x, act, h, sub, row0 + h, a.k_cache, a.k_meta, inv, blk, off,
                                     a.num_kv_heads, a.block_size, sign_bits, a.cR);
      } else {
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
  a.items_per_token = a.q_items + (WRITE ? 2 : 1) * a.kv_items;
  const int64_t blocks = (a.num_tokens * a.items_per_token + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7fffffffll) return cudaErrorNotSupported;
  norm_rope_kernel<D, WRITE, KF, VF, KVARN>
      <<<static_cast<unsigned>(blocks), kRopeWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq

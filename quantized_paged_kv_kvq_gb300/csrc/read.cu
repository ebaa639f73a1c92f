// Rows of the paged cache as bf16 (kvq_read_cache): the inverse of the cache write,
// for every format.
//
//   symmetric   x = code * scale                     (a tensor's, a head's or a page and head's)
//   asymmetric  x = code * scale + zero point        (fp16 fields of the row)
//   KVarN       x = d . (cR * H ((code * scale + zero point) * sigma))
// in float32, rounded once to bf16.
//
// Mapping: a thread makes 16 consecutive elements of a row (32 bytes, two stores);
// a token's rows of all heads lie behind each other in the cache and in the output,
// so consecutive threads read and write whole lines.  K and V are one launch (grid.y).
// Bound by HBM: D codes read and 2 D bytes written per row.
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "mbarrier.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_read)

namespace {

constexpr int kThreads = 256;

// 16 codes as floats (exact).
template <int F>
__device__ __forceinline__ void codes16(const uint8_t* p, float (&x)[16]) {
  if constexpr (F == INT4A) {
    const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = static_cast<float>((w[i >> 3] >> (4 * (i & 7))) & 15u);
  } else if constexpr (F == BF16) {
    const uint4 r[2] = {ldg_stream16(p), ldg_stream16(p + 16)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = bf16_lo(w[e]);
        x[8 * i + 2 * e + 1] = bf16_hi(w[e]);
      }
    }
  } else {
    const uint4 r = ldg_stream16(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F == INT8) x[4 * i + e] = static_cast<float>(static_cast<int8_t>(w[i] >> (8 * e)));
        else if constexpr (F == UINT8A) x[4 * i + e] = static_cast<float>((w[i] >> (8 * e)) & 0xFFu);
      }
      if constexpr (F == E4M3 || F == E5M2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t h = F == E4M3 ? e4m3x2_to_f16x2((w[i] >> (16 * e)) & 0xFFFFu)
                                       : prmt(w[i], 0u, e ? 0x3424 : 0x1404);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          x[4 * i + 2 * e] = f.x;
          x[4 * i + 2 * e + 1] = f.y;
        }
      }
    }
  }
}

template <int D, int F, bool KVARN>
__device__ __forceinline__ void read_rows(const ReadArgs& a, int which) {
  constexpr int P = D / 16, RB = row_bytes(F, D);  // threads and bytes of a row
  const int Hkv = a.num_kv_heads, per_token = Hkv * P;
  const int64_t total = a.num_tokens * per_token, stride = static_cast<int64_t>(gridDim.x) * kThreads;
  const uint8_t* const codes = a.codes[which];
  const int shift = a.block_shift, mask = (1 << shift) - 1;
  // whole warps take part in every turn: KVarN's lanes exchange values
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads; i0 < total; i0 += stride) {
    const int64_t i = i0 + threadIdx.x;
    const int64_t t = i / per_token;
    const int in_token = static_cast<int>(i - t * per_token), h = in_token / P, part = in_token % P;
    const int64_t slot = i < total ? a.slot_mapping[t] : -1;
    bool read = slot >= 0;
    if (read && (slot >> shift) >= a.num_blocks) {
      if (which == 0) raise_error(1u);  // KVQ_DEVERR_SLOT_RANGE
      read = false;
    }
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
    if (read) {
      const int64_t blk = slot >> shift;
      const int off = static_cast<int>(slot) & mask;
      codes16<code_fmt(F)>(codes + (static_cast<size_t>(slot) * Hkv + h) * RB + part * (RB / P), x);
      if constexpr (is_asym(F)) {
        constexpr int NF = KVARN ? 3 : 2;
        const __half* m = static_cast<const __half*>(a.meta[which]) + ((blk * Hkv + h) * NF << shift) + off;
        const float s = __half2float(m[0]), z = __half2float(m[1 << shift]);
        const float g = KVARN ? __half2float(m[2 << shift]) : 1.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = KVARN ? fmaf(x[e], s, z) * g : fmaf(x[e], s, z);
      } else if constexpr (F != BF16) {
        const float s = is_block(F) ? static_cast<const float*>(a.meta[which])[blk * scale_pitch(Hkv) + h]
                        : a.head_scale[which] != nullptr ? a.head_scale[which][h] : a.scale[which];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= s;
      }
    }
    if constexpr (KVARN) {
      fwht_lanes<16, P>(x, part);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] *= a.cR;
        if (a.signs != nullptr && a.signs[part * 16 + e] < 0) x[e] = -x[e];
      }
    }
    if (read) {
      uint4* const to = reinterpret_cast<uint4*>(a.out[which] + t * a.out_stride[which] + h * D + part * 16);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        to[k] = make_uint4(pack_bf162(x[8 * k], x[8 * k + 1]), pack_bf162(x[8 * k + 2], x[8 * k + 3]),
                           pack_bf162(x[8 * k + 4], x[8 * k + 5]), pack_bf162(x[8 * k + 6], x[8 * k + 7]));
    }
  }
}

template <int D, bool KVARN>
__global__ void __launch_bounds__(kThreads) read_cache_kernel(const ReadArgs a) {
  const int which = blockIdx.y;
  if constexpr (KVARN) {
    if (a.fmt[which] == INT4A) read_rows<D, INT4A, true>(a, which);
    else read_rows<D, UINT8A, true>(a, which);
  } else {
    switch (a.fmt[which]) {
      case INT8: read_rows<D, INT8, false>(a, which); break;
      case E4M3: read_rows<D, E4M3, false>(a, which); break;
      case E5M2: read_rows<D, E5M2, false>(a, which); break;
      case INT4A: read_rows<D, INT4A, false>(a, which); break;
      case UINT8A: read_rows<D, UINT8A, false>(a, which); break;
      case INT8B: read_rows<D, INT8B, false>(a, which); break;
      case E4M3B: read_rows<D, E4M3B, false>(a, which); break;
      default: read_rows<D, BF16, false>(a, which); break;
    }
  }
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, int head_dim, bool kvarn, cudaStream_t st, int num_sms) {
  const int64_t threads = a.num_tokens * a.num_kv_heads * (head_dim / 16);
  const int64_t ctas = (threads + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(ctas < 8ll * num_sms ? ctas : 8ll * num_sms), 2, 1);
  if (head_dim == 64 && kvarn) read_cache_kernel<64, true><<<grid, kThreads, 0, st>>>(a);
  else if (head_dim == 64) read_cache_kernel<64, false><<<grid, kThreads, 0, st>>>(a);
  else if (head_dim == 128 && kvarn) read_cache_kernel<128, true><<<grid, kThreads, 0, st>>>(a);
  else if (head_dim == 128) read_cache_kernel<128, false><<<grid, kThreads, 0, st>>>(a);
  else return cudaErrorNotSupported;
  return cudaGetLastError();
}

}  // namespace kvq

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
// Bound by HBM: D codes read and 2 D bytes written per row (65,536 tokens, 8 heads of 128:
// int8 per page 65 us, 6.2 TB/s; int4 64 us, 5.3).
//
// KVarN: H applies to the codes first, H (code * scale + zero) = scale H code + zero D e_0,
// which are whole numbers and so exact in the tensor cores.  Of the log2 D bits of an
// element's number, a warp's mma.sync m16n8k16 (codes by 16 x 8 of +-1, twice) turns four
// and butterflies within a thread the rest: no value goes from lane to lane.  Codes
// enter as 1024 + code, whose part 1024 D comes off element 0.  131,072 tokens, 8 heads of
// 128, int4 K and uint8 V: 160 us, 4.7 TB/s; with a row over 16 lanes and shuffles 254.
// Bound by loads in flight: a third of the warps that fit, and only a row's slot is loaded a
// turn ahead, its codes and fields are waited for (5.5 stalls an issue).
#include <algorithm>

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

template <int D, int F>
__device__ __forceinline__ void read_rows(const ReadArgs& a, int which) {
  constexpr int P = D / 16, RB = row_bytes(F, D);  // threads and bytes of a row
  const int Hkv = a.num_kv_heads, per_token = Hkv * P;
  const int64_t total = a.num_tokens * per_token, stride = static_cast<int64_t>(gridDim.x) * kThreads;
  const uint8_t* const codes = a.codes[which];
  const int shift = a.block_shift, mask = (1 << shift) - 1;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t t = i / per_token;
    const int in_token = static_cast<int>(i - t * per_token), h = in_token / P, part = in_token % P;
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0) continue;
    if ((slot >> shift) >= a.num_blocks) {
      if (which == 0) raise_error(1u);  // KVQ_DEVERR_SLOT_RANGE
      continue;
    }
    float x[16];
    const int64_t blk = slot >> shift;
    const int off = static_cast<int>(slot) & mask;
    codes16<code_fmt(F)>(codes + (static_cast<size_t>(slot) * Hkv + h) * RB + part * (RB / P), x);
    if constexpr (is_asym(F)) {
      const __half* m = static_cast<const __half*>(a.meta[which]) + ((blk * Hkv + h) * 2 << shift) + off;
      const float s = __half2float(m[0]), z = __half2float(m[1 << shift]);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], s, z);
    } else if constexpr (F != BF16) {
      const float s = is_block(F) ? static_cast<const float*>(a.meta[which])[blk * scale_pitch(Hkv) + h]
                      : a.head_scale[which] != nullptr ? a.head_scale[which][h] : a.scale[which];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= s;
    }
    uint4* const to = reinterpret_cast<uint4*>(a.out[which] + t * a.out_stride[which] + h * D + part * 16);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      to[k] = make_uint4(pack_bf162(x[8 * k], x[8 * k + 1]), pack_bf162(x[8 * k + 2], x[8 * k + 3]),
                         pack_bf162(x[8 * k + 4], x[8 * k + 5]), pack_bf162(x[8 * k + 6], x[8 * k + 7]));
  }
}

// Rotated rows: a warp takes 8 consecutive tokens of a kv-head, lanes (g, c) row g's D / 4
// consecutive elements from c D / 4 on.  The bits of an element's number within a lane:
// two are the k-slots' (uint8: b0, b1 of 4 consecutive codes; int4: b2, b0, as a mask takes
// nibbles 4 apart out of a word together), the others number the blocks j, two of which
// make the rows g and g + 8 of a product; c is the k-slots' other two.
// 32 bytes, 32-byte aligned: a whole sector by one thread.
__device__ __forceinline__ void store_sector(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <int D, int F>
__device__ __forceinline__ void read_rotated(const ReadArgs& a, int which) {
  constexpr int E = D / 4, J = E / 4, W = E * (F == INT4A ? 4 : 8) / 32;  // elements, blocks and words of a lane's row
  constexpr uint32_t K64 = 0x64646464u;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int Hkv = a.num_kv_heads, shift = a.block_shift, mask = (1 << shift) - 1;
  const int64_t warps = (a.num_tokens + 7) / 8 * Hkv;
  // B: +-1 of (k-slot (c, s), column (c', s')), c' = column / 2, s' = column % 2 + 2 t
  uint32_t b[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      auto one = [&](int i) {
        return (__popc(c & (g >> 1)) + __popc((i + 2 * q) & ((g & 1) + 2 * t))) & 1 ? 0xBC00u : 0x3C00u;
      };
      b[t][q] = one(0) | one(1) << 16;
    }
  uint32_t flip[E / 2];  // the diagonal's signs of this lane's elements, as pairs of sign bits
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    flip[e] = 0u;
    if (a.signs != nullptr)
      flip[e] = (a.signs[c * E + 2 * e] < 0 ? 0x8000u : 0u) | (a.signs[c * E + 2 * e + 1] < 0 ? 0x80000000u : 0u);
  }
  const bool sectors = reinterpret_cast<uintptr_t>(a.out[which]) % 32 == 0 && a.out_stride[which] % 16 == 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  auto slot_of = [&](int64_t w) {
    const int64_t t = w / Hkv * 8 + g;
    return w < warps && t < a.num_tokens ? a.slot_mapping[t] : -1;
  };
  int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5), next = slot_of(w);
  for (; w < warps; w += step) {
    const int64_t tile = w / Hkv, t = tile * 8 + g, slot = next;
    const int h = static_cast<int>(w - tile * Hkv);
    next = slot_of(w + step);  // a turn ahead: codes and fields wait for it
    bool read = slot >= 0;
    if (read && (slot >> shift) >= a.num_blocks) {
      if (which == 0) raise_error(1u);  // KVQ_DEVERR_SLOT_RANGE
      read = false;
    }
    uint32_t code[W];
#pragma unroll
    for (int i = 0; i < W; ++i) code[i] = 0;
    float scale = 0.f, zero = 0.f;
    if (read) {
      const uint8_t* p = a.codes[which] + (static_cast<size_t>(slot) * Hkv + h) * row_bytes(F, D) + c * (4 * W);
      if constexpr (W >= 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(p + 4 * i));
          code[i] = x.x;
          code[i + 1] = x.y;
          code[i + 2] = x.z;
          code[i + 3] = x.w;
        }
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        code[0] = x.x;
        code[1] = x.y;
      }
      const __half* m = static_cast<const __half*>(a.meta[which]) + (((slot >> shift) * Hkv + h) * 3 << shift) + (slot & mask);
      const float f = __half2float(__ldg(m + (2 << shift))) * a.cR;
      scale = __half2float(__ldg(m)) * f;
      zero = __half2float(__ldg(m + (1 << shift))) * f;
    }
    float v[J][4];  // [j][s']
#pragma unroll
    for (int j = 0; j < J; j += 2) {
      uint32_t x[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (F == INT4A) {
          const uint32_t n = code[j >> 1] >> (8 * r);  // nibbles 2 r and that + 1, and 4 on
          x[r][0] = and_or(n, 0x000F000Fu, 0x64006400u);
          x[r][1] = and_or(n >> 4, 0x000F000Fu, 0x64006400u);
        } else {
          x[r][0] = prmt(code[j + r], K64, 0x4140);
          x[r][1] = prmt(code[j + r], K64, 0x4342);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(d, x[0][0], x[1][0], x[0][1], x[1][1], b[q][0], b[q][1]);
        v[j][2 * q] = d[0];
        v[j][2 * q + 1] = d[1];
        v[j + 1][2 * q] = d[2];
        v[j + 1][2 * q + 1] = d[3];
      }
    }
#pragma unroll
    for (int bit = 1; bit < J; bit <<= 1)
#pragma unroll
      for (int j = 0; j < J; ++j)
        if ((j & bit) == 0)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float p = v[j][e], q = v[j][e + 1], y = v[j + bit][e], z = v[j + bit][e + 1];
            add2(v[j][e], v[j][e + 1], p, q, y, z);
            sub2(v[j + bit][e], v[j + bit][e + 1], p, q, y, z);
          }
    if (c == 0) v[0][0] -= 1024.f * D;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      mul2(v[j][0], v[j][1], v[j][0], v[j][1], scale, scale);
      mul2(v[j][2], v[j][3], v[j][2], v[j][3], scale, scale);
    }
    if (c == 0) v[0][0] = fmaf(zero, static_cast<float>(D), v[0][0]);
    if (read) {
      uint4* const to = reinterpret_cast<uint4*>(a.out[which] + t * a.out_stride[which] + h * D + c * E);
      // element 8 k + e of the lane: block and s' as the bits say
      auto at = [&](int e) {
        if constexpr (F == INT4A) return v[(e >> 1 & 1) + 2 * (e >> 3)][(e >> 2 & 1) + 2 * (e & 1)];
        else return v[e >> 2][e & 3];
      };
#pragma unroll
      for (int k = 0; k < E / 16; ++k) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_bf162(at(16 * k + 2 * i), at(16 * k + 2 * i + 1)) ^ flip[8 * k + i];
        if (sectors) {
          store_sector(to + 2 * k, o);
        } else {
          to[2 * k] = make_uint4(o[0], o[1], o[2], o[3]);
          to[2 * k + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_cache_kernel(const ReadArgs a) {
  const int which = blockIdx.y;
  switch (a.fmt[which]) {
    case INT8: read_rows<D, INT8>(a, which); break;
    case E4M3: read_rows<D, E4M3>(a, which); break;
    case E5M2: read_rows<D, E5M2>(a, which); break;
    case INT4A: read_rows<D, INT4A>(a, which); break;
    case UINT8A: read_rows<D, UINT8A>(a, which); break;
    case INT8B: read_rows<D, INT8B>(a, which); break;
    case E4M3B: read_rows<D, E4M3B>(a, which); break;
    default: read_rows<D, BF16>(a, which); break;
  }
}
template <int D>
__global__ void __launch_bounds__(kThreads, 3) read_rotated_kernel(const ReadArgs a) {
  const int which = blockIdx.y;
  if (a.fmt[which] == INT4A) read_rotated<D, INT4A>(a, which);
  else read_rotated<D, UINT8A>(a, which);
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, int head_dim, bool kvarn, cudaStream_t st, int num_sms) {
  if (head_dim != 64 && head_dim != 128) return cudaErrorNotSupported;
  const int64_t ctas = kvarn ? ((a.num_tokens + 7) / 8 * a.num_kv_heads + kThreads / 32 - 1) / (kThreads / 32)
                             : (a.num_tokens * a.num_kv_heads * (head_dim / 16) + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ctas, 8ll * num_sms)), 2, 1);
  if (kvarn && head_dim == 64) read_rotated_kernel<64><<<grid, kThreads, 0, st>>>(a);
  else if (kvarn) read_rotated_kernel<128><<<grid, kThreads, 0, st>>>(a);
  else if (head_dim == 64) read_cache_kernel<64><<<grid, kThreads, 0, st>>>(a);
  else read_cache_kernel<128><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq

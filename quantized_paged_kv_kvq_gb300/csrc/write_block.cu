// Quantize-and-scatter into a paged cache whose 8-bit codes have one float32
// scale per (page, kv-head): kvq_write_cache of the block formats, and the store
// that kvq_decode_append makes ahead of its attention.
//
// A run is what consecutive tokens of a call put into one page (skipped tokens between
// them, up to 31 in a row, do not part it).  With m the
// largest finite |x| of a head's rows in it, need = max(m / qmax, 2^-126) (0 for
// m = 0), and
//   scale = need                                 where the run reaches offset 0,
//   scale = old * 2^k, least k >= 0, >= need     else (need, if old is 0),
// codes = rounded x / scale, and with k > 0 the codes in front of the run times
// 2^-k, rounded again.  Growth by powers of two keeps those roundings from adding
// up (errors of s/2, s/4, ...: less than one step of the last scale) and is exact
// for e4m3 above its subnormals.
//
// Mapping: a warp holds 16 rows of a run and head in registers (one 16-byte load a
// lane and row piece: the rows are read once), a page of 16 CH tokens takes CH
// warps, which exchange their maxima through shared memory.  K heads and V heads
// share a CTA.  A CTA looks for the runs that begin among its `step` tokens by
// comparing each token's page with that of the token before it, so the slots alone say
// where runs begin and end: no search over sequences, no atomics.  step grows with the
// call from 1 (a decode step: every request's run starts at once) to a page, at least 32
// tokens (so of small pages a CTA stores several runs, one after the other).  A thread a
// token, the CTA loads the places of the tokens around its own and marks, a bit each, which
// are there, begin a run or follow on the offset before: the warps then only read bits.
// Bound by HBM: 4 D bytes read and 2 D written per token and head (16,384 tokens, 8 heads of
// 128, int8, pages of 16: 20.3 us, 5.0 TB/s; of 64: 28.5 us).  Runs at offsets one after the
// other, marked as such, are stored without a look-up per row (else 22.6 us).  A decode
// step's 64 rows take 4.6 us: places, scales and rows are loaded one after the other.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "quant_row.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_write_block)

namespace {

constexpr int kWarps = 8;
constexpr float kSmallest = 1.17549435e-38f;  // 2^-126: 1 / scale stays finite

constexpr int kBack = 32;  // tokens before its own whose places a CTA keeps, too
// Tokens of a CTA at most, pages having 16 CH (or 8) of them.
constexpr int most_tokens(int ch) { return 16 * ch > 32 ? 16 * ch : 32; }

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// (c << 16) | (sat(a) << 8) | sat(b), sat = clamp to [-128, 127]
__device__ __forceinline__ uint32_t pack_sat_s8(int a, int b, uint32_t c) {
  uint32_t d;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Four bf16 values times inv as code bytes (as quantize_store makes them).
template <int F>
__device__ __forceinline__ uint32_t quantize4(uint32_t lo, uint32_t hi, float inv) {
  float a, b, c, d;
  mul2(a, b, bf16_lo(lo), bf16_hi(lo), inv, inv);
  mul2(c, d, bf16_lo(hi), bf16_hi(hi), inv, inv);
  if constexpr (F == INT8)
    return pack_sat_s8(__float2int_rn(b), __float2int_rn(a), pack_sat_s8(__float2int_rn(d), __float2int_rn(c), 0u));
  else
    return f32x2_to_fp8x2<E4M3>(a, b) | f32x2_to_fp8x2<E4M3>(c, d) << 16;
}

// Code bytes times 2^-k (f), rounded again.
template <int F>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t r = 0;
  if constexpr (F == INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
      r |= (static_cast<uint32_t>(__float2int_rn(c * f)) & 0xFFu) << (8 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = e4m3x2_to_f16x2((w >> (16 * i)) & 0xFFFFu);
      const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h));
      r |= f32x2_to_fp8x2<E4M3>(c.x * f, c.y * f) << (16 * i);
    }
  }
  return r;
}

template <int D, int CH>  // head_dim, warps per run and head
__global__ void __launch_bounds__(kWarps * 32, D == 128 ? 3 : 4) write_block_kernel(const WriteArgs a, const AppendSlots ap, int kf, int vf, int step) {
  constexpr int LPR = RowGeom<D>::LPR, RPI = RowGeom<D>::RPI, NP = 16 / RPI;
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kNear = (CH <= 2 ? 1 : 2) * kWarps * 32;  // tokens whose places the CTA keeps
  static_assert(kBack + most_tokens(CH) <= kNear, "its own tokens' among them");
  __shared__ uint32_t most[2][kWarps];
  __shared__ int front[2][kWarps];
  __shared__ uint32_t is_there[kNear / 32], begins[kNear / 32], goes_on[kNear / 32];
  __shared__ int near_page[kNear];
  __shared__ uint8_t near_off[kNear];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR, grp = lane / LPR, chunk = warp % CH;
  const int Hkv = a.num_kv_heads, bs = a.block_size;
  const int vh = blockIdx.y * (kWarps / CH) + warp / CH;  // K heads, then V heads
  const bool active = vh < 2 * Hkv, is_v = vh >= Hkv;
  const int h = is_v ? vh - Hkv : vh;
  const bool append = a.slot_mapping == nullptr;
  const bool int8 = (is_v ? vf : kf) == INT8B;
  uint8_t* const codes = is_v ? a.v_cache : a.k_cache;
  float* const scales = reinterpret_cast<float*>(is_v ? a.v_meta : a.k_meta);
  const int pitch = scale_pitch(Hkv);
  const uint16_t* const rows = (is_v ? a.value : a.key) + static_cast<size_t>(active ? h : 0) * D + sub * 8;
  const int64_t stride = is_v ? a.value_stride : a.key_stride;
  const int64_t n = a.num_tokens, t_begin = static_cast<int64_t>(blockIdx.x) * step, t_end = min(n, t_begin + step);
  const int64_t near0 = t_begin - kBack;
  int parity = 0;

  // Page and offset of token t: page -1 if it is skipped.
  auto place = [&](int64_t t, bool report) {
    int2 p = make_int2(-1, 0);
    if (append) {
      const int len = min(ap.context_lens[t], ap.max_context_len), pos = len - 1;
      if (len > 0) {
        const int blk = ap.block_table[static_cast<size_t>(t) * ap.max_blocks_per_seq + (pos >> a.block_shift)];
        if (blk >= 0 && blk < a.num_blocks) p = make_int2(blk, pos & (bs - 1));
        else if (report) raise_error(2u);  // KVQ_DEVERR_BLOCK_RANGE: nothing written
      }
      return p;
    }
    const int64_t slot = a.slot_mapping[t];
    if (slot >= 0) {
      if ((slot >> a.block_shift) < a.num_blocks) p = make_int2(static_cast<int>(slot >> a.block_shift), static_cast<int>(slot) & (bs - 1));
      else if (report) raise_error(1u);  // KVQ_DEVERR_SLOT_RANGE
    }
    return p;
  };

  // Its tokens' rows on their way into L2 meanwhile: the rows of this warp's share of the heads.
  for (int64_t r = t_begin + chunk * (32 / (D / 64)) + lane / (D / 64); active && r < t_end; r += CH * (32 / (D / 64)))
    asm volatile("prefetch.global.L2 [%0];" ::"l"(rows - sub * 8 + r * stride + lane % (D / 64) * 64));
  // The places of the tokens from kBack before this CTA's first one on (those behind: looked up
  // when they are asked for).
  for (int i = threadIdx.x; i < kNear; i += kWarps * 32) {
    const int64_t t = near0 + i;
    const bool own = t >= t_begin && t < t_end;
    const int2 p = t >= 0 && t < n && (own || !append) ? place(t, blockIdx.y == 0 && own) : make_int2(-1, 0);
    near_page[i] = p.x;
    near_off[i] = static_cast<uint8_t>(p.y);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kNear; i += kWarps * 32) {
    const int page = near_page[i];
    int before = -1;  // page of the last token before it, at most kBack back
    if (page >= 0 && !append && i >= kBack)
      for (int d = 1; d <= kBack && before < 0; ++d) before = near_page[i - d];
    const uint32_t there = __ballot_sync(kAll, page >= 0), first = __ballot_sync(kAll, page >= 0 && i >= kBack && page != before);
    const uint32_t next = __ballot_sync(kAll, page >= 0 && i > 0 && near_page[max(i - 1, 0)] == page &&
                                                  near_off[max(i - 1, 0)] + 1 == near_off[i]);
    if (lane == 0) {
      is_there[i / 32] = there;
      begins[i / 32] = first;
      goes_on[i / 32] = next;  // the next offset of the page of the token before it
    }
  }
  __syncthreads();
  auto place_of = [&](int64_t t) {  // (-1, 0) outside the call
    const int64_t i = t - near0;
    if (i >= 0 && i < kNear) return make_int2(near_page[i], near_off[i]);
    return t >= 0 && t < n ? place(t, false) : make_int2(-1, 0);
  };

  // The run of `len` tokens from near0 + i0 on in `page` (skipped ones among them).  dense: at
  // offsets one after the other, so that nothing has to be looked up row by row.
  auto store_run = [&](int page, int i0, int64_t len, bool dense) {
    const int64_t t0 = near0 + i0;
    float* const scale_at = scales + static_cast<size_t>(page) * pitch + h;
    const float was = active ? *scale_at : 0.0f;  // means nothing where the page is begun
    uint4 v[NP];
    uint32_t m2 = 0;
    const int off0 = near_off[i0];
    int first = dense ? off0 : bs;  // the foremost offset
    const uint16_t* const row0 = rows + t0 * stride;
    uint32_t off[(NP + 3) / 4];  // offsets of the rows, a byte each, 255: not this thread's, or skipped
    auto load = [&](int64_t r0) {  // rows r0 .. r0 + 15 of the run
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int64_t r = r0 + grp + i * RPI;
        const bool read = active && r < len;
        v[i] = read ? ldg_stream16(row0 + r * stride) : make_uint4(0, 0, 0, 0);
      }
      if (dense) return;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int64_t r = r0 + grp + i * RPI;
        const bool read = active && r < len;
        uint32_t o = 255u;
        if (read) {
          if (i0 + r < kNear) {
            if (near_page[i0 + static_cast<int>(r)] == page) o = near_off[i0 + static_cast<int>(r)];
          } else {
            const int2 p = place_of(t0 + r);
            if (p.x == page) o = p.y;
          }
        }
        off[i / 4] = (i % 4 ? off[i / 4] : 0u) | o << (8 * (i % 4));
        first = min(first, static_cast<int>(o));
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if ((off[i / 4] >> (8 * (i % 4)) & 255u) == 255u) v[i] = make_uint4(0, 0, 0, 0);
    };
    auto take_max = [&]() {
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) x = abs_max2(abs_max2(abs_max2(abs_max2(x, v[i].x), v[i].y), v[i].z), v[i].w);
      if ((x & 0xFFFFu) >= 0x7F80u || (x >> 16) >= 0x7F80u) {  // infinities and NaN do not count
        x = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
            x = __vmaxu2(x, (lo < 0x7F80u ? lo : 0u) | (hi < 0x7F80u ? hi << 16 : 0u));
          }
        }
      }
      m2 = __vmaxu2(m2, x);
    };
    // rows of this warp: 16 from 16 chunk on, and again every 16 CH (more only where a
    // call names a slot twice)
    for (int64_t r0 = 16 * (chunk + CH); r0 < len; r0 += 16 * CH) {
      load(r0);
      take_max();
    }
    load(16 * chunk);
    take_max();
    uint32_t m = __reduce_max_sync(kAll, max(m2 & 0xFFFFu, m2 >> 16));
    if (!dense) first = __reduce_min_sync(kAll, first);
    if constexpr (CH > 1) {
      if (lane == 0) {
        most[parity][warp] = m;
        front[parity][warp] = first;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        m = max(m, most[parity][warp / CH * CH + i]);
        first = min(first, front[parity][warp / CH * CH + i]);
      }
      parity ^= 1;
    }
    const float old = first > 0 ? was : 0.0f;
    const float top = __uint_as_float(m << 16);
    const float need = m == 0 ? 0.0f : fmaxf(__fdiv_rn(top, int8 ? 127.0f : 448.0f), kSmallest);
    float scale = need;
    int k = 0;
    if (old >= kSmallest && old < INFINITY) {
      scale = old;
      if (need > old) {
        const uint32_t x = __float_as_uint(need), y = __float_as_uint(old);
        k = static_cast<int>(x >> 23) - static_cast<int>(y >> 23) + ((x & 0x7FFFFFu) > (y & 0x7FFFFFu));
        scale = __uint_as_float(y + (static_cast<uint32_t>(k) << 23));
      }
    }
    if (!active) return;
    if (lane == 0 && chunk == 0 && (k > 0 || scale != old || first == 0)) *scale_at = scale;
    uint8_t* const page_at = codes + (static_cast<size_t>(page) * bs * Hkv + h) * D;  // of the head's first row
    const int row_step = Hkv * D;  // a row's bytes: checked on the host
    if (k > 0) {  // the rows in front, 16 bytes a lane
      constexpr int LP = D / 16;
      const float f = k < 64 ? __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : 0.0f;
      for (int r = chunk * (32 / LP) + lane / LP; r < first; r += CH * (32 / LP)) {
        uint4* const at = reinterpret_cast<uint4*>(page_at + static_cast<size_t>(r) * row_step) + lane % LP;
        uint4 w = *at;
        if (int8) w = make_uint4(rescale4<INT8>(w.x, f), rescale4<INT8>(w.y, f), rescale4<INT8>(w.z, f), rescale4<INT8>(w.w, f));
        else w = make_uint4(rescale4<E4M3>(w.x, f), rescale4<E4M3>(w.y, f), rescale4<E4M3>(w.z, f), rescale4<E4M3>(w.w, f));
        *at = w;
      }
    }
    const float inv = scale > 0.0f ? __frcp_rn(scale) : 0.0f;
    for (int64_t r0 = 16 * chunk; r0 < len; r0 += 16 * CH) {
      if (r0 != 16 * chunk) load(r0);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int64_t r = r0 + grp + i * RPI;
        const uint32_t o = !dense ? off[i / 4] >> (8 * (i % 4)) & 255u : r < len ? off0 + static_cast<uint32_t>(r) : 255u;
        uint2 w;
        if (int8) w = make_uint2(quantize4<INT8>(v[i].x, v[i].y, inv), quantize4<INT8>(v[i].z, v[i].w, inv));
        else w = make_uint2(quantize4<E4M3>(v[i].x, v[i].y, inv), quantize4<E4M3>(v[i].z, v[i].w, inv));
        if (o != 255u) *reinterpret_cast<uint2*>(page_at + static_cast<size_t>(o) * row_step + sub * 8) = w;
      }
    }
  };

  const int own_end = kBack + static_cast<int>(t_end - t_begin);
  for (int w = kBack / 32; 32 * w < own_end; ++w) {
    uint32_t starts = begins[w] & (own_end >= 32 * (w + 1) ? kAll : (1u << (own_end & 31)) - 1u);
    while (starts != 0) {  // the same in every warp
      const int i0 = 32 * w + __ffs(starts) - 1;
      starts &= starts - 1;
      const int page = near_page[i0];
      int64_t len = 1;
      bool dense = true;
      if (!append) {
        // to the last token that is there before the next run begins
        int e = w;
        uint32_t next = begins[w] & ~((2u << (i0 & 31)) - 1u);
        while (next == 0 && e + 1 < kNear / 32) next = begins[++e];
        const int i1 = next != 0 ? 32 * e + __ffs(next) - 1 : kNear;
        uint32_t there = next != 0 ? is_there[e] & ((1u << (i1 & 31)) - 1u) : is_there[e];
        while (there == 0) there = is_there[--e];  // i0 itself at the least
        len = 32 * e + 31 - __clz(there) - i0 + 1;
        // past what the CTA keeps, while no two of its tokens are more than 32 apart
        if (i1 == kNear) {
          int64_t last = near0 + i0 + len - 1;
          for (int64_t more = near0 + kNear; more < n && more <= last + 32; more += 32) {
            const int2 q = place_of(more + lane);
            const unsigned other = __ballot_sync(kAll, q.x >= 0 && q.x != page);
            const unsigned same = __ballot_sync(kAll, q.x == page) & (other != 0 ? (1u << (__ffs(other) - 1)) - 1u : kAll);
            if (same != 0 && more + __ffs(same) - 1 <= last + 32) last = more + 31 - __clz(same);
            else if (same != 0) break;
            if (other != 0) break;
          }
          len = last - (near0 + i0) + 1;
        }
        int g = w;
        uint32_t gap = ~goes_on[w] & ~((2u << (i0 & 31)) - 1u);
        while (gap == 0 && g + 1 < kNear / 32) gap = ~goes_on[++g];
        dense = i0 + len <= (gap != 0 ? 32 * g + __ffs(gap) - 1 : kNear);
      }
      store_run(page, i0, len, dense);
    }
  }
}

template <int D, int CH>
cudaError_t launch_t(const WriteArgs& a, const AppendSlots& s, int kf, int vf, cudaStream_t st, int num_sms) {
  const int y = (2 * a.num_kv_heads * CH + kWarps - 1) / kWarps;
  if (y > 65535) return cudaErrorNotSupported;
  const int64_t step = std::min<int64_t>(std::max<int64_t>(a.num_tokens * y / (6 * num_sms), 1), most_tokens(CH));
  const dim3 grid(static_cast<unsigned>((a.num_tokens + step - 1) / step), y, 1);
  write_block_kernel<D, CH><<<grid, kWarps * 32, 0, st>>>(a, s, kf, vf, static_cast<int>(step));
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const WriteArgs& a, const AppendSlots& s, int kf, int vf, cudaStream_t st, int num_sms) {
  switch (a.block_size) {
    case 32: return launch_t<D, 2>(a, s, kf, vf, st, num_sms);
    case 64: return launch_t<D, 4>(a, s, kf, vf, st, num_sms);
    case 128: return launch_t<D, 8>(a, s, kf, vf, st, num_sms);
    default: return launch_t<D, 1>(a, s, kf, vf, st, num_sms);
  }
}

}  // namespace

cudaError_t launch_write_block(const WriteArgs& a, const AppendSlots& s, int head_dim, int kf, int vf,
                               cudaStream_t st, int num_sms) {
  if (head_dim == 64) return launch_d<64>(a, s, kf, vf, st, num_sms);
  if (head_dim == 128) return launch_d<128>(a, s, kf, vf, st, num_sms);
  return cudaErrorNotSupported;
}

}  // namespace kvq

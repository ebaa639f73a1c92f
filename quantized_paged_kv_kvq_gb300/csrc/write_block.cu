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
// call from 1 (a decode step: every request's run starts at once) to a page.
// Bound by HBM: 4 D bytes read and 2 D written per token and head.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "quant_row.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_write_block)

namespace {

constexpr int kWarps = 8;
constexpr float kSmallest = 1.17549435e-38f;  // 2^-126: 1 / scale stays finite

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

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
__global__ void __launch_bounds__(kWarps * 32) write_block_kernel(const WriteArgs a, const AppendSlots ap, int kf, int vf, int step) {
  constexpr int LPR = RowGeom<D>::LPR, RPI = RowGeom<D>::RPI, NP = 16 / RPI;
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ uint32_t most[2][kWarps];
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
  const int64_t n = a.num_tokens, t_end = min(n, (static_cast<int64_t>(blockIdx.x) + 1) * step);
  const bool reports = blockIdx.y == 0 && warp == 0;
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

  // The run of `len` tokens from t0 on in `page`, the foremost of them at offset `first`.
  auto store_run = [&](int page, int64_t t0, int64_t len, int first) {
    float* const scale_at = scales + static_cast<size_t>(page) * pitch + h;
    const float old = active && first > 0 ? *scale_at : 0.0f;
    uint4 v[NP];
    uint32_t m2 = 0;
    int off[NP];  // of the rows, -1: not this thread's, or skipped
    auto load = [&](int64_t r0) {  // rows r0 .. r0 + 15 of the run
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int64_t r = r0 + i * RPI + grp;
        const bool read = active && r < len;
        v[i] = read ? ldg_stream16(rows + (t0 + r) * stride) : make_uint4(0, 0, 0, 0);
        const int64_t slot = read && !append ? a.slot_mapping[t0 + r] : -1;
        off[i] = append && read ? first : (slot >> a.block_shift) == page ? static_cast<int>(slot) & (bs - 1) : -1;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (off[i] < 0) v[i] = make_uint4(0, 0, 0, 0);
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
    if constexpr (CH > 1) {
      if (lane == 0) most[parity][warp] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CH; ++i) m = max(m, most[parity][warp / CH * CH + i]);
      parity ^= 1;
    }
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
    const size_t page_row = static_cast<size_t>(page) * bs;
    if (k > 0) {  // the rows in front, 16 bytes a lane
      constexpr int LP = D / 16;
      const float f = k < 64 ? __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : 0.0f;
      for (int r = chunk * (32 / LP) + lane / LP; r < first; r += CH * (32 / LP)) {
        uint4* const at = reinterpret_cast<uint4*>(codes + ((page_row + r) * Hkv + h) * D) + lane % LP;
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
        const bool mine = off[i] >= 0;
        float x[8];
        unpack8(v[i], x);
        const size_t row = (page_row + max(off[i], 0)) * Hkv + h;
        if (int8) quantize_store<D, INT8, false>(x, mine, h, sub, row, codes, nullptr, inv, 0, 0, 0, 0, 0u, 0.f);
        else quantize_store<D, E4M3, false>(x, mine, h, sub, row, codes, nullptr, inv, 0, 0, 0, 0, 0u, 0.f);
      }
    }
  };

  for (int64_t base = static_cast<int64_t>(blockIdx.x) * step; base < t_end; base += 32) {
    const int64_t t = base + lane;
    const int2 p = t < n ? place(t, reports && t < t_end) : make_int2(-1, 0);
    unsigned begins = __ballot_sync(kAll, t < t_end && p.x >= 0);
    if (!append) {  // but not those whose page is that of the last token before them, at most 32 back
      const int2 q = t >= 32 ? place(t - 32, false) : make_int2(-1, 0);
      const unsigned here = __ballot_sync(kAll, p.x >= 0) & ((1u << lane) - 1u), there = __ballot_sync(kAll, q.x >= 0);
      const int from = here != 0 ? 31 - __clz(here) : there != 0 ? 31 - __clz(there) : 0;
      const int x = __shfl_sync(kAll, p.x, from), y = __shfl_sync(kAll, q.x, from);
      const int before = here != 0 ? x : from >= lane ? y : -1;
      begins &= __ballot_sync(kAll, p.x != before);
    }
    while (begins != 0) {  // the same in every warp
      const int src = __ffs(begins) - 1;
      begins &= begins - 1;
      const int page = __shfl_sync(kAll, p.x, src);
      int64_t len = 1;
      int first = __shfl_sync(kAll, p.y, src);
      if (!append) {
        // its tokens up to the first of another page: among these 32, and on while none is 32 apart
        unsigned other = __ballot_sync(kAll, lane > src && p.x >= 0 && p.x != page);
        unsigned same = __ballot_sync(kAll, lane >= src && p.x == page) & (other != 0 ? (1u << (__ffs(other) - 1)) - 1u : kAll);
        first = __reduce_min_sync(kAll, same >> lane & 1 ? p.y : 0x7fffffff);
        int64_t last = base + 31 - __clz(same);
        for (int64_t more = base + 32; other == 0 && more < n && more <= last + 32; more += 32) {
          const int2 q = more + lane < n ? place(more + lane, false) : make_int2(-1, 0);
          other = __ballot_sync(kAll, q.x >= 0 && q.x != page);
          same = __ballot_sync(kAll, q.x == page) & (other != 0 ? (1u << (__ffs(other) - 1)) - 1u : kAll);
          if (same == 0) continue;
          if (more + __ffs(same) - 1 > last + 32) break;
          first = min(first, __reduce_min_sync(kAll, same >> lane & 1 ? q.y : 0x7fffffff));
          last = more + 31 - __clz(same);
        }
        len = last - (base + src) + 1;
      }
      store_run(page, base + src, len, first);
    }
  }
}

template <int D, int CH>
cudaError_t launch_t(const WriteArgs& a, const AppendSlots& s, int kf, int vf, cudaStream_t st, int num_sms) {
  const int y = (2 * a.num_kv_heads * CH + kWarps - 1) / kWarps;
  if (y > 65535) return cudaErrorNotSupported;
  const int64_t step = std::min<int64_t>(std::max<int64_t>(a.num_tokens * y / (6 * num_sms), 1), a.block_size);
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

// Attention of each sequence's new tokens to its paged, quantized context
// (kvq_paged_prefill).  One warp per (token, query head), each lane D/32
// consecutive elements; online softmax over the visible positions.
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_prefill)

namespace {

// Element e of a row (kv-head `h` of token offset `off` in block `blk`), dequantized.
__device__ __forceinline__ float cached_value(const uint8_t* cache, const __half* meta, int fmt, int kvarn,
                                              int d, int hkv, int bs, int blk, int off, int h, int e) {
  const size_t row = ((static_cast<size_t>(blk) * bs + off) * hkv + h) * row_bytes(fmt, d);
  if (fmt == BF16) return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(cache + row)[e]) << 16);
  if (fmt == INT8) return static_cast<float>(reinterpret_cast<const int8_t*>(cache + row)[e]);
  if (fmt == E4M3) {
    const uint32_t h2 = e4m3x2_to_f16x2(cache[row + e]);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h2 & 0xFFFFu)));
  }
  if (fmt == E5M2) return __half2float(__ushort_as_half(static_cast<uint16_t>(cache[row + e] << 8)));
  const int code = fmt == INT4A ? (cache[row + e / 2] >> (4 * (e & 1))) & 15 : cache[row + e];
  const __half* m = meta + (static_cast<size_t>(blk) * hkv + h) * (kvarn ? 3 : 2) * bs + off;
  const float x = code * __half2float(m[0]) + __half2float(m[bs]);
  return kvarn ? x * __half2float(m[2 * bs]) : x;
}

template <int D>
__global__ void __launch_bounds__(128) prefill_kernel(const PrefillArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t t = item / a.num_q_heads;
  const int hq = static_cast<int>(item - t * a.num_q_heads), h = hq / a.gqa;
  if (t >= a.total_q) return;
  // the sequence whose rows hold t
  int s = -1, j = 0, q = 0;
  for (int i = 0; i < a.num_seqs; ++i) {
    const int c0 = a.cu_query[i], c1 = a.cu_query[i + 1];
    if (c0 < 0 || c1 < c0 || c1 > a.total_q || c1 - c0 > a.max_query_len) {
      raise_error(256u);
      continue;
    }
    if (c0 <= t && t < c1) {
      s = i;
      j = static_cast<int>(t - c0);
      q = c1 - c0;
    }
  }
  if (s < 0) return;
  int n = a.context_lens[s];
  if (n < 0 || n > a.max_context_len) {
    raise_error(4u);
    n = min(max(n, 0), a.max_context_len);
  }
  const int p = n - q + j;
  if (p < 0) raise_error(4u);
  float x[E], o[E];
  const uint16_t* src = a.query + (t * a.num_q_heads + hq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = __uint_as_float(static_cast<uint32_t>(src[e]) << 16);
    if (a.kvarn && a.signs != nullptr && a.signs[lane * E + e] < 0) x[e] = -x[e];
    o[e] = 0.f;
  }
  if (a.kvarn) {
    fwht_lanes<E, 32>(x, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= a.cR;
  }
  if (a.k_fmt != BF16) {
    bool bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) bad |= !isfinite(__half2float(__float2half_rn(x[e])));
    if (bad) raise_error(64u);
  }
  const int bs = 1 << a.block_shift;
  const float ks = a.k_head_scale ? a.k_head_scale[h] : a.k_scale;
  const float vs = a.v_head_scale ? a.v_head_scale[h] : a.v_scale;
  float m = -INFINITY, l = 0.f;
  const int w0 = a.window > 0 ? max(p - a.window + 1, 0) : 0;
  for (int k = 0; k <= p; ++k) {
    if (k < w0 && k >= a.sinks) k = w0;
    const int b = a.block_table[static_cast<size_t>(s) * a.max_blocks_per_seq + (k >> a.block_shift)];
    int blk = b;
    if (b < 0 || b >= a.num_blocks) {
      raise_error(2u);
      blk = 0;
    }
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      dot += x[e] * cached_value(a.k_cache, a.k_meta, a.k_fmt, a.kvarn, D, a.num_kv_heads, bs, blk,
                                 k & (bs - 1), h, lane * E + e);
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
    const float z = dot * a.sm_scale_log2 * ks;
    const float mn = fmaxf(m, z);
    const float al = exp2f(m - mn), pr = exp2f(z - mn);
    m = mn;
    l = l * al + pr;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * al + pr * cached_value(a.v_cache, a.v_meta, a.v_fmt, a.kvarn, D, a.num_kv_heads, bs,
                                           blk, k & (bs - 1), h, lane * E + e);
  }
  const float il = l > 0.f ? vs / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] *= il;
  if (a.kvarn) {
    fwht_lanes<E, 32>(o, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] *= a.cR;
      if (a.signs != nullptr && a.signs[lane * E + e] < 0) o[e] = -o[e];
    }
  }
  uint16_t* dst = a.out + (t * a.num_q_heads + hq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e]));
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, int head_dim, cudaStream_t st) {
  const int64_t grid = (a.total_q * a.num_q_heads + 3) / 4;
  if (grid > 0x7fffffffll) return cudaErrorNotSupported;
  if (head_dim == 64) prefill_kernel<64><<<static_cast<unsigned>(grid), 128, 0, st>>>(a);
  else if (head_dim == 128) prefill_kernel<128><<<static_cast<unsigned>(grid), 128, 0, st>>>(a);
  else return cudaErrorNotSupported;
  return cudaGetLastError();
}

}  // namespace kvq

// Tables of cos and sin for rotary positions (kvq_rope_table).
//
// Entry (p, i) is amplitude * (cos, sin)(p * theta_i).  theta_i / (2 pi) is the
// number of turns a position adds; held as a 64-bit fraction of a turn, p times
// it wraps modulo one turn by itself, so the angle's reduction is one integer
// product and exact however far the position is (float32 angles lose all digits
// past a few thousand radians; float64 ones cost this part's slow pipe).  What
// is left is the eighth of a turn nearest zero, converted to float32 with its
// full relative precision, and sincospif on it.
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// (cos, sin) of `turn` / 2^64 turns
__device__ __forceinline__ float2 cos_sin_turn(unsigned long long turn) {
  const unsigned q = static_cast<unsigned>((turn + (1ull << 61)) >> 62);  // nearest quarter
  const long long rest = static_cast<long long>(turn - (static_cast<unsigned long long>(q) << 62));
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);  // pi * (2 * turns), |.| <= pi / 4
  const float x = (q & 1) ? s : c, y = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -x : x, (q >= 2) ? -y : y);
}

__global__ void __launch_bounds__(256) rope_table_kernel(float2* table, int64_t entries, int pairs,
                                                         float amplitude,
                                                         const __grid_constant__ RopeTurns turns) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < entries; e += step) {
    const int64_t p = e / pairs;
    const int i = static_cast<int>(e - p * pairs);
    float2 v = cos_sin_turn(static_cast<unsigned long long>(p) * turns.t[i]);
    v.x *= amplitude;
    v.y *= amplitude;
    table[e] = v;
  }
}

}  // namespace

cudaError_t launch_rope_table(float* table, int64_t num_positions, int pairs, float amplitude,
                              const RopeTurns& turns, cudaStream_t st) {
  const int64_t entries = num_positions * pairs;
  const int64_t want = (entries + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want < 65536 ? want : 65536);
  rope_table_kernel<<<grid, 256, 0, st>>>(reinterpret_cast<float2*>(table), entries, pairs, amplitude, turns);
  return cudaGetLastError();
}

}  // namespace kvq

// Tables of cos and sin for rotary positions (kvq_rope_table).
//
// Entry (p, i) is amplitude * (cos, sin)(p * theta_i).  theta_i / (2 pi) is the
// number of turns a position adds; held as a 64-bit fraction of a turn, p times
// it wraps modulo one turn by itself, so the angle's reduction is one integer
// product and exact however far the position is (float32 angles lose all digits
// past a few thousand radians; float64 ones cost this part's slow pipe).  What
// is left after the nearest quarter turn goes through sincospif.
//
// A thread makes a run of 8 positions of one pair: the first angle's cos and sin,
// turned by 0 .. 7 positions' (kept in registers for all of the thread's runs):
// one complex product in place of a sincospif, 2^-23 more of error.  Threads of a
// warp hold neighbouring pairs, so each store is a row's consecutive bytes.  Bound by
// its writes and its instructions alike: 131,072 positions of 64 pairs, 67 MB, take
// 12.7 to 13.6 us from box to box, 73 to 78 % of the copy rate (a sincospif per entry: 73 us
// with its divisions).
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRun = 8;        // positions per thread and step
constexpr int kThreads = 256;

// (cos, sin) of `turn` / 2^64 turns.  The part beyond a quarter turn is rounded to 32
// bits of a turn: off by 2^-33 turns, 7e-10 radians, at most.
__device__ __forceinline__ float2 cos_sin_turn(unsigned long long turn) {
  const unsigned q = static_cast<unsigned>((turn + (1ull << 61)) >> 62);  // nearest quarter
  const long long beyond = static_cast<long long>(turn - (static_cast<unsigned long long>(q) << 62));  // |.| <= 2^61
  const int rest = static_cast<int>((beyond + (1ll << 31)) >> 32);
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);  // pi * (2 * turns), |.| <= pi / 4
  const float x = (q & 1) ? s : c, y = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -x : x, (q >= 2) ? -y : y);
}

__global__ void __launch_bounds__(kThreads) rope_table_kernel(float2* table, int64_t positions, int pairs,
                                                              float amplitude,
                                                              const __grid_constant__ RopeTurns turns) {
  const int rows = kThreads / pairs;  // runs of positions per CTA and step
  const int r = threadIdx.x / pairs, i = threadIdx.x - r * pairs;
  if (r >= rows) return;
  const unsigned long long t = turns.t[i];
  float2 fine[kRun];
#pragma unroll
  for (int k = 0; k < kRun; ++k) fine[k] = cos_sin_turn(k * t);
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows * kRun;
  for (int64_t p = (static_cast<int64_t>(blockIdx.x) * rows + r) * kRun; p < positions; p += step) {
    float2 v = cos_sin_turn(static_cast<unsigned long long>(p) * t);
    v.x *= amplitude;
    v.y *= amplitude;
    float2* dst = table + p * pairs + i;
    const int n = static_cast<int>(min(positions - p, static_cast<int64_t>(kRun)));
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const float c = v.x * fine[k].x - v.y * fine[k].y, s = v.y * fine[k].x + v.x * fine[k].y;
      if (k < n) dst[k * pairs] = make_float2(c, s);
    }
  }
}

}  // namespace

cudaError_t launch_rope_table(float* table, int64_t num_positions, int pairs, float amplitude,
                              const RopeTurns& turns, cudaStream_t st, int num_sms) {
  const int64_t per = static_cast<int64_t>(kThreads / pairs) * kRun;
  const int64_t want = (num_positions + per - 1) / per;
  const int64_t most = 3ll * num_sms;  // 8: 14.3 us for 131,072 x 64 pairs, 3: 12.9 (each thread makes its turns once)
  rope_table_kernel<<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, st>>>(
      reinterpret_cast<float2*>(table), num_positions, pairs, amplitude, turns);
  return cudaGetLastError();
}

}  // namespace kvq

// Decode instances: head_dim 128, 8-bit codes with a scale per (page, kv-head).
// One translation unit per group of instances keeps the build parallel.
#include "decode_launch.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_decode_d128_block)

cudaError_t launch_decode_d128_block(const DecodeArgs& a, int head_dim, int kf, int vf, bool kvarn,
                                     cudaStream_t st) {
  if (head_dim != 128 || kvarn) return cudaErrorNotSupported;
#define KVQ_D(KF_, VF_) \
  if (kf == KF_ && vf == VF_) return launch_decode_t<128, KF_, VF_, false>(a, st);
  KVQ_D(INT8B, INT8B)
  KVQ_D(INT8B, E4M3B)
  KVQ_D(E4M3B, INT8B)
  KVQ_D(E4M3B, E4M3B)
#undef KVQ_D
  return cudaErrorNotSupported;
}

}  // namespace kvq

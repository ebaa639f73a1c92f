// kvq_norm_rope (no cache) and kvq_norm_rope_write for the symmetric formats
// and the 16-bit cache.
#include "norm_rope.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_norm_rope)

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, cudaStream_t st) {
  switch (head_dim) {
    case 64: return launch_norm_rope_t<64, false, BF16, BF16, false>(a, st);
    case 128: return launch_norm_rope_t<128, false, BF16, BF16, false>(a, st);
    case 256: return launch_norm_rope_t<256, false, BF16, BF16, false>(a, st);
    default: return cudaErrorNotSupported;
  }
}

namespace {
template <int D>
cudaError_t dispatch_d(const NormRopeArgs& a, int kf, int vf, cudaStream_t st) {
#define KVQ_W(KF_, VF_) \
  if (kf == KF_ && vf == VF_) return launch_norm_rope_t<D, true, KF_, VF_, false>(a, st);
  KVQ_W(INT8, INT8)
  KVQ_W(INT8, E4M3)
  KVQ_W(INT8, E5M2)
  KVQ_W(E4M3, INT8)
  KVQ_W(E4M3, E4M3)
  KVQ_W(E4M3, E5M2)
  KVQ_W(E5M2, INT8)
  KVQ_W(E5M2, E4M3)
  KVQ_W(E5M2, E5M2)
  KVQ_W(BF16, BF16)
#undef KVQ_W
  return cudaErrorNotSupported;
}
}  // namespace

cudaError_t launch_norm_rope_write(const NormRopeArgs& a, int head_dim, int kf, int vf, bool kvarn,
                                   cudaStream_t st) {
  if (is_asym(kf) || is_asym(vf)) return launch_norm_rope_write_asym(a, head_dim, kf, vf, kvarn, st);
  if (head_dim == 64) return dispatch_d<64>(a, kf, vf, st);
  if (head_dim == 128) return dispatch_d<128>(a, kf, vf, st);
  return cudaErrorNotSupported;
}

}  // namespace kvq

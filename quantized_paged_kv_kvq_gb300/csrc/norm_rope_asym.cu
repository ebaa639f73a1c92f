// kvq_norm_rope_write for the asymmetric formats, with or without KVarN.
#include "norm_rope.cuh"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_norm_rope_asym)

namespace {
template <int D>
cudaError_t dispatch_d(const NormRopeArgs& a, int kf, int vf, bool kvarn, cudaStream_t st) {
#define KVQ_W(KF_, VF_, KV_) \
  if (kf == KF_ && vf == VF_ && kvarn == KV_) return launch_norm_rope_t<D, true, KF_, VF_, KV_>(a, st);
  KVQ_W(INT4A, INT4A, false)
  KVQ_W(INT4A, UINT8A, false)
  KVQ_W(UINT8A, INT4A, false)
  KVQ_W(UINT8A, UINT8A, false)
  KVQ_W(INT4A, INT4A, true)
  KVQ_W(INT4A, UINT8A, true)
  KVQ_W(UINT8A, INT4A, true)
  KVQ_W(UINT8A, UINT8A, true)
#undef KVQ_W
  return cudaErrorNotSupported;
}
}  // namespace

cudaError_t launch_norm_rope_write_asym(const NormRopeArgs& a, int head_dim, int kf, int vf, bool kvarn,
                                        cudaStream_t st) {
  if (head_dim == 64) return dispatch_d<64>(a, kf, vf, kvarn, st);
  if (head_dim == 128) return dispatch_d<128>(a, kf, vf, kvarn, st);
  return cudaErrorNotSupported;
}

}  // namespace kvq

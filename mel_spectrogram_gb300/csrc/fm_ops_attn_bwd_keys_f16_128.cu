#include "fm_ops_attn_bwd.cuh"
namespace fm {
fm_status attn_bwd_keys_f16_128(const TcParams& t, const bwd::Extra& x, int mode, cudaStream_t st) {
  return bwd::launch<128, false, true>(t, x, mode, st);
}
}  // namespace fm

#include "fm_ops_attn_fwd.cuh"
namespace fm {
fm_status attn_fwd_f16_64(const TcParams& t, int mode, cudaStream_t st) { return fwd::launch<64, false>(t, mode, st); }
}  // namespace fm

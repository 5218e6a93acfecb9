#include "fm_ops_attn_fwd.cuh"
namespace fm {
fm_status attn_fwd_bf16_128(const TcParams& t, int mode, cudaStream_t st) { return fwd::launch<128, true>(t, mode, st); }
}  // namespace fm

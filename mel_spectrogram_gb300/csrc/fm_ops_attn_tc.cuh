// Parameters of the tensor-core attention kernels (fm_ops_attn_fwd*.cu,
// fm_ops_attn_bwd*.cu).
#pragma once

#include "fm_ops_attn.cuh"
#include "fm_tc.cuh"

namespace fm {

constexpr int kTile = 128;      // rows of a tile: the lanes of tensor memory
constexpr int kBiasPad = 256;   // copies of the end values beside the bias by offset

// Which documents the 128 frames of a tile hold: lowest and highest id, and
// whether all its frames carry that one id. No documents: every tile is {0, 0, 1}.
struct DocRange {
  int lo, hi, uniform;
};

struct TcParams {
  AttnParams p;
  CUtensorMap qm, km, vm, gm;  // q, k, v, dout as {dim, token, head, batch}
  // coordinates step by 0 along broadcast heads or batches
  int q_mh, q_mb, k_mh, k_mb, v_mh, v_mb, g_mh, g_mb;
  const int4* q_ranges;  // [batch][q tiles] (lo, hi, uniform, 0), NULL without documents
  const int4* k_ranges;  // [batch][k tiles]
  int q_tiles, k_tiles;  // of 128
  int dim16;             // dim rounded up to 16
  int splits, split_tiles;  // the key tiles of one split; splits > 1: partial results
  float* part_o;         // [splits][batch][heads][q_len][dim]
  float* part_lse;       // [splits][batch][heads][q_len], base 2
  unsigned* err;
};

// the device's error word for the operators, NULL if there is none
unsigned* ops_error_word();

// Bytes of workspace of the tensor-core passes, and whether they take this
// call: 16-bit types, dim a multiple of 8 up to 128, and tensors whose rows
// start on 16-byte boundaries. ws may be NULL to ask only.
// The few-query kernel: its splits of the key axis.
struct StepPlan {
  int splits, split_keys, row_tiles;
};
StepPlan step_plan(const AttnParams& p);
fm_status attn_step(const AttnParams& p, int64_t dtype, const StepPlan& w, float* part_o, float* part_lse,
                    cudaStream_t st);

struct TcPlan {
  StepPlan step;  // step.splits > 0: the forward pass takes the few-query kernel
  int splits, split_tiles, q_tiles, k_tiles;
  int64_t ranges, part_o, part_lse, stats, peak, bias, total;
};
bool tc_layout_ok(const AttnParams& p, int64_t dtype, bool backward);
TcPlan tc_plan(const AttnParams& p, bool backward);  // backward needs heads, q_len, map and grad only
fm_status attn_tc_forward(const AttnParams& p, int64_t dtype, char* ws, cudaStream_t st);
// grad: the bias gradient is wanted (p.part is set here; its rows are p.batch * q_tiles of tile kTile)
fm_status attn_tc_backward(AttnParams& p, int64_t dtype, bool grad, char* ws, cudaStream_t st);

#ifdef __CUDACC__
// The key tiles a tile of queries [i0, i0 + n) has to visit, as one range:
// below the lengths, causality and, with documents, from the first to the last
// tile that shares an id.
struct TileRange {
  int begin, end;
};
__device__ __forceinline__ int key_end(const AttnParams& p, const RowInfo& r, int i0, int n) {
  int end = r.len;
  if (p.causal) end = min(end, max(r.start + i0 + n, r.prefix));
  return max(end, 0);
}

// The head's bias by offset, in units of log2, padded by copies of its ends:
// bias[o + max_distance + kBiasPad] for |o| <= max_distance + kBiasPad.
template <bool BF16>
__device__ __forceinline__ void fill_bias(const AttnParams& p, int h, float* bias, int tid, int threads) {
  const int D = p.max_distance;
  for (int i = tid; i < 2 * (D + kBiasPad) + 1; i += threads) {
    const int at = min(max(i - kBiasPad, 0), 2 * D);
    bias[i] = kLog2e * table_value(p, (long long)p.map[at] * p.heads + h, BF16);
  }
}
#endif

}  // namespace fm

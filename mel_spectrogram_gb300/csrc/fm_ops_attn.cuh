// What the attention kernels share: one launch's parameters and the score's
// definition (fm_ops.h).
#pragma once

#include "fm_ops.cuh"

namespace fm {

struct Strides {
  long long b, t, h;
};

struct AttnParams {
  int batch, q_len, k_len, heads, kv_heads, group, dim;
  int causal;
  float scale, cap;
  const void *q, *k, *v, *dout;
  const void* out_in;  // the forward's output, read by the backward
  void *out, *dq, *dk, *dv;
  Strides qs, ks, vs, os, dos, dqs, dks, dvs;
  float* lse;
  void* rest;  // what rounding took from the output, in the output's layout; NULL: not wanted
  const int32_t *q_docs, *k_docs, *k_lens, *q_start, *prefix;
  int start_end, start_all;  // where q_start is NULL: queries end with the keys, or start at start_all
  const int32_t* map;        // NULL: no bucket bias
  int max_distance;
  const void* table;
  int table_f32;
  const float* slopes;
  float* delta;  // [batch][heads][q_len]: sum of dout * out
  float* part;   // partial bias gradients: [batch * q tiles][heads][2 * max_distance + 1]
  int q_tiles;
  int f16;  // the inputs' type: the backward pass on the tensor cores scales dS
};

// Rows of one batch entry: how many keys count, where the queries stand.
struct RowInfo {
  int len, start, prefix;
};
__device__ __forceinline__ RowInfo row_info(const AttnParams& p, int b) {
  RowInfo r;
  r.len = p.k_lens ? min(max(p.k_lens[b], 0), p.k_len) : p.k_len;
  r.start = p.q_start ? p.q_start[b] : p.start_end ? r.len - p.q_len : p.start_all;
  r.start = min(max(r.start, -(1 << 29)), 1 << 29);
  r.prefix = p.causal && p.prefix ? p.prefix[b] : 0;
  return r;
}
__device__ __forceinline__ float table_value(const AttnParams& p, long long at, int dtype_bf16) {
  if (p.table_f32) return ((const float*)p.table)[at];
  return dtype_bf16 ? to_f(((const __nv_bfloat16*)p.table)[at]) : to_f(((const __half*)p.table)[at]);
}

// kernels for any type, head size and stride (fm_ops_attn_any.cu)
fm_status attn_any_forward(const AttnParams& p, int64_t dtype, cudaStream_t st);
fm_status attn_any_backward(const AttnParams& p, int64_t dtype, cudaStream_t st);
int any_rows(const AttnParams& p);  // queries a block takes, and per row of AttnParams::part

}  // namespace fm

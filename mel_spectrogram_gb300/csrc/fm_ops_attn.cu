// C entry points of attention (fm_ops.h): argument checks, workspaces and the
// choice of kernels.
#include "fm_ops_attn_tc.cuh"

namespace fm {
namespace {

constexpr int64_t kMaxLen = (1 << 29) - 1;
int64_t align256(int64_t n) { return (n + 255) & ~(int64_t)255; }

fm_status check(const fm_attention_args* a) {
  if (a == nullptr) return FM_ERR_INVALID_ARG;
  if (a->batch < 0 || a->batch > 65535 || a->q_len < 0 || a->q_len > kMaxLen || a->k_len < 0 || a->k_len > kMaxLen)
    return FM_ERR_INVALID_ARG;
  if (a->heads < 1 || a->heads > 65535 || a->kv_heads < 1 || a->heads % a->kv_heads) return FM_ERR_INVALID_ARG;
  if (a->dim < 1) return FM_ERR_INVALID_ARG;
  if (a->dim > 256) return FM_ERR_UNSUPPORTED;
  if (!is_float_type(a->dtype)) return FM_ERR_INVALID_ARG;
  const double big = 3e38;
  if (!(a->scale >= -big && a->scale <= big) || !(a->softcap >= 0 && a->softcap <= big)) return FM_ERR_INVALID_ARG;
  if ((a->q_docs == nullptr) != (a->k_docs == nullptr)) return FM_ERR_INVALID_ARG;
  if (a->buckets != nullptr && a->table_dtype != a->dtype && a->table_dtype != FM_F32) return FM_ERR_INVALID_ARG;
  // one 31-bit index counts the rows of statistics
  if (a->batch * a->heads > 0x7fffffffLL || a->batch * a->heads * ((a->q_len + 7) / 8) > 0x7fffffffLL)
    return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

Strides strides(const int64_t* s) { return Strides{s[0], s[1], s[2]}; }

AttnParams params(const fm_attention_args* a) {
  AttnParams p{};
  p.batch = (int)a->batch;
  p.q_len = (int)a->q_len;
  p.k_len = (int)a->k_len;
  p.heads = (int)a->heads;
  p.kv_heads = (int)a->kv_heads;
  p.group = p.heads / p.kv_heads;
  p.dim = (int)a->dim;
  p.causal = a->causal != 0;
  p.scale = (float)a->scale;
  // smaller caps make all scores equal to 32 bits as this one does, but could
  // round to 0, which means no cap, or leave the range of floats as scale / cap
  p.cap = a->softcap > 0 ? (float)(a->softcap > 1e-30 ? a->softcap : 1e-30) : 0.f;
  p.q = a->q, p.k = a->k, p.v = a->v;
  p.qs = strides(a->q_s), p.ks = strides(a->k_s), p.vs = strides(a->v_s), p.os = strides(a->out_s);
  p.lse = a->lse;
  p.rest = a->dtype == FM_F32 ? nullptr : a->out_rest;
  p.q_docs = a->q_docs, p.k_docs = a->k_docs, p.k_lens = a->k_lens, p.q_start = a->q_start, p.prefix = a->prefix;
  p.start_end = a->q_start_all == FM_Q_START_END;
  const int64_t far = 1 << 29;
  p.start_all = p.start_end ? 0 : (int)(a->q_start_all > far ? far : a->q_start_all < -far ? -far : a->q_start_all);
  if (a->buckets) {
    p.map = a->buckets->map;
    p.max_distance = a->buckets->max_distance;
    p.table = a->table;
    p.table_f32 = a->table_dtype == FM_F32;
  }
  p.slopes = a->slopes;
  p.f16 = a->dtype == FM_F16;
  return p;
}

// Layout of the backward workspace for the kernels of any type; the
// tensor-core kernels' own (tc_plan) is followed by partial bias gradients too.
struct Workspace {
  int64_t delta, part, total;
  int q_tiles;
};
int64_t part_bytes(const fm_attention_args* a, int q_tiles) {
  if (a->buckets == nullptr || a->dtable == nullptr) return 0;
  return align256(sizeof(float) * a->batch * q_tiles * a->heads * (2 * (int64_t)a->buckets->max_distance + 1));
}
Workspace any_layout(const fm_attention_args* a) {
  Workspace w{};
  const int rows = any_rows(params(a));
  w.q_tiles = (int)((a->q_len + rows - 1) / rows);
  w.part = align256(sizeof(float) * a->batch * a->heads * a->q_len);
  w.total = w.part + part_bytes(a, w.q_tiles) + 256;
  return w;
}
int64_t backward_bytes(const fm_attention_args* a) {
  int64_t n = any_layout(a).total;
  if (a->dtype != FM_F32 && a->dim <= 128 && a->dim % 8 == 0) {
    // whichever kernels the pointers' alignment lets run
    const TcPlan w = tc_plan(params(a), true);
    const int64_t tc = w.total + part_bytes(a, w.q_tiles);
    if (tc > n) n = tc;
  }
  return n;
}
bool same_device(const fm_buckets* b) {
  int dev = -1;
  return b == nullptr || (cudaGetDevice(&dev) == cudaSuccess && dev == b->device);
}
}  // namespace
}  // namespace fm

using namespace fm;

extern "C" int64_t fm_attention_workspace(const fm_attention_args* a, int backward) {
  if (check(a) != FM_OK) return -1;
  if (a->batch == 0 || a->q_len == 0) return backward ? backward_bytes(a) : 0;
  if (!backward) return a->dtype == FM_F32 || a->dim > 128 || a->dim % 8 ? 0 : tc_plan(params(a), false).total;
  return backward_bytes(a);
}

extern "C" fm_status fm_attention_forward(const fm_attention_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->batch == 0 || a->q_len == 0) return FM_OK;
  if (a->q == nullptr || a->out == nullptr || (a->k_len > 0 && (a->k == nullptr || a->v == nullptr)))
    return FM_ERR_INVALID_ARG;
  if ((a->buckets && a->table == nullptr) || !same_device(a->buckets)) return FM_ERR_INVALID_ARG;
  if (fm_status s = ops_error_seen()) return s;
  AttnParams p = params(a);
  p.out = a->out;
  if (tc_layout_ok(p, a->dtype, false)) {
    const TcPlan w = tc_plan(p, false);
    if (w.total > 0 && (a->workspace == nullptr || a->workspace_bytes < w.total || ((uintptr_t)a->workspace & 15)))
      return FM_ERR_INVALID_ARG;
    return attn_tc_forward(p, a->dtype, (char*)a->workspace, (cudaStream_t)stream);
  }
  return attn_any_forward(p, a->dtype, (cudaStream_t)stream);
}

extern "C" fm_status fm_attention_backward(const fm_attention_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->batch == 0 || (a->q_len == 0 && a->k_len == 0)) {
    if (a->dtable && a->buckets) {
      const size_t n = (size_t)a->buckets->num_buckets * a->heads * item_size(a->table_dtype);
      if (cudaMemsetAsync(a->dtable, 0, n, (cudaStream_t)stream) != cudaSuccess) return FM_ERR_CUDA;
    }
    return FM_OK;
  }
  if (a->q_len > 0 && (a->q == nullptr || a->dout == nullptr || a->out == nullptr || a->dq == nullptr ||
                       a->lse == nullptr))
    return FM_ERR_INVALID_ARG;
  if (a->k_len > 0 && (a->k == nullptr || a->v == nullptr || a->dk == nullptr || a->dv == nullptr))
    return FM_ERR_INVALID_ARG;
  if ((a->buckets && a->table == nullptr) || !same_device(a->buckets)) return FM_ERR_INVALID_ARG;
  if (a->workspace == nullptr || a->workspace_bytes < backward_bytes(a) || ((uintptr_t)a->workspace & 15))
    return FM_ERR_INVALID_ARG;
  if (fm_status s = ops_error_seen()) return s;
  AttnParams p = params(a);
  p.out_in = a->out;
  p.dout = a->dout;
  p.dos = strides(a->dout_s);
  p.dq = a->dq, p.dk = a->dk, p.dv = a->dv;
  p.dqs = strides(a->dq_s), p.dks = strides(a->dk_s), p.dvs = strides(a->dv_s);
  const bool grad = a->buckets && a->dtable;
  char* ws = (char*)a->workspace;
  if (tc_layout_ok(p, a->dtype, true)) {
    p.q_tiles = tc_plan(p, true).q_tiles;
    if (fm_status s = attn_tc_backward(p, a->dtype, grad, ws, (cudaStream_t)stream)) return s;
  } else {
    const Workspace w = any_layout(a);
    p.delta = (float*)ws;
    p.q_tiles = w.q_tiles;
    if (grad) p.part = (float*)(ws + w.part);
    if (fm_status s = attn_any_backward(p, a->dtype, (cudaStream_t)stream)) return s;
  }
  if (!grad) return FM_OK;
  const int W = 2 * p.max_distance + 1;
  return bucket_sums_launch(a->buckets, p.part, (long long)p.batch * p.q_tiles, (long long)p.heads * W, W,
                            -p.max_distance, W, p.heads, a->dtable, a->table_dtype, (cudaStream_t)stream);
}

// Gated linear recurrence over frames: checks of arguments (fm_ops.h); the kernels, and
// the reasons for their shape, are in fm_ops_scan.cuh, one translation unit per type.
#include "fm_ops_scan.cuh"

namespace fm {
fm_status scan_f32(const scan::ScanParams& p, bool backward, cudaStream_t st);
fm_status scan_f16(const scan::ScanParams& p, bool backward, cudaStream_t st);
fm_status scan_bf16(const scan::ScanParams& p, bool backward, cudaStream_t st);

bool ops_error_words(tc::ErrorWords* words);
fm_status ops_error_seen();

namespace {
using scan::ScanParams;

fm_status check(const fm_scan_args* a) {
  if (a == nullptr || a->batch < 0 || a->batch > 0x7fffffffLL || a->frames < 0 || a->frames > (1LL << 30) ||
      a->channels < 1 || a->channels > (1 << 24) || !is_float_type(a->dtype))
    return FM_ERR_INVALID_ARG;
  return FM_OK;
}

ScanParams params(const fm_scan_args* a) {
  ScanParams p{};
  p.batch = a->batch, p.frames = a->frames;
  p.channels = (int)a->channels;
  p.reverse = a->reverse != 0;
  for (int i = 0; i < 2; ++i) p.x_s[i] = a->x_s[i], p.g_s[i] = a->gate_s[i];
  p.x = a->x, p.g = a->gate;
  p.lens = a->lens, p.docs = a->docs;
  p.marks = a->marks;
  // calls that need none take none: what they were handed may hold less than they would write
  const int64_t need = fm_scan_workspace(a);
  if (need > 0 && a->workspace_bytes >= need) p.sums = (float2*)a->workspace;
  return p;
}
}  // namespace
}  // namespace fm

using namespace fm;

extern "C" int64_t fm_scan_marks(const fm_scan_args* a) {
  if (check(a) != FM_OK) return -1;
  return (a->frames + scan::kMark - 1) / scan::kMark * a->batch * a->channels * (int64_t)sizeof(float);
}

// Rows that may be worth stretches: long, and of few enough channels to leave the device
// half empty.
extern "C" int64_t fm_scan_workspace(const fm_scan_args* a) {
  if (check(a) != FM_OK) return -1;
  if (a->frames < 4096 || a->batch > 8192 / a->channels) return 0;
  return (scan::kMaxStretches + 1) * a->batch * a->channels * (int64_t)sizeof(float2);
}

extern "C" fm_status fm_scan_forward(const fm_scan_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->batch == 0) return FM_OK;
  if (a->frames > 0 && (a->x == nullptr || a->gate == nullptr || a->y == nullptr)) return FM_ERR_INVALID_ARG;
  if (((uintptr_t)a->marks | (uintptr_t)a->workspace) & 15) return FM_ERR_INVALID_ARG;
  if (fm_status s = ops_error_seen()) return s;
  ScanParams p = params(a);
  if (!ops_error_words(&p.err)) return FM_ERR_CUDA;
  for (int i = 0; i < 2; ++i) p.y_s[i] = a->y_s[i];
  p.y = a->y;
  p.state = a->state, p.end = a->end;
  cudaStream_t st = (cudaStream_t)stream;
  return a->dtype == FM_F32 ? scan_f32(p, false, st) : a->dtype == FM_F16 ? scan_f16(p, false, st) : scan_bf16(p, false, st);
}

extern "C" fm_status fm_scan_backward(const fm_scan_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->batch == 0) return FM_OK;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->frames == 0) {
    if (a->dstate == nullptr) return FM_OK;
    const size_t n = (size_t)(a->batch * a->channels) * sizeof(float);
    const cudaError_t e = a->dend ? cudaMemcpyAsync(a->dstate, a->dend, n, cudaMemcpyDeviceToDevice, st)
                                  : cudaMemsetAsync(a->dstate, 0, n, st);
    return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
  }
  if (a->x == nullptr || a->gate == nullptr || a->dy == nullptr || a->marks == nullptr || (((uintptr_t)a->marks | (uintptr_t)a->workspace) & 15))
    return FM_ERR_INVALID_ARG;
  if (!a->dx && !a->dgate && !a->dstate) return FM_OK;
  if (fm_status s = ops_error_seen()) return s;
  ScanParams p = params(a);
  if (!ops_error_words(&p.err)) return FM_ERR_CUDA;
  for (int i = 0; i < 2; ++i) p.dy_s[i] = a->dy_s[i], p.dx_s[i] = a->dx_s[i], p.dg_s[i] = a->dgate_s[i];
  p.dy = a->dy;
  p.dx = a->dx, p.dg = a->dgate;
  p.dend = a->dend, p.dstate = a->dstate;
  return a->dtype == FM_F32 ? scan_f32(p, true, st) : a->dtype == FM_F16 ? scan_f16(p, true, st) : scan_bf16(p, true, st);
}

// Gated linear layer (fm_ops.h): checks, choice of kernels, and the kernels for 32-bit
// tensors, on the FP32 pipes.
//
// Those are products in square tiles, whose sums stay in registers: 8 x 8 a thread
// in tiles of 128, or 4 x 4 in tiles of 64 where 128 would leave SMs without one. The
// forward pass (and the backward pass's first product) fills half of a tile's columns
// with rows of w_gate and half with the same rows of w_up, so that g and u of an element
// meet in one thread. dg and du stay in 32 bits, side by side in rows of 2 * hidden; dx
// is one product over both, and one product over the rows gives both weights' gradients.
// Where those two have fewer tiles than SMs, each tile's sum is cut into stretches, whose
// results another kernel adds up in order: dx of 258 rows, 256 to 1024, went through 128
// steps in 20 blocks otherwise, 90 of the 174 us that the whole step took. Bound by the
// FP32 pipes and what feeds them: 2048 rows, 512 to 2048 forward 235 us, 36 TFLOP/s.
#include <type_traits>

#include "fm_ops_gated.cuh"
#include "fm_tc.cuh"

namespace fm {

bool gated_step_takes(const fm_gated_args* a);
fm_status gated_step_forward(const fm_gated_args* a, const GatedParams& p, cudaStream_t st);
int64_t gated_tc_workspace(const fm_gated_args* a, bool backward);
fm_status gated_tc_forward(const fm_gated_args* a, GatedParams p, cudaStream_t st);
fm_status gated_tc_backward(const fm_gated_args* a, GatedParams p, cudaStream_t st);

namespace {

constexpr int kDepth = 16, kThreads = 256;
constexpr int kMostCuts = 16;  // stretches of a sum

enum Product { kForward, kGrads, kDx, kDw };
constexpr bool pairs(Product P) { return P == kForward || P == kGrads; }

// C[m][n] = sum over k of A(m, k) B(n, k), in steps of kDepth terms; kDx goes through
// w_gate's rows and then through w_up's, each padded to whole steps. d: dg and du. parts:
// where stretch blockIdx.y (of `stretch` steps) leaves its sums, NULL for one.
template <Product P, int ACT, int TILE>
__global__ void __launch_bounds__(kThreads) gated_f32(const GatedParams p, float* d, long long tiles_n, long long stretch,
                                                      float* parts) {
  constexpr int kHalf = TILE / 2, N = TILE / 16, kLoads = TILE * kDepth / kThreads, kPad = 4;
  __shared__ __align__(16) float as[2][kDepth][TILE + kPad], bs[2][kDepth][TILE + kPad];
  const long long tile_m = blockIdx.x / tiles_n, tile_n = blockIdx.x % tiles_n;
  const int F = p.hidden;
  const long long F2 = 2LL * F;
  const long long M = P == kDw ? F2 : p.rows;                                     // rows of C
  const long long K = P == kDx ? F : P == kDw ? p.rows : (long long)p.width;      // terms (kDx: of either half)
  const long long m0 = tile_m * TILE, n0 = tile_n * (pairs(P) ? kHalf : TILE);    // n0: hidden unit, or column of C
  const long long each = (K + kDepth - 1) / kDepth, steps = P == kDx ? 2 * each : each;
  const long long begin = blockIdx.y * stretch, end = begin + stretch < steps ? begin + stretch : steps;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const float *x = (const float*)p.x, *wg = (const float*)p.wg, *wu = (const float*)p.wu;

  // Neighbouring threads read neighbouring elements: along k (a thread's elements are
  // kRowStep rows apart), or along the rows (kDeepStep terms apart).
  constexpr int kRowStep = kThreads / 16, kDeepStep = kThreads / TILE;
  constexpr bool kADeep = P == kDw, kBDeep = !pairs(P);
  const int across = tid % TILE, deep = tid / TILE, row = tid / 16, col = tid % 16;
  const float *pa, *pb, *pu = nullptr;     // this thread's first elements of the next step; pu: pairs, of w_up
  long long next_a, next_b, next_u = 0;    // to the same of the step after
  long long far_a, far_b, far_u = 0;       // to a thread's next element
  unsigned a_here = 0, b_here = 0;         // which of a thread's rows exist; all or none where deep
  long long k_next = 0;
  auto start = [&](long long step) {
    const bool up = P == kDx && step >= each;
    k_next = (up ? step - each : step) * kDepth;
    if (P == kDw) pa = d + (k_next + deep) * F2 + m0 + across, far_a = kDeepStep * F2, next_a = kDepth * F2;
    else if (P == kDx) pa = d + (m0 + row) * F2 + (up ? F : 0) + k_next + col, far_a = kRowStep * F2, next_a = kDepth;
    else pa = x + (m0 + row) * p.xs + k_next + col, far_a = kRowStep * p.xs, next_a = kDepth;
    if (pairs(P)) {
      pb = wg + (n0 + row) * p.gs + k_next + col, far_b = kRowStep * p.gs, next_b = kDepth;
      pu = wu + (n0 + row) * p.us + k_next + col, far_u = kRowStep * p.us, next_u = kDepth;
    } else if (P == kDx) {
      const long long stride = up ? p.us : p.gs;
      pb = (up ? wu : wg) + (k_next + deep) * stride + n0 + across, far_b = kDeepStep * stride, next_b = kDepth * stride;
    } else {
      pb = x + (k_next + deep) * p.xs + n0 + across, far_b = kDeepStep * p.xs, next_b = kDepth * p.xs;
    }
  };
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    if (kADeep ? m0 + across < M : m0 + row + kRowStep * i < M) a_here |= 1u << i;
    if (kBDeep ? n0 + across < p.width : n0 + (row + kRowStep * i) % kHalf < F) b_here |= 1u << i;
  }
  float ra[kLoads], rb[kLoads];
  auto read = [&](long long step) {
    if (P == kDx && step == each) start(step);
    const float *qa = pa, *qb = pb;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool in_a = k_next + (kADeep ? deep + kDeepStep * i : col) < K;
      const bool in_b = k_next + (kBDeep ? deep + kDeepStep * i : col) < K;
      if (pairs(P) && i == kLoads / 2) qb = pu;
      ra[i] = in_a && (a_here >> i & 1) ? *qa : 0.f;
      rb[i] = in_b && (b_here >> i & 1) ? *qb : 0.f;
      qa += far_a;
      qb += pairs(P) && i >= kLoads / 2 ? far_u : far_b;
    }
    pa += next_a, pb += next_b, pu += next_u;
    k_next += kDepth;
  };
  auto write = [&](int slot) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (kADeep) as[slot][deep + kDeepStep * i][across] = ra[i];
      else as[slot][col][row + kRowStep * i] = ra[i];
      if (kBDeep) bs[slot][deep + kDeepStep * i][across] = rb[i];
      else bs[slot][col][row + kRowStep * i] = rb[i];
    }
  };

  float2 acc[N][N / 2];  // pairs of columns
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < N / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
  start(begin);
  read(begin);
  write(0);
  for (long long step = begin; step < end; ++step) {
    const int slot = (int)(step - begin) & 1;
    __syncthreads();  // this step's operands are there, and all are done with the other slot
    if (step + 1 < end) read(step + 1);
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      float a[N];
      float2 b[N / 2];
#pragma unroll
      for (int i = 0; i < N; i += 4) *(float4*)&a[i] = *(const float4*)&as[slot][k][ty * N + i];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < N / 4; ++j) b[h * (N / 4) + j] = *(const float2*)&bs[slot][k][h * kHalf + tx * (N / 2) + 2 * j];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) acc[i][j] = tc::fma2(tc::both(a[i]), b[j], acc[i][j]);
    }
    if (step + 1 < end) write(slot ^ 1);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long m = m0 + ty * N + i;
    if (m >= M) break;
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const float lo[2] = {acc[i][j].x, acc[i][j].y}, hi[2] = {acc[i][N / 4 + j].x, acc[i][N / 4 + j].y};
      const int at = tx * (N / 2) + 2 * j;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (pairs(P)) {  // lo is g, hi is u
          const long long f = n0 + at + e;
          if (f >= F) continue;
          if (P == kForward) {
            ((float*)p.h)[m * p.hs + f] = act_of<ACT>(lo[e]) * hi[e];
          } else {
            float a, slope;
            act_and_slope<ACT>(lo[e], a, slope);
            const float dh = ((const float*)p.dh)[m * p.dhs + f];
            d[m * F2 + f] = dh * hi[e] * slope;
            d[m * F2 + F + f] = dh * a;
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const long long c = n0 + h * kHalf + at + e;
            if (c >= p.width) continue;
            const float v = h ? hi[e] : lo[e];
            if (parts) parts[(blockIdx.y * M + m) * p.width + c] = v;
            else if (P == kDx) ((float*)p.dx)[m * p.dxs + c] = v;
            else if (m < F) { if (p.dwg) ((float*)p.dwg)[m * p.dgs + c] = v; }
            else if (p.dwu) ((float*)p.dwu)[(m - F) * p.dus + c] = v;
          }
        }
      }
    }
  }
}

// The stretches' sums, one after another. to: rows < split at a, the others at b.
__global__ void __launch_bounds__(256) add_parts(const float* parts, int cuts, long long rows, int cols, long long split,
                                                 float* a, long long a_stride, float* b, long long b_stride) {
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x, n = rows * cols;
  if (at >= n) return;
  const long long m = at / cols, c = at % cols;
  float* to = m < split ? a : b;
  if (!to) return;
  float s = parts[at];
#pragma unroll 4
  for (int i = 1; i < cuts; ++i) s += parts[i * n + at];
  to[(m < split ? m * a_stride : (m - split) * b_stride) + c] = s;
}

// How a product of M rows, N columns and K terms is laid out.
struct Plan {
  int tile, cuts;
  long long tiles_n, tiles, stretch;  // stretch: steps of a cut
};
Plan plan_of(Product P, const GatedParams& p) {
  const long long M = P == kDw ? 2LL * p.hidden : p.rows, K = P == kDx ? p.hidden : P == kDw ? p.rows : p.width;
  const long long steps = (K + kDepth - 1) / kDepth * (P == kDx ? 2 : 1);
  const int N = pairs(P) ? p.hidden : p.width;
  auto count = [&](int tile, long long* tiles_n) {
    const int step = pairs(P) ? tile / 2 : tile;
    *tiles_n = (N + step - 1) / step;
    return (M + tile - 1) / tile * *tiles_n;
  };
  Plan w{};
  w.tile = 128;
  w.tiles = count(w.tile, &w.tiles_n);
  if (w.tiles < num_sms()) w.tile = 64, w.tiles = count(w.tile, &w.tiles_n);
  // at least eight steps a stretch: each costs a pass of its results through memory
  long long cuts = 1;
  if (!pairs(P) && w.tiles < num_sms()) {
    cuts = (2 * num_sms() + w.tiles - 1) / w.tiles;
    const long long most = steps / 8 < kMostCuts ? steps / 8 : kMostCuts;
    if (cuts > most) cuts = most;
    if (cuts < 1) cuts = 1;
  }
  w.stretch = (steps + cuts - 1) / cuts;
  w.cuts = (int)((steps + w.stretch - 1) / w.stretch);
  return w;
}

template <Product P, int ACT>
fm_status f32_launch(const GatedParams& p, float* d, float* parts, cudaStream_t st) {
  const Plan w = plan_of(P, p);
  if (w.tiles > 0x7fffffffLL) return FM_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)w.tiles, (unsigned)w.cuts);
  float* to = w.cuts > 1 ? parts : nullptr;
  if (w.tile == 128) gated_f32<P, ACT, 128><<<grid, kThreads, 0, st>>>(p, d, w.tiles_n, w.stretch, to);
  else gated_f32<P, ACT, 64><<<grid, kThreads, 0, st>>>(p, d, w.tiles_n, w.stretch, to);
  if (to) {
    const long long M = P == kDw ? 2LL * p.hidden : p.rows, n = M * p.width;
    if (P == kDx) add_parts<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(to, w.cuts, M, p.width, M, (float*)p.dx, p.dxs, nullptr, 0);
    else
      add_parts<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(to, w.cuts, M, p.width, p.hidden, (float*)p.dwg, p.dgs,
                                                             (float*)p.dwu, p.dus);
  }
  return launch_status();
}
fm_status f32_forward(const GatedParams& p, cudaStream_t st) {
  fm_status s = FM_OK;
  with_act(p.act, [&](auto act) { s = f32_launch<kForward, decltype(act)::value>(p, nullptr, nullptr, st); });
  return s;
}
int64_t f32_d_bytes(const GatedParams& p) { return (p.rows * 2 * (int64_t)p.hidden * (int64_t)sizeof(float) + 255) / 256 * 256; }
int64_t f32_workspace(const GatedParams& p) {
  const Plan x = plan_of(kDx, p), w = plan_of(kDw, p);
  const int64_t a = x.cuts > 1 ? x.cuts * p.rows : 0, b = w.cuts > 1 ? w.cuts * 2LL * p.hidden : 0;
  return f32_d_bytes(p) + (a > b ? a : b) * p.width * (int64_t)sizeof(float);
}
fm_status f32_backward(const GatedParams& p, char* ws, cudaStream_t st) {
  float *d = (float*)ws, *parts = (float*)(ws + f32_d_bytes(p));
  fm_status s = FM_OK;
  with_act(p.act, [&](auto act) { s = f32_launch<kGrads, decltype(act)::value>(p, d, nullptr, st); });
  if (s == FM_OK && p.dx) s = f32_launch<kDx, 0>(p, d, parts, st);
  if (s == FM_OK && (p.dwg || p.dwu)) s = f32_launch<kDw, 0>(p, d, parts, st);
  return s;
}

fm_status check(const fm_gated_args* a) {
  if (a == nullptr) return FM_ERR_INVALID_ARG;
  auto side = [](int64_t n) { return n >= 1 && n <= (1 << 24); };
  if (a->rows < 0 || a->rows > (1LL << 30) || !side(a->width) || !side(a->hidden)) return FM_ERR_INVALID_ARG;
  if (!is_float_type(a->dtype) || (a->in_dtype != a->dtype && a->in_dtype != FM_E4M3)) return FM_ERR_INVALID_ARG;
  if (a->act < FM_ACT_SILU || a->act > FM_ACT_RELU) return FM_ERR_INVALID_ARG;
  return FM_OK;
}
bool apart(int64_t rows, int64_t stride, int64_t length) { return rows <= 1 || stride >= length; }

GatedParams params(const fm_gated_args* a) {
  GatedParams p{};
  p.rows = a->rows;
  p.width = (int)a->width, p.hidden = (int)a->hidden;
  p.act = (int)a->act;
  p.xs = a->x_stride, p.gs = a->gate_stride, p.us = a->up_stride;
  p.x = a->x, p.wg = a->w_gate, p.wu = a->w_up;
  if (a->in_dtype == FM_E4M3) p.x_scales = a->x_scales, p.g_scales = a->gate_scales, p.u_scales = a->up_scales;
  return p;
}
bool workspace_ok(const fm_gated_args* a, int backward) {
  const int64_t need = fm_gated_workspace(a, backward);
  return need == 0 || (need > 0 && a->workspace && a->workspace_bytes >= need && ((uintptr_t)a->workspace & 15) == 0);
}
}  // namespace
}  // namespace fm

using namespace fm;

extern "C" int64_t fm_gated_workspace(const fm_gated_args* a, int backward) {
  if (check(a) != FM_OK || (backward && a->in_dtype == FM_E4M3)) return -1;
  if (a->rows == 0 || (!backward && gated_step_takes(a))) return 0;
  if (a->in_dtype != FM_F32) return gated_tc_workspace(a, backward);
  return backward ? f32_workspace(params(a)) : 0;
}

extern "C" fm_status fm_gated_forward(const fm_gated_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  const bool eight = a->in_dtype == FM_E4M3;
  if (!apart(a->rows, a->x_stride, a->width) || !apart(a->hidden, a->gate_stride, a->width) ||
      !apart(a->hidden, a->up_stride, a->width) || !apart(a->rows, a->h_stride, a->hidden))
    return FM_ERR_INVALID_ARG;
  if (a->rows == 0) return FM_OK;
  if (!a->x || !a->w_gate || !a->w_up || !a->h) return FM_ERR_INVALID_ARG;
  if (eight && (!a->x_scales || !a->gate_scales || !a->up_scales)) return FM_ERR_INVALID_ARG;
  if (!workspace_ok(a, 0)) return FM_ERR_INVALID_ARG;
  GatedParams p = params(a);
  p.h = a->h, p.hs = a->h_stride;
  cudaStream_t st = (cudaStream_t)stream;
  if (gated_step_takes(a)) return gated_step_forward(a, p, st);
  return a->in_dtype == FM_F32 ? f32_forward(p, st) : gated_tc_forward(a, p, st);
}

extern "C" fm_status fm_gated_backward(const fm_gated_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->in_dtype == FM_E4M3) return FM_ERR_INVALID_ARG;
  if (!apart(a->rows, a->x_stride, a->width) || !apart(a->hidden, a->gate_stride, a->width) ||
      !apart(a->hidden, a->up_stride, a->width) || !apart(a->rows, a->dh_stride, a->hidden) ||
      (a->dx && !apart(a->rows, a->dx_stride, a->width)) || (a->dw_gate && !apart(a->hidden, a->dgate_stride, a->width)) ||
      (a->dw_up && !apart(a->hidden, a->dup_stride, a->width)))
    return FM_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->rows == 0) {
    const size_t item = (size_t)item_size(a->dtype), width = (size_t)a->width * item;
    auto clear = [&](void* w, int64_t stride) {
      return !w || cudaMemset2DAsync(w, (size_t)(a->hidden > 1 ? stride : a->width) * item, 0, width, (size_t)a->hidden,
                                     st) == cudaSuccess;
    };
    return clear(a->dw_gate, a->dgate_stride) && clear(a->dw_up, a->dup_stride) ? FM_OK : FM_ERR_CUDA;
  }
  if (!a->x || !a->w_gate || !a->w_up || !a->dh) return FM_ERR_INVALID_ARG;
  if (!a->dx && !a->dw_gate && !a->dw_up) return FM_OK;
  if (!workspace_ok(a, 1)) return FM_ERR_INVALID_ARG;
  GatedParams p = params(a);
  p.dh = a->dh, p.dhs = a->dh_stride;
  p.dx = a->dx, p.dxs = a->dx_stride;
  p.dwg = a->dw_gate, p.dgs = a->dgate_stride;
  p.dwu = a->dw_up, p.dus = a->dup_stride;
  return a->in_dtype == FM_F32 ? f32_backward(p, (char*)a->workspace, st) : gated_tc_backward(a, p, st);
}

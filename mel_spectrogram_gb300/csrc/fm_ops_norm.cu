// Layer norm, forward and backward (fm_ops.h).
//
// Both passes are memory bound: 8 operations per element read or written. A
// row lives in the registers of TPR threads (a warp, or a block for wide
// rows) from its one read to its one write, so x crosses HBM once in the
// forward pass and x and dy once each in the backward pass. The variance is
// the mean of squared deviations from the finished mean (two passes over
// registers), never a difference of sums. Measured for 82688 rows of 1024 in
// bf16: forward 60 us (5.6 TB/s), backward 113 (4.5 TB/s) and 6 for its columns.
#include "fm_ops.cuh"

namespace fm {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxWidth = 8192;  // of the kernels that keep a row in registers
constexpr int kMaxPerSm = 6;     // blocks of the backward kernel an SM, at most

struct NormParams {
  long long rows;
  int width;
  long long xs, ys, dys, dxs;
  float eps;
  const void *x, *w, *b, *dy;
  void *y, *dx;
  float *mean, *rstd;
  float* part;  // [blocks][2][width]: partial dweight, dbias
};

// Sum over the TPR threads that share a row; every thread gets it.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = warp_sum(x);
  if (TPR > 32) {
    const int w = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[w] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) x += red[i];
  }
  return x;
}
// Two sums at once (the backward pass needs both before it can go on).
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (TPR > 32) {
    const int w = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[w] = a, red[32 + w] = b;
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) a += red[i], b += red[32 + i];
  }
}

template <typename T, typename P, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBlock) norm_fwd(const NormParams p) {
  __shared__ float red[64];
  constexpr int kRows = kBlock / TPR;
  const int lane = threadIdx.x % TPR;
  const int nvec = p.width / VEC;
  const float inv = 1.f / (float)p.width;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole row groups leave: with TPR > 32 a block is one row
  const T* x = (const T*)p.x + row * p.xs;
  float v[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int at = n * TPR + lane;
    if (at < nvec) {
      const Pack<T, VEC> q = *(const Pack<T, VEC>*)(x + (long long)at * VEC);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[n][k] = to_f(q.v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[n][k] = 0.f;
    }
  }
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int k = 0; k < VEC; ++k) s += v[n][k];
  const float mean = row_sum<TPR>(s, red) * inv;
  s = 0.f;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    if (n * TPR + lane < nvec) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        v[n][k] -= mean;
        s = fmaf(v[n][k], v[n][k], s);
      }
    }
  }
  const float rstd = 1.f / sqrtf(row_sum<TPR>(s, red) * inv + p.eps);
  if (lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  T* y = (T*)p.y + row * p.ys;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int at = n * TPR + lane;
    if (at < nvec) {
      Pack<P, VEC> w, b;
      if (p.w) w = ((const Pack<P, VEC>*)p.w)[at];
      if (p.b) b = ((const Pack<P, VEC>*)p.b)[at];
      Pack<T, VEC> q;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float r = v[n][k] * rstd;
        if (p.w) r *= to_f(w.v[k]);
        if (p.b) r += to_f(b.v[k]);
        q.v[k] = from_f<T>(r);
      }
      *(Pack<T, VEC>*)(y + (long long)at * VEC) = q;
    }
  }
}

// Rows too wide for registers: three passes over the row, which stays in L2.
template <typename T, typename P>
__global__ void __launch_bounds__(kBlock) norm_fwd_wide(const NormParams p) {
  __shared__ float red[64];
  const long long row = blockIdx.x;
  const T* x = (const T*)p.x + row * p.xs;
  float s = 0.f;
  for (int i = threadIdx.x; i < p.width; i += kBlock) s += to_f(x[i]);
  const float inv = 1.f / (float)p.width;
  const float mean = row_sum<kBlock>(s, red) * inv;
  s = 0.f;
  for (int i = threadIdx.x; i < p.width; i += kBlock) {
    const float d = to_f(x[i]) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.f / sqrtf(row_sum<kBlock>(s, red) * inv + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  T* y = (T*)p.y + row * p.ys;
  for (int i = threadIdx.x; i < p.width; i += kBlock) {
    float r = (to_f(x[i]) - mean) * rstd;
    if (p.w) r *= to_f(((const P*)p.w)[i]);
    if (p.b) r += to_f(((const P*)p.b)[i]);
    y[i] = from_f<T>(r);
  }
}

// dx = rstd * (h - mean(h) - n * mean(h n)), h = dy * weight, n = (x - mean) * rstd;
// every thread also sums dy * n and dy of its own columns over the rows its
// block takes (block, block + grid, ...), and the block writes one partial
// row of each. Fixed order throughout.
//
// A warp keeps a row's 64 sums per lane of 32 elements, so registers leave
// twelve warps an SM; their reads and the arithmetic between them take turns.
// Compared for 82688 rows of 1024 in bf16 (508 MB), by itself over and over on the
// same inputs, which leaves some of them in L2 (113 us from a cold one): 100 us in
// blocks of four warps, three to an SM; 127 in blocks of eight (one and a half
// fit); 103 with the next row's reads ahead (254 registers, eight warps); 106 to
// 123 with two or four warps a row, whose sums then need barriers.
constexpr int kBwdWarps = 4;
template <int TPR, int E>  // threads of a block, and blocks meant to fit an SM
constexpr int kBwdThreads = TPR == 32 ? 32 * kBwdWarps : TPR;
template <int TPR, int E>
constexpr int kBwdBlocks = (E > 16 ? 384 : E > 8 ? 512 : 768) / kBwdThreads<TPR, E>;
template <typename T, typename P, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBwdThreads<TPR, NV * VEC>, kBwdBlocks<TPR, NV * VEC>) norm_bwd(const NormParams p) {
  __shared__ float red[64];
  extern __shared__ float cols[];  // [kRows][width], TPR == 32 only
  constexpr int kThreads = kBwdThreads<TPR, NV * VEC>, kRows = kThreads / TPR;
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nvec = p.width / VEC;
  const float inv = 1.f / (float)p.width;
  float dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw[n][k] = db[n][k] = 0.f;

  for (long long row = (long long)blockIdx.x * kRows + sub; row < p.rows; row += (long long)gridDim.x * kRows) {
    const T* x = (const T*)p.x + row * p.xs;
    const T* dy = (const T*)p.dy + row * p.dys;
    Pack<T, VEC> qx[NV], qd[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        qx[n] = *(const Pack<T, VEC>*)(x + (long long)at * VEC);
        qd[n] = *(const Pack<T, VEC>*)(dy + (long long)at * VEC);
      }
    }
    const float mean = p.mean[row], rstd = p.rstd[row];
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        Pack<P, VEC> w;
        if (p.w) w = ((const Pack<P, VEC>*)p.w)[at];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float d = to_f(qd[n].v[k]), xn = (to_f(qx[n].v[k]) - mean) * rstd;
          dw[n][k] = fmaf(d, xn, dw[n][k]);
          db[n][k] += d;
          const float h = p.w ? d * to_f(w.v[k]) : d;
          a += h;
          b = fmaf(h, xn, b);
        }
      }
    }
    if (p.dx) {
      row_sum2<TPR>(a, b, red);
      a *= inv;
      b *= inv;
      T* dx = (T*)p.dx + row * p.dxs;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int at = n * TPR + lane;
        if (at < nvec) {
          Pack<P, VEC> w;
          if (p.w) w = ((const Pack<P, VEC>*)p.w)[at];
          Pack<T, VEC> q;
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float d = to_f(qd[n].v[k]), xn = (to_f(qx[n].v[k]) - mean) * rstd;
            const float h = p.w ? d * to_f(w.v[k]) : d;
            q.v[k] = from_f<T>(rstd * (h - a - xn * b));
          }
          *(Pack<T, VEC>*)(dx + (long long)at * VEC) = q;
        }
      }
    }
  }
  if (p.part == nullptr) return;
  float* out = p.part + (long long)blockIdx.x * 2 * p.width;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (TPR == 32) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int at = n * TPR + lane;
        if (at < nvec)
#pragma unroll
          for (int k = 0; k < VEC; ++k) cols[sub * p.width + at * VEC + k] = which ? db[n][k] : dw[n][k];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < p.width; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += cols[r * p.width + i];
        out[which * p.width + i] = s;
      }
    } else {
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int at = n * TPR + lane;
        if (at < nvec)
#pragma unroll
          for (int k = 0; k < VEC; ++k) out[which * p.width + at * VEC + k] = which ? db[n][k] : dw[n][k];
      }
    }
  }
}

// Wide rows: dx from three reads of the row, one block a row ...
template <typename T, typename P>
__global__ void __launch_bounds__(kBlock) norm_bwd_wide(const NormParams p) {
  __shared__ float red[64];
  const long long row = blockIdx.x;
  const T* x = (const T*)p.x + row * p.xs;
  const T* dy = (const T*)p.dy + row * p.dys;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float a = 0.f, b = 0.f;
  for (int i = threadIdx.x; i < p.width; i += kBlock) {
    const float h = to_f(dy[i]) * (p.w ? to_f(((const P*)p.w)[i]) : 1.f);
    a += h;
    b = fmaf(h, (to_f(x[i]) - mean) * rstd, b);
  }
  row_sum2<kBlock>(a, b, red);
  a /= (float)p.width;
  b /= (float)p.width;
  T* dx = (T*)p.dx + row * p.dxs;
  for (int i = threadIdx.x; i < p.width; i += kBlock) {
    const float h = to_f(dy[i]) * (p.w ? to_f(((const P*)p.w)[i]) : 1.f);
    dx[i] = from_f<T>(rstd * (h - a - (to_f(x[i]) - mean) * rstd * b));
  }
}
// ... and the column sums by a thread per column over a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kBlock) norm_cols_wide(const NormParams p) {
  const int i = blockIdx.x * kBlock + threadIdx.x;
  if (i >= p.width) return;
  float dw = 0.f, db = 0.f;
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float d = to_f(((const T*)p.dy)[row * p.dys + i]);
    const float xn = (to_f(((const T*)p.x)[row * p.xs + i]) - p.mean[row]) * p.rstd[row];
    dw = fmaf(d, xn, dw);
    db += d;
  }
  float* out = p.part + (long long)blockIdx.y * 2 * p.width;
  out[i] = dw;
  out[p.width + i] = db;
}

// Sum of the partial rows: 32 columns a block, 32 row groups, then the groups.
template <typename P>
__global__ void __launch_bounds__(1024) norm_cols(const float* part, int blocks, int width, void* dw, void* db) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const long long n2 = 2LL * width;
  const long long col = (long long)blockIdx.x * 32 + c;
  float a = 0.f;
  if (col < n2) {
#pragma unroll 8
    for (int r = g; r < blocks; r += 32) a += part[r * n2 + col];
  }
  s[g][c] = a;
  __syncthreads();
  if (g == 0 && col < n2) {
    a = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) a += s[r][c];
    void* to = col < width ? dw : db;
    if (to) ((P*)to)[col < width ? col : col - width] = from_f<P>(a);
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// 16-byte accesses where every row of every array starts on such a boundary;
// one element at a time otherwise (odd widths, views at odd offsets).
template <typename T>
bool vector_ok(const NormParams& p, int vec, int64_t param_item) {
  auto row_ok = [&](const void* q, long long s) { return q == nullptr || (aligned16(q) && s % vec == 0); };
  auto par_ok = [&](const void* q) { return q == nullptr || ((uintptr_t)q % (vec * param_item)) == 0; };
  return p.width % vec == 0 && row_ok(p.x, p.xs) && row_ok(p.y, p.ys) && row_ok(p.dy, p.dys) &&
         row_ok(p.dx, p.dxs) && par_ok(p.w) && par_ok(p.b);
}

template <typename T, typename P, int VEC, int TPR, int NV>
void fwd_launch(const NormParams& p, cudaStream_t st) {
  const long long blocks = (p.rows * TPR + kBlock - 1) / kBlock;
  norm_fwd<T, P, VEC, TPR, NV><<<(unsigned)blocks, kBlock, 0, st>>>(p);
}
template <typename T, typename P, int VEC>
bool fwd_vec(const NormParams& p, cudaStream_t st) {
  constexpr bool kNarrow = VEC < 8;  // eight packs of eight would spill
  const int n = p.width / VEC;
  if (n <= 32) fwd_launch<T, P, VEC, 32, 1>(p, st);
  else if (n <= 64) fwd_launch<T, P, VEC, 32, 2>(p, st);
  else if (n <= 128) fwd_launch<T, P, VEC, 32, 4>(p, st);
  else if (n <= 256 && kNarrow) fwd_launch<T, P, VEC, 32, kNarrow ? 8 : 1>(p, st);
  else if (n <= 256) fwd_launch<T, P, VEC, 256, 1>(p, st);
  else if (n <= 512) fwd_launch<T, P, VEC, 256, 2>(p, st);
  else if (n <= 1024) fwd_launch<T, P, VEC, 256, 4>(p, st);
  else if (n <= 2048 && kNarrow) fwd_launch<T, P, VEC, 256, kNarrow ? 8 : 1>(p, st);
  else return false;
  return true;
}
template <typename T, typename P>
void fwd_typed(const NormParams& p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool done = vector_ok<T>(p, V, sizeof(P)) ? fwd_vec<T, P, V>(p, st) : fwd_vec<T, P, 1>(p, st);
  if (!done) norm_fwd_wide<T, P><<<(unsigned)p.rows, kBlock, 0, st>>>(p);
}

// Blocks of the backward kernel: enough to fill the SMs, few enough that the
// partial rows stay small beside the rows themselves.
int partial_blocks(long long rows, int rows_per_block, int per_sm) {
  const long long want = (rows + rows_per_block - 1) / rows_per_block;
  const long long most = (long long)per_sm * num_sms();
  return (int)(want < most ? (want < 1 ? 1 : want) : most);
}

// Slices of the rows for the column sums of wide rows.
int wide_blocks(long long rows, int width) {
  const long long columns = (width + kBlock - 1) / kBlock, want = (2LL * num_sms() + columns - 1) / columns;
  const long long most = (rows + 7) / 8;
  return (int)(want < most ? want : most < 1 ? 1 : most);
}

template <typename T, typename P, int VEC, int TPR, int NV>
int bwd_launch(const NormParams& p, cudaStream_t st) {
  constexpr int threads = kBwdThreads<TPR, NV * VEC>, rows = threads / TPR;
  const int blocks = partial_blocks(p.rows, rows, kBwdBlocks<TPR, NV * VEC>);
  const size_t smem = TPR == 32 ? sizeof(float) * rows * p.width : 0;
  auto k = norm_bwd<T, P, VEC, TPR, NV>;
  if (!allow_smem(k, smem)) return -1;
  k<<<blocks, threads, smem, st>>>(p);
  return blocks;
}
template <typename T, typename P, int VEC>
int bwd_vec(const NormParams& p, cudaStream_t st) {
  constexpr bool kNarrow = VEC < 8;  // eight packs of eight would spill
  const int n = p.width / VEC;
  if (n <= 32) return bwd_launch<T, P, VEC, 32, 1>(p, st);
  if (n <= 64) return bwd_launch<T, P, VEC, 32, 2>(p, st);
  if (n <= 128) return bwd_launch<T, P, VEC, 32, 4>(p, st);
  if (n <= 256 && kNarrow) return bwd_launch<T, P, VEC, 32, kNarrow ? 8 : 1>(p, st);
  if (n <= 256) return bwd_launch<T, P, VEC, 256, 1>(p, st);
  if (n <= 512) return bwd_launch<T, P, VEC, 256, 2>(p, st);
  if (n <= 1024) return bwd_launch<T, P, VEC, 256, 4>(p, st);
  if (n <= 2048 && kNarrow) return bwd_launch<T, P, VEC, 256, kNarrow ? 8 : 1>(p, st);
  return 0;
}
template <typename T, typename P>
fm_status bwd_typed(const NormParams& p, void* dw, void* db, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  int blocks = vector_ok<T>(p, V, sizeof(P)) ? bwd_vec<T, P, V>(p, st) : bwd_vec<T, P, 1>(p, st);
  if (blocks < 0) return FM_ERR_CUDA;
  if (blocks == 0) {
    if (p.dx) norm_bwd_wide<T, P><<<(unsigned)p.rows, kBlock, 0, st>>>(p);
    if (p.part) {
      blocks = wide_blocks(p.rows, p.width);
      norm_cols_wide<T><<<dim3((p.width + kBlock - 1) / kBlock, blocks), kBlock, 0, st>>>(p);
    }
  }
  if (p.part)
    norm_cols<P><<<(unsigned)((2LL * p.width + 31) / 32), 1024, 0, st>>>(p.part, blocks, p.width, dw, db);
  return launch_status();
}

fm_status check(const fm_layer_norm_args* a) {
  if (a == nullptr) return FM_ERR_INVALID_ARG;
  if (a->rows < 0 || a->rows > 0x7fffffffLL || a->width < 1 || a->width > (1 << 24)) return FM_ERR_INVALID_ARG;
  if (!is_float_type(a->dtype) || (a->param_dtype != a->dtype && a->param_dtype != FM_F32))
    return FM_ERR_INVALID_ARG;
  if (!(a->eps >= 0)) return FM_ERR_INVALID_ARG;
  return FM_OK;
}
bool stride_ok(const fm_layer_norm_args* a, int64_t s) { return a->rows <= 1 || s >= a->width; }

NormParams params(const fm_layer_norm_args* a) {
  NormParams p{};
  p.rows = a->rows;
  p.width = (int)a->width;
  p.xs = a->x_stride;
  p.eps = (float)a->eps;
  p.x = a->x;
  p.w = a->weight;
  p.mean = a->mean;
  p.rstd = a->rstd;
  return p;
}
}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status fm_layer_norm_forward(const fm_layer_norm_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (!stride_ok(a, a->x_stride) || !stride_ok(a, a->y_stride)) return FM_ERR_INVALID_ARG;
  if (a->rows == 0) return FM_OK;
  if (a->x == nullptr || a->y == nullptr) return FM_ERR_INVALID_ARG;
  NormParams p = params(a);
  p.ys = a->y_stride;
  p.b = a->bias;
  p.y = a->y;
  cudaStream_t st = (cudaStream_t)stream;
  const bool wide = a->param_dtype == FM_F32;
  if (a->dtype == FM_F32) fwd_typed<float, float>(p, st);
  else if (a->dtype == FM_F16) wide ? fwd_typed<__half, float>(p, st) : fwd_typed<__half, __half>(p, st);
  else wide ? fwd_typed<__nv_bfloat16, float>(p, st) : fwd_typed<__nv_bfloat16, __nv_bfloat16>(p, st);
  return launch_status();
}

extern "C" int64_t fm_layer_norm_workspace(const fm_layer_norm_args* a) {
  if (check(a) != FM_OK) return -1;
  // one partial row of each gradient per block, whichever variant runs
  int64_t blocks = wide_blocks(a->rows, (int)a->width);
  if (a->width <= kMaxWidth) {
    const int64_t n = partial_blocks(a->rows, 1, kMaxPerSm);
    if (n > blocks) blocks = n;
  }
  return blocks * 2 * a->width * (int64_t)sizeof(float);
}

extern "C" fm_status fm_layer_norm_backward(const fm_layer_norm_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (!stride_ok(a, a->x_stride) || !stride_ok(a, a->dy_stride) || (a->dx && !stride_ok(a, a->dx_stride)))
    return FM_ERR_INVALID_ARG;
  const bool sums = a->dweight != nullptr || a->dbias != nullptr;
  if (a->rows > 0 && (a->x == nullptr || a->dy == nullptr || a->mean == nullptr || a->rstd == nullptr))
    return FM_ERR_INVALID_ARG;
  if (sums && (a->workspace == nullptr || a->workspace_bytes < fm_layer_norm_workspace(a) ||
               ((uintptr_t)a->workspace & 15)))
    return FM_ERR_INVALID_ARG;
  if (!sums && a->dx == nullptr) return FM_OK;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->rows == 0) {
    const size_t n = (size_t)a->width * item_size(a->param_dtype);
    if (a->dweight && cudaMemsetAsync(a->dweight, 0, n, st) != cudaSuccess) return FM_ERR_CUDA;
    if (a->dbias && cudaMemsetAsync(a->dbias, 0, n, st) != cudaSuccess) return FM_ERR_CUDA;
    return FM_OK;
  }
  NormParams p = params(a);
  p.dys = a->dy_stride;
  p.dxs = a->dx_stride;
  p.dy = a->dy;
  p.dx = a->dx;
  p.part = sums ? (float*)a->workspace : nullptr;
  const bool wide = a->param_dtype == FM_F32;
  if (a->dtype == FM_F32) return bwd_typed<float, float>(p, a->dweight, a->dbias, st);
  if (a->dtype == FM_F16)
    return wide ? bwd_typed<__half, float>(p, a->dweight, a->dbias, st)
                : bwd_typed<__half, __half>(p, a->dweight, a->dbias, st);
  return wide ? bwd_typed<__nv_bfloat16, float>(p, a->dweight, a->dbias, st)
              : bwd_typed<__nv_bfloat16, __nv_bfloat16>(p, a->dweight, a->dbias, st);
}

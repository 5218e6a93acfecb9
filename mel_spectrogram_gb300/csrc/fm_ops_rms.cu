// Root-mean-square norm with the residual's addition, forward and backward, and
// rows in 8 bits (fm_ops.h).
//
// Memory bound: 6 operations per element. A row lives in the registers of TPR
// threads (a warp, or a block for wide rows) from its one read to its one write:
// x and residual are read once, total and y written once; the 8-bit form takes the
// largest |y| of a row from the same registers, so that y is never held in 16 bits.
// Measured for 82688 rows of 1024 in bf16: forward 105 us (6.4 TB/s), in 8 bits 100
// (5.9 TB/s), backward 117 (5.8 TB/s) and 5 for its columns.
#include <cuda_fp8.h>

#include "fm_ops_rows.cuh"
#include "fm_tc.cuh"

namespace fm {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxWidth = 8192;  // of the kernels that keep a row in registers
constexpr int kMaxPerSm = 6;     // blocks of the backward kernel an SM, at most
constexpr float kLargest = 448.f;

struct RmsParams {
  long long rows;
  int width;
  long long xs, rs, ts, ys, dys, dts, dxs;
  float eps;
  const void *x, *res, *w, *dy, *dt;
  void *total, *y, *dx;
  float *scales, *rstd;
  float* part;  // [blocks][width]: partial dweight
};

struct E4M3 {
  uint8_t bits;
};
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ E4M3 e4m3(float x) { return E4M3{__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3)}; }

// 16 bytes to shared memory, without waiting
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from)
               : "memory");
}

// Largest |x| over the threads that share a row, by bits: infinities and then NaN
// are the largest of all.
__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
template <int TPR>
__device__ __forceinline__ unsigned row_max(unsigned x, unsigned* red) {
  x = __reduce_max_sync(0xffffffffu, x);
  if (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) x = max(x, red[i]);
  }
  return x;
}
// 2^-126 at the least, so that no value overflows in the division by it; NaN where
// the row holds an infinity or NaN
__device__ __forceinline__ float scale_of(unsigned largest) {
  return largest >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                                : fmaxf(__uint_as_float(largest) / kLargest, 1.17549435e-38f);
}

// v / scale by the reciprocal's two halves: it is known to 46 bits (29 for scales beyond
// 2^120), so that the one rounding of the sum gives the rounded quotient but for borders
// closer than that. The first half is rounded down, which keeps both of one sign and a -0
// one. 82688 rows of 1024 in bf16 with the norm (without): 104 us (45), by the rounded reciprocal
// alone, whose quotients are off by one and a half last places, 104 (43), by divisions 125 (55).
struct Inverse {
  float first, rest;
  __device__ explicit Inverse(float scale) {
    first = __frcp_rd(scale);
    rest = fmaf(-first, scale, 1.f) * first;
  }
  __device__ float2 times(float2 v) const {
    return tc::fma2(v, tc::both(first), tc::mul2(v, tc::both(rest)));
  }
  __device__ float times(float v) const { return fmaf(v, first, v * rest); }
};

// total = x + residual as it is held
template <typename T>
__device__ __forceinline__ T sum_of(T x, T r) {
  return from_f<T>(to_f(x) + to_f(r));
}

// NORM: the norm; otherwise y is x. EIGHT: y in 8 bits.
template <typename T, typename P, int VEC, int TPR, int NV, bool NORM, bool EIGHT>
__global__ void __launch_bounds__(kBlock) rms_fwd(const RmsParams p) {
  __shared__ float red[64];
  constexpr int kRows = kBlock / TPR;
  const int lane = threadIdx.x % TPR;
  const int nvec = p.width / VEC;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole row groups leave: with TPR > 32 a block is one row
  const T* x = (const T*)p.x + row * p.xs;
  float v[NV][VEC];
  if (NORM && p.res) {
    const T* res = (const T*)p.res + row * p.rs;
    Pack<T, VEC> q[NV], r[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        q[n] = *(const Pack<T, VEC>*)(x + (long long)at * VEC);
        r[n] = *(const Pack<T, VEC>*)(res + (long long)at * VEC);
      }
    }
    T* total = (T*)p.total + row * p.ts;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        q[n].v[k] = sum_of(q[n].v[k], r[n].v[k]);
        v[n][k] = at < nvec ? to_f(q[n].v[k]) : 0.f;
      }
      if (at < nvec) *(Pack<T, VEC>*)(total + (long long)at * VEC) = q[n];
    }
  } else {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      Pack<T, VEC> q;
      if (at < nvec) q = *(const Pack<T, VEC>*)(x + (long long)at * VEC);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[n][k] = at < nvec ? to_f(q.v[k]) : 0.f;
    }
  }
  if (NORM) {
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) s = fmaf(v[n][k], v[n][k], s);
    const float rstd = 1.f / sqrtf(row_sum<TPR>(s, red) / (float)p.width + p.eps);
    if (lane == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        Pack<P, VEC> w;
        if (p.w) w = ((const Pack<P, VEC>*)p.w)[at];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          v[n][k] *= rstd;
          if (p.w) v[n][k] *= to_f(w.v[k]);
        }
      }
    }
  }
  if (EIGHT) {
    unsigned m = 0;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) m = max(m, abs_bits(v[n][k]));
    const float scale = scale_of(row_max<TPR>(m, (unsigned*)red));
    if (lane == 0) p.scales[row] = scale;
    const Inverse inv(scale);
    E4M3* y = (E4M3*)p.y + row * p.ys;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        if (VEC == 1) {
          y[at] = e4m3(inv.times(v[n][0]));
        } else {
          Pack<uint16_t, (VEC + 1) / 2> q;
#pragma unroll
          for (int k = 0; k < VEC / 2; ++k) {
            const float2 two = inv.times(make_float2(v[n][2 * k], v[n][(2 * k + 1) % VEC]));
            q.v[k] = e4m3x2(two.x, two.y);
          }
          *(Pack<uint16_t, (VEC + 1) / 2>*)(y + (long long)at * VEC) = q;
        }
      }
    }
  } else {
    T* y = (T*)p.y + row * p.ys;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        Pack<T, VEC> q;
#pragma unroll
        for (int k = 0; k < VEC; ++k) q.v[k] = from_f<T>(v[n][k]);
        *(Pack<T, VEC>*)(y + (long long)at * VEC) = q;
      }
    }
  }
}

// Rows too wide for registers: further passes over the row, which stays in L2.
template <typename T, typename P, bool NORM, bool EIGHT>
__global__ void __launch_bounds__(kBlock) rms_fwd_wide(const RmsParams p) {
  __shared__ float red[64];
  const long long row = blockIdx.x;
  const T* x = (const T*)p.x + row * p.xs;
  float s = 0.f;
  if (NORM && p.res) {  // every thread reads again only what it wrote itself
    const T* res = (const T*)p.res + row * p.rs;
    T* total = (T*)p.total + row * p.ts;
    for (int i = threadIdx.x; i < p.width; i += kBlock) {
      total[i] = sum_of(x[i], res[i]);
      const float v = to_f(total[i]);
      s = fmaf(v, v, s);
    }
    x = total;
  } else if (NORM) {
    for (int i = threadIdx.x; i < p.width; i += kBlock) {
      const float v = to_f(x[i]);
      s = fmaf(v, v, s);
    }
  }
  float rstd = 1.f;
  if (NORM) {
    rstd = 1.f / sqrtf(row_sum<kBlock>(s, red) / (float)p.width + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
  }
  auto value = [&](int i) {
    float v = to_f(x[i]);
    if (NORM) v *= rstd;
    if (NORM && p.w) v *= to_f(((const P*)p.w)[i]);
    return v;
  };
  float scale = 1.f;
  if (EIGHT) {
    unsigned m = 0;
    for (int i = threadIdx.x; i < p.width; i += kBlock) m = max(m, abs_bits(value(i)));
    scale = scale_of(row_max<kBlock>(m, (unsigned*)red));
    if (threadIdx.x == 0) p.scales[row] = scale;
  }
  const Inverse inv(scale);
  for (int i = threadIdx.x; i < p.width; i += kBlock) {
    if (EIGHT) ((E4M3*)p.y)[row * p.ys + i] = e4m3(inv.times(value(i)));
    else ((T*)p.y)[row * p.ys + i] = from_f<T>(value(i));
  }
}

// dx = dtotal + rstd * (h - n * mean(h n)), h = dy * weight, n = total * rstd; every
// thread also sums dy * n of its own columns over the rows its block takes (block,
// block + grid, ...), and the block writes one partial row. Fixed order throughout.
constexpr int kBwdWarps = 4;
template <int TPR>
constexpr int kBwdThreads = TPR == 32 ? 32 * kBwdWarps : TPR;
template <int TPR, int E>  // blocks meant to fit an SM
constexpr int kBwdBlocks = (E > 16 ? 384 : E > 8 ? 512 : 768) / kBwdThreads<TPR>;
template <typename T, typename P, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBwdThreads<TPR>, kBwdBlocks<TPR, NV * VEC>) rms_bwd(const RmsParams p) {
  __shared__ float red[64];
  extern __shared__ float cols[];  // [kRows][width], TPR == 32 only
  constexpr int kThreads = kBwdThreads<TPR>, kRows = kThreads / TPR;
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nvec = p.width / VEC;
  const float inv = 1.f / (float)p.width;
  float dw[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw[n][k] = 0.f;

  for (long long row = (long long)blockIdx.x * kRows + sub; row < p.rows; row += (long long)gridDim.x * kRows) {
    const T* x = (const T*)p.x + row * p.xs;
    const T* dy = (const T*)p.dy + row * p.dys;
    const T* dt = p.dt ? (const T*)p.dt + row * p.dts : nullptr;
    Pack<T, VEC> qx[NV], qd[NV], qt[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        qx[n] = *(const Pack<T, VEC>*)(x + (long long)at * VEC);
        qd[n] = *(const Pack<T, VEC>*)(dy + (long long)at * VEC);
        if (dt) qt[n] = *(const Pack<T, VEC>*)(dt + (long long)at * VEC);
      }
    }
    const float rstd = p.rstd[row];
    float b = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec) {
        Pack<P, VEC> w;
        if (p.w) w = ((const Pack<P, VEC>*)p.w)[at];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float dn = to_f(qd[n].v[k]) * (to_f(qx[n].v[k]) * rstd);
          dw[n][k] += dn;
          b = p.w ? fmaf(dn, to_f(w.v[k]), b) : b + dn;
        }
      }
    }
    if (p.dx) {
      b = row_sum<TPR>(b, red) * inv;
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
            const float d = to_f(qd[n].v[k]), h = p.w ? d * to_f(w.v[k]) : d;
            float g = rstd * (h - to_f(qx[n].v[k]) * rstd * b);
            if (dt) g += to_f(qt[n].v[k]);
            q.v[k] = from_f<T>(g);
          }
          *(Pack<T, VEC>*)(dx + (long long)at * VEC) = q;
        }
      }
    }
  }
  if (p.part == nullptr) return;
  float* out = p.part + (long long)blockIdx.x * p.width;
  if (TPR == 32) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec)
#pragma unroll
        for (int k = 0; k < VEC; ++k) cols[sub * p.width + at * VEC + k] = dw[n][k];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.width; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += cols[r * p.width + i];
      out[i] = s;
    }
  } else {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = n * TPR + lane;
      if (at < nvec)
#pragma unroll
        for (int k = 0; k < VEC; ++k) out[at * VEC + k] = dw[n][k];
    }
  }
}

// The same where rows are read 16 bytes at a time: the next rows come to shared memory
// (each thread's own places) while one is worked on, so that a warp always has reads
// under way and a row takes no registers between the two passes over it. In registers
// alone, 82688 rows of 1024 in bf16 took 205 us, their reads and the arithmetic between
// them taking turns; this way 117. With three rows ahead in three blocks an SM 126.
template <int NV>
constexpr int kAhead = NV <= 2 ? 4 : 2;  // rows of a thread in shared memory
template <int TPR, int NV>
constexpr int kRingBytes = kAhead<NV> * 3 * NV * 16 * kBwdThreads<TPR>;
template <typename T, typename P, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBwdThreads<TPR>, 512 / kBwdThreads<TPR>) rms_bwd_ring(const RmsParams p) {
  __shared__ float red[64];
  extern __shared__ __align__(16) unsigned char raw[];
  constexpr int kThreads = kBwdThreads<TPR>, kRows = kThreads / TPR, kDeep = kAhead<NV>;
  uint4* ring = (uint4*)raw + threadIdx.x;  // [kDeep][3][NV][kThreads]
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nvec = p.width / VEC;
  const float inv = 1.f / (float)p.width;
  const long long step = (long long)gridDim.x * kRows;
  float dw[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw[n][k] = 0.f;

  auto at = [&](int slot, int array, int n) { return ring + ((slot * 3 + array) * NV + n) * kThreads; };
  auto fetch = [&](long long row, int slot) {
    if (row < p.rows) {
      const T *x = (const T*)p.x + row * p.xs, *dy = (const T*)p.dy + row * p.dys;
      const T* dt = p.dt ? (const T*)p.dt + row * p.dts : nullptr;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = n * TPR + lane;
        if (i < nvec) {
          copy16(at(slot, 0, n), x + (long long)i * VEC);
          copy16(at(slot, 1, n), dy + (long long)i * VEC);
          if (dt) copy16(at(slot, 2, n), dt + (long long)i * VEC);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  long long row = (long long)blockIdx.x * kRows + sub;
#pragma unroll
  for (int i = 0; i < kDeep - 1; ++i) fetch(row + i * step, i);
  float next_rstd = row < p.rows ? p.rstd[row] : 0.f;
  int slot = 0;
  // with TPR > 32 a block is one row, and its threads take as many turns
  for (; row < p.rows; row += step) {
    const int last = slot == 0 ? kDeep - 1 : slot - 1;  // of the row before this one: free
    fetch(row + (kDeep - 1) * step, last);
    const float rstd = next_rstd;
    if (row + step < p.rows) next_rstd = p.rstd[row + step];
    asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
    float b = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = n * TPR + lane;
      if (i < nvec) {
        const Pack<T, VEC> qx = *(const Pack<T, VEC>*)at(slot, 0, n), qd = *(const Pack<T, VEC>*)at(slot, 1, n);
        Pack<P, VEC> w;
        if (p.w) w = ((const Pack<P, VEC>*)p.w)[i];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float dn = to_f(qd.v[k]) * (to_f(qx.v[k]) * rstd);
          dw[n][k] += dn;
          b = p.w ? fmaf(dn, to_f(w.v[k]), b) : b + dn;
        }
      }
    }
    if (p.dx) {
      b = row_sum<TPR>(b, red) * inv * rstd;
      T* dx = (T*)p.dx + row * p.dxs;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int i = n * TPR + lane;
        if (i < nvec) {
          const Pack<T, VEC> qx = *(const Pack<T, VEC>*)at(slot, 0, n), qd = *(const Pack<T, VEC>*)at(slot, 1, n);
          Pack<T, VEC> q;
          if (p.dt) q = *(const Pack<T, VEC>*)at(slot, 2, n);
          Pack<P, VEC> w;
          if (p.w) w = ((const Pack<P, VEC>*)p.w)[i];
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float d = to_f(qd.v[k]), h = p.w ? d * to_f(w.v[k]) : d;
            float g = rstd * fmaf(-to_f(qx.v[k]), b, h);
            if (p.dt) g += to_f(q.v[k]);
            q.v[k] = from_f<T>(g);
          }
          *(Pack<T, VEC>*)(dx + (long long)i * VEC) = q;
        }
      }
    }
    slot = slot + 1 == kDeep ? 0 : slot + 1;
  }
  if (p.part == nullptr) return;
  float* out = p.part + (long long)blockIdx.x * p.width;
  if (TPR == 32) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the ring becomes [kRows][width] sums
    float* cols = (float*)raw;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = n * TPR + lane;
      if (i < nvec)
#pragma unroll
        for (int k = 0; k < VEC; ++k) cols[sub * p.width + i * VEC + k] = dw[n][k];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.width; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += cols[r * p.width + i];
      out[i] = s;
    }
  } else {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = n * TPR + lane;
      if (i < nvec)
#pragma unroll
        for (int k = 0; k < VEC; ++k) out[i * VEC + k] = dw[n][k];
    }
  }
}

// Wide rows: dx from two reads of the row, one block a row ...
template <typename T, typename P>
__global__ void __launch_bounds__(kBlock) rms_bwd_wide(const RmsParams p) {
  __shared__ float red[64];
  const long long row = blockIdx.x;
  const T* x = (const T*)p.x + row * p.xs;
  const T* dy = (const T*)p.dy + row * p.dys;
  const T* dt = p.dt ? (const T*)p.dt + row * p.dts : nullptr;
  const float rstd = p.rstd[row];
  auto h = [&](int i) { return to_f(dy[i]) * (p.w ? to_f(((const P*)p.w)[i]) : 1.f); };
  float b = 0.f;
  for (int i = threadIdx.x; i < p.width; i += kBlock) b = fmaf(h(i), to_f(x[i]) * rstd, b);
  b = row_sum<kBlock>(b, red) / (float)p.width;
  T* dx = (T*)p.dx + row * p.dxs;
  for (int i = threadIdx.x; i < p.width; i += kBlock) {
    float g = rstd * (h(i) - to_f(x[i]) * rstd * b);
    if (dt) g += to_f(dt[i]);
    dx[i] = from_f<T>(g);
  }
}
// ... and the column sums by a thread per column over a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kBlock) rms_cols_wide(const RmsParams p) {
  const int i = blockIdx.x * kBlock + threadIdx.x;
  if (i >= p.width) return;
  float dw = 0.f;
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y)
    dw = fmaf(to_f(((const T*)p.dy)[row * p.dys + i]), to_f(((const T*)p.x)[row * p.xs + i]) * p.rstd[row], dw);
  p.part[(long long)blockIdx.y * p.width + i] = dw;
}

// 16-byte accesses where every row of every array starts on such a boundary (of
// half as many bytes for 8-bit values); one element at a time otherwise (odd widths,
// views at odd offsets).
template <typename T>
bool vector_ok(const RmsParams& p, int vec, int64_t param_item, bool eight) {
  auto row_ok = [&](const void* q, long long s) { return q == nullptr || (aligned16(q) && s % vec == 0); };
  const bool y = eight ? ((uintptr_t)p.y % vec) == 0 && p.ys % vec == 0 : row_ok(p.y, p.ys);
  return p.width % vec == 0 && row_ok(p.x, p.xs) && row_ok(p.res, p.rs) && row_ok(p.total, p.ts) && y &&
         row_ok(p.dy, p.dys) && row_ok(p.dt, p.dts) && row_ok(p.dx, p.dxs) &&
         (p.w == nullptr || ((uintptr_t)p.w % (vec * param_item)) == 0);
}

template <typename T, typename P, int VEC, int TPR, int NV, bool NORM, bool EIGHT>
void fwd_launch(const RmsParams& p, cudaStream_t st) {
  const long long blocks = (p.rows * TPR + kBlock - 1) / kBlock;
  rms_fwd<T, P, VEC, TPR, NV, NORM, EIGHT><<<(unsigned)blocks, kBlock, 0, st>>>(p);
}
template <typename T, typename P, int VEC, bool NORM, bool EIGHT>
bool fwd_vec(const RmsParams& p, cudaStream_t st) {
  constexpr bool kNarrow = VEC < 8;  // eight packs of eight would spill
  const int n = p.width / VEC;
  if (n <= 32) fwd_launch<T, P, VEC, 32, 1, NORM, EIGHT>(p, st);
  else if (n <= 64) fwd_launch<T, P, VEC, 32, 2, NORM, EIGHT>(p, st);
  else if (n <= 128) fwd_launch<T, P, VEC, 32, 4, NORM, EIGHT>(p, st);
  else if (n <= 256 && kNarrow) fwd_launch<T, P, VEC, 32, kNarrow ? 8 : 1, NORM, EIGHT>(p, st);
  else if (n <= 256) fwd_launch<T, P, VEC, 256, 1, NORM, EIGHT>(p, st);
  else if (n <= 512) fwd_launch<T, P, VEC, 256, 2, NORM, EIGHT>(p, st);
  else if (n <= 1024) fwd_launch<T, P, VEC, 256, 4, NORM, EIGHT>(p, st);
  else if (n <= 2048 && kNarrow) fwd_launch<T, P, VEC, 256, kNarrow ? 8 : 1, NORM, EIGHT>(p, st);
  else return false;
  return true;
}
template <typename T, typename P, bool NORM, bool EIGHT>
void fwd_typed(const RmsParams& p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool done = vector_ok<T>(p, V, sizeof(P), EIGHT) ? fwd_vec<T, P, V, NORM, EIGHT>(p, st)
                                                         : fwd_vec<T, P, 1, NORM, EIGHT>(p, st);
  if (!done) rms_fwd_wide<T, P, NORM, EIGHT><<<(unsigned)p.rows, kBlock, 0, st>>>(p);
}
template <typename T, typename P>
void fwd_norm(const RmsParams& p, bool eight, cudaStream_t st) {
  eight ? fwd_typed<T, P, true, true>(p, st) : fwd_typed<T, P, true, false>(p, st);
}

template <typename T, typename P, int VEC, int TPR, int NV>
int bwd_launch(const RmsParams& p, cudaStream_t st) {
  constexpr int threads = kBwdThreads<TPR>, rows = threads / TPR;
  if constexpr (VEC > 1) {
    // as many blocks as an SM's shared memory holds, four at most (registers)
    constexpr int bytes = kRingBytes<TPR, NV>, by_regs = 512 / threads, by_smem = 220 * 1024 / (bytes + 1024);
    static_assert(bytes >= (TPR == 32 ? 4 * rows * 32 * NV * VEC : 0), "the sums fit the ring");
    const int blocks = partial_blocks(p.rows, rows, by_regs < by_smem ? by_regs : by_smem);
    auto k = rms_bwd_ring<T, P, VEC, TPR, NV>;
    if (!allow_smem(k, bytes)) return -1;
    k<<<blocks, threads, bytes, st>>>(p);
    return blocks;
  } else {
    const int blocks = partial_blocks(p.rows, rows, kBwdBlocks<TPR, NV * VEC>);
    const size_t smem = TPR == 32 ? sizeof(float) * rows * p.width : 0;
    auto k = rms_bwd<T, P, VEC, TPR, NV>;
    if (!allow_smem(k, smem)) return -1;
    k<<<blocks, threads, smem, st>>>(p);
    return blocks;
  }
}
template <typename T, typename P, int VEC>
int bwd_vec(const RmsParams& p, cudaStream_t st) {
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
fm_status bwd_typed(const RmsParams& p, void* dw, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  int blocks = vector_ok<T>(p, V, sizeof(P), false) ? bwd_vec<T, P, V>(p, st) : bwd_vec<T, P, 1>(p, st);
  if (blocks < 0) return FM_ERR_CUDA;
  if (blocks == 0) {
    if (p.dx) rms_bwd_wide<T, P><<<(unsigned)p.rows, kBlock, 0, st>>>(p);
    if (p.part) {
      blocks = wide_blocks(p.rows, p.width, kBlock);
      rms_cols_wide<T><<<dim3((p.width + kBlock - 1) / kBlock, blocks), kBlock, 0, st>>>(p);
    }
  }
  if (p.part)
    column_sums<P><<<(unsigned)((p.width + 31) / 32), 1024, 0, st>>>(p.part, blocks, p.width, p.width, dw, nullptr);
  return launch_status();
}

bool rows_ok(int64_t rows, int64_t width) {
  return rows >= 0 && rows <= 0x7fffffffLL && width >= 1 && width <= (1 << 24);
}
fm_status check(const fm_rms_norm_args* a) {
  if (a == nullptr || !rows_ok(a->rows, a->width)) return FM_ERR_INVALID_ARG;
  if (!is_float_type(a->dtype) || (a->param_dtype != a->dtype && a->param_dtype != FM_F32))
    return FM_ERR_INVALID_ARG;
  if (a->y_dtype != a->dtype && a->y_dtype != FM_E4M3) return FM_ERR_INVALID_ARG;
  if (!(a->eps >= 0)) return FM_ERR_INVALID_ARG;
  return FM_OK;
}
bool stride_ok(const fm_rms_norm_args* a, int64_t s) { return a->rows <= 1 || s >= a->width; }

RmsParams params(const fm_rms_norm_args* a) {
  RmsParams p{};
  p.rows = a->rows;
  p.width = (int)a->width;
  p.xs = a->x_stride;
  p.eps = (float)a->eps;
  p.x = a->x;
  p.w = a->weight;
  p.rstd = a->rstd;
  return p;
}
}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status fm_rms_norm_forward(const fm_rms_norm_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  const bool eight = a->y_dtype == FM_E4M3;
  if (!stride_ok(a, a->x_stride) || !stride_ok(a, a->y_stride)) return FM_ERR_INVALID_ARG;
  if (a->residual && (!stride_ok(a, a->residual_stride) || !stride_ok(a, a->total_stride))) return FM_ERR_INVALID_ARG;
  if (a->rows == 0) return FM_OK;
  if (a->x == nullptr || a->y == nullptr || (eight && a->scales == nullptr) || (a->residual && a->total == nullptr))
    return FM_ERR_INVALID_ARG;
  RmsParams p = params(a);
  p.ys = a->y_stride;
  p.y = a->y;
  p.scales = a->scales;
  if (a->residual) p.res = a->residual, p.rs = a->residual_stride, p.total = a->total, p.ts = a->total_stride;
  cudaStream_t st = (cudaStream_t)stream;
  const bool wide = a->param_dtype == FM_F32;
  if (a->dtype == FM_F32) fwd_norm<float, float>(p, eight, st);
  else if (a->dtype == FM_F16) wide ? fwd_norm<__half, float>(p, eight, st) : fwd_norm<__half, __half>(p, eight, st);
  else wide ? fwd_norm<__nv_bfloat16, float>(p, eight, st) : fwd_norm<__nv_bfloat16, __nv_bfloat16>(p, eight, st);
  return launch_status();
}

extern "C" int64_t fm_rms_norm_workspace(const fm_rms_norm_args* a) {
  if (check(a) != FM_OK) return -1;
  // one partial row per block, whichever variant runs
  int64_t blocks = wide_blocks(a->rows, (int)a->width, kBlock);
  if (a->width <= kMaxWidth) {
    const int64_t n = partial_blocks(a->rows, 1, kMaxPerSm);
    if (n > blocks) blocks = n;
  }
  return blocks * a->width * (int64_t)sizeof(float);
}

extern "C" fm_status fm_rms_norm_backward(const fm_rms_norm_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->y_dtype != a->dtype) return FM_ERR_INVALID_ARG;
  if (!stride_ok(a, a->x_stride) || !stride_ok(a, a->dy_stride) || (a->dx && !stride_ok(a, a->dx_stride)) ||
      (a->dtotal && !stride_ok(a, a->dtotal_stride)))
    return FM_ERR_INVALID_ARG;
  if (a->rows > 0 && (a->x == nullptr || a->dy == nullptr || a->rstd == nullptr)) return FM_ERR_INVALID_ARG;
  if (a->dweight && (a->workspace == nullptr || a->workspace_bytes < fm_rms_norm_workspace(a) ||
                     ((uintptr_t)a->workspace & 15)))
    return FM_ERR_INVALID_ARG;
  if (!a->dweight && a->dx == nullptr) return FM_OK;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->rows == 0) {
    const size_t n = (size_t)a->width * item_size(a->param_dtype);
    return !a->dweight || cudaMemsetAsync(a->dweight, 0, n, st) == cudaSuccess ? FM_OK : FM_ERR_CUDA;
  }
  RmsParams p = params(a);
  p.dys = a->dy_stride;
  p.dxs = a->dx_stride;
  p.dts = a->dtotal_stride;
  p.dy = a->dy;
  p.dt = a->dx ? a->dtotal : nullptr;
  p.dx = a->dx;
  p.part = a->dweight ? (float*)a->workspace : nullptr;
  const bool wide = a->param_dtype == FM_F32;
  if (a->dtype == FM_F32) return bwd_typed<float, float>(p, a->dweight, st);
  if (a->dtype == FM_F16)
    return wide ? bwd_typed<__half, float>(p, a->dweight, st) : bwd_typed<__half, __half>(p, a->dweight, st);
  return wide ? bwd_typed<__nv_bfloat16, float>(p, a->dweight, st)
              : bwd_typed<__nv_bfloat16, __nv_bfloat16>(p, a->dweight, st);
}

extern "C" fm_status fm_rows_8bit(const fm_rows_8bit_args* a, fm_stream_t stream) {
  if (a == nullptr || !rows_ok(a->rows, a->width) || !is_float_type(a->dtype)) return FM_ERR_INVALID_ARG;
  if (a->rows > 1 && (a->x_stride < a->width || a->values_stride < a->width)) return FM_ERR_INVALID_ARG;
  if (a->rows == 0) return FM_OK;
  if (a->x == nullptr || a->values == nullptr || a->scales == nullptr) return FM_ERR_INVALID_ARG;
  RmsParams p{};
  p.rows = a->rows;
  p.width = (int)a->width;
  p.xs = a->x_stride;
  p.ys = a->values_stride;
  p.x = a->x;
  p.y = a->values;
  p.scales = a->scales;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->dtype == FM_F32) fwd_typed<float, float, false, true>(p, st);
  else if (a->dtype == FM_F16) fwd_typed<__half, __half, false, true>(p, st);
  else fwd_typed<__nv_bfloat16, __nv_bfloat16, false, true>(p, st);
  return launch_status();
}

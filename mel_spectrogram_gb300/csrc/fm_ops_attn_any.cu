// Attention on the FP32 pipes, for what the tensor cores cannot take: 32-bit
// inputs (their products are exact to 32 bits here), head sizes and strides
// that do not fit 16-byte tiles. Forward: a running maximum and sum over key
// tiles of 64. Backward: one kernel per owner (a tile of keys sums dk and dv
// over the queries and the heads that share it, a tile of queries sums dq and
// the bias), each recomputing the scores, so that every sum has one owner and
// one order. Bound by the FP32 pipes' shared-memory operands: 4 x 4 products
// per thread and step. Small problems are bound by latency: 2 rows of 129
// frames, 4 heads of 40, train in 115 us of kernels (forward 27, backward 4, 42
// and 37, the bias's sums 4), five tiles one after another in each.
#include "fm_ops_attn.cuh"

#include <cmath>

namespace fm {
namespace {

constexpr int kThreads = 256;  // 16 x 16: a thread has R rows and columns 16 apart

// Floats between rows of a staged tile: padded to whole float4, an odd number
// of them, so that float4 reads down a column of rows hit distinct banks.
__host__ __device__ inline int pitch_of(int dim) {
  const int d4 = (dim + 3) / 4;
  return 4 * (d4 | 1);
}

// Stages ROWS rows of up to 64 G elements: 16 threads a row, and every thread
// has all its loads of 16 rows under way before it writes the first (one load
// at a time, each waiting for the last, took most of a small problem's time).
//
// bad: where not every query sees the same keys, a row that is not finite must
// not reach the rows that do not see it, but a weight of 0 times it would; such
// elements are staged as zeros and their row is marked, and a weight for it
// becomes NaN. NULL: no matter.
template <typename T, int G, int ROWS>
__device__ __forceinline__ void stage(float* to, const T* from, long long stride, int n, int dim, int pitch,
                                      const int32_t* docs, int* bad = nullptr) {
  // rows at or past n, and padding frames, arrive as zeros whatever memory holds
  const int lane = threadIdx.x & 15, sub = threadIdx.x >> 4;
#pragma unroll
  for (int r0 = 0; r0 < ROWS; r0 += kThreads / 16) {
    const int r = r0 + sub;
    const bool real = r < n && (docs == nullptr || docs[r] >= 0);
    const T* row = from + r * stride;
    float v[4 * G];
#pragma unroll
    for (int k = 0; k < 4 * G; ++k) v[k] = real && lane + 16 * k < dim ? to_f(row[lane + 16 * k]) : 0.f;
    if (bad) {
      bool any = false;
#pragma unroll
      for (int k = 0; k < 4 * G; ++k) {
        const bool wrong = !(fabsf(v[k]) <= 3.402823466e38f);
        v[k] = wrong ? 0.f : v[k];
        any |= wrong;
      }
      if (any) bad[r] = 1;
    }
#pragma unroll
    for (int k = 0; k < 4 * G; ++k)
      if (lane + 16 * k < pitch) to[r * pitch + lane + 16 * k] = v[k];
    // a pitch one float4 past 64 G: its last four
    if (pitch > 64 * G && lane < pitch - 64 * G) to[r * pitch + 64 * G + lane] = 0.f;
  }
}

struct Score {
  float z;      // the biased score, or -inf where unseen
  float slope;  // d(capped)/d(scaled): 1 - tanh^2
  bool seen;
};

template <typename T>
struct ScoreOf {
  const AttnParams& p;
  RowInfo r;
  int h;
  float slope_h;
  const int32_t *qd, *kd;
  __device__ ScoreOf(const AttnParams& p_, int b, int h_) : p(p_), r(row_info(p_, b)), h(h_) {
    slope_h = p.slopes ? p.slopes[h] : 0.f;
    qd = p.q_docs ? p.q_docs + (long long)b * p.q_len : nullptr;
    kd = p.k_docs ? p.k_docs + (long long)b * p.k_len : nullptr;
  }
  __device__ __forceinline__ Score operator()(float dot, int i, int j) const {
    Score s;
    s.seen = i < p.q_len && j < r.len;
    s.slope = 1.f;
    s.z = dot * p.scale;
    if (!s.seen) {
      s.z = -INFINITY;
      return s;
    }
    if (p.cap > 0.f) {
      const float t = tanhf(s.z / p.cap);
      s.slope = 1.f - t * t;
      s.z = p.cap * t;
    }
    const int o = j - (r.start + i);
    if (p.map) {
      const int D = p.max_distance, c = o < -D ? -D : o > D ? D : o;
      const long long at = (long long)p.map[c + D] * p.heads + h;
      s.z += p.table_f32 ? ((const float*)p.table)[at] : to_f(((const T*)p.table)[at]);
    }
    if (p.slopes) s.z -= slope_h * fabsf((float)o);
    if (p.causal && o > 0 && j >= r.prefix) s.seen = false;
    if (qd) {
      const int d = qd[i];
      if (d < 0 || d != kd[j]) s.seen = false;
    }
    if (!s.seen) s.z = -INFINITY;
    return s;
  }
};

__device__ __forceinline__ float half_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// s[r][c] = A row (ty*R + r) . B row (tx + 16 c)
template <int R, int C>
__device__ __forceinline__ void products(const float* A, const float* B, int dim, int pitch, int tx, int ty,
                                         float (&s)[R][C]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) s[r][c] = 0.f;
  const int d4 = (dim + 3) / 4;
  for (int d = 0; d < d4; ++d) {
    float4 a[R], b[C];
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = *(const float4*)(A + (ty * R + r) * pitch + 4 * d);
#pragma unroll
    for (int c = 0; c < C; ++c) b[c] = *(const float4*)(B + (tx + 16 * c) * pitch + 4 * d);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        s[r][c] = fmaf(a[r].x, b[c].x, s[r][c]);
        s[r][c] = fmaf(a[r].y, b[c].y, s[r][c]);
        s[r][c] = fmaf(a[r].z, b[c].z, s[r][c]);
        s[r][c] = fmaf(a[r].w, b[c].w, s[r][c]);
      }
  }
}

// acc[r][g] += sum_j W[(ty*R + r)][j] * V[j][4 tx + 64 g ..]
template <int R, int G>
__device__ __forceinline__ void accumulate(float4 (&acc)[R][G], const float* W, int wpitch, const float* V, int n,
                                           int dim, int pitch, int tx, int ty) {
  for (int j = 0; j < n; ++j) {
    float w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = W[(ty * R + r) * wpitch + j];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int d = 4 * tx + 64 * g;
      if (d >= dim) continue;
      const float4 v = *(const float4*)(V + j * pitch + d);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r][g].x = fmaf(w[r], v.x, acc[r][g].x);
        acc[r][g].y = fmaf(w[r], v.y, acc[r][g].y);
        acc[r][g].z = fmaf(w[r], v.z, acc[r][g].z);
        acc[r][g].w = fmaf(w[r], v.w, acc[r][g].w);
      }
    }
  }
}
template <int R, int G>
__device__ __forceinline__ void clear(float4 (&acc)[R][G]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int g = 0; g < G; ++g) acc[r][g] = make_float4(0.f, 0.f, 0.f, 0.f);
}
template <typename T, int R, int G>
__device__ __forceinline__ void put(T* to, long long stride, int n, int dim, const float4 (&acc)[R][G],
                                    const float (&f)[R], int tx, int ty, T* rest = nullptr) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = ty * R + r;
    if (row >= n) continue;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int d = 4 * tx + 64 * g;
      const float v[4] = {acc[r][g].x, acc[r][g].y, acc[r][g].z, acc[r][g].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (d + k < dim) {
          const T rounded = from_f<T>(v[k] * f[r]);
          to[row * stride + d + k] = rounded;
          if (rest) rest[row * stride + d + k] = from_f<T>(v[k] * f[r] - to_f(rounded));
        }
    }
  }
}

constexpr int kFwdKeys = 64;

template <typename T, int G, int R>
__global__ void __launch_bounds__(kThreads) any_fwd(const AttnParams p) {
  extern __shared__ float sm[];
  constexpr int kRows = 16 * R;
  const int pitch = pitch_of(p.dim);
  float *Q = sm, *K = Q + kRows * pitch, *V = K + kFwdKeys * pitch, *P = V + kFwdKeys * pitch;
  constexpr int wp = kFwdKeys + 4;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = blockIdx.x * kRows, h = blockIdx.y, b = blockIdx.z, hk = h / p.group;
  __shared__ int bad_rows[kFwdKeys];
  int* bad = p.causal || p.k_docs ? bad_rows : nullptr;
  const ScoreOf<T> score(p, b, h);
  const T* q = (const T*)p.q + b * p.qs.b + i0 * p.qs.t + h * p.qs.h;
  const T* k = (const T*)p.k + b * p.ks.b + hk * p.ks.h;
  const T* v = (const T*)p.v + b * p.vs.b + hk * p.vs.h;
  const int nq = min(kRows, p.q_len - i0);
  stage<T, G, kRows>(Q, q, p.qs.t, nq, p.dim, pitch, score.qd ? score.qd + i0 : nullptr);
  float4 acc[R][G];
  clear(acc);
  float m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = -INFINITY, l[r] = 0.f;
  int end = score.r.len;
  if (p.causal) end = min(end, max(score.r.start + i0 + nq, score.r.prefix));
  for (int j0 = 0; j0 < end; j0 += kFwdKeys) {
    const int n = min(kFwdKeys, score.r.len - j0);
    __syncthreads();
    if (bad) {
      if (threadIdx.x < kFwdKeys) bad[threadIdx.x] = 0;
      __syncthreads();
    }
    stage<T, G, kFwdKeys>(K, k + j0 * p.ks.t, p.ks.t, n, p.dim, pitch, score.kd ? score.kd + j0 : nullptr);
    stage<T, G, kFwdKeys>(V, v + j0 * p.vs.t, p.vs.t, n, p.dim, pitch, score.kd ? score.kd + j0 : nullptr,
                          bad);
    __syncthreads();
    float s[R][4];
    products<R, 4>(Q, K, p.dim, pitch, tx, ty, s);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = m[r];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const Score z = score(s[r][c], i0 + ty * R + r, j0 + tx + 16 * c);
        s[r][c] = z.seen && bad && bad[tx + 16 * c] ? NAN : z.z;
        top = fmaxf(top, s[r][c]);
      }
      top = half_max(top);
      const float base = top == -INFINITY ? 0.f : top;  // nothing seen yet: exp(-inf - 0) = 0
      const float f = expf(m[r] - base);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float e = expf(s[r][c] - base);
        sum += e;
        P[(ty * R + r) * wp + tx + 16 * c] = e;
      }
      l[r] = l[r] * f + half_sum(sum);
      m[r] = top;
#pragma unroll
      for (int g = 0; g < G; ++g) acc[r][g].x *= f, acc[r][g].y *= f, acc[r][g].z *= f, acc[r][g].w *= f;
    }
    __syncwarp();  // a row's weights come from the 16 lanes of its half warp
    accumulate<R, G>(acc, P, wp, V, n, p.dim, pitch, tx, ty);
  }
  float f[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    f[r] = l[r] == 0.f ? 0.f : 1.f / l[r];
    const int i = i0 + ty * R + r;
    if (p.lse && tx == 0 && i < p.q_len)
      p.lse[((long long)b * p.heads + h) * p.q_len + i] = l[r] == 0.f ? -INFINITY : m[r] + logf(l[r]);
  }
  const long long at = b * p.os.b + i0 * p.os.t + h * p.os.h;
  put((T*)p.out + at, p.os.t, nq, p.dim, acc, f, tx, ty, p.rest ? (T*)p.rest + at : nullptr);
}

constexpr int kBwdCols = 32;  // rows of the streamed tile

// OF_KEYS: the block owns keys and streams queries (dk, dv); otherwise it
// owns queries and streams keys (dq and the bias).
template <typename T, int G, int R, bool OF_KEYS>
__global__ void __launch_bounds__(kThreads) any_bwd(const AttnParams p) {
  extern __shared__ float sm[];
  constexpr int kRows = 16 * R;
  const int pitch = pitch_of(p.dim);
  float *R1 = sm, *R2 = R1 + kRows * pitch;              // owned: (K, V) or (Q, dout)
  float *C1 = R2 + kRows * pitch, *C2 = C1 + kBwdCols * pitch;  // streamed: (Q, dout) or (K, V)
  float *W1 = C2 + kBwdCols * pitch, *W2 = W1 + kRows * (kBwdCols + 4);
  constexpr int wp = kBwdCols + 4;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r0 = blockIdx.x * kRows, b = blockIdx.z;
  const int hk = OF_KEYS ? blockIdx.y : blockIdx.y / p.group;
  const int h0 = OF_KEYS ? hk * p.group : blockIdx.y, h1 = OF_KEYS ? h0 + p.group : h0 + 1;
  const T* k = (const T*)p.k + b * p.ks.b + hk * p.ks.h;
  const T* v = (const T*)p.v + b * p.vs.b + hk * p.vs.h;
  __shared__ int bad_rows[kBwdCols];
  int* bad = p.causal || p.k_docs ? bad_rows : nullptr;
  const RowInfo info = row_info(p, b);
  const int32_t* kd = p.k_docs ? p.k_docs + (long long)b * p.k_len : nullptr;
  const int32_t* qd = p.q_docs ? p.q_docs + (long long)b * p.q_len : nullptr;
  const int owned = min(kRows, (OF_KEYS ? p.k_len : p.q_len) - r0);
  if (OF_KEYS) {
    const int n = min(owned, info.len - r0);
    stage<T, G, kRows>(R1, k + r0 * p.ks.t, p.ks.t, n, p.dim, pitch, kd ? kd + r0 : nullptr);
    stage<T, G, kRows>(R2, v + r0 * p.vs.t, p.vs.t, n, p.dim, pitch, kd ? kd + r0 : nullptr);
  }
  float4 a1[R][G], a2[R][G];
  clear(a1);
  clear(a2);
  float* part = nullptr;
  const int D = p.max_distance;
  if (!OF_KEYS && p.part) {
    part = p.part + (((long long)b * p.q_tiles + blockIdx.x) * p.heads + h0) * (2 * D + 1);
    for (int i = threadIdx.x; i <= 2 * D; i += kThreads) part[i] = 0.f;
  }
  for (int h = h0; h < h1; ++h) {
    const ScoreOf<T> score(p, b, h);
    const T* q = (const T*)p.q + b * p.qs.b + h * p.qs.h;
    const T* g = (const T*)p.dout + b * p.dos.b + h * p.dos.h;
    const float* lse = p.lse + ((long long)b * p.heads + h) * p.q_len;
    const float* delta = p.delta + ((long long)b * p.heads + h) * p.q_len;
    if (!OF_KEYS) {
      stage<T, G, kRows>(R1, q + r0 * p.qs.t, p.qs.t, owned, p.dim, pitch, qd ? qd + r0 : nullptr);
      stage<T, G, kRows>(R2, g + r0 * p.dos.t, p.dos.t, owned, p.dim, pitch, qd ? qd + r0 : nullptr);
    }
    int begin = 0, end = OF_KEYS ? p.q_len : info.len;
    if (p.causal && !OF_KEYS) end = min(end, max(info.start + r0 + owned, info.prefix));
    if (OF_KEYS && p.causal && r0 >= info.prefix) begin = max(0, r0 - info.start) / kBwdCols * kBwdCols;
    if (OF_KEYS && r0 >= info.len) end = 0;
    for (int c0 = begin; c0 < end; c0 += kBwdCols) {
      const int n = min(kBwdCols, end - c0);
      __syncthreads();
      if (bad) {
        if (threadIdx.x < kBwdCols) bad[threadIdx.x] = 0;
        __syncthreads();
      }
      if (OF_KEYS) {
        stage<T, G, kBwdCols>(C1, q + c0 * p.qs.t, p.qs.t, n, p.dim, pitch, qd ? qd + c0 : nullptr, bad);
        stage<T, G, kBwdCols>(C2, g + c0 * p.dos.t, p.dos.t, n, p.dim, pitch, qd ? qd + c0 : nullptr, bad);
      } else {
        stage<T, G, kBwdCols>(C1, k + c0 * p.ks.t, p.ks.t, n, p.dim, pitch, kd ? kd + c0 : nullptr, bad);
        stage<T, G, kBwdCols>(C2, v + c0 * p.vs.t, p.vs.t, n, p.dim, pitch, kd ? kd + c0 : nullptr);
      }
      __syncthreads();
      float s[R][2], dp[R][2];
      products<R, 2>(R1, C1, p.dim, pitch, tx, ty, s);
      products<R, 2>(R2, C2, p.dim, pitch, tx, ty, dp);
      float bias_grad[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = r0 + ty * R + r, col = c0 + tx + 16 * c;
          const int i = OF_KEYS ? col : row, j = OF_KEYS ? row : col;
          const Score z = score(s[r][c], i, j);
          float w = 0.f, d = 0.f;
          if (z.seen) {
            w = bad && bad[tx + 16 * c] ? NAN : expf(z.z - lse[i]);
            d = w * (dp[r][c] - delta[i]);
          }
          bias_grad[r][c] = d;
          W1[(ty * R + r) * wp + tx + 16 * c] = w;
          W2[(ty * R + r) * wp + tx + 16 * c] = d * z.slope;
        }
      __syncwarp();
      if (OF_KEYS) accumulate<R, G>(a1, W1, wp, C2, n, p.dim, pitch, tx, ty);  // dv
      accumulate<R, G>(a2, W2, wp, C1, n, p.dim, pitch, tx, ty);               // dk or dq
      if (part) {
        // the tile's diagonals, one thread each; the clamped ends one each
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < 2; ++c) W1[(ty * R + r) * wp + tx + 16 * c] = bias_grad[r][c];
        __syncthreads();
        constexpr int kDiag = kRows + kBwdCols - 1;
        const int base = c0 - (info.start + r0) - (kRows - 1);  // offset of diagonal 0
        const int t = threadIdx.x;
        float sum = 0.f;
        if (t < kDiag) {
          for (int i = 0; i < kRows; ++i) {
            const int j = t - (kRows - 1) + i;
            if (j >= 0 && j < kBwdCols) sum += W1[i * wp + j];
          }
        }
        __syncthreads();
        if (t < kDiag) W2[t] = sum;
        __syncthreads();
        if (t < kDiag && base + t > -D && base + t < D) {
          part[base + t + D] += sum;
        } else if (t == kDiag || t == kDiag + 1) {
          float far = 0.f;
          for (int e = 0; e < kDiag; ++e)
            if (t == kDiag ? base + e <= -D : base + e >= D) far += W2[e];
          part[t == kDiag ? 0 : 2 * D] += far;
        }
      }
    }
  }
  float one[R], sc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) one[r] = 1.f, sc[r] = p.scale;
  if (OF_KEYS) {
    put((T*)p.dv + b * p.dvs.b + r0 * p.dvs.t + hk * p.dvs.h, p.dvs.t, owned, p.dim, a1, one, tx, ty);
    put((T*)p.dk + b * p.dks.b + r0 * p.dks.t + hk * p.dks.h, p.dks.t, owned, p.dim, a2, sc, tx, ty);
  } else {
    put((T*)p.dq + b * p.dqs.b + r0 * p.dqs.t + h0 * p.dqs.h, p.dqs.t, owned, p.dim, a2, sc, tx, ty);
  }
}

// delta[b][h][i] = dout . out, a warp per row; 0 for padding frames, whose
// dout may hold anything
template <typename T>
__global__ void __launch_bounds__(256) any_delta(const AttnParams p) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long rows = (long long)p.batch * p.heads * p.q_len;
  if (row >= rows) return;
  const int i = (int)(row % p.q_len), h = (int)(row / p.q_len % p.heads), b = (int)(row / p.q_len / p.heads);
  const T* g = (const T*)p.dout + b * p.dos.b + i * p.dos.t + h * p.dos.h;
  const T* o = (const T*)p.out_in + b * p.os.b + i * p.os.t + h * p.os.h;
  const T* rest = p.rest ? (const T*)p.rest + b * p.os.b + i * p.os.t + h * p.os.h : nullptr;
  float s = 0.f;
  if (p.q_docs == nullptr || p.q_docs[(long long)b * p.q_len + i] >= 0)
    for (int d = threadIdx.x & 31; d < p.dim; d += 32)
      s = fmaf(to_f(g[d]), to_f(o[d]) + (rest ? to_f(rest[d]) : 0.f), s);
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) p.delta[row] = s;
}

size_t fwd_smem(int dim, int rows) {
  return sizeof(float) * ((size_t)(rows + 2 * kFwdKeys) * pitch_of(dim) + rows * (kFwdKeys + 4));
}
size_t bwd_smem(int dim, int rows) {
  return sizeof(float) * ((size_t)(2 * rows + 2 * kBwdCols) * pitch_of(dim) + 2 * rows * (kBwdCols + 4));
}

template <typename T, int G, int R>
fm_status fwd(const AttnParams& p, cudaStream_t st) {
  const dim3 grid((p.q_len + 16 * R - 1) / (16 * R), p.heads, p.batch);
  const size_t smem = fwd_smem(p.dim, 16 * R);
  if (!allow_smem(any_fwd<T, G, R>, smem)) return FM_ERR_CUDA;
  any_fwd<T, G, R><<<grid, kThreads, smem, st>>>(p);
  return launch_status();
}
template <typename T, int G, int R>
fm_status bwd(const AttnParams& p, cudaStream_t st) {
  const int tile = 16 * R;
  const size_t smem = bwd_smem(p.dim, tile);
  if (!allow_smem(any_bwd<T, G, R, true>, smem) || !allow_smem(any_bwd<T, G, R, false>, smem)) return FM_ERR_CUDA;
  if (p.q_len > 0) {
    const long long rows = (long long)p.batch * p.heads * p.q_len;
    any_delta<T><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p);
    any_bwd<T, G, R, false><<<dim3((p.q_len + tile - 1) / tile, p.heads, p.batch), kThreads, smem, st>>>(p);
  }
  if (p.k_len > 0)
    any_bwd<T, G, R, true><<<dim3((p.k_len + tile - 1) / tile, p.kv_heads, p.batch), kThreads, smem, st>>>(p);
  return launch_status();
}
template <typename T, int R>
fm_status fwd_g(const AttnParams& p, cudaStream_t st) {
  return p.dim <= 64 ? fwd<T, 1, R>(p, st) : p.dim <= 128 ? fwd<T, 2, R>(p, st) : fwd<T, 4, R>(p, st);
}
template <typename T, int R>
fm_status bwd_g(const AttnParams& p, cudaStream_t st) {
  return p.dim <= 64 ? bwd<T, 1, R>(p, st) : p.dim <= 128 ? bwd<T, 2, R>(p, st) : bwd<T, 4, R>(p, st);
}
}  // namespace

int any_rows(const AttnParams& p) {
  // 64 rows a block make four times the products of an operand read; 32 make
  // twice the blocks, for problems that would leave SMs without one
  const long long blocks = (long long)((p.q_len + 63) / 64) * p.heads * p.batch;
  return blocks < num_sms() ? 32 : 64;
}
template <typename T>
static fm_status any_forward(const AttnParams& p, cudaStream_t st) {
  return any_rows(p) == 32 ? fwd_g<T, 2>(p, st) : fwd_g<T, 4>(p, st);
}
template <typename T>
static fm_status any_backward(const AttnParams& p, cudaStream_t st) {
  return any_rows(p) == 32 ? bwd_g<T, 2>(p, st) : bwd_g<T, 4>(p, st);
}
fm_status attn_any_forward(const AttnParams& p, int64_t dtype, cudaStream_t st) {
  return dtype == FM_F32 ? any_forward<float>(p, st)
                         : dtype == FM_F16 ? any_forward<__half>(p, st) : any_forward<__nv_bfloat16>(p, st);
}
fm_status attn_any_backward(const AttnParams& p, int64_t dtype, cudaStream_t st) {
  return dtype == FM_F32 ? any_backward<float>(p, st)
                         : dtype == FM_F16 ? any_backward<__half>(p, st) : any_backward<__nv_bfloat16>(p, st);
}
}  // namespace fm

// Distance buckets, the dense position bias and its gradient (fm_ops.h).
#include "fm_ops.cuh"

#include <cmath>
#include <new>
#include <vector>

namespace fm {

int num_sms() {
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (known[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    known[dev] = n;
  }
  return known[dev];
}

namespace {

// Whole numbers as base-2^32 digits, for the one comparison below.
using Digits = std::vector<uint32_t>;
void times(Digits& d, uint32_t f) {
  uint64_t carry = 0;
  for (uint32_t& x : d) {
    carry += (uint64_t)x * f;
    x = (uint32_t)carry;
    carry >>= 32;
  }
  if (carry) d.push_back((uint32_t)carry);
}
int compare(const Digits& a, const Digits& b) {
  if (a.size() != b.size()) return a.size() < b.size() ? -1 : 1;
  for (size_t i = a.size(); i-- > 0;)
    if (a[i] != b[i]) return a[i] < b[i] ? -1 : 1;
  return 0;
}

// n^L >= e^(L-m) M^m. Logarithms settle all but the near ties, which are
// multiplied out.
bool reaches(int n, int L, int e, int M, int m) {
  const double left = L * std::log((double)n), right = (L - m) * std::log((double)e) + m * std::log((double)M);
  if (std::fabs(left - right) > 1e-9 * (1.0 + std::fabs(right))) return left > right;
  Digits a{1}, b{1};
  for (int i = 0; i < L; ++i) times(a, (uint32_t)n);
  for (int i = 0; i < L - m; ++i) times(b, (uint32_t)e);
  for (int i = 0; i < m; ++i) times(b, (uint32_t)M);
  return compare(a, b) >= 0;
}

struct BiasParams {
  int heads, q_len, k_len, q_start, max_distance;
  const int32_t* map;
  const void* table;
  void* out;
  const void* dout;
  float* part;  // [chunks][heads][2 * max_distance + 1]
  int rows_per_chunk, near_blocks;
};

constexpr int kFillThreads = 256;
constexpr int kFillPacks = 16;  // packs of 16 bytes a thread writes

// The bias by offset in shared memory, as V copies (V elements make 16 bytes)
// shifted by one element each: the V neighbours from any offset on are then one
// aligned 16-byte read. Copy c holds offset -max_distance - V - c at its start;
// V copies of the end values stand at either end.
template <int V>
__host__ __device__ inline int fill_pitch(int max_distance) {
  return (2 * max_distance + 1 + 3 * V + V - 1) / V * V;
}

// Write bound. A block writes a flat run of one head's matrix with 16-byte
// stores. A pack far from the diagonal is one value, one near it one shared
// read; an element at a time (an index, two clamps and a 2-byte read each) the
// kernel took 86 us for 16 x 3001 x 3001 in 16 bits, bound by instructions; so
// it takes 56 (288 MB, 5.1 TB/s).
template <typename T>
__global__ void __launch_bounds__(kFillThreads) bias_fill(const BiasParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  constexpr int V = 16 / sizeof(T);
  T* val = (T*)raw;
  const int h = blockIdx.y, D = p.max_distance, pitch = fill_pitch<V>(D);
  for (int i = threadIdx.x; i < pitch + V; i += kFillThreads) {
    const T v = ((const T*)p.table)[(long long)p.map[min(max(i - 2 * V, 0), 2 * D)] * p.heads + h];
    // element i of the row that starts at offset -D - 2 V
#pragma unroll
    for (int c = 0; c < V; ++c)
      if (i - V + c >= 0 && i - V + c < pitch) val[c * pitch + i - V + c] = v;
  }
  __syncthreads();
  const long long n = (long long)p.q_len * p.k_len;
  T* out = (T*)p.out + h * n;
  // elements before the first 16-byte boundary, at most V - 1, go to block 0
  const int head = (int)((16 - ((uintptr_t)out & 15)) & 15) / (int)sizeof(T);
  auto value = [&](int i, int j) {
    const int o = min(max(j - i - p.q_start, -D), D);
    return val[o + D + V];  // copy 0
  };
  const long long run = (long long)kFillThreads * kFillPacks * V;
  const long long begin = head + blockIdx.x * run;
  if (blockIdx.x == 0 && threadIdx.x < head && threadIdx.x < n) {
    const int i = threadIdx.x / p.k_len;
    out[threadIdx.x] = value(i, threadIdx.x - i * p.k_len);
  }
  if (begin >= n) return;
  const int i0 = (int)(begin / p.k_len), j0 = (int)(begin - (long long)i0 * p.k_len);
#pragma unroll 4
  for (int s = 0; s < kFillPacks; ++s) {
    const int local = (s * kFillThreads + threadIdx.x) * V;
    const long long at = begin + local;
    if (at >= n) break;
    const unsigned u = (unsigned)j0 + (unsigned)local;
    const unsigned r = u / (unsigned)p.k_len;
    int i = i0 + (int)r, j = (int)(u - r * (unsigned)p.k_len);
    Pack<T, V> q;
    if (j + V <= p.k_len) {
      // offsets o .. o + V - 1, clamped to where the ends' copies begin
      const int o = min(max(j - i - p.q_start, -D - V), D + 1) + D + V;  // element of copy 0
      const int c = (V - (o & (V - 1))) & (V - 1);
      q = *(const Pack<T, V>*)(val + c * pitch + o + c);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        q.v[k] = value(i, j);
        if (++j == p.k_len) j = 0, ++i;
      }
    }
    if (at + V <= n) {
      *(Pack<T, V>*)(out + at) = q;
    } else {
      for (int k = 0; k < V && at + k < n; ++k) out[at + k] = q.v[k];
    }
  }
}

// Read bound. Near the diagonal (|offset| < max_distance) a thread owns an
// offset and walks down its diagonal over the rows of a chunk, 16 reads under
// way, so neighbouring threads read neighbouring elements and a sum stays in
// one register; beyond, where one bucket holds all, the last block sums whole
// stretches of rows with 16-byte reads. No atomics, one fixed order. 86 us for
// 16 x 3001 x 3001 in 16 bits with 800 places either way (288 MB, 3.3 TB/s); by
// themselves the walk takes 46 of a cold cache and the stretches 57. (The band
// staged in shared memory instead took 62 us where the walk takes 35.)
template <typename T>
__global__ void __launch_bounds__(256) bias_diagonals(const BiasParams p) {
  const int D = p.max_distance, W = 2 * D + 1;
  const int h = blockIdx.z, r0 = blockIdx.y * p.rows_per_chunk, r1 = min(r0 + p.rows_per_chunk, p.q_len);
  const T* x = (const T*)p.dout + (long long)h * p.q_len * p.k_len;
  float* part = p.part + ((long long)blockIdx.y * p.heads + h) * W;
  if ((int)blockIdx.x < p.near_blocks) {
    const int t = blockIdx.x * 256 + threadIdx.x;  // offset t - (D - 1)
    if (t > 2 * (D - 1)) return;
    const int c = t - (D - 1) + p.q_start;  // j - i
    const int lo = max(r0, -c), hi = min(r1, p.k_len - c);
    float s = 0.f;
    const long long step = (long long)p.k_len + 1;
    const T* at = x + (long long)lo * step + c;
    int i = lo;
    for (; i + 16 <= hi; i += 16) {
      T v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = at[k * step];
#pragma unroll
      for (int k = 0; k < 16; ++k) s += to_f(v[k]);
      at += 16 * step;
    }
    for (; i < hi; ++i, at += step) s += to_f(*at);
    part[t + 1] = s;
    return;
  }
  // ---- far: a warp a row, the stretches before and after in one run of packs,
  // so that all of a row's reads are under way at once
  __shared__ float sums[2][8];
  constexpr int V = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float total[2] = {0.f, 0.f};
  for (int i = r0 + warp; i < r1; i += 8) {
    const T* row = x + (long long)i * p.k_len;
    const long long near = (long long)i + p.q_start;
    const int b[2] = {0, (int)min(max(near + D, 0LL), (long long)p.k_len)};
    const int e[2] = {(int)min(max(near - D + 1, 0LL), (long long)p.k_len), p.k_len};
    int first[2], packs[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int n = max(e[w] - b[w], 0);
      const int skip = min((int)((16 - ((uintptr_t)(row + b[w]) & 15)) & 15) / (int)sizeof(T), n);
      first[w] = b[w] + skip;
      packs[w] = (n - skip) / V;
      const int done = first[w] + packs[w] * V;  // fewer than V elements before the first pack and after the last
      if (lane < skip) total[w] += to_f(row[b[w] + lane]);
      if (done + lane < e[w]) total[w] += to_f(row[done + lane]);
    }
#pragma unroll 8
    for (int k = lane; k < packs[0] + packs[1]; k += 32) {
      const bool after = k >= packs[0];
      const Pack<T, V> v = *(const Pack<T, V>*)(row + (after ? first[1] + (k - packs[0]) * V : first[0] + k * V));
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int y = 0; y < V; ++y) s[y & 1] += to_f(v.v[y]);
      s[0] += s[1];
      total[0] += after ? 0.f : s[0];
      total[1] += after ? s[0] : 0.f;
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float s = warp_sum(total[w]);
    if (lane == 0) sums[w][warp] = s;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sums[threadIdx.x][k];
    part[threadIdx.x ? 2 * D : 0] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) bucket_sums(const int32_t* ranges, int max_distance, const float* part,
                                                   long long rows, long long row_stride, long long head_stride,
                                                   int first, int count, int heads, T* dtable) {
  __shared__ float red[8];
  const int c = blockIdx.x, h = blockIdx.y;
  int lo = ranges[2 * c], hi = ranges[2 * c + 1];
  float s = 0.f;
  if (lo <= hi) {
    if (lo == -max_distance || lo < first) lo = first;
    if (hi == max_distance || hi > first + count - 1) hi = first + count - 1;
    const int n = hi - lo + 1;
    if (n > 0) {
      // element t of the bucket: row t / n, column t % n, both followed without a
      // division (their product may pass 2^32)
      const int r = threadIdx.x / n, dr = 256 / n, dc = 256 - dr * n;
      int col = threadIdx.x - r * n;
      const float* at = part + h * head_stride + (lo - first) + r * row_stride + col;
      const long long total = rows * n, step = dr * row_stride + dc, next = row_stride - n;
#pragma unroll 8
      for (long long t = threadIdx.x; t < total; t += 256) {
        s += *at;
        at += step;
        col += dc;
        if (col >= n) col -= n, at += next;
      }
    }
  }
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i];
    dtable[(long long)c * heads + h] = from_f<T>(s);
  }
}

// Host memory to the device, there before this returns, whichever stream reads
// it next: on a stream of its own, which waits for none and none for it. (A plain
// copy from pageable memory may return before the device has it, and torch's
// side streams do not wait for the default one.) Allocation and copy are allowed
// while this or another thread records a graph.
cudaError_t upload(int32_t** to, const int32_t* from, size_t bytes) {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t err = cudaThreadExchangeStreamCaptureMode(&mode);
  if (err != cudaSuccess) return err;
  cudaStream_t st = nullptr;
  *to = nullptr;
  err = cudaMalloc(to, bytes);
  if (err == cudaSuccess) err = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
  if (err == cudaSuccess) err = cudaMemcpyAsync(*to, from, bytes, cudaMemcpyHostToDevice, st);
  if (err == cudaSuccess) err = cudaStreamSynchronize(st);
  if (st) cudaStreamDestroy(st);
  if (err != cudaSuccess && *to) cudaFree(*to);
  cudaThreadExchangeStreamCaptureMode(&mode);
  return err;
}

constexpr int kMaxLen = (1 << 29) - 1;

fm_status check(const fm_relative_bias_args* a) {
  if (a == nullptr || a->buckets == nullptr) return FM_ERR_INVALID_ARG;
  if (a->heads < 1 || a->heads > 65535 || a->q_len < 0 || a->q_len > kMaxLen || a->k_len < 0 || a->k_len > kMaxLen)
    return FM_ERR_INVALID_ARG;
  if (!is_float_type(a->dtype)) return FM_ERR_INVALID_ARG;
  return FM_OK;
}
// Rows of a chunk of bias_diagonals: shorter chunks for fewer rows, so that
// there are blocks enough, while the partial sums stay far below the matrix.
int chunk_rows(const fm_relative_bias_args* a) { return a->q_len >= 1024 ? 32 : 16; }
int chunks_of(const fm_relative_bias_args* a) {
  const int r = chunk_rows(a);
  return (int)((a->q_len + r - 1) / r);
}
BiasParams params(const fm_relative_bias_args* a) {
  BiasParams p{};
  p.heads = (int)a->heads;
  p.q_len = (int)a->q_len;
  p.k_len = (int)a->k_len;
  // beyond 2^30 every offset is past max_distance: the same bias
  const int64_t far = 1 << 30;
  p.q_start = (int)(a->q_start > far ? far : a->q_start < -far ? -far : a->q_start);
  p.max_distance = a->buckets->max_distance;
  p.map = a->buckets->map;
  return p;
}
bool same_device(const fm_buckets* b) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == b->device;
}
}  // namespace

fm_status bucket_sums_launch(const fm_buckets* b, const float* part, long long rows, long long row_stride,
                             long long head_stride, int first, int count, int heads, void* dtable, int64_t dtype,
                             cudaStream_t st) {
  const dim3 grid(b->num_buckets, heads);
  if (dtype == FM_F32)
    bucket_sums<float><<<grid, 256, 0, st>>>(b->ranges, b->max_distance, part, rows, row_stride, head_stride, first,
                                             count, heads, (float*)dtable);
  else if (dtype == FM_F16)
    bucket_sums<__half><<<grid, 256, 0, st>>>(b->ranges, b->max_distance, part, rows, row_stride, head_stride, first,
                                              count, heads, (__half*)dtable);
  else
    bucket_sums<__nv_bfloat16><<<grid, 256, 0, st>>>(b->ranges, b->max_distance, part, rows, row_stride, head_stride,
                                                     first, count, heads, (__nv_bfloat16*)dtable);
  return launch_status();
}
}  // namespace fm

using namespace fm;

extern "C" fm_status fm_buckets_create(fm_buckets** out, int num_buckets, int max_distance, int bidirectional) {
  if (out == nullptr) return FM_ERR_INVALID_ARG;
  *out = nullptr;
  if (num_buckets > 4096 || num_buckets < (bidirectional ? 4 : 2) || (bidirectional && num_buckets % 2))
    return FM_ERR_INVALID_ARG;
  const int side = bidirectional ? num_buckets / 2 : num_buckets, e = side / 2, L = side - e;
  if (max_distance <= e || max_distance > 2048) return FM_ERR_INVALID_ARG;
  fm_buckets* b = new (std::nothrow) fm_buckets{};
  const int n_map = 2 * max_distance + 1, n_all = n_map + 2 * num_buckets;
  int32_t* host = new (std::nothrow) int32_t[n_all];
  if (b == nullptr || host == nullptr) {
    delete b;
    delete[] host;
    return FM_ERR_OOM;
  }
  b->num_buckets = num_buckets;
  b->max_distance = max_distance;
  b->bidirectional = bidirectional ? 1 : 0;
  b->host = host;
  try {  // the digits' vectors may throw
    int m = 0;
    for (int n = 0; n <= max_distance; ++n) {
      if (n >= e)
        while (m < L - 1 && reaches(n, L, e, max_distance, m + 1)) ++m;
      const int c = n < e ? n : e + m;
      host[max_distance - n] = c;
      host[max_distance + n] = b->bidirectional ? c + (n > 0 ? side : 0) : 0;
    }
  } catch (...) {
    delete[] host;
    delete b;
    return FM_ERR_OOM;
  }
  for (int c = 0; c < num_buckets; ++c) host[n_map + 2 * c] = 1, host[n_map + 2 * c + 1] = 0;
  for (int i = 0; i < n_map; ++i) {
    int32_t* r = host + n_map + 2 * host[i];
    if (r[0] > r[1]) r[0] = i - max_distance;
    r[1] = i - max_distance;
  }
  fm_status st = FM_ERR_CUDA;
  if (cudaGetDevice(&b->device) == cudaSuccess) {
    const cudaError_t err = upload(&b->map, host, sizeof(int32_t) * n_all);
    st = err == cudaSuccess ? FM_OK : err == cudaErrorMemoryAllocation ? FM_ERR_OOM : FM_ERR_CUDA;
  }
  if (st != FM_OK) {
    cudaGetLastError();  // an allocation failure stays out of later calls' status
    delete[] host;
    delete b;
    return st;
  }
  b->ranges = b->map + n_map;
  *out = b;
  return FM_OK;
}

extern "C" fm_status fm_buckets_map(const fm_buckets* b, int32_t* map) {
  if (b == nullptr || map == nullptr) return FM_ERR_INVALID_ARG;
  for (int i = 0; i <= 2 * b->max_distance; ++i) map[i] = b->host[i];
  return FM_OK;
}

extern "C" fm_status fm_buckets_destroy(fm_buckets* b) {
  if (b == nullptr) return FM_OK;
  const bool ok = cudaFree(b->map) == cudaSuccess;
  delete[] b->host;
  delete b;
  return ok ? FM_OK : FM_ERR_CUDA;
}

extern "C" fm_status fm_relative_bias_forward(const fm_relative_bias_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->q_len == 0 || a->k_len == 0) return FM_OK;
  if (a->table == nullptr || a->out == nullptr || ((uintptr_t)a->out % item_size(a->dtype)) ||
      !same_device(a->buckets))
    return FM_ERR_INVALID_ARG;
  BiasParams p = params(a);
  p.table = a->table;
  p.out = a->out;
  const int64_t item = item_size(a->dtype);
  const long long run = (long long)kFillThreads * kFillPacks * (16 / item);
  const long long blocks = ((long long)a->q_len * a->k_len + run - 1) / run;
  if (blocks > 0x7fffffffLL) return FM_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks, (unsigned)a->heads);
  const size_t smem = 16 * (size_t)(item == 4 ? fill_pitch<4>(p.max_distance) : fill_pitch<8>(p.max_distance));
  cudaStream_t st = (cudaStream_t)stream;
  if (!allow_smem(bias_fill<float>, smem) || !allow_smem(bias_fill<__half>, smem) ||
      !allow_smem(bias_fill<__nv_bfloat16>, smem))
    return FM_ERR_CUDA;
  if (a->dtype == FM_F32) bias_fill<float><<<grid, kFillThreads, smem, st>>>(p);
  else if (a->dtype == FM_F16) bias_fill<__half><<<grid, kFillThreads, smem, st>>>(p);
  else bias_fill<__nv_bfloat16><<<grid, kFillThreads, smem, st>>>(p);
  return launch_status();
}

extern "C" int64_t fm_relative_bias_workspace(const fm_relative_bias_args* a) {
  if (check(a) != FM_OK) return -1;
  return (int64_t)chunks_of(a) * a->heads * (2 * (int64_t)a->buckets->max_distance + 1) * (int64_t)sizeof(float) + 16;
}

extern "C" fm_status fm_relative_bias_backward(const fm_relative_bias_args* a, fm_stream_t stream) {
  if (fm_status s = check(a)) return s;
  if (a->dtable == nullptr || !same_device(a->buckets)) return FM_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->q_len == 0 || a->k_len == 0) {
    const size_t n = (size_t)a->buckets->num_buckets * a->heads * item_size(a->dtype);
    return cudaMemsetAsync(a->dtable, 0, n, st) == cudaSuccess ? FM_OK : FM_ERR_CUDA;
  }
  if (a->dout == nullptr || a->workspace == nullptr || a->workspace_bytes < fm_relative_bias_workspace(a) ||
      ((uintptr_t)a->workspace & 15))
    return FM_ERR_INVALID_ARG;
  BiasParams p = params(a);
  p.dout = a->dout;
  p.part = (float*)a->workspace;
  p.rows_per_chunk = chunk_rows(a);
  const int W = 2 * p.max_distance + 1, chunks = chunks_of(a);
  if (chunks > 65535) return FM_ERR_UNSUPPORTED;
  p.near_blocks = (2 * p.max_distance - 1 + 255) / 256;
  const dim3 grid(p.near_blocks + 1, chunks, p.heads);
  if (a->dtype == FM_F32) bias_diagonals<float><<<grid, 256, 0, st>>>(p);
  else if (a->dtype == FM_F16) bias_diagonals<__half><<<grid, 256, 0, st>>>(p);
  else bias_diagonals<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
  if (fm_status s = launch_status()) return s;
  return bucket_sums_launch(a->buckets, p.part, chunks, (long long)p.heads * W, W, -p.max_distance, W, p.heads,
                            a->dtable, a->dtype, st);
}

// Host side of the gated linear layer on the tensor cores, and the small kernels
// around it: rows that TMA cannot read are copied to ones that it can, and the
// gradients of FM_F16 are scaled by powers of two.
#include <cudaTypedefs.h>

#include <climits>

#include "fm_ops_gated_tc.cuh"

namespace fm {

fm_status gated_tc_bf16(gated::Op op, const gated::TcArgs& t, int bn, cudaStream_t st);
fm_status gated_tc_f16(gated::Op op, const gated::TcArgs& t, int bn, cudaStream_t st);
fm_status gated_tc_e4m3(int64_t dtype, const gated::TcArgs& t, int bn, cudaStream_t st);

namespace {
using namespace gated;

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// [rows][cols] with rows `stride` elements apart, in boxes of 128 bytes x box_rows.
// The encoder is a driver call: it needs the device's context on this thread, which
// a thread that only took cached memory so far does not have.
bool encode(CUtensorMap* m, const void* base, int64_t dtype, long long rows, long long cols, long long stride,
            int box_rows) {
  const int item = dtype == FM_E4M3 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)((rows > 1 ? stride * item : (cols * item + 15) / 16 * 16))};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / item), (cuuint32_t)box_rows}, step[2] = {1, 1};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess || encoder() == nullptr) return false;
  const CUtensorMapDataType type = dtype == FM_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == FM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encoder()(m, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t align256(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Rows that TMA cannot read (off the 16-byte grid), for a copy that it can.
template <typename T>
__global__ void __launch_bounds__(256) copy_rows(const T* from, long long stride, long long rows, int cols, T* to,
                                                 long long to_stride) {
  for (long long r = blockIdx.y; r < rows; r += gridDim.y)
    for (int c = blockIdx.x * 256 + threadIdx.x; c < cols; c += gridDim.x * 256) to[r * to_stride + c] = from[r * stride + c];
}

// FM_F16: dg and du of a row are scaled by a power of two, so that what they can reach at
// most is just below what f16 holds: no product is lost to infinity that its sum is not,
// and digits are lost below 2^-24 of that alone. With |dh| < 2^(e + 1) in the row,
// |u| <= |x| max |w_up| in 2-norms, |act(g)| <= |g| (1: sigmoid) and slopes up to 1.13, both
// stay below 1.13 * 2^(e + 1 + reach), where the two norms' product is below 2^reach.
// What is not finite, in dh, x or the weights, does not count: it ends in its own row.
// 24008 rows of 1024 to 4096: 41 us, memory bound (263 MB), and scale_rows 16.
struct RowSize {
  short dh, x;  // the largest |dh| is in 2^dh .. 2^(dh + 1), |x| alike; kLeast for a row of zeros
  short norm;   // |x| in the 2-norm is below 2^norm
  short down;   // for the weights' gradients D's row is 2^-down of what it is for dx
};
struct Loudest {
  int up, gate;        // bits of the largest squared norm of w_up's and w_gate's rows
  int by_norm, by_x;   // largest dh + x + norm, and dh + x, of the rows that have both
  int scaled;          // exponent that the weights' gradients are multiplied by (see scale_rows)
};
constexpr int kNone = -30;  // exponent of a norm of zero: below that of any other
// the least power of two above the norm, whose square may be off by a thousandth and more for
// long rows
__device__ __forceinline__ int norm_exponent(float square) {
  int e = kNone;
  if (square > 0.f) frexpf(sqrtf(square) * 1.05f, &e);
  return e;
}
__device__ __forceinline__ int reach(int norm, const Loudest& all, int act, int width) {
  const int up = norm_exponent(__int_as_float(max(all.up, 0))), gate = norm_exponent(__int_as_float(max(all.gate, 0)));
  const int most = act == FM_ACT_SIGMOID ? max(norm + up, 0) : norm + max(up, gate);
  return most + (width >> 20 != 0);  // sums of so many terms may be off by as much as they are
}

// The largest finite magnitude of a lane's part of a row, and its squares' sum.
template <int VEC>
__device__ __forceinline__ void measure(const __half* row, int cols, int lane, unsigned& most, float& square) {
  most = 0, square = 0.f;
#pragma unroll 4
  for (int c = lane * VEC; c < cols; c += 32 * VEC) {
    const Pack<__half, VEC> q = *(const Pack<__half, VEC>*)(row + c);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const unsigned v = __half_as_ushort(q.v[k]) & 0x7fffu;
      if (v < 0x7c00u) {
        const float f = __half2float(q.v[k]);
        most = max(most, v), square = fmaf(f, f, square);
      }
    }
  }
}
// A warp a row of dh and x, and then a warp a row of either weight.
__global__ void __launch_bounds__(256) row_sizes(const GatedParams p, int vec_dh, int vec_x, RowSize* sizes, Loudest* all) {
  __shared__ int red[4][8];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long n = (long long)blockIdx.x * 8 + warp;
  int found[4] = {INT_MIN, INT_MIN, INT_MIN, INT_MIN};  // as in Loudest
  unsigned most;
  float square;
  if (n < p.rows) {
    const __half *dh = (const __half*)p.dh + n * p.dhs, *x = (const __half*)p.x + n * p.xs;
    if (vec_dh) measure<8>(dh, p.hidden, lane, most, square);
    else measure<1>(dh, p.hidden, lane, most, square);
    const unsigned of_dh = __reduce_max_sync(0xffffffffu, most);
    if (vec_x) measure<8>(x, p.width, lane, most, square);
    else measure<1>(x, p.width, lane, most, square);
    const unsigned of_x = __reduce_max_sync(0xffffffffu, most);
    auto exponent = [](unsigned largest) {
      int e = kLeast + 1;
      if (largest) frexpf(__half2float(__ushort_as_half((unsigned short)largest)), &e);
      return e - 1;
    };
    const int e = exponent(of_dh), ex = exponent(of_x), norm = norm_exponent(warp_sum(square));
    if (lane == 0) sizes[n] = RowSize{(short)e, (short)ex, (short)norm, 0};
    if (of_dh && of_x) found[2] = e + ex + norm, found[3] = e + ex;
  } else if (n < p.rows + 2LL * p.hidden) {
    const long long f = n - p.rows;
    const bool up = f >= p.hidden;
    const __half* w = up ? (const __half*)p.wu + (f - p.hidden) * p.us : (const __half*)p.wg + f * p.gs;
    if (vec_x) measure<8>(w, p.width, lane, most, square);
    else measure<1>(w, p.width, lane, most, square);
    found[up ? 0 : 1] = __float_as_int(warp_sum(square));
  }
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[i][warp] = found[i];
  __syncthreads();
  if (threadIdx.x < 4) {
    int v = INT_MIN;
#pragma unroll
    for (int w = 0; w < 8; ++w) v = max(v, red[threadIdx.x][w]);
    if (v != INT_MIN) atomicMax((int*)all + threadIdx.x, v);
  }
}
// What each row of dh is multiplied by. X: and x, for the product that sums over rows, so that
// all rows' terms have one scale. The rows with the largest terms have both factors' largest
// at 2^14; what another's terms are smaller by, x takes up to 2^14 of, and the two share the
// rest: terms keep their digits, relative to their own row's largest, to 2^-(32 - n / 2) where
// that is 2^-n of the largest of all. On x alone, from 1 on, 2^-24 below the largest row
// nothing would be left, also in columns to which only the small ones add. A warp a row.
template <int VEC, bool X>
__global__ void __launch_bounds__(256) scale_rows(const GatedParams p, RowSize* sizes, Loudest* all, float* scale,
                                                  __half* to, long long to_stride) {
  const long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  if (r >= p.rows) return;
  const RowSize size = sizes[r];
  const int s = size.dh + reach(size.norm, *all, p.act, p.width) - 14;
  if constexpr (X) {
    // the largest of s + x over the rows that have terms: reach() by parts
    const int up = norm_exponent(__int_as_float(max(all->up, 0))), gate = norm_exponent(__int_as_float(max(all->gate, 0)));
    int top = all->by_norm + (p.act == FM_ACT_SIGMOID ? up : max(up, gate));
    if (p.act == FM_ACT_SIGMOID) top = max(top, all->by_x);
    top += (p.width >> 20 != 0) - 14;
    if (all->by_x < 2 * kLeast) top = 0;  // there are none
    if (r == 0 && threadIdx.x == 0) all->scaled = top - 14;
    const int below = max(top - s - size.x, 0), down = max(below - 14, 0) / 2;
    if (threadIdx.x % 32 == 0) sizes[r].down = (short)down;
    const float f = power_of_two(max(14 - size.x - (below - down), -126));
    const __half* x = (const __half*)p.x + r * p.xs;
#pragma unroll 4
    for (int c = threadIdx.x % 32 * VEC; c < p.width; c += 32 * VEC) {
      Pack<__half, VEC> q = *(const Pack<__half, VEC>*)(x + c);
#pragma unroll
      for (int k = 0; k < VEC; ++k) q.v[k] = __float2half_rn(__half2float(q.v[k]) * f);
      *(Pack<__half, VEC>*)(to + r * to_stride + c) = q;
    }
  }
  if (threadIdx.x % 32 == 0) scale[r] = power_of_two(-s);
}
// D's rows that are far below the largest, after dx, which asks nothing of other rows. Where
// none is, this reads the sizes alone. A warp a row.
__global__ void __launch_bounds__(256) lower_rows(const RowSize* sizes, long long rows, __half* d, long long ld) {
  const long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int down = r < rows ? sizes[r].down : 0;
  if (down == 0) return;
  const float f = power_of_two(max(-down, -126));
  for (long long c = threadIdx.x % 32 * 8; c < ld; c += 32 * 8) {
    Pack<__half, 8> q = *(const Pack<__half, 8>*)(d + r * ld + c);
#pragma unroll
    for (int k = 0; k < 8; ++k) q.v[k] = __float2half_rn(__half2float(q.v[k]) * f);
    *(Pack<__half, 8>*)(d + r * ld + c) = q;
  }
}

dim3 copy_grid(long long rows, int cols) {
  return dim3((unsigned)((cols + 255) / 256), (unsigned)(rows < 4096 ? rows : 4096));
}

// at least one, where there is no device to ask as well
long long sm_pairs() { return num_sms() > 1 ? num_sms() / 2 : 1; }

// The widest tile whose sums, over all waves of tiles, take least: a step of 128 bytes
// takes the matrix unit BN * 2 cycles, and L2 some (16 KB + BN / 2 * 128) / 64.
int columns_of(long long tiles_m, int units, bool pairs) {
  int best = 256;
  double least = 1e300;
  for (int bn = 256; bn >= (pairs ? 64 : 128); bn /= 2) {
    const long long tiles = tiles_m * ((units + (pairs ? bn / 2 : bn) - 1) / (pairs ? bn / 2 : bn));
    const long long waves = (tiles + sm_pairs() - 1) / sm_pairs();
    const double steps = (double)waves * (bn * 2 > 256 + bn ? bn * 2 : 256 + bn);
    if (steps < least) least = steps, best = bn;
  }
  return best;
}

// A product of few tiles leaves pairs of SMs idle: its sum is then cut into stretches, each
// with tiles of its own, whose 32-bit results add_parts adds up in order: dx of 200 rows,
// 1024 to 4096, 33 us whole and 16 cut, the weights' gradients of 24008 rows, 256 to 1024,
// 96 and 38. Where it saves less than 48 steps it does not pay (1292 rows, 512 to 2048: 20
// and 21). No stretch is longer than 2^18 steps, far less than the two seconds after
// which a wait gives up, however many rows there are.
struct Cut {
  int bn, tiles_n, steps;  // of a stretch
  long long tiles_m;
  int cuts;
};
constexpr int kMostSteps = 1 << 18;
Cut cut_of(long long rows, int width, int steps) {
  Cut c{};
  c.tiles_m = (rows + 2 * kRows - 1) / (2 * kRows);
  c.bn = columns_of(c.tiles_m, width, false);
  c.tiles_n = (width + c.bn - 1) / c.bn;
  long long cuts = sm_pairs() / (c.tiles_m * c.tiles_n);
  if (cuts > steps / 8) cuts = steps / 8;
  if (cuts > 16) cuts = 16;
  if (cuts < 1 || steps - steps / cuts < 48) cuts = 1;
  const int least = (steps + kMostSteps - 1) / kMostSteps;
  if (cuts < least) cuts = least;
  c.steps = (int)((steps + cuts - 1) / cuts);
  c.cuts = (steps + c.steps - 1) / c.steps;
  return c;
}
// D's rows of hidden units, padded: dg's, then du's
struct Sums {
  Cut x, w;
};
Sums sums_of(const fm_gated_args* a, int fpad) {
  return Sums{cut_of(a->rows, (int)a->width, 2 * fpad / 64),
              cut_of(2LL * fpad, (int)a->width, (int)((a->rows + 63) / 64))};
}
// The stretches' sums, one after another. Rows below `split` go to a, those from there on to
// b, each as long as the first `exist` of them.
template <typename T>
__global__ void __launch_bounds__(256) add_parts(const float* parts, int cuts, long long rows, int cols, long long split,
                                                 long long exist, T* a, long long a_stride, T* b, long long b_stride) {
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x, n = rows * cols;
  if (at >= n) return;
  const long long m = at / cols, c = at % cols, r = m < split ? m : m - split;
  T* to = m < split ? a : b;
  if (to == nullptr || r >= exist) return;
  float s = parts[at];
#pragma unroll 4
  for (int i = 1; i < cuts; ++i) s += parts[i * n + at];
  to[r * (m < split ? a_stride : b_stride) + c] = from_f<T>(s);
}
template <typename T>
fm_status add(const TcArgs& t, int cuts, long long rows, long long split, long long exist, void* a, long long a_stride,
              void* b, long long b_stride, cudaStream_t st) {
  const long long n = rows * t.p.width;
  add_parts<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(t.parts, cuts, rows, t.p.width, split, exist, (T*)a, a_stride,
                                                           (T*)b, b_stride);
  return launch_status();
}

struct Plan {
  int64_t x, g, u;  // copies of rows, -1 for none
  int64_t d, scales, sizes, all, scaled, parts, total;
  long long stride;  // of copied rows
  int fpad;
};
bool readable(const void* base, int64_t stride, int64_t rows, int item) {
  return ((uintptr_t)base & 15) == 0 && (rows <= 1 || (stride * item) % 16 == 0);
}
Plan plan_of(const fm_gated_args* a, bool backward) {
  const int item = a->in_dtype == FM_E4M3 ? 1 : 2;
  Plan w{};
  w.stride = (a->width + 15) / 16 * 16;
  w.fpad = (int)((a->hidden + 63) / 64 * 64);
  int64_t at = 0;
  auto copy = [&](const void* base, int64_t stride, int64_t rows) {
    if (readable(base, stride, rows, item)) return (int64_t)-1;
    const int64_t here = at;
    at += align256(rows * w.stride * item);
    return here;
  };
  w.x = copy(a->x, a->x_stride, a->rows);
  w.g = copy(a->w_gate, a->gate_stride, a->hidden);
  w.u = copy(a->w_up, a->up_stride, a->hidden);
  if (backward) {
    w.d = at;
    at += align256(a->rows * 2 * (int64_t)w.fpad * 2);
    if (a->dtype == FM_F16) {
      w.scales = at;
      at += align256(a->rows * (int64_t)sizeof(float));
      w.sizes = at;
      at += align256(a->rows * (int64_t)sizeof(RowSize));
      w.all = at;
      at += 256;
      w.scaled = at;
      if (a->dw_gate || a->dw_up) at += align256(a->rows * w.stride * 2);
    }
    w.parts = at;
    const Sums s = sums_of(a, w.fpad);
    const int64_t x = a->dx && s.x.cuts > 1 ? s.x.cuts * a->rows : 0;
    const int64_t dw = (a->dw_gate || a->dw_up) && s.w.cuts > 1 ? s.w.cuts * 2LL * w.fpad : 0;
    at += align256((x > dw ? x : dw) * a->width * (int64_t)sizeof(float));
  }
  w.total = at;
  return w;
}

template <typename T>
fm_status copied(const void*& base, long long& stride, int64_t at, char* ws, long long rows, int cols, long long to_stride,
                 cudaStream_t st) {
  if (at < 0) return FM_OK;
  copy_rows<T><<<copy_grid(rows, cols), 256, 0, st>>>((const T*)base, stride, rows, cols, (T*)(ws + at), to_stride);
  base = ws + at;
  stride = to_stride;
  return launch_status();
}
fm_status copies(GatedParams& p, const Plan& w, int64_t in_dtype, char* ws, cudaStream_t st) {
  auto one = [&](const void*& base, long long& stride, int64_t at, long long rows) {
    return in_dtype == FM_E4M3 ? copied<uint8_t>(base, stride, at, ws, rows, p.width, w.stride, st)
                               : copied<uint16_t>(base, stride, at, ws, rows, p.width, w.stride, st);
  };
  if (fm_status s = one(p.x, p.xs, w.x, p.rows)) return s;
  if (fm_status s = one(p.wg, p.gs, w.g, p.hidden)) return s;
  return one(p.wu, p.us, w.u, p.hidden);
}

bool lines(const void* base, long long stride, long long rows, int item) { return readable(base, stride, rows, item); }

fm_status start(TcArgs& t, const GatedParams& p) {
  t.p = p;
  if (fm_status s = ops_error_seen()) return s;
  return ops_error_words(&t.err) ? FM_OK : FM_ERR_CUDA;
}
// kForward and kGrads: x against rows of both weights, `units` of each
fm_status pair_product(TcArgs& t, int64_t in_dtype, int units, int* bn) {
  const GatedParams& p = t.p;
  t.tiles_m = (p.rows + 2 * kRows - 1) / (2 * kRows);
  *bn = columns_of(t.tiles_m, units, true);
  t.tiles_n = (units + *bn / 2 - 1) / (*bn / 2);
  t.tiles = t.tiles_m * t.tiles_n;
  const int step = in_dtype == FM_E4M3 ? 128 : 64;
  t.steps = t.cut_steps = (p.width + step - 1) / step;
  return encode(&t.a, p.x, in_dtype, p.rows, p.width, p.xs, kRows) &&
                 encode(&t.b0, p.wg, in_dtype, p.hidden, p.width, p.gs, *bn / 2) &&
                 encode(&t.b1, p.wu, in_dtype, p.hidden, p.width, p.us, *bn / 2)
             ? FM_OK
             : FM_ERR_CUDA;
}
}  // namespace

int64_t gated_tc_workspace(const fm_gated_args* a, bool backward) { return plan_of(a, backward).total; }

fm_status gated_tc_forward(const fm_gated_args* a, GatedParams p, cudaStream_t st) {
  const Plan w = plan_of(a, false);
  if (fm_status s = copies(p, w, a->in_dtype, (char*)a->workspace, st)) return s;
  TcArgs t{};
  int bn = 0;
  if (fm_status s = start(t, p)) return s;
  if (fm_status s = pair_product(t, a->in_dtype, p.hidden, &bn)) return s;
  t.vec_out = lines(p.h, p.hs, p.rows, a->dtype == FM_F32 ? 4 : 2);
  if (a->in_dtype == FM_E4M3) return gated_tc_e4m3(a->dtype, t, bn, st);
  return a->dtype == FM_BF16 ? gated_tc_bf16(kForward, t, bn, st) : gated_tc_f16(kForward, t, bn, st);
}

fm_status gated_tc_backward(const fm_gated_args* a, GatedParams p, cudaStream_t st) {
  const Plan w = plan_of(a, true);
  char* ws = (char*)a->workspace;
  if (fm_status s = copies(p, w, a->in_dtype, ws, st)) return s;
  const bool f16 = a->dtype == FM_F16;
  const auto run = f16 ? gated_tc_f16 : gated_tc_bf16;
  TcArgs t{};
  if (fm_status s = start(t, p)) return s;
  t.fpad = w.fpad;
  t.d = ws + w.d;
  if (f16) {
    float* scales = (float*)(ws + w.scales);
    RowSize* sizes = (RowSize*)(ws + w.sizes);
    Loudest* all = (Loudest*)(ws + w.all);
    if (cudaMemsetAsync(all, 0x80, sizeof(Loudest), st) != cudaSuccess) return FM_ERR_CUDA;  // below all that is found
    const bool dw = p.dwg || p.dwu, vec_x = p.width % 8 == 0;  // x and the weights are on the 16-byte grid by now
    const bool vec_dh = lines(p.dh, p.dhs, p.rows, 2) && p.hidden % 8 == 0;
    row_sizes<<<(unsigned)((p.rows + 2LL * p.hidden + 7) / 8), 256, 0, st>>>(p, vec_dh, vec_x, sizes, all);
    auto k = !dw ? scale_rows<1, false> : vec_x ? scale_rows<8, true> : scale_rows<1, true>;
    k<<<(unsigned)((p.rows + 7) / 8), 256, 0, st>>>(p, sizes, all, scales, (__half*)(ws + w.scaled), w.stride);
    t.row_scale = scales;
    t.scaled = &all->scaled;
    if (fm_status s = launch_status()) return s;
  }
  int bn = 0;
  // all of D's columns are written: zeros in those that pad, which meet rows of zeros later
  if (fm_status s = pair_product(t, a->dtype, w.fpad, &bn)) return s;
  t.vec_dh = lines(p.dh, p.dhs, p.rows, 2);
  if (fm_status s = run(kGrads, t, bn, st)) return s;

  const long long ld = 2LL * w.fpad;
  const Sums sums = sums_of(a, w.fpad);
  auto set = [&](const Cut& c, int steps) {
    t.tiles_m = c.tiles_m, t.tiles_n = c.tiles_n;
    t.tiles = c.tiles_m * c.tiles_n * c.cuts;
    t.steps = steps, t.cut_steps = c.steps;
    t.parts = c.cuts > 1 ? (float*)(ws + w.parts) : nullptr;
  };
  if (p.dx) {
    t.half_steps = w.fpad / 64;
    set(sums.x, 2 * t.half_steps);
    t.vec_out = t.parts ? p.width % 4 == 0 : lines(p.dx, p.dxs, p.rows, 2);
    if (!encode(&t.a, t.d, a->dtype, p.rows, ld, ld, kRows) || !encode(&t.b0, p.wg, a->dtype, p.hidden, p.width, p.gs, 64) ||
        !encode(&t.b1, p.wu, a->dtype, p.hidden, p.width, p.us, 64))
      return FM_ERR_CUDA;
    if (fm_status s = run(kDx, t, sums.x.bn, st)) return s;
    if (t.parts) {
      const auto join = f16 ? add<__half> : add<__nv_bfloat16>;
      if (fm_status s = join(t, sums.x.cuts, p.rows, p.rows, p.rows, p.dx, p.dxs, nullptr, 0, st)) return s;
    }
  }
  if (p.dwg || p.dwu) {
    if (f16) {
      lower_rows<<<(unsigned)((p.rows + 7) / 8), 256, 0, st>>>((const RowSize*)(ws + w.sizes), p.rows, (__half*)t.d, ld);
      if (fm_status s = launch_status()) return s;
    }
    set(sums.w, (int)((p.rows + 63) / 64));
    t.vec_out = t.parts ? p.width % 4 == 0
                        : (!p.dwg || lines(p.dwg, p.dgs, p.hidden, 2)) && (!p.dwu || lines(p.dwu, p.dus, p.hidden, 2));
    const void* x = f16 ? (const void*)(ws + w.scaled) : p.x;
    if (!encode(&t.a, t.d, a->dtype, p.rows, ld, ld, 64) ||
        !encode(&t.b0, x, a->dtype, p.rows, p.width, f16 ? w.stride : p.xs, 64))
      return FM_ERR_CUDA;
    t.b1 = t.b0;
    if (fm_status s = run(kDw, t, sums.w.bn, st)) return s;
    if (t.parts) {
      const auto join = f16 ? add<__half> : add<__nv_bfloat16>;
      return join(t, sums.w.cuts, ld, w.fpad, p.hidden, p.dwg, p.dgs, p.dwu, p.dus, st);
    }
  }
  return FM_OK;
}
}  // namespace fm

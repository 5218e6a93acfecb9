// Gated linear layer, few rows (fm_ops.h): one new frame of each of a few streams.
//
// Memory bound: every weight is read once, for 2 operations a row. A block has UNITS
// groups of 8 hidden units; its eight warps take turns along the sum, so that a small
// layer's whole weights are under way at once (hidden / 8 blocks of eight warps), and
// their sums are added up in order in shared memory. The products go to mma.sync, whose
// 16 rows are the 8 units' rows of w_gate and the same of w_up: g and u of a unit and a
// row of x then meet in one thread. (A tile of tcgen05 is 128 rows, of which a few would
// be used.) Which terms of the sum a lane multiplies is free as long as both operands
// agree, so lanes read 16 bytes at a time straight into their operands, nothing through
// shared memory.
#include "fm_ops_gated.cuh"

namespace fm {
namespace {

constexpr int kWarps = 8;

template <typename T>
__device__ __forceinline__ void multiply(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (sizeof(T) == 1)
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ROWS groups of 8 rows of x, UNITS groups of 8 hidden units.
template <typename T, typename TO, int ROWS, int UNITS>
__global__ void __launch_bounds__(32 * kWarps) gated_step(const GatedParams p) {
  extern __shared__ float4 parts[];  // [kWarps][UNITS][ROWS][32]
  constexpr int kPer = 16 / (int)sizeof(T), kChunk = 4 * kPer;  // terms of a lane, of a step
  // steps under way at once: their reads fill about half of the registers
  constexpr int kAhead = ROWS + 2 * UNITS <= 3 ? 4 : ROWS + 2 * UNITS <= 6 ? 2 : 1;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, row = lane / 4;
  const int f0 = blockIdx.x * UNITS * 8;
  const T* x = (const T*)p.x + lane % 4 * kPer;
  const T *wg = (const T*)p.wg + lane % 4 * kPer, *wu = (const T*)p.wu + lane % 4 * kPer;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  float c[UNITS][ROWS][4];
#pragma unroll
  for (int i = 0; i < UNITS; ++i)
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) c[i][j][k] = 0.f;
#pragma unroll 1
  for (int k0 = warp * kChunk; k0 < p.width; k0 += kAhead * kWarps * kChunk) {
    uint4 qg[kAhead][UNITS], qu[kAhead][UNITS], qx[kAhead][ROWS];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int k = k0 + a * kWarps * kChunk;
      const bool in = k + lane % 4 * kPer < p.width;  // whole packs: width is a multiple of kPer
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const long long f = f0 + i * 8 + row;
        const bool here = in && f < p.hidden;
        qg[a][i] = here ? *(const uint4*)(wg + f * p.gs + k) : zero;
        qu[a][i] = here ? *(const uint4*)(wu + f * p.us + k) : zero;
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const long long r = j * 8 + row;
        qx[a][j] = in && r < p.rows ? *(const uint4*)(x + r * p.xs + k) : zero;
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (k0 + a * kWarps * kChunk >= p.width) break;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const uint4 b = qx[a][j];
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
          const uint4 g = qg[a][i], u = qu[a][i];
          multiply<T>(c[i][j], g.x, u.x, g.y, u.y, b.x, b.y);
          multiply<T>(c[i][j], g.z, u.z, g.w, u.w, b.z, b.w);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i)
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
      parts[((warp * UNITS + i) * ROWS + j) * 32 + lane] = make_float4(c[i][j][0], c[i][j][1], c[i][j][2], c[i][j][3]);
  __syncthreads();
  // a thread has g and u of one unit and two rows of x
  for (int at = threadIdx.x; at < UNITS * ROWS * 32; at += 32 * kWarps) {
    float4 s = parts[at];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = parts[w * UNITS * ROWS * 32 + at];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const int l = at % 32, j = at / 32 % ROWS, i = at / 32 / ROWS;
    const long long f = f0 + i * 8 + l / 4;
    if (f >= p.hidden) continue;
    const float g2[2] = {s.x, s.y}, u2[2] = {s.z, s.w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long r = j * 8 + l % 4 * 2 + k;
      if (r >= p.rows) continue;
      float g = g2[k], u = u2[k];
      if (sizeof(T) == 1) {  // one after the other: their product may be out of range where g is not
        const float xs = p.x_scales[r];
        g = g * xs * p.g_scales[f];
        u = u * xs * p.u_scales[f];
      }
      float h = 0.f;
      if (p.act == FM_ACT_SILU) h = act_of<FM_ACT_SILU>(g);
      else if (p.act == FM_ACT_GELU) h = act_of<FM_ACT_GELU>(g);
      else if (p.act == FM_ACT_SIGMOID) h = act_of<FM_ACT_SIGMOID>(g);
      else h = act_of<FM_ACT_RELU>(g);
      ((TO*)p.h)[r * p.hs + f] = from_f<TO>(h * u);
    }
  }
}

template <typename T, typename TO, int ROWS, int UNITS>
fm_status launch(const GatedParams& p, cudaStream_t st) {
  constexpr size_t bytes = sizeof(float4) * kWarps * UNITS * ROWS * 32;
  auto k = gated_step<T, TO, ROWS, UNITS>;
  if (!allow_smem(k, bytes)) return FM_ERR_CUDA;
  k<<<(unsigned)((p.hidden + 8 * UNITS - 1) / (8 * UNITS)), 32 * kWarps, bytes, st>>>(p);
  return launch_status();
}
// Two groups of units a block where x has many rows, all of which each block reads, and
// where one group would leave a block little to read (a kilobyte or less a unit) and make
// more blocks than run at once: 4096 units of 1024 take 5.4 us with one and 4.7 with two
// in 8 bits, 5.1 and 5.6 in 16.
template <typename T, typename TO>
fm_status sized(const GatedParams& p, cudaStream_t st) {
  const bool many = p.hidden > 16 * num_sms() && p.width * (int)sizeof(T) <= 1024;
  if (p.rows <= 8) return many ? launch<T, TO, 1, 2>(p, st) : launch<T, TO, 1, 1>(p, st);
  if (p.rows <= 16) return many ? launch<T, TO, 2, 2>(p, st) : launch<T, TO, 2, 1>(p, st);
  return launch<T, TO, 4, 2>(p, st);
}
}  // namespace

// Up to 32 rows. For 1024 to 4096 in 16 bits (8 bits) this takes 5.1 us (4.7) for one row, 5.6
// (4.9) for 16 and 9.4 (5.8) for 32; the tiles of the tensor cores 9 to 12 (7.7) for any
// number up to 128. At 64 rows this would take 15 (11).
constexpr int kFewRows = 32;

bool gated_step_takes(const fm_gated_args* a) {
  const int item = a->in_dtype == FM_E4M3 ? 1 : 2, per = 16 / item;
  auto ok = [&](const void* q, int64_t stride, int64_t rows) {
    return ((uintptr_t)q & 15) == 0 && (rows <= 1 || stride % per == 0);
  };
  return (a->in_dtype == FM_E4M3 || a->dtype != FM_F32) && a->rows <= kFewRows && a->width % per == 0 &&
         ok(a->x, a->x_stride, a->rows) && ok(a->w_gate, a->gate_stride, a->hidden) &&
         ok(a->w_up, a->up_stride, a->hidden);
}

fm_status gated_step_forward(const fm_gated_args* a, const GatedParams& p, cudaStream_t st) {
  if (a->in_dtype != FM_E4M3)
    return a->dtype == FM_F16 ? sized<__half, __half>(p, st) : sized<__nv_bfloat16, __nv_bfloat16>(p, st);
  return a->dtype == FM_F32   ? sized<E4M3, float>(p, st)
         : a->dtype == FM_F16 ? sized<E4M3, __half>(p, st) : sized<E4M3, __nv_bfloat16>(p, st);
}
}  // namespace fm

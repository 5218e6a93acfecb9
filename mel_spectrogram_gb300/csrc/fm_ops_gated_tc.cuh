// Gated linear layer on the tensor cores: one persistent kernel for its four products.
//
//   kForward  g | u = x [w_gate | w_up]^T  ->  h = act(g) u
//   kGrads    the same product             ->  D = [dg | du], from dh
//   kDx       dx = D [w_gate ; w_up]
//   kDw       [dw_gate ; dw_up] = D^T x
//
// A pair of SMs (a cluster of two blocks) works on a tile of 256 rows and BN columns:
// tcgen05.mma over both, each block holding 128 rows of A and half of B's columns in
// shared memory, so that a step of 128 bytes along the sum costs each SM 16 KB of A and
// BN / 2 * 128 bytes of B. One SM alone would read B whole: at 128 x 256 that is 96
// bytes a cycle at the matrix unit's full rate, more than L2 gives an SM (64 at most);
// the pair needs 64. For kForward and kGrads one block of the pair reads rows of
// w_gate and the other the same rows of w_up: both then hold g and u of their rows.
//
// Sums are 32-bit, in tensor memory, two buffers of BN columns in turn: eight warps
// read out one tile while the next is summed. Results go through shared memory, a
// warp's 32 rows at a time, and leave in whole lines.
//
// A and B are K-major (rows along the sum) in kForward and kGrads; in kDx the weights,
// and in kDw both, have the sum along their rows and are read as they lie (MN-major).
//
// Bound by the matrix unit: 92 % of its cycles in kForward, kDx and kDw. Measured for 24008
// rows, 1024 to 4096 in bf16, each product by itself: kForward 202 us (1.99 PFLOP/s),
// kGrads 240 (1.68: it also reads dh and writes D, 590 MB), kDx 204 (1.97), kDw 223 (1.81:
// 1.7 waves of tiles). In 8 bits kForward 118 us with silu (3.4 PFLOP/s), 134 with gelu.
#pragma once

#include "fm_ops_gated.cuh"
#include "fm_tc.cuh"

namespace fm {

bool ops_error_words(tc::ErrorWords* words);
fm_status ops_error_seen();

namespace gated {
using namespace tc;

enum Op { kForward, kGrads, kDx, kDw };

struct TcArgs {
  CUtensorMap a, b0, b1;
  ErrorWords err;
  GatedParams p;
  long long tiles_m, tiles;
  int tiles_n;
  int steps;        // steps of 128 bytes along the sum
  int half_steps;   // kDx: those over w_gate's rows
  int cut_steps;    // of a stretch of the sum (kDx, kDw); stretches are tiles of their own
  float* parts;     // [stretch][rows of the result][width]: where they leave their sums, NULL for one
  int fpad;         // hidden units rounded up to whole steps of 64: du's place in a row of D
  void* d;          // [rows][2 * fpad]
  const float* row_scale;  // FM_F16: what each row of dh is multiplied by
  const int* scaled;       // FM_F16: exponent that the weights' gradients are multiplied by
  int vec_out, vec_dh;     // whether rows of the result (of dh) allow 16-byte accesses
};

constexpr int kLeast = -24;       // exponent of the smallest magnitude in FM_F16
constexpr int kRows = 128;        // of a block
constexpr int kStepBytes = 128;   // along the sum
constexpr int kOperandA = kRows * kStepBytes;
constexpr int kGroup = 8;         // tiles of rows that are worked on before the next columns

// Warps that read out: a warp has 32 rows and its share of the columns. Sixteen where
// an activation is worked out for every element (eight took 259 us for 24008 rows of
// 1024 to 4096 in 8 bits with gelu, 207 with silu, the products alone about 110).
template <Op OP, int BN>
constexpr int kOutWarps = (OP == kForward || OP == kGrads) && BN >= 128 ? 16 : 8;
template <Op OP, int BN>
constexpr int kThreads = 64 + 32 * kOutWarps<OP, BN>;  // one that copies, one that issues products, those

template <Op OP, typename TO, int BN>
struct Layout {
  static constexpr int kUnits = OP == kForward || OP == kGrads ? BN / 2 : BN;   // columns of a tile's results
  static constexpr int kMine = kUnits / (kOutWarps<OP, BN> / 4);                // of a warp
  static constexpr int kOnce = kMine < 128 / (int)sizeof(TO) ? kMine : 128 / (int)sizeof(TO);  // of them at a time
  static constexpr int kPitch = kOnce * (int)sizeof(TO);                        // bytes of a row in shared memory
  // 32 rows (kGrads: twice, of dg and du; kForward: the scales of 8-bit rows before)
  static constexpr int kStaging = 32 * kPitch * (OP == kGrads ? 2 : 1);
  static constexpr int kOperandB = BN / 2 * kStepBytes;
  static constexpr int kSlot = kOperandA + kOperandB;
  static constexpr int kSlots = (227 * 1024 - 1536 - kOutWarps<OP, BN> * kStaging) / kSlot < 8
                                    ? (227 * 1024 - 1536 - kOutWarps<OP, BN> * kStaging) / kSlot
                                    : 8;
  static constexpr int kStage = kSlots * kSlot;
  static constexpr int kBars = kStage + kOutWarps<OP, BN> * kStaging;
  static constexpr int kBytes = kBars + 8 * (2 * kSlots + 4) + 1024;  // and what aligning takes
  static_assert(kSlots >= 4 && kBytes <= 227 * 1024 - 64, "fits an SM");
};

// ---- what two blocks need ---------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// an address in the pair's first block
constexpr uint32_t kFirstBlock = 0xfeffffffu;
__device__ __forceinline__ void tma_load_pair(uint32_t to, const CUtensorMap* m, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(to),
      "l"(m), "r"(bar & kFirstBlock), "r"(x), "r"(y)
      : "memory");
}
// The scope of its release is left at the block: what it orders are reads of tensor
// memory, by the fence before it. A release to the cluster would wait until all results
// stored so far are in global memory.
__device__ __forceinline__ void bar_arrive_first(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
template <bool EIGHT>
__device__ __forceinline__ void mma_pair(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if (EIGHT)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
        : "memory");
}
// arrives on both blocks' bar once every product issued so far is done
__device__ __forceinline__ void mma_commit_pair(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\tsetp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          bar),
      "r"(lead)
      : "memory");
}

// ---- reading out ------------------------------------------------------------
// A warp's 32 rows of PITCH bytes in shared memory, in pieces of 16 bytes whose place
// within a row is turned by the row, so that neither a lane's own row nor a line's
// lanes meet in a bank.
template <int PITCH>
__device__ __forceinline__ uint32_t piece(uint32_t base, int row, int n) {
  constexpr int kPieces = PITCH / 16, kRowsOfLine = 128 / PITCH;
  static_assert(PITCH == 32 || PITCH == 64 || PITCH == 128, "whole lines");
  return base + row * PITCH + ((n ^ (row / kRowsOfLine & (kPieces - 1))) << 4);
}
__device__ __forceinline__ void put16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 get16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const uint32_t* v) {  // 16 bytes of T from 32-bit floats
  if constexpr (sizeof(T) == 4) {
    return make_uint4(v[0], v[1], v[2], v[3]);
  } else {
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    auto two = [&](int k) { return pack2<BF16>(__uint_as_float(v[k]), __uint_as_float(v[k + 1])); };
    return make_uint4(two(0), two(2), two(4), two(6));
  }
}
// element k of 16-bit ones packed in words
template <typename T>
__device__ __forceinline__ float element(const uint32_t* w, int k) {
  const uint32_t v = k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(v << 16);
  else return __half2float(__ushort_as_half((unsigned short)v));
}

// Copies COLS columns of the warp's 32 rows from shared memory to where row(r) is
// (NULL: nowhere), columns c0 .. of which those below `end` exist.
template <typename T, int COLS, typename Row>
__device__ __forceinline__ void write_rows(uint32_t base, int lane, int c0, int end, bool vec, Row row) {
  constexpr int kPer = 16 / sizeof(T), kPieces = COLS / kPer, kAtOnce = 32 / kPieces;
  static_assert(COLS * sizeof(T) <= 128 && COLS % kPer == 0, "a row fits its place");
#pragma unroll
  for (int i = 0; i < 32; i += kAtOnce) {
    const int r = i + lane / kPieces, n = lane % kPieces, c = c0 + n * kPer;
    T* to = row(r);
    const uint4 v = get16(piece<COLS * sizeof(T)>(base, r, n));
    if (to == nullptr || c >= end) continue;
    if (vec && c + kPer <= end) {
      *(uint4*)(to + c) = v;
    } else {
      const T* e = (const T*)&v;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (c + k < end) to[c + k] = e[k];
    }
  }
}
// The other way, in two steps: read, zeros in the place of what does not exist; and put.
template <typename T, int COLS>
constexpr int kRowPieces = COLS * (int)sizeof(T) / 16;  // a row's; a lane gets as many
template <typename T, int COLS, typename Row>
__device__ __forceinline__ void read_rows(uint4 (&v)[kRowPieces<T, COLS>], int lane, int c0, int end, bool vec, Row row) {
  constexpr int kPer = 16 / (int)sizeof(T), kPieces = kRowPieces<T, COLS>;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = c0 + lane % kPieces * kPer;
    const T* from = row((32 * i + lane) / kPieces);
    v[i] = make_uint4(0, 0, 0, 0);
    if (from == nullptr || c >= end) continue;
    if (vec && c + kPer <= end) {
      v[i] = *(const uint4*)(from + c);
    } else {
      T e[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) e[k] = c + k < end ? from[c + k] : from_f<T>(0.f);
      v[i] = *(const uint4*)e;
    }
  }
}
template <typename T, int COLS>
__device__ __forceinline__ void put_rows(uint32_t base, int lane, const uint4 (&v)[kRowPieces<T, COLS>]) {
  constexpr int kPieces = kRowPieces<T, COLS>;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) put16(piece<COLS * sizeof(T)>(base, (32 * i + lane) / kPieces, lane % kPieces), v[i]);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t* r) {
  if (N == 32) tmem_ld32(addr, r);
  else tmem_ld16(addr, r);
}
template <int N>
__device__ __forceinline__ void tie(uint32_t* r) {
  if (N == 32) tie32(r);
  else tie16(r);
}

// ---- activations of pairs -----------------------------------------------------
__device__ __forceinline__ float2 pair_of(const uint32_t* v) { return make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])); }
__device__ __forceinline__ void set_pair(uint32_t* v, float2 x) { v[0] = __float_as_uint(x.x), v[1] = __float_as_uint(x.y); }
// and e = exp(-g)
__device__ __forceinline__ float2 sigmoids(float2 g, float2& e) {
  g = mul2(g, both(-kLog2e));
  e = make_float2(ex2(g.x), ex2(g.y));
  const float2 d = add2(e, both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float2 sigmoids(float2 g) {
  float2 e;
  return sigmoids(g, e);
}
// The normal distribution's integral up to g, and e = exp(-g^2 / 2): of |g| from 1, or of
// g itself, erfc(|g| / sqrt 2) / 2 = e t P(t) with t = 1 / (1 + 0.304 |g|); P of degree 7
// fitted for the least relative error up to |g| = 14 (1.4e-7), so that the tail that gelu
// multiplies by a large g keeps its digits. The exponent's three roundings add up to
// 9e-8 g^2, 2e-5 at 14, to e's.
__device__ __forceinline__ float2 normal_integrals(float2 g, float2& e) {
  constexpr float c[8] = {0.12126036f, 0.122141108f, 0.102763310f, 0.122487135f, -0.0411235951f, 0.189988881f,
                          -0.154114947f, 0.0365977213f};
  const float2 size = make_float2(fabsf(g.x), fabsf(g.y));
  float2 t = fma2(size, both(0.304055929f), both(1.f));
  t = make_float2(rcp(t.x), rcp(t.y));
  float2 q = both(c[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) q = fma2(q, t, both(c[i]));
  const float2 s = mul2(mul2(g, g), both(-0.5f * kLog2e));
  e = make_float2(ex2(s.x), ex2(s.y));
  q = mul2(mul2(q, t), e);
  const float2 r = fma2(q, both(-1.f), both(1.f));
  return make_float2(g.x > 0.f ? r.x : q.x, g.y > 0.f ? r.y : q.y);
}
__device__ __forceinline__ float2 positive(float2 g) {  // a NaN stays one
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(g.x) : "f"(0.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(g.y) : "f"(0.f));
  return g;
}
template <int ACT>
__device__ __forceinline__ float2 acts(float2 g) {
  if (ACT == FM_ACT_SILU) return mul2(g, sigmoids(g));
  if (ACT == FM_ACT_SIGMOID) return sigmoids(g);
  if (ACT == FM_ACT_RELU) return positive(g);
  float2 e;
  return mul2(g, normal_integrals(g, e));
}
template <int ACT>
__device__ __forceinline__ void acts_and_slopes(float2 g, float2& a, float2& slope) {
  if (ACT == FM_ACT_SILU) {
    const float2 s = sigmoids(g), r = fma2(s, both(-1.f), both(1.f));
    a = mul2(g, s);
    slope = fma2(a, r, s);  // s + g s (1 - s)
  } else if (ACT == FM_ACT_SIGMOID) {
    // s (1 - s). Above zero 1 - s is e^-g s: taken from one, it would be 1 % off at g = 12
    // and nothing from 17 on.
    float2 e;
    a = sigmoids(g, e);
    const float2 r = fma2(a, both(-1.f), both(1.f)), q = mul2(e, a);
    slope = mul2(a, make_float2(g.x > 0.f ? q.x : r.x, g.y > 0.f ? q.y : r.y));
  } else if (ACT == FM_ACT_RELU) {
    a = positive(g);
    slope = make_float2(g.x > 0.f ? 1.f : 0.f, g.y > 0.f ? 1.f : 0.f);
  } else {
    float2 e;
    const float2 c = normal_integrals(g, e);
    a = mul2(g, c);
    slope = fma2(mul2(g, both(0.398942280f)), e, c);
  }
}
// f(act) with the activation as a constant
template <typename F>
__device__ __forceinline__ void by_act(int act, F f) {
  if (act == FM_ACT_SILU) f(std::integral_constant<int, FM_ACT_SILU>());
  else if (act == FM_ACT_GELU) f(std::integral_constant<int, FM_ACT_GELU>());
  else if (act == FM_ACT_SIGMOID) f(std::integral_constant<int, FM_ACT_SIGMOID>());
  else f(std::integral_constant<int, FM_ACT_RELU>());
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// T: inputs, TO: results, BN: columns of a tile's sums.
template <Op OP, typename T, typename TO, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<OP, BN>, 1) product(const __grid_constant__ TcArgs t) {
  using L = Layout<OP, TO, BN>;
  constexpr bool kEight = sizeof(T) == 1, kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kPairs = OP == kForward || OP == kGrads;  // columns are g | u
  constexpr int kUnits = L::kUnits, kMine = L::kMine, kOnce = L::kOnce;
  constexpr int kStep = kStepBytes / (int)sizeof(T);       // terms of a step
  extern __shared__ unsigned char raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int dead;
  const GatedParams& p = t.p;
  const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_rank();
  auto full = [&](int s) { return base + L::kBars + 8 * s; };
  auto empty = [&](int s) { return base + L::kBars + 8 * (L::kSlots + s); };
  auto sums_full = [&](int b) { return base + L::kBars + 8 * (2 * L::kSlots + b); };
  auto sums_empty = [&](int b) { return base + L::kBars + 8 * (2 * L::kSlots + 2 + b); };

  if (tid == 0) {
    for (int s = 0; s < L::kSlots; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(sums_full(b), 1), bar_init(sums_empty(b), 2 * kOutWarps<OP, BN>);
    fence_bar_init();
    dead = 0;
    tma_prefetch(&t.a);
    tma_prefetch(&t.b0);
    tma_prefetch(&t.b1);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), 2 * BN);
  fence_before();
  __syncthreads();
  cluster_sync();  // the other block's barriers and tensor memory are there
  fence_after();
  const uint32_t tmem = tmem_slot;

  const long long pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  // first row and column of a tile; which stretch of the sum
  const long long flat = t.tiles_m * t.tiles_n;
  auto cut_of = [&](long long tile) { return kPairs ? 0 : (int)(tile / flat); };
  auto place = [&](long long tile, long long& m0, int& n0) {
    if (!kPairs) tile %= flat;
    const long long group = tile / ((long long)kGroup * t.tiles_n), in = tile - group * kGroup * t.tiles_n;
    const long long left = t.tiles_m - group * kGroup, tall = left < kGroup ? left : kGroup;
    m0 = (group * kGroup + in % tall) * 2 * kRows;
    n0 = (int)(in / tall) * kUnits;
  };

  if (warp == 0) {
    if (lane == 0) {  // ---- copies of this block's operands
      int slot = 0, turn = 1;
      bool ok = true;
      for (long long tile = pair; ok && tile < t.tiles; tile += pairs) {
        long long m0;
        int n0;
        place(tile, m0, n0);
        const int row = (int)(m0 + rank * kRows);
        const int begin = cut_of(tile) * t.cut_steps, end = min(begin + t.cut_steps, t.steps);
        for (int s = begin; s < end; ++s) {
          ok = bar_wait(empty(slot), turn, &dead, t.err);
          if (!ok) break;
          if (rank == 0) bar_expect(full(slot), 2 * L::kSlot);
          const uint32_t a = base + slot * L::kSlot, b = a + kOperandA;
          if (kPairs) {
            tma_load_pair(a, &t.a, full(slot), s * kStep, row);
            tma_load_pair(b, rank == 0 ? &t.b0 : &t.b1, full(slot), s * kStep, n0);
          } else {
            constexpr int kBox = 64 * kStepBytes;  // 64 columns of 64 rows
            const int first = n0 + (int)rank * (BN / 2);
            if (OP == kDx) {
              tma_load_pair(a, &t.a, full(slot), s * kStep, row);
              const bool up = s >= t.half_steps;
              const int y = (up ? s - t.half_steps : s) * kStep;
#pragma unroll
              for (int i = 0; i < (BN / 2 + 63) / 64; ++i)
                tma_load_pair(b + i * kBox, up ? &t.b1 : &t.b0, full(slot), first + 64 * i, y);
            } else {
#pragma unroll
              for (int i = 0; i < kRows / 64; ++i)
                tma_load_pair(a + i * kBox, &t.a, full(slot), row + 64 * i, s * kStep);
#pragma unroll
              for (int i = 0; i < (BN / 2 + 63) / 64; ++i)
                tma_load_pair(b + i * kBox, &t.b0, full(slot), first + 64 * i, s * kStep);
            }
          }
          if (++slot == L::kSlots) slot = 0, turn ^= 1;
        }
      }
      // the other block's last arrivals here come before this one ends
      for (int s = 0; ok && s < L::kSlots; ++s) {
        ok = bar_wait(empty(slot), turn, &dead, t.err);
        if (++slot == L::kSlots) slot = 0, turn ^= 1;
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {  // ---- products, for both blocks
      const uint32_t lead = elect();
      const uint32_t idesc = instr_desc(2 * kRows, BN, kBf16, !kPairs) | (OP == kDw ? 1u << 15 : 0u);
      int slot = 0, turn = 0, buffer = 0, used = 1;
      bool ok = true;
      for (long long tile = pair; ok && tile < t.tiles; tile += pairs) {
        ok = bar_wait(sums_empty(buffer), used, &dead, t.err);
        if (!ok) break;
        fence_after();
        const uint32_t d = tmem + buffer * BN;
        const int begin = cut_of(tile) * t.cut_steps, end = min(begin + t.cut_steps, t.steps);
        for (int s = begin; s < end; ++s) {
          ok = bar_wait(full(slot), turn, &dead, t.err);
          if (!ok) break;
          fence_after();
          const uint32_t a = base + slot * L::kSlot, b = a + kOperandA;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t da = OP == kDw ? desc_mn(a + 2048 * k, 64 * kStepBytes) : desc_k(a + 32 * k);
            const uint64_t db = kPairs ? desc_k(b + 32 * k) : desc_mn(b + 2048 * k, 64 * kStepBytes);
            mma_pair<kEight>(lead, d, da, db, idesc, s > begin || k > 0);
          }
          mma_commit_pair(lead, empty(slot));
          if (++slot == L::kSlots) slot = 0, turn ^= 1;
        }
        if (!ok) break;
        mma_commit_pair(lead, sums_full(buffer));
        buffer ^= 1;
        if (buffer == 0) used ^= 1;
      }
    }
    __syncwarp();
  } else {  // ---- results: a warp has 32 rows and its share of the columns
    const int quarter = warp & 3, share = (warp - 2) >> 2;
    const uint32_t stage = base + L::kStage + (warp - 2) * L::kStaging;
    const uint32_t lanes = (uint32_t)quarter << 21;
    int buffer = 0, turn = 0;
    bool ok = true;
    // this warp has all it needs of a tile's sums: the next but one may come there
    auto taken = [&] {
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_first(sums_empty(buffer));
    };
    // kGrads: dh of the next tile, read while this one is worked on
    uint4 ahead[OP == kGrads ? kRowPieces<TO, kMine> : 1];
    auto read_dh = [&](auto& v, long long row, int column) {
      read_rows<TO, kMine>(v, lane, column, p.hidden, t.vec_dh, [&](int i) {
        return row + i < p.rows ? (const TO*)p.dh + (row + i) * p.dhs : (const TO*)nullptr;
      });
    };
    for (long long tile = pair; ok && tile < t.tiles; tile += pairs) {
      long long m0;
      int n0;
      place(tile, m0, n0);
      const long long r0 = m0 + rank * kRows + quarter * 32, r = r0 + lane;
      const int c0 = n0 + share * kMine;
      const uint32_t sums = tmem + lanes + buffer * BN + share * kMine;
      if constexpr (OP == kForward) {
        constexpr int kPer = 16 / (int)sizeof(TO);
        static_assert(kOnce == kMine && kMine <= 32, "a warp's columns at once");
        float xs = 1.f;
        if (kEight) {
          xs = r < p.rows ? p.x_scales[r] : 1.f;
          const int f = c0 + lane;
          float gs = 0.f, us = 0.f;
          if (lane < kMine && f < p.hidden) gs = p.g_scales[f], us = p.u_scales[f];
          if (lane < kMine)
            asm volatile("st.shared.f32 [%0], %2;\n\tst.shared.f32 [%1], %3;" ::"r"(stage + 4 * lane),
                         "r"(stage + 4 * (kMine + lane)), "f"(gs), "f"(us)
                         : "memory");
          __syncwarp();
        }
        ok = bar_wait(sums_full(buffer), turn, &dead, t.err);
        if (!ok) break;
        fence_after();
        uint32_t g[kMine], u[kMine];
        tmem_ld<kMine>(sums, g);
        tmem_ld<kMine>(sums + BN / 2, u);
        wait_ld();
        tie<kMine>(g);
        tie<kMine>(u);
        taken();
        if (kEight) {
#pragma unroll
          for (int k = 0; k < kMine; k += 4) {
            const uint4 gs = get16(stage + 4 * k), us = get16(stage + 4 * (kMine + k));
            const uint32_t gw[4] = {gs.x, gs.y, gs.z, gs.w}, uw[4] = {us.x, us.y, us.z, us.w};
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              set_pair(g + k + j, mul2(mul2(pair_of(g + k + j), both(xs)), pair_of(gw + j)));
              set_pair(u + k + j, mul2(mul2(pair_of(u + k + j), both(xs)), pair_of(uw + j)));
            }
          }
          __syncwarp();
        }
        by_act(p.act, [&](auto act) {
#pragma unroll
          for (int k = 0; k < kMine; k += 2)
            set_pair(g + k, mul2(acts<decltype(act)::value>(pair_of(g + k)), pair_of(u + k)));
        });
#pragma unroll
        for (int k = 0; k < kMine; k += kPer) put16(piece<L::kPitch>(stage, lane, k / kPer), pack16<TO>(g + k));
        __syncwarp();
        write_rows<TO, kMine>(stage, lane, c0, p.hidden, t.vec_out, [&](int i) {
          return r0 + i < p.rows ? (TO*)p.h + (r0 + i) * p.hs : (TO*)nullptr;
        });
      } else if constexpr (OP == kGrads) {
        static_assert(kOnce == kMine && kMine <= 32, "a warp's columns at once");
        const uint32_t other = stage + 32 * L::kPitch;
        const float scale = t.row_scale && r < p.rows ? t.row_scale[r] : 1.f;
        const long long ld = 2LL * t.fpad;
        TO* d = (TO*)t.d;
        if (tile == pair) read_dh(ahead, r0, c0);
        put_rows<TO, kMine>(stage, lane, ahead);
        __syncwarp();
        uint32_t dh[kMine / 2];
#pragma unroll
        for (int k = 0; k < kMine / 8; ++k) {
          const uint4 v = get16(piece<L::kPitch>(stage, lane, k));
          dh[4 * k] = v.x, dh[4 * k + 1] = v.y, dh[4 * k + 2] = v.z, dh[4 * k + 3] = v.w;
        }
        if (tile + pairs < t.tiles) {
          long long m1;
          int n1;
          place(tile + pairs, m1, n1);
          read_dh(ahead, m1 + rank * kRows + quarter * 32, n1 + share * kMine);
        }
        ok = bar_wait(sums_full(buffer), turn, &dead, t.err);
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int c = 0; c < kMine; c += 16) {
          uint32_t g[16], u[16];
          tmem_ld<16>(sums + c, g);
          tmem_ld<16>(sums + BN / 2 + c, u);
          wait_ld();
          tie<16>(g);
          tie<16>(u);
          if (c + 16 == kMine) taken();
          by_act(p.act, [&](auto act) {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float2 a, slope, s = make_float2(element<TO>(dh, c + k), element<TO>(dh, c + k + 1));
              if (!kBf16) s = mul2(s, both(scale));
              acts_and_slopes<decltype(act)::value>(pair_of(g + k), a, slope);
              set_pair(g + k, mul2(mul2(s, pair_of(u + k)), slope));
              set_pair(u + k, mul2(s, a));
            }
          });
#pragma unroll
          for (int k = 0; k < 16; k += 8) {  // a lane's own row: nobody else reads it before the warp meets
            put16(piece<L::kPitch>(stage, lane, (c + k) / 8), pack16<TO>(g + k));
            put16(piece<L::kPitch>(other, lane, (c + k) / 8), pack16<TO>(u + k));
          }
        }
        __syncwarp();
#pragma unroll
        for (int which = 0; which < 2; ++which)
          write_rows<TO, kMine>(which ? other : stage, lane, c0, t.fpad, true, [&](int i) {
            return r0 + i < p.rows ? d + (r0 + i) * ld + which * t.fpad : (TO*)nullptr;
          });
      } else {
        constexpr int kLd = kOnce < 32 ? kOnce : 32;
        float scale = 1.f;
        if (OP == kDx && t.row_scale && r < p.rows) scale = 1.f / t.row_scale[r];
        if (OP == kDw && t.scaled) scale = power_of_two(min(max(*t.scaled, -126), 126));
        ok = bar_wait(sums_full(buffer), turn, &dead, t.err);
        if (!ok) break;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < kMine; c += kOnce) {
#pragma unroll
          for (int q = 0; q < kOnce; q += kLd) {
            uint32_t v[kLd];
            tmem_ld<kLd>(sums + c + q, v);
            wait_ld();
            tie<kLd>(v);
            if (c + q + kLd == kMine) taken();
            if (std::is_same<T, __half>::value) {
#pragma unroll
              for (int k = 0; k < kLd; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * scale);
            }
#pragma unroll
            for (int k = 0; k < kLd; k += 16 / (int)sizeof(TO))
              put16(piece<L::kPitch>(stage, lane, (q + k) * (int)sizeof(TO) / 16), pack16<TO>(v + k));
          }
          __syncwarp();
          write_rows<TO, kOnce>(stage, lane, c0 + c, p.width, t.vec_out, [&](int i) {
            const long long m = r0 + i;
            if constexpr (std::is_same<TO, float>::value) {
              const long long rows = OP == kDx ? p.rows : 2LL * t.fpad;
              return m < rows ? t.parts + (cut_of(tile) * rows + m) * p.width : (float*)nullptr;
            }
            if (OP == kDx) return m < p.rows ? (TO*)p.dx + m * p.dxs : (TO*)nullptr;
            const bool up = m >= t.fpad;
            const long long f = up ? m - t.fpad : m;
            TO* to = (TO*)(up ? p.dwu : p.dwg);
            return to && f < p.hidden ? to + f * (up ? p.dus : p.dgs) : (TO*)nullptr;
          });
          __syncwarp();
        }
      }
      __syncwarp();
      buffer ^= 1;
      if (buffer == 0) turn ^= 1;
    }
  }
  __syncthreads();
  if (dead && tid == 0) {
    // copies still in flight land in this block's memory: give them time
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  __syncthreads();
  fence_before();
  cluster_sync();  // neither block's memory goes while the other may reach for it
  if (warp == 1) {
    __syncwarp();
    fence_after();
    tmem_free_pair(tmem, 2 * BN);
  }
}

template <Op OP, typename T, typename TO, int BN>
fm_status launch(const TcArgs& t, cudaStream_t st) {
  constexpr int kBytes = Layout<OP, TO, BN>::kBytes;
  auto k = product<OP, T, TO, BN>;
  if (!allow_smem(k, kBytes)) return FM_ERR_CUDA;
  const long long most = num_sms() / 2, pairs = t.tiles < most ? t.tiles : most;
  k<<<(unsigned)(2 * pairs), kThreads<OP, BN>, kBytes, st>>>(t);
  return launch_status();
}
template <Op OP, typename T, typename TO>
fm_status launch(const TcArgs& t, int bn, cudaStream_t st) {
  if (bn == 256) return launch<OP, T, TO, 256>(t, st);
  if constexpr (OP == kForward || OP == kGrads) {
    if (bn == 64) return launch<OP, T, TO, 64>(t, st);
  }
  return launch<OP, T, TO, 128>(t, st);
}

}  // namespace gated
}  // namespace fm

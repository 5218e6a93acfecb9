// Parameters of the tensor-core attention kernels (fm_ops_attn_fwd*.cu,
// fm_ops_attn_bwd*.cu).
#pragma once

#include "fm_ops_attn.cuh"
#include "fm_tc.cuh"

namespace fm {

constexpr int kTile = 128;      // rows of a tile: the lanes of tensor memory
constexpr int kBiasPad = 128;   // copies of the end values beside the bias by offset: a warp's rows and a
                                // thread's columns reach 94 past an end when one of them is inside

// Which documents the 128 frames of a tile hold: lowest and highest id, and
// whether all its frames carry that one id. No documents: every tile is {0, 0, 1}.
struct DocRange {
  int lo, hi, uniform;
};

struct TcParams {
  AttnParams p;
  CUtensorMap qm, km, vm, gm;  // q, k, v, dout as {dim, token, head, batch}
  // coordinates step by 0 along broadcast heads or batches
  int q_mh, q_mb, k_mh, k_mb, v_mh, v_mb, g_mh, g_mb;
  const int4* q_ranges;  // [batch][q tiles] (lo, hi, uniform, 0), NULL without documents
  const int4* k_ranges;  // [batch][k tiles]
  int q_tiles, k_tiles;  // of 128
  int dim16;             // dim rounded up to 16
  int splits, split_tiles;  // the key tiles of one split; splits > 1: partial results
  const float* bias;     // [heads][2 * max_distance + 1]: the bias by offset, base 2
  float* part_o;         // [splits][batch][heads][q_len][dim]
  float* part_lse;       // [splits][batch][heads][q_len], base 2
  tc::ErrorWords err;
  // Where masks may hide a key from one query of a tile and not from another, a
  // block notes here whether its results were all finite, and a second launch
  // runs the others again, looking at every streamed row (clean_row): nearly
  // always it has nothing to do. To look at the rows at once cost a sixth of the
  // time of packed training; a second run inside the block cost as much in
  // registers. NULL: no such masks.
  int* flags;  // [blocks]
  int blocks[3];  // of the first launch
  int raw;        // it ran as MODE 0: the second has to round as it did
};

constexpr int kScan = 3;  // in place of a mode: the second launch

// The current device's error words, NULL if there are none: made by the first
// call, also while a graph is being recorded.
bool ops_error_words(tc::ErrorWords* words);

// Bytes of workspace of the tensor-core passes, and whether they take this
// call: 16-bit types, dim a multiple of 8 up to 128, and tensors whose rows
// start on 16-byte boundaries. ws may be NULL to ask only.
// The few-query kernel: its splits of the key axis.
struct StepPlan {
  int splits, split_keys, row_tiles;
};
bool tc_encode(CUtensorMap* m, const void* base, const Strides& s, int batch, int len, int heads, int dim, int rows,
               bool bf16, int* mh, int* mb);
StepPlan step_plan(const AttnParams& p);
fm_status attn_step(const AttnParams& p, int64_t dtype, const StepPlan& w, float* part_o, float* part_lse,
                    cudaStream_t st);

struct TcPlan {
  StepPlan step;  // step.splits > 0: the forward pass takes the few-query kernel
  int splits, split_tiles, q_tiles, k_tiles;
  int64_t ranges, part_o, part_lse, stats, scales, bias, flags, flags_keys, total;
};
bool tc_layout_ok(const AttnParams& p, int64_t dtype, bool backward);
TcPlan tc_plan(const AttnParams& p, bool backward);  // backward needs heads, q_len, map and grad only
// FM_ERR_KERNEL_TIMEOUT where a wait gave up since the words were last taken: its
// call's results are not valid, and nothing more is started on top of them
fm_status ops_error_seen();
fm_status attn_tc_forward(const AttnParams& p, int64_t dtype, char* ws, cudaStream_t st);
// grad: the bias gradient is wanted (p.part is set here; its rows are p.batch * q_tiles of tile kTile)
fm_status attn_tc_backward(AttnParams& p, int64_t dtype, bool grad, char* ws, cudaStream_t st);

#ifdef __CUDACC__
// The key tiles a tile of queries [i0, i0 + n) has to visit, as one range:
// below the lengths, causality and, with documents, from the first to the last
// tile that shares an id.
struct TileRange {
  int begin, end;
};
__device__ __forceinline__ int key_end(const AttnParams& p, const RowInfo& r, int i0, int n) {
  int end = r.len;
  if (p.causal) end = min(end, max(r.start + i0 + n, r.prefix));
  return max(end, 0);
}

// The head's bias by offset, in units of log2, padded by copies of its ends:
// bias[o + max_distance + kBiasPad] for |o| <= max_distance + kBiasPad.
__device__ __forceinline__ void fill_bias(const TcParams& t, int h, float* bias, int tid, int threads) {
  const int D = t.p.max_distance;
  const float* from = t.bias + (long long)h * (2 * D + 1);
  for (int i = tid; i < 2 * (D + kBiasPad) + 1; i += threads) bias[i] = from[min(max(i - kBiasPad, 0), 2 * D)];
}

// 16 bits x 16 columns of this thread's row, staged so that a warp writes whole
// lines: rows of `stage` are 128 bytes, their 16-byte pieces in an order that
// keeps eight rows' same pieces on different banks.
__device__ __forceinline__ void stage_piece(unsigned char* stage, int row, int piece, uint4 v) {
  *(uint4*)(stage + row * 128 + ((piece ^ (row & 7)) << 4)) = v;
}
// The warp's 32 rows of PIECES 16-byte pieces each, from `first` on, to rows of
// `stride` elements at `to`; `rows` of them exist, and `pieces` of their pieces.
template <int PIECES>
__device__ __forceinline__ void write_rows(const unsigned char* stage, int first, uint16_t* to, long long stride,
                                           int rows, int pieces) {
  const int lane = threadIdx.x & 31, piece = lane % PIECES;
#pragma unroll
  for (int r = lane / PIECES; r < 32; r += 32 / PIECES)
    if (r < rows && piece < pieces)
      *(uint4*)(to + r * stride + 8 * piece) = *(const uint4*)(stage + r * 128 + (((first + piece) ^ (r & 7)) << 4));
}

// A row's N raw products of one tile, to scores in base 2: scaled or capped,
// and biased. MODE 0 leaves them raw (the weights' exponent scales them), 1 is
// scale and bucket bias, 2 anything. Column j has offset o0 + j, or o0 - j
// where REV. CAP_SLOPE: also 1 - tanh^2, the cap's derivative, into slope.
//
// tanh: where every score of the warp's rows is small against the cap
// (kTanhSmall, the usual case) the polynomial alone: four multiply-adds and two
// products instead of two trips to the special-function unit, which the
// weights' 2^z needs. Elsewhere each score takes the form that its own size
// asks for, so that its value does not depend on its neighbours', which may be
// hidden from it.
template <int N, int MODE, bool REV, bool CAP_SLOPE>
__device__ __forceinline__ void tile_scores(float (&s)[N], float (&slope)[CAP_SLOPE ? N : 1], const AttnParams& p,
                                            float c, const float* bias, float slope2, int o0) {
  using namespace tc;
  if (MODE == 0) return;
  const int D = p.max_distance, last = REV ? o0 - (N - 1) : o0 + (N - 1);
  if (MODE == 2 && !(p.cap > 0.f) && p.slopes == nullptr) {
    // as MODE 1, or a scale alone
    if (CAP_SLOPE) {
#pragma unroll
      for (int j = 0; j < N; ++j) slope[j] = 1.f;
    }
    if (p.map == nullptr) {
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] *= c;
    }
  } else if (MODE == 2) {
    // a slope's share is linear in the column where all offsets have one sign
    const bool ahead = __all_sync(0xffffffffu, min(o0, last) >= 0), back = __all_sync(0xffffffffu, max(o0, last) <= 0);
    const bool linear = p.slopes && (ahead || back);
    const float g = !linear ? 0.f : ahead ? -slope2 : slope2;
    const float2 g2 = both(REV ? -g : g), base = both(linear ? g * (float)o0 : 0.f);
    if (p.cap > 0.f) {
      const float k = p.scale / p.cap, out = p.cap * kLog2e;
      const float2 in = both(1.f / out), k2 = both(k);
      float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) top[j & 3] = fmaxf(top[j & 3], fabsf(s[j]));
      const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const bool small = __all_sync(0xffffffffu, most * fabsf(k) <= kTanhSmall);
      // of the polynomial, times what takes a raw product to base 2 (k's powers
      // in them would leave the range of floats at large and at tiny caps)
      float2 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = both(tanh_over_x(i) * c);
      auto polynomial = [&](float2 x) {
        const float2 y = mul2(x, k2), q = mul2(y, y);
        return mul2(fma2(fma2(fma2(a[3], q, a[2]), q, a[1]), q, a[0]), x);
      };
      auto finish = [&](int j, float2 t) {
        if (CAP_SLOPE) {
          const float2 th = mul2(t, in), f = fma2(make_float2(-th.x, -th.y), th, both(1.f));
          slope[j] = f.x;
          slope[j + 1] = f.y;
        }
        const float2 z = add2(t, fma2(g2, make_float2((float)j, (float)(j + 1)), base));
        s[j] = z.x;
        s[j + 1] = z.y;
      };
      // two loops: with the choice inside one, its branches kept the columns'
      // chains of multiply-adds from overlapping (four times slower)
      if (small) {
#pragma unroll
        for (int j = 0; j < N; j += 2) finish(j, polynomial(make_float2(s[j], s[j + 1])));
      } else {
        const float c2 = 2.f * kLog2e * k;
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const float2 x = make_float2(s[j], s[j + 1]);
          float2 t = polynomial(x);
          if (fabsf(x.x * k) > kTanhSmall) t.x = out * tanh_from(x.x * c2);
          if (fabsf(x.y * k) > kTanhSmall) t.y = out * tanh_from(x.y * c2);
          finish(j, t);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float2 z = fma2(make_float2(s[j], s[j + 1]), both(c),
                              fma2(g2, make_float2((float)j, (float)(j + 1)), base));
        s[j] = z.x;
        s[j + 1] = z.y;
        if (CAP_SLOPE) slope[j] = slope[j + 1] = 1.f;
      }
    }
    if (p.slopes && !linear) {
      const float f0 = (float)o0;
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = fmaf(-slope2, fabsf(REV ? f0 - (float)j : f0 + (float)j), s[j]);
    }
    c = 1.f;
  }
  if (MODE == 1 || p.map) {
    // rows of a warp differ by 31 in o0: one choice for all of them (the array
    // holds copies of its ends far enough)
    const bool above = __all_sync(0xffffffffu, min(o0, last) >= D), below = __all_sync(0xffffffffu, max(o0, last) <= -D);
    if (above || below) {
      const float2 b = both(bias[above ? 2 * (D + kBiasPad) : 0]);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float2 z = fma2(make_float2(s[j], s[j + 1]), both(c), b);
        s[j] = z.x;
        s[j + 1] = z.y;
      }
    } else {
      const float* at = bias + (o0 + D + kBiasPad);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float2 b = REV ? make_float2(at[-j], at[-j - 1]) : make_float2(at[j], at[j + 1]);
        const float2 z = fma2(make_float2(s[j], s[j + 1]), both(c), b);
        s[j] = z.x;
        s[j + 1] = z.y;
      }
    }
  }
}

// Whether any of eight 16-bit floats is infinite or NaN: an exponent of ones
// overflows into the sign's place when one is added to it.
template <bool BF16>
__device__ __forceinline__ bool not_finite(uint4 v) {
  constexpr uint32_t one = BF16 ? 0x00800080u : 0x04000400u, m = 0x7fff7fffu;
  return ((((v.x & m) + one) | ((v.y & m) + one) | ((v.z & m) + one) | ((v.w & m) + one)) & 0x80008000u) != 0;
}
// adds 0, or NaN for a value that is not finite
__device__ __forceinline__ float taint(float sum, float v) { return fmaf(v, 0.f, sum); }
// zeros for four 16-byte pieces of a row in each of BOXES boxes
template <int BOXES>
__device__ __forceinline__ void clear_row(unsigned char* row, int box, int first) {
#pragma unroll
  for (int x = 0; x < BOXES; ++x)
#pragma unroll
    for (int e = first; e < first + 4; ++e) *(uint4*)(row + x * box + 16 * e) = make_uint4(0, 0, 0, 0);
}
// In a tile with masked pairs a streamed row must not reach the rows that do
// not see it, but a weight of 0 times infinity or NaN would. Four 16-byte
// pieces of a row in each of BOXES boxes: all zeros if the row is unused, and
// pieces that are not finite become zeros; whether there were any. A row that
// sees such a row gets a NaN as its weight, and so a result of NaN. mark: set
// before a piece is cleared, for others who scan the same row.
template <bool BF16, int BOXES>
__device__ __forceinline__ bool clean_row(unsigned char* row, int box, int first, bool unused,
                                          uint32_t* mark = nullptr, uint32_t bit = 0) {
  bool bad = false;
#pragma unroll
  for (int x = 0; x < BOXES; ++x)
#pragma unroll
    for (int e = first; e < first + 4; ++e) {
      uint4* at = (uint4*)(row + x * box + 16 * e);
      const bool wrong = !unused && not_finite<BF16>(*at);
      if (wrong && mark) {
        atomicOr(mark, bit);
        __threadfence_block();
      }
      if (unused || wrong) *at = make_uint4(0, 0, 0, 0);
      bad |= wrong;
    }
  return bad;
}

// The second launch (TcParams::flags): this block's share of the flagged blocks'
// work, one after another, work(place in the grid, index, tensor memory). A
// block may allocate tensor memory only once, and nearly all have nothing to
// do: the first flagged one allocates, after the last it is freed. Ends early
// where a wait gave up, whose products and copies may still be under way.
template <typename Work>
__device__ __forceinline__ void scan_blocks(const TcParams& t, Work work) {
  using namespace tc;
  __shared__ uint32_t slot;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), x = t.blocks[0], y = t.blocks[1];
  uint32_t tmem = 0;
  bool held = false;
  for (int i = blockIdx.x; i < x * y * t.blocks[2]; i += gridDim.x) {
    if (!t.flags[i]) continue;  // the same for the whole block
    if (!held) {
      if (warp == 17) tmem_alloc(smem_u32(&slot), 512);
      fence_before();
      __syncthreads();
      fence_after();
      tmem = slot;
      held = true;
    }
    if (!work(dim3(i % x, i / x % y, i / x / y), i, tmem)) break;
  }
  if (!held) return;
  __syncthreads();
  if (warp == 17) {
    __syncwarp();
    fence_after();
    tmem_free(tmem, 512);
  }
}

// Bits of the N columns whose document is this row's. ids: the columns'
// documents, `there` of them exist; own: the row's (-2: none matches). A warp
// goes through the distinct ids of the tile, usually one or two.
template <int N>
__device__ __forceinline__ uint64_t same_document(const int32_t* ids, int there, int own) {
  const int lane = threadIdx.x & 31;
  const int v0 = lane < there ? __ldg(ids + lane) : -1;
  const int v1 = N > 32 && lane + 32 < there ? __ldg(ids + lane + 32) : -1;
  uint64_t left = (uint64_t)__ballot_sync(0xffffffffu, v0 >= 0) | (uint64_t)__ballot_sync(0xffffffffu, v1 >= 0) << 32;
  uint64_t same = 0;
  while (left != 0) {
    const int j = __ffsll((long long)left) - 1;
    const int id = __shfl_sync(0xffffffffu, j < 32 ? v0 : v1, j & 31);
    const uint64_t m = (uint64_t)__ballot_sync(0xffffffffu, v0 == id) | (uint64_t)__ballot_sync(0xffffffffu, v1 == id) << 32;
    if (own == id) same = m;
    left &= ~m;
  }
  return same;
}
// bits [lo, hi) of N columns
template <int N>
__device__ __forceinline__ uint64_t column_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, N);
  return lo < hi ? (~0ull >> (64 - (hi - lo))) << lo : 0ull;
}
#endif

}  // namespace fm

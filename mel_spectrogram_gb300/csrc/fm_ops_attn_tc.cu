// Host side of the tensor-core attention kernels, and the small kernels around
// them: document ranges of tiles before, the join of split results after.
#include "fm_ops_attn_bwd.cuh"

#include <cudaTypedefs.h>

#include <mutex>

namespace fm {

__device__ unsigned g_ops_error;

bool ops_error_words(tc::ErrorWords* words) {
  static std::mutex mu;
  static tc::ErrorWords known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev].host == nullptr) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return false;
    void *d = nullptr, *h = nullptr;
    // addressed the same from the device: a 64-bit process has one address space
    const bool ok = cudaGetSymbolAddress(&d, g_ops_error) == cudaSuccess &&
                    cudaHostAlloc(&h, sizeof(unsigned), cudaHostAllocPortable | cudaHostAllocMapped) == cudaSuccess;
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (!ok) return false;
    *(volatile unsigned*)h = 0;
    known[dev] = tc::ErrorWords{(unsigned*)d, (unsigned*)h};
  }
  *words = known[dev];
  return true;
}

fm_status ops_error_seen() {
  tc::ErrorWords w;
  if (!ops_error_words(&w)) return FM_ERR_CUDA;
  return *(volatile unsigned*)w.host ? FM_ERR_KERNEL_TIMEOUT : FM_OK;
}

fm_status attn_fwd_bf16_64(const TcParams& t, int mode, cudaStream_t st);
fm_status attn_fwd_bf16_128(const TcParams& t, int mode, cudaStream_t st);
fm_status attn_fwd_f16_64(const TcParams& t, int mode, cudaStream_t st);
fm_status attn_fwd_f16_128(const TcParams& t, int mode, cudaStream_t st);

#define FM_BWD(name) fm_status name(const TcParams& t, const bwd::Extra& x, int mode, cudaStream_t st)
FM_BWD(attn_bwd_keys_bf16_64);
FM_BWD(attn_bwd_keys_bf16_128);
FM_BWD(attn_bwd_keys_f16_64);
FM_BWD(attn_bwd_keys_f16_128);
FM_BWD(attn_bwd_queries_bf16_64);
FM_BWD(attn_bwd_queries_bf16_128);
FM_BWD(attn_bwd_queries_f16_64);
FM_BWD(attn_bwd_queries_f16_128);

namespace {

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

// Whether a tensor [batch][len][heads][dim] can be read by 16-byte rows: a
// stride of 0 (a broadcast head or batch) becomes a dimension of one entry.
bool rows_ok(const void* base, const Strides& s, int batch, int len, int heads) {
  auto ok = [](long long stride, int extent, bool broadcast) {
    return extent <= 1 || (broadcast && stride == 0) || (stride > 0 && stride % 8 == 0 && stride < (1LL << 38));
  };
  return ((uintptr_t)base & 15) == 0 && ok(s.t, len, false) && ok(s.h, heads, true) && ok(s.b, batch, true);
}

// Before the tiles' kernels, in one launch: the documents of each tile of 128
// frames ({lowest, highest, all one id}; padding frames count only against the
// last), by blocks x < tiles of row y = batch entry; and the bias by offset in
// base 2, by the blocks after them with y = head.
__global__ void __launch_bounds__(kTile) prepare(const AttnParams p, int q_tiles, int k_tiles, int4* ranges, int bf16,
                                                 float* bias) {
  __shared__ int lo, hi, valid;
  const int tiles = ranges ? q_tiles + k_tiles : 0, x = blockIdx.x;
  if (x >= tiles) {
    const int W = 2 * p.max_distance + 1, i = (x - tiles) * kTile + threadIdx.x, h = blockIdx.y;
    if (i < W && h < p.heads) bias[(long long)h * W + i] = kLog2e * table_value(p, (long long)p.map[i] * p.heads + h, bf16);
    return;
  }
  const int b = blockIdx.y;
  if (b >= p.batch) return;
  const bool keys = x >= q_tiles;
  const int tile = keys ? x - q_tiles : x, len = keys ? p.k_len : p.q_len;
  const int at = tile * kTile + threadIdx.x;
  const int id = at < len ? (keys ? p.k_docs : p.q_docs)[(long long)b * len + at] : -1;
  if (threadIdx.x == 0) lo = 0x7fffffff, hi = -1, valid = 0;
  __syncthreads();
  if (id >= 0) {
    atomicMin(&lo, id);
    atomicMax(&hi, id);
    atomicAdd(&valid, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int4* to = keys ? ranges + (long long)p.batch * q_tiles + (long long)b * k_tiles : ranges + (long long)b * q_tiles;
    to[tile] = make_int4(lo, hi, valid == kTile && lo == hi, 0);
  }
}

// out = sum of the splits' results, weighted by 2^(lse - highest lse). A block
// a row: its warps take splits in turn, four elements a lane, and are added up
// in order. Eight warps for few splits; 32 for many, whose reads one after
// another would otherwise be what takes the time.
template <bool BF16, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) join(const AttnParams p, int splits, const float* part_o, const float* part_lse) {
  __shared__ float tops[WARPS], totals[WARPS];
  __shared__ float4 sums[WARPS][32];
  const long long rows = (long long)p.batch * p.heads * p.q_len, row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < splits; s += 32 * WARPS) top = fmaxf(top, part_lse[s * rows + row]);
  top = warp_max(top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
  top = tops[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) top = fmaxf(top, tops[w]);
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);  // dim <= 128
  const bool mine = 4 * lane < p.dim;
#pragma unroll 8
  for (int s = warp; s < splits; s += WARPS) {
    const float lse = part_lse[s * rows + row], w = lse == -INFINITY ? 0.f : exp2f(lse - base);
    total += w;
    if (mine) {
      const float4 o = *(const float4*)(part_o + (s * rows + row) * p.dim + 4 * lane);
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
    }
  }
  sums[warp][lane] = acc;
  if (lane == 0) totals[warp] = total;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) {
    const float4 o = sums[w][lane];
    acc.x += o.x;
    acc.y += o.y;
    acc.z += o.z;
    acc.w += o.w;
    total += totals[w];
  }
  const int i = (int)(row % p.q_len), h = (int)(row / p.q_len % p.heads), b = (int)(row / p.q_len / p.heads);
  const float f = total == 0.f ? 0.f : 1.f / total;
  if (p.lse && lane == 0) p.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
  if (mine) {
    const long long at = b * p.os.b + i * p.os.t + h * p.os.h + 4 * lane;
    const uint2 r = make_uint2(tc::pack2<BF16>(acc.x * f, acc.y * f), tc::pack2<BF16>(acc.z * f, acc.w * f));
    *(uint2*)((uint16_t*)p.out + at) = r;
    if (p.rest)
      *(uint2*)((uint16_t*)p.rest + at) =
          make_uint2(tc::rest2<BF16>(acc.x * f, acc.y * f, r.x), tc::rest2<BF16>(acc.z * f, acc.w * f, r.y));
  }
}

// Statistics of the backward pass by query, padded to whole tiles of 64:
// base-2 lse (+inf where a query sees nothing or is padding: every weight
// 2^(z - inf) is 0) less `lift`, and delta = dout . out. LANES threads a row, 8
// elements each, kStatsParts rows in turn; block (x, head, batch entry). norms
// (f16, zeros before): a query's largest squared norm of dout over the heads that
// share keys; what is not finite counts as 0.
constexpr int kStatsParts = 4;
template <typename T, int LANES>
__global__ void __launch_bounds__(256) bwd_stats(const AttnParams p, int q_pad, float lift, float* lse2, float* delta,
                                                 float* norms, int norm_pad) {
  const int lane = threadIdx.x % LANES, h = blockIdx.y, b = blockIdx.z;
#pragma unroll 2
  for (int part = 0; part < kStatsParts; ++part) {
    const int i = (blockIdx.x * kStatsParts + part) * (256 / LANES) + threadIdx.x / LANES;
    const bool there = i < p.q_len && (p.q_docs == nullptr || p.q_docs[(long long)b * p.q_len + i] >= 0);
    const long long row = (long long)b * p.heads + h;
    float s = 0.f, norm = 0.f, l = -INFINITY;
    if (there) {
      l = p.lse[row * p.q_len + i];
      if (lane * 8 < p.dim) {
        const Pack<T, 8> g = *(const Pack<T, 8>*)((const T*)p.dout + b * p.dos.b + i * p.dos.t + h * p.dos.h + lane * 8);
        const long long at = b * p.os.b + i * p.os.t + h * p.os.h + lane * 8;
        const Pack<T, 8> o = *(const Pack<T, 8>*)((const T*)p.out_in + at);
        Pack<T, 8> rest{};
        if (p.rest) rest = *(const Pack<T, 8>*)((const T*)p.rest + at);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = to_f(g.v[k]);
          s = fmaf(d, to_f(o.v[k]) + to_f(rest.v[k]), s);
          norm = fmaf(d, d, norm);
        }
      }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o, LANES);
      norm += __shfl_xor_sync(0xffffffffu, norm, o, LANES);
    }
    if (lane == 0 && i < q_pad) {
      lse2[row * q_pad + i] = l == -INFINITY ? INFINITY : l * kLog2e - lift;
      delta[row * q_pad + i] = s;
      // bits of floats that are not negative are ordered as ints; a maximum has no order
      if (norms && norm <= 3.402823466e38f)
        atomicMax((int*)norms + ((long long)b * p.kv_heads + h / p.group) * norm_pad + i, __float_as_int(norm));
    }
  }
}

// Squared norms of v by key, whole tiles of 128; 0 for what does not count or is
// not finite. 16 threads a key, 16 keys a block.
__global__ void __launch_bounds__(256) bwd_v_norms(const AttnParams p, float* norms, int pad) {
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 15, j = blockIdx.x * 16 + (threadIdx.x >> 4);
  float norm = 0.f;
  if (j < row_info(p, b).len && lane * 8 < p.dim && (p.k_docs == nullptr || p.k_docs[(long long)b * p.k_len + j] >= 0)) {
    const Pack<__half, 8> v =
        *(const Pack<__half, 8>*)((const __half*)p.v + b * p.vs.b + j * p.vs.t + h * p.vs.h + lane * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) norm = fmaf(to_f(v.v[k]), to_f(v.v[k]), norm);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, o, 16);
  if (lane == 0) norms[((long long)b * p.kv_heads + h) * pad + j] = norm <= 3.402823466e38f ? norm : 0.f;
}

// The power of two for each row of dS: 2^14 over the bound 2 |dout| |v| of the
// row's own norm and the largest one that it sees. A block takes the 128 queries
// or keys of a tile, a thread a row. Of a tile that all of them see a thread reads
// one norm; of one cut by lengths or causality a row needs the largest norm up to,
// or from, one column, which the block makes once for all; only where documents
// meet each thread goes through the tile's norms and ids. 6 us for causal
// training's 8 x 4 x 1292 rows (17 with each thread going through every cut tile).
__global__ void __launch_bounds__(kTile) bwd_scales(const __grid_constant__ TcParams t, const float* q_norms,
                                                    const float* k_norms, float* q_scale, float* k_scale) {
  __shared__ float norm[kTile], tops[kTile / 32];
  __shared__ int id[kTile];
  const AttnParams& p = t.p;
  const bool keys = (int)blockIdx.x >= t.q_tiles;
  const int b = blockIdx.z, tile = keys ? blockIdx.x - t.q_tiles : blockIdx.x, r0 = tile * kTile, tid = threadIdx.x;
  const RowInfo info = row_info(p, b);
  const long long head = (long long)b * p.kv_heads + blockIdx.y;
  const long long q_at = head * t.q_tiles * kTile, k_at = head * t.k_tiles * kTile;
  const float *own = keys ? k_norms + k_at : q_norms + q_at, *other = keys ? q_norms + q_at : k_norms + k_at;
  const int row = r0 + tid, s_len = keys ? p.q_len : p.k_len, own_len = keys ? p.k_len : p.q_len;
  // columns [lo, hi) are seen by length and causality; tiles [begin, end) hold some of any row's
  int lo = 0, hi = keys ? p.q_len : info.len, begin = 0, end = keys ? t.q_tiles : 0;
  int all_lo = 0, all_hi = hi;  // of all rows
  if (keys) {
    if (p.causal) {
      if (row >= info.prefix) lo = row - info.start;
      if (r0 + kTile > info.prefix) all_lo = r0 + kTile - 1 - info.start;
      if (r0 >= info.prefix) begin = min(end, max(0, r0 - info.start) / kTile);
    }
  } else {
    if (p.causal) {
      hi = min(hi, max(info.start + row + 1, info.prefix));
      all_hi = min(all_hi, max(info.start + r0 + 1, info.prefix));
    }
    end = (key_end(p, info, r0, min(kTile, p.q_len - r0)) + kTile - 1) / kTile;
  }
  const int32_t* docs = nullptr;
  int4 own_range = make_int4(0, 0, 1, 0);
  int doc = -2;  // matches none
  if (t.k_ranges) {
    docs = keys ? p.q_docs + (long long)b * p.q_len : p.k_docs + (long long)b * p.k_len;
    own_range = keys ? t.k_ranges[b * t.k_tiles + tile] : t.q_ranges[b * t.q_tiles + tile];
    if (row < own_len) doc = (keys ? p.k_docs + (long long)b * p.k_len : p.q_docs + (long long)b * p.q_len)[row];
    if (doc < 0) doc = -2;
  }
  float all = 0.f, mine = 0.f;  // of this thread's column of tiles that all see; of this row's
  // without documents those tiles follow one another
  const int whole_begin = docs ? begin : max(begin, (all_lo + kTile - 1) / kTile);
  const int whole_end = docs ? begin : min(end, all_hi / kTile);
#pragma unroll 8
  for (int i = whole_begin; i < whole_end; ++i) all = fmaxf(all, other[i * kTile + tid]);
  for (int i = begin; i < end; ++i) {
    const int c0 = i * kTile, c = c0 + tid;
    bool same = true;
    if (docs) {
      const int4 o = keys ? t.q_ranges[b * t.q_tiles + i] : t.k_ranges[b * t.k_tiles + i];
      if (o.x > own_range.y || o.y < own_range.x) continue;
      same = o.z && own_range.z && o.x == own_range.x;
      if (same && c0 >= all_lo && c0 + kTile <= all_hi) {
        all = fmaxf(all, other[c]);
        continue;
      }
    } else if (i >= whole_begin && i < whole_end) {
      i = whole_end - 1;
      continue;
    }
    float v = other[c];
    __syncthreads();
    if (same) {
      // a query sees the tile's keys before its `hi`, a key the queries from its
      // `lo` on: the largest of a warp's columns up to, or from, each one
      const int lane = tid & 31;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const float o = keys ? __shfl_down_sync(0xffffffffu, v, d) : __shfl_up_sync(0xffffffffu, v, d);
        if (keys ? lane + d < 32 : lane >= d) v = fmaxf(v, o);
      }
      norm[tid] = v;
      __syncthreads();
      const int first = max(lo - c0, 0), last = min(hi - c0, kTile) - 1;
      if (first <= last) {
        const int at = keys ? first : last;
        mine = fmaxf(mine, norm[at]);
        for (int w = keys ? (at | 31) + 1 : (at & ~31) - 1; w >= 0 && w < kTile; w += keys ? 32 : -32)
          mine = fmaxf(mine, norm[w]);
      }
      continue;
    }
    norm[tid] = v;
    id[tid] = c < s_len ? docs[c] : -1;
    __syncthreads();
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
    for (int k = 0; k < kTile; ++k)
      m[k & 3] = fmaxf(m[k & 3], c0 + k >= lo && c0 + k < hi && id[k] == doc ? norm[k] : 0.f);
    mine = fmaxf(mine, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
  }
  all = warp_max(all);
  if ((tid & 31) == 0) tops[tid >> 5] = all;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTile / 32; ++w) mine = fmaxf(mine, tops[w]);
  const float e = floorf(13.f - 0.5f * log2f(own[row]) - 0.5f * log2f(mine));
  (keys ? k_scale + k_at : q_scale + q_at)[row] = fabsf(e) < 120.f ? exp2f(e) : 1.f;  // of nothing: as it is
}

// Whether the few-query kernel runs. It takes time with its operands of 16 rows
// (queries x heads that share a key head), the tiled kernel with its heads, each a
// tile of 256 rows however few queries fill it; a row costs the first less at head
// size 64 than at 128. Measured, bf16, few-query / tiled in us (batch x key heads x
// heads that share one, keys):
//  16 queries: 35 / 38 and 52 / 46 (32x4x1, 3001; size 64 and 128), 63 / 137 and
//   153 / 167 (32x16x1), 74 / 236 and 138 / 286 (32x4x8), 19 / 17 and 23 / 19
//   (64x1x2, 800), 14 / 19 and 17 / 21 (1x1x1, 30001).
//  17 to 32, size 64: 43 / 72 (64x4x1, 3001), 81 / 137 (32x16x1), 41 to 52 / 70
//   (32x4x2), 29 to 43 / 37 (8x2x8), 28 to 31 / 37 (24x4x1), 41 to 45 / 38
//   (32x4x1), 21 to 25 / 17 (64x1x2, 800).
//  17 to 32, size 128: where four or more heads share keys, 98 to 138 / 165 (32x4x4),
//   17 to 25 / 27 (3x8x8, 600), 55 to 71 / 86 (1x2x32, 12001), but 52 to 66 / 45
//   (8x2x8) and 45 to 66 / 43 (2x1x64), where the tiled kernel's blocks are one full
//   wave of the SMs and split no keys; where fewer share, 156 / 167 (32x16x1), but
//   101 to 114 / 87 (64x4x1), 52 to 64 / 37 (64x4x1, 800), 52 to 105 / 86 (32x4x2).
//  40 and more: 92 / 71 and 98 / 87 (64x4x1), 51 / 40 and 70 / 49 (40x4x1, 1500),
//   174 / 235 and 282 / 285 (32x4x8), at 64 queries 253 / 235 and 431 / 286.
bool takes_step(const AttnParams& p) {
  if (p.q_len <= 16 || p.q_len > 32) return p.q_len <= 16;
  const long long blocks = (long long)p.batch * p.heads;
  const bool one_wave = 2 * blocks > num_sms() && blocks <= num_sms();
  return p.dim <= 64 || (p.group >= 4 && !one_wave);
}

int mode_of(const AttnParams& p) {
  if (p.cap > 0.f || p.slopes || !(p.scale > 0.f)) return 2;
  return p.map ? 1 : 0;
}
int64_t align256(int64_t n) { return (n + 255) & ~(int64_t)255; }
}  // namespace

// The tensor [batch][len][heads][dim] to TMA as {dim, len, heads, batch}, boxes of
// 64 x rows. The encoder is a driver call: it needs the device's context on
// this thread, which a thread that only took cached memory so far does not
// have.
bool tc_encode(CUtensorMap* m, const void* base, const Strides& s, int batch, int len, int heads, int dim, int rows,
               bool bf16, int* mh, int* mb) {
  *mh = heads > 1 && s.h != 0;
  *mb = batch > 1 && s.b != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)len, (cuuint64_t)(*mh ? heads : 1),
                              (cuuint64_t)(*mb ? batch : 1)};
  auto bytes = [&](long long stride, bool used) { return (cuuint64_t)(used ? stride * 2 : 16); };
  const cuuint64_t strides[3] = {bytes(s.t, len > 1), bytes(s.h, *mh), bytes(s.b, *mb)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, step[4] = {1, 1, 1, 1};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
  return encoder() != nullptr &&
         encoder()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tc_layout_ok(const AttnParams& p, int64_t dtype, bool backward) {
  if (dtype == FM_F32 || p.dim > 128 || p.dim % 8 || p.k_len == 0 || encoder() == nullptr) return false;
  if (backward && !(p.q_len > 0 && rows_ok(p.dout, p.dos, p.batch, p.q_len, p.heads) &&
                    rows_ok(p.out_in, p.os, p.batch, p.q_len, p.heads) &&
                    rows_ok(p.dq, p.dqs, p.batch, p.q_len, p.heads) &&
                    rows_ok(p.dk, p.dks, p.batch, p.k_len, p.kv_heads) &&
                    rows_ok(p.dv, p.dvs, p.batch, p.k_len, p.kv_heads)))
    return false;
  if (((uintptr_t)p.rest & 15) != 0) return false;
  return rows_ok(p.q, p.qs, p.batch, p.q_len, p.heads) && rows_ok(p.k, p.ks, p.batch, p.k_len, p.kv_heads) &&
         rows_ok(p.v, p.vs, p.batch, p.k_len, p.kv_heads) && rows_ok(p.out, p.os, p.batch, p.q_len, p.heads);
}

TcPlan tc_plan(const AttnParams& p, bool backward) {
  TcPlan w{};
  w.q_tiles = (p.q_len + kTile - 1) / kTile;
  w.k_tiles = (p.k_len + kTile - 1) / kTile;
  w.splits = 1;
  w.split_tiles = w.k_tiles;
  if (!backward && takes_step(p)) {
    w.step = step_plan(p);
    w.splits = w.step.splits;
  } else if (!backward) {
    // Too few blocks for the SMs and a long key axis: split it, four tiles a
    // split at least (a split costs a pass of its rows through the join).
    const long long blocks = (long long)((w.q_tiles + 1) / 2) * p.heads * p.batch;
    const int sms = num_sms();
    if (blocks * 2 <= sms && w.k_tiles >= 8) {
      long long s = sms / blocks;
      if (s > w.k_tiles / 4) s = w.k_tiles / 4;
      w.split_tiles = (int)((w.k_tiles + s - 1) / s);
      w.splits = (w.k_tiles + w.split_tiles - 1) / w.split_tiles;
    }
  }
  int64_t at = 0;
  w.ranges = at;
  if (p.q_docs) at += align256((int64_t)sizeof(int4) * p.batch * (w.q_tiles + w.k_tiles));
  const int64_t rows = (int64_t)p.batch * p.heads * p.q_len;
  w.part_o = at;
  if (w.splits > 1) at += align256(rows * w.splits * p.dim * (int64_t)sizeof(float));
  w.part_lse = at;
  if (w.splits > 1) at += align256(rows * w.splits * (int64_t)sizeof(float));
  w.stats = at;
  if (backward) at += align256((int64_t)sizeof(float) * 2 * p.batch * p.heads * ((p.q_len + 63) / 64 * 64));
  w.scales = at;  // norms of queries and keys, then the powers of two
  if (backward && p.f16)
    at += align256((int64_t)sizeof(float) * 2 * p.batch * p.kv_heads * kTile * ((int64_t)w.q_tiles + w.k_tiles));
  w.bias = at;
  if (p.map && w.step.splits == 0) at += align256((int64_t)sizeof(float) * p.heads * (2 * (int64_t)p.max_distance + 1));
  w.flags = at;
  if (p.causal || p.q_docs) {
    const int64_t q_blocks = backward ? w.q_tiles : (w.q_tiles + 1) / 2;
    w.flags_keys = at + align256((int64_t)sizeof(int) * q_blocks * p.heads * p.batch * w.splits);
    at = w.flags_keys + (backward ? align256((int64_t)sizeof(int) * w.k_tiles * p.kv_heads * p.batch) : 0);
  }
  w.total = at;
  return w;
}

fm_status tc_setup(TcParams& t, const AttnParams& p, int64_t dtype, const TcPlan& w, char* ws, int q_rows, int k_rows,
                   cudaStream_t st) {
  const bool bf16 = dtype == FM_BF16;
  t.p = p;
  if (!ops_error_words(&t.err)) return FM_ERR_CUDA;
  t.raw = mode_of(p) == 0;
  t.q_tiles = w.q_tiles;
  t.k_tiles = w.k_tiles;
  t.dim16 = (p.dim + 15) / 16 * 16;
  t.splits = w.splits;
  t.split_tiles = w.split_tiles;
  if (!tc_encode(&t.qm, p.q, p.qs, p.batch, p.q_len, p.heads, p.dim, q_rows, bf16, &t.q_mh, &t.q_mb) ||
      !tc_encode(&t.km, p.k, p.ks, p.batch, p.k_len, p.kv_heads, p.dim, k_rows, bf16, &t.k_mh, &t.k_mb) ||
      !tc_encode(&t.vm, p.v, p.vs, p.batch, p.k_len, p.kv_heads, p.dim, k_rows, bf16, &t.v_mh, &t.v_mb))
    return FM_ERR_CUDA;
  if (p.dout && !tc_encode(&t.gm, p.dout, p.dos, p.batch, p.q_len, p.heads, p.dim, q_rows, bf16, &t.g_mh, &t.g_mb))
    return FM_ERR_CUDA;
  if (p.q_docs || p.map) {
    int4* r = p.q_docs ? (int4*)(ws + w.ranges) : nullptr;
    float* bias = p.map ? (float*)(ws + w.bias) : nullptr;
    const int tiles = r ? w.q_tiles + w.k_tiles : 0, spans = bias ? (2 * p.max_distance + kTile) / kTile : 0;
    const int rows = r && bias ? (p.batch > p.heads ? p.batch : p.heads) : r ? p.batch : p.heads;
    prepare<<<dim3(tiles + spans, rows), kTile, 0, st>>>(p, w.q_tiles, w.k_tiles, r, bf16, bias);
    t.q_ranges = r;
    t.k_ranges = r ? r + (int64_t)p.batch * w.q_tiles : nullptr;
    t.bias = bias;
  }
  return FM_OK;
}

fm_status attn_tc_forward(const AttnParams& p, int64_t dtype, char* ws, cudaStream_t st) {
  const TcPlan w = tc_plan(p, false);
  const bool bf16 = dtype == FM_BF16;
  TcParams t{};
  t.part_o = (float*)(ws + w.part_o);
  t.part_lse = (float*)(ws + w.part_lse);
  fm_status s = FM_OK;
  if (w.step.splits > 0) {
    s = attn_step(p, dtype, w.step, t.part_o, t.part_lse, st);
  } else {
    s = tc_setup(t, p, dtype, w, ws, kTile, kTile, st);
    const int mode = mode_of(p);
    if (p.causal || p.q_docs) t.flags = (int*)(ws + w.flags);
    if (s == FM_OK)
      s = p.dim <= 64 ? (bf16 ? attn_fwd_bf16_64(t, mode, st) : attn_fwd_f16_64(t, mode, st))
                      : (bf16 ? attn_fwd_bf16_128(t, mode, st) : attn_fwd_f16_128(t, mode, st));
  }
  if (s != FM_OK || w.splits == 1) return s;
  const long long rows = (long long)p.batch * p.heads * p.q_len;
  const unsigned blocks = (unsigned)rows;
  const bool many = w.splits >= 64;
  auto k = many ? (bf16 ? join<true, 32> : join<false, 32>) : (bf16 ? join<true, 8> : join<false, 8>);
  k<<<blocks, many ? 1024 : 256, 0, st>>>(p, w.splits, t.part_o, t.part_lse);
  return launch_status();
}

fm_status attn_tc_backward(AttnParams& p, int64_t dtype, bool grad, char* ws, cudaStream_t st) {
  const TcPlan w = tc_plan(p, true);
  TcParams t{};
  if (grad) p.part = (float*)(ws + w.total);
  if (fm_status s = tc_setup(t, p, dtype, w, ws, bwd::kCols, bwd::kCols, st)) return s;
  const bool bf16 = dtype == FM_BF16;
  bwd::Extra x{};
  x.q_pad = (p.q_len + 63) / 64 * 64;
  const long long rows = (long long)p.batch * p.heads * x.q_pad;
  float* lse2 = (float*)(ws + w.stats);
  x.lse2 = lse2;
  x.delta = lse2 + rows;
  const bool narrow = p.dim <= 64;
  const int per_block = kStatsParts * (narrow ? 32 : 16);
  const dim3 grid((x.q_pad + per_block - 1) / per_block, p.heads, p.batch);
  float *delta = lse2 + rows, *q_norms = nullptr;
  const int q_rows = w.q_tiles * kTile, k_rows = w.k_tiles * kTile;
  const long long heads = (long long)p.batch * p.kv_heads;
  if (!bf16) {
    q_norms = (float*)(ws + w.scales);
    if (cudaMemsetAsync(q_norms, 0, sizeof(float) * heads * q_rows, st) != cudaSuccess) return FM_ERR_CUDA;
  }
  if (bf16 && narrow) bwd_stats<__nv_bfloat16, 8><<<grid, 256, 0, st>>>(p, x.q_pad, 0.f, lse2, delta, nullptr, 0);
  else if (bf16) bwd_stats<__nv_bfloat16, 16><<<grid, 256, 0, st>>>(p, x.q_pad, 0.f, lse2, delta, nullptr, 0);
  else if (narrow) bwd_stats<__half, 8><<<grid, 256, 0, st>>>(p, x.q_pad, bwd::kLift<false>, lse2, delta, q_norms, q_rows);
  else bwd_stats<__half, 16><<<grid, 256, 0, st>>>(p, x.q_pad, bwd::kLift<false>, lse2, delta, q_norms, q_rows);
  if (!bf16) {
    float *k_norms = q_norms + heads * q_rows, *q_scale = k_norms + heads * k_rows, *k_scale = q_scale + heads * q_rows;
    bwd_v_norms<<<dim3(k_rows / 16, p.kv_heads, p.batch), 256, 0, st>>>(p, k_norms, k_rows);
    bwd_scales<<<dim3(w.q_tiles + w.k_tiles, p.kv_heads, p.batch), kTile, 0, st>>>(t, q_norms, k_norms, q_scale, k_scale);
    x.q_scale = q_scale;
    x.k_scale = k_scale;
  }
  const int mode = mode_of(p);
  using Fn = fm_status (*)(const TcParams&, const bwd::Extra&, int, cudaStream_t);
  const bool small = p.dim <= 64;
  const Fn queries = small ? (bf16 ? attn_bwd_queries_bf16_64 : attn_bwd_queries_f16_64)
                           : (bf16 ? attn_bwd_queries_bf16_128 : attn_bwd_queries_f16_128);
  const Fn keys = small ? (bf16 ? attn_bwd_keys_bf16_64 : attn_bwd_keys_f16_64)
                        : (bf16 ? attn_bwd_keys_bf16_128 : attn_bwd_keys_f16_128);
  const bool masks = p.causal || p.q_docs;
  // the second launches (kScan, see TcParams::flags) come after both first ones,
  // which run beside one another
  for (int m : {mode, kScan}) {
    if (m == kScan && !masks) break;
    t.flags = masks ? (int*)(ws + w.flags) : nullptr;
    if (fm_status s = queries(t, x, m, st)) return s;
    t.flags = masks ? (int*)(ws + w.flags_keys) : nullptr;
    if (fm_status s = keys(t, x, m, st)) return s;
  }
  return FM_OK;
}
}  // namespace fm

namespace {
// a wait for an arrival that never comes
__global__ void wait_for_nothing(fm::tc::ErrorWords err) {
  __shared__ uint64_t bar;
  __shared__ volatile int dead;
  if (threadIdx.x == 0) {
    fm::tc::bar_init(fm::tc::smem_u32(&bar), 1);
    fm::tc::fence_bar_init();
    dead = 0;
  }
  __syncthreads();
  fm::tc::bar_wait(fm::tc::smem_u32(&bar), 0, &dead, err);
}
}  // namespace

extern "C" fm_status fm_ops_selftest_wait(fm_stream_t stream) {
  fm::tc::ErrorWords w;
  if (!fm::ops_error_words(&w)) return FM_ERR_CUDA;
  wait_for_nothing<<<1, 32, 0, (cudaStream_t)stream>>>(w);
  return fm::launch_status();
}

extern "C" fm_status fm_ops_poll_error(void) {
  fm::tc::ErrorWords w;
  // the whole device: a copy would not wait for streams that do not wait for the default one
  if (!fm::ops_error_words(&w) || cudaDeviceSynchronize() != cudaSuccess) return FM_ERR_CUDA;
  unsigned v = 0;
  if (cudaMemcpy(&v, w.device, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return FM_ERR_CUDA;
  if (v != 0 && cudaMemset(w.device, 0, sizeof v) != cudaSuccess) return FM_ERR_CUDA;
  *(volatile unsigned*)w.host = 0;
  return (fm_status)v;
}

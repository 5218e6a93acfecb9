// Attention backward on the fifth-generation tensor cores.
//
// Two kernels of one shape, so that every sum has one owner and one order:
//   KEYS     a block owns 128 keys of one key head and streams the queries of
//            all heads that share it: dv += P^T dout, dk += dS^T q.
//   queries  a block owns 128 queries of one head and streams the keys:
//            dq += dS k, and the bias gradient, sums of dS along diagonals.
// Both recompute scores and weights P = 2^(z - lse) with dP = dout v^T and
// dS = P (dP - delta). Seven products instead of the five of a single kernel,
// but no partial dq in memory and no atomics.
//
// An owned row is a lane of tensor memory. Streamed tiles are 64 wide, and
// two groups of 256 threads take them in turn, two threads a row with 32
// columns each: a thread reads its S and dP, and writes P and dS (16 bits)
// over them, from where the second products take them as their A operand.
// Warp 16 copies, warp 17 issues products, so one group's arithmetic runs
// beside the other group's products. (With one thread a row a tile's
// arithmetic took twice its products' time, and the code of the biased modes
// did not stay in the instruction cache.)
//
// Bound: a group's chain on a tile. At head size 64 with a bias its arithmetic
// takes about 2300 cycles (3300 where the bias gradient's diagonals are added
// too), while the products of two tiles take 1000 to 1300; at 128 the score
// products count as well: their 128 x 64 x 16 steps read 6 KB of shared memory
// for 32 cycles of arithmetic (the tensor unit takes 128 bytes a cycle).
// Measured: 8 packed rows of 3001 frames, 8 heads of 64, bf16, bias of 320
// buckets up to 800: 205 us for the queries, 186 for the keys; 8 rows of 1292,
// 16 heads of 128 on 4 key heads, f16, causal, capped: 177 and 237.
#pragma once

#include "fm_ops_attn_tc.cuh"

namespace fm {
namespace bwd {

using namespace tc;

constexpr int kThreads = 640;
constexpr int kGroup = 256;
constexpr int kCols = 64;      // rows of a streamed tile
constexpr int kColumns = kCols / 2;  // a thread's share
constexpr int kDiagPad = 192;  // room beside the bias gradient for a tile's diagonals
constexpr int kChains = 4, kChainEntries = 48;
// f16 operands: P is kept 2^15 larger (weights are at most 1), and each row of dS
// (a query's, or a key's in the keys' kernel) times a power of two that brings
// its bound 2 |dout| |v| to 2^14, so that small weights and small gradients stay
// normal numbers and large ones in range. The bound takes what the row sees and
// no more (bwd_scales): what is hidden from it changes none of its bits. The
// products' results are scaled back in 32 bits. bf16 has the range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 15.f;

template <int DP, bool KEYS>
struct Smem {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kOwnBox = kTile * 128;
  static constexpr int kOwn = kBoxes * kOwnBox;  // one owned operand
  static constexpr int kBox = kCols * 128;
  static constexpr int kHalf = kBoxes * kBox;  // one streamed operand
  static constexpr int kStats = 2 * kHalf;     // lse and delta of the slot's queries
  static constexpr int kSlot = 2 * kHalf + 1024;
  static constexpr int kMaxSlots = 6;
  static constexpr int kBars = 2 * kOwn;
  static constexpr int kRing = kBars + 1024;
  // floats, whole 16-byte units: the bias by offset, the bias gradient by offset
  __host__ __device__ static int bias_floats(int max_distance) { return (2 * (max_distance + kBiasPad) + 4) & ~3; }
  __host__ __device__ static int diag_floats(int max_distance) { return (2 * (max_distance + kDiagPad) + 4) & ~3; }
  // what follows the ring: the bias (a copy for each group where heads change
  // on the way), the bias gradient by offset for each group, the chains'
  // results (and at the end the far sums, in their place)
  static size_t tail(int max_distance, bool bias, bool grad) {
    size_t n = 0;
    if (bias) n += sizeof(float) * (KEYS ? 2 : 1) * bias_floats(max_distance);
    if (grad) n += sizeof(float) * (2 * diag_floats(max_distance) + 8 * kChains * kChainEntries);
    return n;
  }
  // streamed tiles the ring holds: what shared memory (227 KB, less a little
  // for static variables and the base's alignment) has room for. Three at least
  // for any map; with three a tile's copy starts only when the tile three
  // before it is summed.
  static int slots(int max_distance, bool bias, bool grad) {
    const int n = (int)((227 * 1024 - 256 - 1024 - kRing - tail(max_distance, bias, grad)) / kSlot);
    return n < kMaxSlots ? n : kMaxSlots;
  }
  static size_t bytes(int max_distance, bool bias, bool grad) {
    return 1024 + kRing + (size_t)slots(max_distance, bias, grad) * kSlot + tail(max_distance, bias, grad);
  }
};
enum { kFull = 0, kEmpty = 8, kOwnFull = 16, kSFull = 17, kPReady = 20, kDone = 23, kScanned = 24, kBarCount = 26 };
// Buffers of 128 columns for a streamed tile's scores and dP, taken in turn:
// with three, a tile's scores are there before the group that will take it has
// finished its last one. Beside dk and dv of 128 columns only two fit.
template <int DP, bool KEYS>
constexpr int kBuffers = DP == 128 && KEYS ? 2 : 3;

// a barrier of a group's 256 threads that also tells whether all are well
__device__ __forceinline__ bool group_ok(int group, bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, %2, 256, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)ok), "r"(group + 1)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "l"(from), "r"(bytes), "r"(bar)
               : "memory");
}

// What the kernels need beside TcParams.
struct Extra {
  const float* lse2;   // [batch * heads][q_pad]: base-2 lse, +inf for rows that see nothing or are not there
  const float* delta;  // [batch * heads][q_pad]
  int q_pad;           // q_len rounded up to 64
  // f16: powers of two for the rows of dS, [batch][kv_heads][tiles of 128 queries or keys]
  const float *q_scale, *k_scale;
  int slots;  // tiles of the ring
};
// One block's work; SCAN: of the second launch, on tensor memory that its block
// holds (held), as in the forward pass. False: a wait gave up.
template <int DP, bool BF16, int MODE, bool KEYS, bool SCAN>
__device__ __forceinline__ bool block(const TcParams& t, const Extra& x, const dim3 at, const int index,
                                      const uint32_t held) {
  using L = Smem<DP, KEYS>;
  extern __shared__ unsigned char raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int dead;
  __shared__ int range[2];
  __shared__ int tainted;                            // a result is not finite
  __shared__ uint32_t bad_rows[SCAN ? 2 : 1][2][8];  // [parity][group][warp]: streamed rows that are not finite
  const AttnParams& p = t.p;
  const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
  unsigned char* mem = raw + (base - smem_u32(raw));
  auto bar = [&](int n) { return base + L::kBars + 8 * n; };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one per warp
  const bool has_bias = MODE == 1 || (MODE == 2 && p.map);
  const int D = p.max_distance, nbias = L::bias_floats(D);
  const bool grad = !KEYS && p.part != nullptr;
  // the group's threads meet at barriers: then they also leave together
  const bool joined = grad || (KEYS && has_bias);
  float* bias_mem = (float*)(mem + L::kRing + x.slots * L::kSlot);
  float* diag_mem = bias_mem + (has_bias ? (KEYS ? 2 : 1) * nbias : 0);  // [2][ndiag]
  const int ndiag = L::diag_floats(D);
  float* chain_mem = diag_mem + 2 * ndiag;  // [group][quarter of the rows][kChains][kChainEntries]
  float* far_mem = chain_mem;  // [2][512], after the last chain

  const int b = at.z;
  const int r0 = (!KEYS && p.causal ? t.blocks[0] - 1 - (int)at.x : (int)at.x) * kTile;
  const int hk = KEYS ? at.y : at.y / p.group;
  const int h0 = KEYS ? hk * p.group : at.y;
  const RowInfo info = row_info(p, b);
  const int owned = min(kTile, (KEYS ? p.k_len : p.q_len) - r0);

  if (tid == 0) {
    for (int i = 0; i < x.slots; ++i) bar_init(bar(kFull + i), 1), bar_init(bar(kEmpty + i), 1);
    bar_init(bar(kOwnFull), 1);
    for (int w = 0; w < 3; ++w) bar_init(bar(kSFull + w), 1), bar_init(bar(kPReady + w), 8);
    for (int w = 0; w < 2; ++w) bar_init(bar(kScanned + w), 8);
    bar_init(bar(kDone), 1);
    fence_bar_init();
    dead = 0;
    tainted = 0;
    range[0] = 0x7fffffff;
    range[1] = 0;
    tma_prefetch(&t.qm);
    tma_prefetch(&t.km);
    tma_prefetch(&t.vm);
    tma_prefetch(&t.gm);
  }
  if (!SCAN && warp == 17) tmem_alloc(smem_u32(&tmem_slot), 512);
  if (has_bias && !KEYS) fill_bias(t, h0, bias_mem, tid, kThreads);
  if (grad)
    for (int i = tid; i < 2 * ndiag; i += kThreads) diag_mem[i] = 0.f;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = SCAN ? held : tmem_slot;
  // The keys' kernel needs nothing of the queries' one: its blocks may start on
  // SMs that have no more blocks of this one.
  if (!KEYS && !SCAN) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // the streamed tiles [sb, se), in steps of 64, of each head
  int sb = 0, se;
  if (KEYS) {
    se = r0 < info.len ? (p.q_len + kCols - 1) / kCols : 0;
    if (p.causal && r0 >= info.prefix) sb = min(se, max(0, r0 - info.start) / kCols);
  } else {
    se = (key_end(p, info, r0, owned) + kCols - 1) / kCols;
  }
  if (t.k_ranges) {
    const int4 own = KEYS ? t.k_ranges[b * t.k_tiles + r0 / kTile] : t.q_ranges[b * t.q_tiles + r0 / kTile];
    const int4* other = KEYS ? t.q_ranges + (long long)b * t.q_tiles : t.k_ranges + (long long)b * t.k_tiles;
    for (int i = sb / 2 + tid; i < (se + 1) / 2; i += kThreads) {
      const int4 o = other[i];
      if (o.x <= own.y && o.y >= own.x) {
        atomicMin(&range[0], 2 * i);
        atomicMax(&range[1], 2 * i + 2);
      }
    }
    __syncthreads();
    sb = max(sb, range[0]);
    se = min(se, range[1]);
  }
  const int per_head = max(se - sb, 0), n = per_head * (KEYS ? p.group : 1);

  constexpr int NB = kBuffers<DP, KEYS>;
  float far_lo = 0.f, far_hi = 0.f;  // bias gradients beyond the map, of this thread's row
  // columns: buffers of S and dP (64 each), then dv and dk, or dq
  constexpr uint32_t kAcc = NB * 128, kAcc2 = kAcc + (KEYS ? DP : 0);
  // registers: 5 groups of warps x 96 at the start; 4 x 104 + 64 = 480
  if (warp < 16) {
    if (!SCAN) take_registers<104>();
    const int w = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, lane = tid & 31;
    const int lane_row = quarter * 32 + lane, in_group = half * 128 + lane_row;
    const uint32_t lanes = (uint32_t)quarter << 21;
    const int row = r0 + lane_row;  // the key or the query
    const float c = p.scale * kLog2e;
    const bool raw = MODE == 0 || (SCAN && t.raw);
    const int row_tiles = KEYS ? t.k_tiles : t.q_tiles;
    const float sigma =
        BF16 ? 1.f : (KEYS ? x.k_scale : x.q_scale)[((long long)b * p.kv_heads + hk) * row_tiles * kTile + row];
    const float tau = BF16 ? 1.f : sigma * exp2f(-kLift<BF16>);
    const int32_t* kdocs = p.k_docs ? p.k_docs + (long long)b * p.k_len : nullptr;
    const int32_t* qdocs = p.q_docs ? p.q_docs + (long long)b * p.q_len : nullptr;
    const int32_t* sdocs = KEYS ? qdocs : kdocs;  // of the streamed side
    int rd = -2;                                   // this row's document; matches none if padding
    int4 own_range = make_int4(0, 0, 1, 0);
    if (kdocs) {
      own_range = KEYS ? t.k_ranges[b * t.k_tiles + r0 / kTile] : t.q_ranges[b * t.q_tiles + r0 / kTile];
      if (lane_row < owned) {
        const int d = (KEYS ? kdocs : qdocs)[row];
        if (d >= 0) rd = d;
      }
    }
    float row_lse = 0.f, row_delta = 0.f;
    if (!KEYS) {
      const long long at = ((long long)b * p.heads + h0) * x.q_pad + row;
      const bool there = row < x.q_pad;
      row_lse = there ? x.lse2[at] : INFINITY;
      row_delta = there ? x.delta[at] : 0.f;
    }
    float* bias = bias_mem + (KEYS ? w * nbias : 0);
    float* diag = diag_mem + w * ndiag;
    int buffer = w, turn = 0, slot = w, round = 0, scan = 0;
    int head = -1, hh = 0, tile = sb + w;  // the streamed tile, and the head of the group it is of
    bool ok = true;
    for (int it = w; it < n; it += 2, tile += 2) {
      if (KEYS) {
        while (tile >= se) tile -= per_head, ++hh;
      }
      const int first = tile * kCols, c0 = first + half * kColumns, h = h0 + hh;
      const uint32_t ts = tmem + lanes + buffer * 128 + half * kColumns, tt = ts + 64;
      if (KEYS && has_bias && h != head) {
        // every thread of the group is done with the head before
        if (!group_ok(w, ok)) break;
        fill_bias(t, h, bias, in_group, kGroup);
        if (!group_ok(w, ok)) break;
      }
      head = h;
      const float slope2 = MODE == 2 && p.slopes ? p.slopes[h] * kLog2e : 0.f;
      // columns [lo, hi) of this half are seen by length and causality
      int lo = 0, hi = kColumns;
      bool masked = false, clean = false, docs = false;
      if (KEYS) {
        if (row >= info.len) hi = 0;
        if (p.causal && row >= info.prefix) lo = row - info.start - c0;
        masked = r0 + kTile > info.len;
        if (p.causal && r0 + kTile > info.prefix) masked |= r0 + kTile - 1 - info.start > first;
      } else {
        int end = info.len, all = info.len;
        if (p.causal) {
          end = min(end, max(info.start + row + 1, info.prefix));
          all = min(all, max(info.start + r0 + 1, info.prefix));
        }
        hi = end - c0;
        masked = first + kCols > all;
        clean = first + kCols > info.len && info.len < p.k_len;
      }
      if (kdocs) {
        const int4 o = KEYS ? t.q_ranges[b * t.q_tiles + first / kTile] : t.k_ranges[b * t.k_tiles + first / kTile];
        if (!(o.z && own_range.z && o.x == own_range.x)) docs = masked = true;
        if (!o.z) clean = true;
      }
      const int s_len = KEYS ? p.q_len : p.k_len;
      uint32_t seen = ~0u;  // bit j: column j is seen
      if (masked) {
        seen = (uint32_t)column_range<kColumns>(lo, min(hi, s_len - c0));
        if (docs) seen &= (uint32_t)same_document<kColumns>(sdocs + c0, s_len - c0, rd);
      }

      unsigned char* smem_slot = mem + L::kRing + slot * L::kSlot;
      // this thread's half of a streamed row: of q or dout, or of k
      const int s_op = (in_group >> 6) & 1, s_frame = first + (in_group & 63);
      unsigned char* s_row = smem_slot + s_op * L::kHalf + (in_group & 63) * 128;
      uint32_t bad_seen = 0;  // columns seen by this row that are not finite
      bool well = true;
      if constexpr (SCAN) {
        if (masked) {
          well = bar_wait(bar(kFull + slot), round, &dead, t.err);
          bool bad = false;
          if (well && (KEYS || s_op == 0))
            bad = clean_row<BF16, L::kBoxes>(
                s_row, L::kBox, 4 * half,
                s_frame < s_len && ((!KEYS && s_frame >= info.len) || (kdocs && sdocs[s_frame] < 0)));
          fence_async();
          const uint32_t rows = __ballot_sync(0xffffffffu, bad);
          if (lane == 0) {
            bad_rows[scan][w][half * 4 + quarter] = rows;
            bar_arrive(bar(kScanned + w));
          }
          well = bar_wait(bar(kScanned + w), scan, &dead, t.err) && well;
          const uint32_t* all = bad_rows[scan][w] + half;  // rows 32 half ..: every second warp's
          bad_seen = seen & (all[0] | all[2] | all[4] | all[6]);
          scan ^= 1;
        }
        clean = false;
      }
      ok = bar_wait(bar(kSFull + buffer), turn, &dead, t.err) && well;
      fence_after();
      if (clean || KEYS) ok = bar_wait(bar(kFull + slot), round, &dead, t.err) && ok;
      if (joined) {
        if (!group_ok(w, ok)) break;
      } else if (!__all_sync(0xffffffffu, ok)) {
        break;
      }
      if (clean) {
        // streamed frames that nothing may use become zeros before the second
        // products read them: q and dout, or k
        const bool unused = s_frame < s_len && ((!KEYS && s_frame >= info.len) || (kdocs && sdocs[s_frame] < 0));
        if (unused && (KEYS || s_op == 0)) clear_row<L::kBoxes>(s_row, L::kBox, 4 * half);
        fence_async();
      }
      const float* lse = (const float*)(smem_slot + L::kStats) + half * kColumns;
      const float* delta = lse + kCols;

      float s[kColumns], slope[MODE == 2 ? kColumns : 1];
      uint32_t dp[kColumns];
      uint32_t* u = (uint32_t*)s;
      tmem_ld32(ts, u);
      if (MODE != 2) tmem_ld32(tt, dp);
      wait_ld();
      tie32(u);
      if (MODE != 2) tie32(dp);
      if (SCAN && raw) {
#pragma unroll
        for (int j = 0; j < (MODE == 2 ? kColumns : 1); ++j) slope[j] = 1.f;
      }
      if (!raw) tile_scores<kColumns, MODE, KEYS, MODE == 2>(s, slope, p, c, bias, slope2,
                                                   KEYS ? row - (info.start + c0) : c0 - (info.start + row));
#pragma unroll
      for (int j = 0; j < kColumns; j += 4) {
        float4 q = make_float4(row_lse, row_lse, row_lse, row_lse);
        if (KEYS) q = *(const float4*)(lse + j);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 z = make_float2(s[j + e], s[j + e + 1]), n2 = e ? make_float2(-q.z, -q.w) : make_float2(-q.x, -q.y);
          const float2 a = raw ? fma2(z, both(c), n2) : add2(z, n2);
          s[j + e] = ex2(a.x);
          s[j + e + 1] = ex2(a.y);
        }
      }
      if (masked) {
#pragma unroll
        for (int j = 0; j < kColumns; ++j) s[j] = (seen >> j & 1) ? s[j] : 0.f;
      }
      if (SCAN) {
#pragma unroll
        for (int j = 0; j < kColumns; ++j) s[j] = (bad_seen >> j & 1) ? NAN : s[j];
      }
      uint32_t pk[kColumns / 2];
      if (KEYS) {
#pragma unroll
        for (int j = 0; j < kColumns / 2; ++j) pk[j] = pack2<BF16>(s[2 * j], s[2 * j + 1]);
        tmem_st16(ts, pk);
      }
      if (MODE == 2) {  // beside the cap's derivatives there were no registers for it
        tmem_ld32(tt, dp);
        wait_ld();
        tie32(dp);
      }
#pragma unroll
      for (int j = 0; j < kColumns; j += 4) {
        float4 q = make_float4(row_delta, row_delta, row_delta, row_delta);
        if (KEYS) q = *(const float4*)(delta + j);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 g = add2(make_float2(__uint_as_float(dp[j + e]), __uint_as_float(dp[j + e + 1])),
                                e ? make_float2(-q.z, -q.w) : make_float2(-q.x, -q.y));
          const float2 f = mul2(make_float2(s[j + e], s[j + e + 1]), g);
          s[j + e] = f.x;
          s[j + e + 1] = f.y;
        }
      }
      if (masked) {  // 0 times what an unused frame's dP holds
#pragma unroll
        for (int j = 0; j < kColumns; ++j) s[j] = (seen >> j & 1) ? s[j] : 0.f;
      }
      // dS goes to the products in the inputs' type; the bias gradient below
      // sums it in 32 bits
#pragma unroll
      for (int j = 0; j < kColumns / 2; ++j) {
        float2 a = make_float2(s[2 * j], s[2 * j + 1]);
        if (!BF16) a = mul2(a, both(tau));
        if (MODE == 2) a = mul2(a, make_float2(slope[2 * j], slope[2 * j + 1]));
        pk[j] = pack2<BF16>(a.x, a.y);
      }
      tmem_st16(tt, pk);
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kPReady + buffer));
      buffer += 2;
      if (buffer >= NB) buffer -= NB, turn ^= 1;
      slot += 2;
      if (slot >= x.slots) slot -= x.slots, round ^= 1;

      if (grad) {
        // offsets of the tile: o = (first - start - r0) + column - row
        const int t0 = first - info.start - r0;
        if (t0 - (kTile - 1) >= D || t0 + kCols - 1 <= -D) {
          float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
          for (int j = 0; j < kColumns; j += 2) sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], make_float2(s[j], s[j + 1]));
          sum[0] = add2(sum[0], sum[1]);
          if (t0 > 0) far_hi += sum[0].x + sum[0].y;
          else far_lo += sum[0].x + sum[0].y;
        } else {
          // Diagonal sums of the warp's 32 x 32: in two chains of 16 columns,
          // each step hands a lane's sum to the next row's lane, which adds its
          // element of the next column. Lane 31 finishes one diagonal a step;
          // at the end lane r holds that of column 15 - row r.
          float* mine = chain_mem + ((w * 4 + quarter) * kChains + 2 * half) * kChainEntries;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float f[16];
            f[0] = s[16 * g];
#pragma unroll
            for (int k = 1; k < 16; ++k) {
              const float up = __shfl_up_sync(0xffffffffu, f[k - 1], 1);
              f[k] = s[16 * g + k] + (lane ? up : 0.f);
            }
            float* e = mine + g * kChainEntries;
            if (lane == 31) {
#pragma unroll
              for (int k = 0; k < 16; k += 4) *(float4*)(e + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
            } else {
              e[46 - lane] = f[15];
            }
          }
          ok = group_ok(w, ok);
          // the rows' quarters and their chains, diagonal by diagonal
          const int d = in_group;  // column - row + 127
          if (d < kTile + kCols - 1) {
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int g = 0; g < kChains; ++g) {
                const int e = d - 96 - 16 * g + 32 * q;
                if (e >= 0 && e < 47) sum += chain_mem[((w * 4 + q) * kChains + g) * kChainEntries + e];
              }
            diag[t0 + d - 127 + D + kDiagPad] += sum;
          }
        }
      }
    }
    // ---- results: a group each for dv and dk, or half of dq's columns each,
    // and half of those a thread
    if (n > 0) ok = __all_sync(0xffffffffu, ok && bar_wait(bar(kDone), 0, &dead, t.err));
    if (ok) {
      fence_after();
      const bool is_dv = KEYS && w == 0;
      const Strides st = KEYS ? (is_dv ? p.dvs : p.dks) : p.dqs;
      uint16_t* out = (uint16_t*)(KEYS ? (is_dv ? p.dv : p.dk) : p.dq) + b * st.b + (row - lane) * st.t +
                      (KEYS ? hk : h0) * st.h;
      const uint32_t from = tmem + lanes + (is_dv ? kAcc : kAcc2);
      const float f = is_dv ? exp2f(-kLift<BF16>) : p.scale / sigma;
      constexpr int kShare = KEYS ? DP / 2 : DP / 4;
      const int begin = (KEYS ? half : 2 * w + half) * kShare;
      // through shared memory (rows of the owned tile, which no product reads any
      // more), to be written by lines
      constexpr int kPieces = kShare / 8;
      unsigned char* stage = mem + warp * 32 * 128;
      float taints = 0.f;
#pragma unroll
      for (int y = 0; y < kShare; y += 16) {
        uint32_t o[16];
        if (n > 0) tmem_ld16(from + begin + y, o);
        wait_ld();
        tie16(o);
        uint32_t v[8];
        if (n > 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) taints = taint(taints, __uint_as_float(o[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = n > 0 ? pack2<BF16>(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f) : 0u;
        stage_piece(stage, lane, y / 8, make_uint4(v[0], v[1], v[2], v[3]));
        stage_piece(stage, lane, y / 8 + 1, make_uint4(v[4], v[5], v[6], v[7]));
      }
      __syncwarp();
      if (lane_row < owned && taints != 0.f) tainted = 1;  // NaN
      write_rows<kPieces>(stage, 0, out + begin, st.t, owned - quarter * 32, min(kPieces, (p.dim - begin) / 8));
      fence_before();
    }
  } else {
    if (!SCAN) give_registers<64>();
    const uint32_t lead = elect();
    if (warp == 16 && n > 0) {
      // ---- copies: the owned tile once, then streamed tiles
      if (lead) {
        const uint32_t own = bar(kOwnFull);
        bar_expect(own, 2 * L::kOwn);
        for (int y = 0; y < L::kBoxes; ++y)
          for (int half = 0; half < 2; ++half) {
            const uint32_t to = base + y * L::kOwnBox + half * (kCols * 128);
            const int row = r0 + half * kCols;
            if (KEYS) {
              tma_load(to, &t.km, own, 64 * y, row, hk * t.k_mh, b * t.k_mb);
              tma_load(to + L::kOwn, &t.vm, own, 64 * y, row, hk * t.v_mh, b * t.v_mb);
            } else {
              tma_load(to, &t.qm, own, 64 * y, row, h0 * t.q_mh, b * t.q_mb);
              tma_load(to + L::kOwn, &t.gm, own, 64 * y, row, h0 * t.g_mh, b * t.g_mb);
            }
          }
      }
      int tile = sb, h = h0;
      int s = 0, round = 1;
      for (int it = 0; it < n; ++it) {
        const bool ok = bar_wait(bar(kEmpty + s), round, &dead, t.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lead) {
          const uint32_t full = bar(kFull + s), to = base + L::kRing + s * L::kSlot;
          const int c0 = tile * kCols;
          bar_expect(full, 2 * L::kHalf + (KEYS ? 2 * kCols * 4 : 0));
#pragma unroll
          for (int y = 0; y < L::kBoxes; ++y) {
            if (KEYS) {
              tma_load(to + y * L::kBox, &t.qm, full, 64 * y, c0, h * t.q_mh, b * t.q_mb);
              tma_load(to + L::kHalf + y * L::kBox, &t.gm, full, 64 * y, c0, h * t.g_mh, b * t.g_mb);
            } else {
              tma_load(to + y * L::kBox, &t.km, full, 64 * y, c0, hk * t.k_mh, b * t.k_mb);
              tma_load(to + L::kHalf + y * L::kBox, &t.vm, full, 64 * y, c0, hk * t.v_mh, b * t.v_mb);
            }
          }
          if (KEYS) {
            const long long at = ((long long)b * p.heads + h) * x.q_pad + c0;
            bulk_load(to + L::kStats, x.lse2 + at, kCols * 4, full);
            bulk_load(to + L::kStats + kCols * 4, x.delta + at, kCols * 4, full);
          }
        }
        __syncwarp();
        if (++tile == se) tile = sb, ++h;
        if (++s == x.slots) s = 0, round ^= 1;
      }
      if (SCAN) {  // the last arrival on every slot's barrier, before their memory serves others
        for (int it = max(n - x.slots, 0); it < n; ++it)
          if (!bar_wait(bar(kEmpty + it % x.slots), (it / x.slots) & 1, &dead, t.err)) break;
        __syncwarp();
      }
    } else if (warp == 17 && n > 0) {
      // ---- products
      const uint32_t id_s = instr_desc(kTile, kCols, BF16, false), id_a = instr_desc(kTile, t.dim16, BF16, true);
      const int ksteps = t.dim16 / 16;
      auto wait = [&](int n_bar, uint32_t parity) {
        const bool ok = bar_wait(bar(n_bar), parity, &dead, t.err);
        return __all_sync(0xffffffffu, ok) != 0;
      };
      auto scores = [&](int buffer, int slot) {
        const uint32_t d = tmem + buffer * 128, from = base + L::kRing + slot * L::kSlot;
#pragma unroll
        for (int op = 0; op < 2; ++op)
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            mma_ss(k < ksteps ? lead : 0u, d + op * 64,
                   desc_k(base + op * L::kOwn + (k / 4) * L::kOwnBox + (k % 4) * 32),
                   desc_k(from + op * L::kHalf + (k / 4) * L::kBox + (k % 4) * 32), id_s, k > 0);
        mma_commit(lead, bar(kSFull + buffer));
      };
      // each half's 16-bit weights start where its scores did
      auto p_at = [](int k) { return (uint32_t)((k >> 1) * kColumns + (k & 1) * 8); };
      // slot, round and buffer of the next tile to get scores, and of the one
      // being summed
      int ahead = 0, ahead_slot = 0, ahead_round = 0, fill = 0;
      int slot = 0, buffer = 0, turn = 0;
      bool ok = wait(kOwnFull, 0);
      auto next_scores = [&]() {
        ok = ok && wait(kFull + ahead_slot, ahead_round);
        if (!ok) return;
        scores(fill, ahead_slot);
        ++ahead;
        if (++ahead_slot == x.slots) ahead_slot = 0, ahead_round ^= 1;
        if (++fill == NB) fill = 0;
      };
      for (int i = 0; i < NB && i < n; ++i) next_scores();
      for (int it = 0; ok && it < n; ++it) {
        ok = wait(kPReady + buffer, turn);
        if (!ok) break;
        fence_after();
        const uint32_t from = base + L::kRing + slot * L::kSlot, p_from = tmem + buffer * 128;
        if (KEYS) {
#pragma unroll
          for (int k = 0; k < kCols / 16; ++k)
            mma_ts(lead, tmem + kAcc, p_from + p_at(k), desc_mn(from + L::kHalf + k * 2048, L::kBox), id_a,
                   it > 0 || k > 0);
        }
#pragma unroll
        for (int k = 0; k < kCols / 16; ++k)
          mma_ts(lead, tmem + kAcc2, p_from + 64 + p_at(k), desc_mn(from + k * 2048, L::kBox), id_a, it > 0 || k > 0);
        mma_commit(lead, bar(kEmpty + slot));
        if (++slot == x.slots) slot = 0;
        if (++buffer == NB) buffer = 0, turn ^= 1;
        // in order of issue: these scores replace P and dS only after the
        // products above have read them
        if (ahead < n) next_scores();
      }
      if (ok) mma_commit(lead, bar(kDone));
    }
  }
  __syncthreads();
  if (!SCAN && t.flags && tid == 0) t.flags[index] = tainted;
  if (grad) {
    if (warp < 16) far_mem[tid] = far_lo, far_mem[512 + tid] = far_hi;
    __syncthreads();
    // this tile's row of partial bias gradients: the two groups, and at the
    // ends of the map what lay beyond them
    float* part = p.part + (((long long)b * t.q_tiles + r0 / kTile) * p.heads + h0) * (2 * D + 1);
    const float unit = BF16 ? 1.f : exp2f(-kLift<BF16>);
    auto both = [&](int i) { return (diag_mem[i] + diag_mem[ndiag + i]) * unit; };
    for (int i = tid + 1; i < 2 * D; i += kThreads) part[i] = both(i + kDiagPad);
    if (warp < 2) {
      float s = 0.f;
      const int lane = tid & 31;
      for (int i = lane; i < 512; i += 32) s += far_mem[warp * 512 + i] * unit;
      for (int i = lane; i <= kDiagPad; i += 32) s += both(warp ? 2 * D + kDiagPad + i : i);
      s = warp_sum(s);
      if (lane == 0) part[warp ? 2 * D : 0] = s;
    }
  }
  if (dead && tid == 0) {
    // copies still in flight land in this block's memory: give them time
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  __syncthreads();
  if (!SCAN && warp == 17) {
    __syncwarp();
    fence_after();
    tmem_free(tmem, 512);
  }
  // what follows in the stream waits for this kernel: one block of it waits
  // for the queries' kernel
  if (KEYS && !SCAN && index == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool well = !dead;
  if (SCAN && well) {  // another block's work may follow
    if (tid == 0) {
      for (int i = 0; i < x.slots; ++i) bar_free(bar(kFull + i)), bar_free(bar(kEmpty + i));
      for (int i = kOwnFull; i < kBarCount; ++i) bar_free(bar(i));
    }
    fence_async();
    __syncthreads();
  }
  return well;
}

template <int DP, bool BF16, int MODE, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) kernel(const __grid_constant__ TcParams t,
                                                      const __grid_constant__ Extra x) {
  block<DP, BF16, MODE, KEYS, false>(t, x, blockIdx, (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x, 0);
}
template <int DP, bool BF16, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) scan_kernel(const __grid_constant__ TcParams t,
                                                           const __grid_constant__ Extra x) {
  scan_blocks(t, [&](const dim3 at, int index, uint32_t tmem) {
    return block<DP, BF16, 2, KEYS, true>(t, x, at, index, tmem);
  });
}

template <int DP, bool BF16, bool KEYS>
fm_status launch(TcParams t, Extra x, int mode, cudaStream_t st) {
  const int rows = KEYS ? t.p.k_len : t.p.q_len;
  const dim3 grid((rows + kTile - 1) / kTile, KEYS ? t.p.kv_heads : t.p.heads, t.p.batch);
  const bool bias = t.p.map != nullptr, grad = !KEYS && t.p.part != nullptr;
  const size_t smem = Smem<DP, KEYS>::bytes(t.p.max_distance, bias, grad);
  x.slots = Smem<DP, KEYS>::slots(t.p.max_distance, bias, grad);
  if (x.slots < 3) return FM_ERR_UNSUPPORTED;
  t.blocks[0] = grid.x, t.blocks[1] = grid.y, t.blocks[2] = grid.z;
  if (mode == kScan) {
    const long long blocks = (long long)grid.x * grid.y * grid.z;
    if (!allow_smem(scan_kernel<DP, BF16, KEYS>, smem)) return FM_ERR_CUDA;
    scan_kernel<DP, BF16, KEYS><<<(unsigned)(blocks < num_sms() ? blocks : num_sms()), kThreads, smem, st>>>(t, x);
    return launch_status();
  }
  auto k = mode == 0 ? kernel<DP, BF16, 0, KEYS> : mode == 1 ? kernel<DP, BF16, 1, KEYS> : kernel<DP, BF16, 2, KEYS>;
  if (!allow_smem(k, smem)) return FM_ERR_CUDA;
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = smem;
  config.stream = st;
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &early;
  config.numAttrs = KEYS ? 1 : 0;  // launched right after the queries' kernel
  return cudaLaunchKernelEx(&config, k, t, (const Extra)x) == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // namespace bwd
}  // namespace fm

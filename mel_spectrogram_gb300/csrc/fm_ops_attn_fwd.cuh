// Attention forward on the fifth-generation tensor cores.
//
// A block owns 256 queries of one head, as two tiles of 128, and streams the
// keys in tiles of 128. Scores S = Q K^T and the output O += P V are tcgen05
// products with accumulators in tensor memory; a thread reads its scores,
// keeps its row's running maximum and its own sum in registers, and writes its
// 16-bit weights P back over them, from where the second product takes them.
// Warps: 0-7 and 8-15 do the softmax of one query tile each, two threads a row
// with 64 columns each; warp 16 copies tiles by TMA into a ring, warp 17 issues
// products. While one tile's softmax runs, the products of the other do.
//
// Bound: a key tile costs 2 x 2 products of 128 x 128 x dim (2048 cycles of the
// tensor unit at dim 128) for 2 x 16384 exponentials, and takes about 3200: a
// tile's own chain (scores, 1500 cycles of softmax, products) is longer than
// its share of the tensor unit, and tensor memory has no room for a third score
// buffer beside two outputs of 128 columns. Measured: 374 us for 8 rows of up
// to 3001 frames, 16 heads of 128, bf16 (447 GFLOP: 1200 TFLOP/s, 0.61 of the
// measured matrix rate). With a bias by distance at head size 64 the shared
// reads of the bias, the exponentials and the products want about 1000 cycles
// of a tile each, and a tile takes 3300.
// What made it faster: products issued by a converged warp (472 to 363 us, see
// mma_ss); two threads a row, for the biased modes, whose code with a row's 128
// columns unrolled did not stay in the instruction cache (199 to 147 us of
// packed training's forward pass); the third score buffer at head size 64 and
// results written by lines (147 to 128).
//
// Rescaling O when the maximum rises is put off until it has risen by 2^8:
// weights then stay below 2^8, the same factor divides out of sum and output,
// and O is touched a few times per row instead of once per tile.
#pragma once

#include "fm_ops_attn_tc.cuh"

namespace fm {
namespace fwd {

using namespace tc;

constexpr int kThreads = 640;  // warps 18 and 19 only complete a group of four
constexpr int kColumns = kTile / 2;  // a thread's share of a tile
constexpr float kRise = 8.f;
// f16 weights are kept 2^7 larger, up to 2^15, so that small ones stay normal
// numbers; the factor divides out with the sum. bf16 has the range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

template <int DP>
struct Smem {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kBox = kTile * 128;        // bytes of one 64-column box
  static constexpr int kOperand = kBoxes * kBox;  // one 128-row tile
  static constexpr int kSlots = DP == 64 ? 6 : 4;
  static constexpr int kRing = 2 * kOperand;
  static constexpr int kBars = kRing + kSlots * kOperand;
  static constexpr int kBias = kBars + 256;
  static size_t bytes(int max_distance, bool bias) {
    return 1024 + kBias + (bias ? sizeof(float) * (2 * (max_distance + kBiasPad) + 1) : 0);
  }
};
enum { kFull = 0, kEmpty = 8, kQFull = 16, kSFull = 17, kPReady = 20, kOFull = 23, kOReady = 25, kScanned = 27, kBarCount = 29 };
// Score buffers of 128 columns. The tiles (key tile j, query tile w) are taken
// in the order i = 2 j + w, buffer i % kBuffers. With three of them the scores
// of a tile's successor are there before its softmax ends; beside two outputs
// of 128 columns only two fit.
template <int DP>
constexpr int kBuffers = DP == 64 ? 3 : 2;

// a barrier of the two warps that share 32 rows, which also tells whether both
// are well: they leave together
__device__ __forceinline__ bool pair_ok(int pair, bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, %2, 64, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)ok), "r"(pair + 1)
      : "memory");
  return r != 0;
}

// One block's work; SCAN: of the second launch (TcParams::flags), whose blocks
// run several of these one after another, on tensor memory that they hold from
// the first to the last (held). False: a wait gave up.
template <int DP, bool BF16, int MODE, bool SCAN>
__device__ __forceinline__ bool block(const TcParams& t, const dim3 at, const int index, const uint32_t held) {
  using L = Smem<DP>;
  extern __shared__ unsigned char raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int dead;
  __shared__ int range[2];
  __shared__ float row_stat[2][2][2][kTile];  // [tile parity][query tile][half][row]
  __shared__ int tainted;                      // a result is not finite
  __shared__ uint32_t bad_rows[SCAN ? L::kSlots : 1][4];  // of the slot's V: rows that are not finite
  const AttnParams& p = t.p;
  const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
  unsigned char* mem = raw + (base - smem_u32(raw));
  float* bias = (float*)(mem + L::kBias);
  auto bar = [&](int n) { return base + L::kBars + 8 * n; };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one per warp

  const int split = at.z % t.splits, b = at.z / t.splits, h = at.y, hk = h / p.group;
  // causal rows late in the sequence see the most keys: they go first
  const int q0 = (p.causal ? t.blocks[0] - 1 - (int)at.x : (int)at.x) * 2 * kTile;
  const RowInfo info = row_info(p, b);
  const int nq = min(2 * kTile, p.q_len - q0);

  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) bar_init(bar(kFull + i), 1), bar_init(bar(kEmpty + i), 1);
    bar_init(bar(kQFull), 1);
    for (int w = 0; w < 3; ++w) bar_init(bar(kSFull + w), 1), bar_init(bar(kPReady + w), 8);
    for (int w = 0; w < 2; ++w) bar_init(bar(kOFull + w), 1), bar_init(bar(kOReady + w), 1), bar_init(bar(kScanned + w), 8);
    fence_bar_init();
    dead = 0;
    tainted = 0;
    range[0] = 0x7fffffff;
    range[1] = 0;
    tma_prefetch(&t.qm);
    tma_prefetch(&t.km);
    tma_prefetch(&t.vm);
  }
  if (!SCAN && warp == 17) tmem_alloc(smem_u32(&tmem_slot), 512);
  if (MODE == 1 || (MODE == 2 && p.map)) fill_bias(t, h, bias, tid, kThreads);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = SCAN ? held : tmem_slot;

  // the key tiles this block visits
  int tb = split * t.split_tiles, te = (key_end(p, info, q0, nq) + kTile - 1) / kTile;
  te = min(te, tb + t.split_tiles);
  if (t.k_ranges) {
    const int4 a = t.q_ranges[b * t.q_tiles + q0 / kTile];
    const int4 c = q0 + kTile < p.q_len ? t.q_ranges[b * t.q_tiles + q0 / kTile + 1] : make_int4(0x7fffffff, -1, 0, 0);
    const int lo = min(a.x, c.x), hi = max(a.y, c.y);
    for (int i = tb + tid; i < te; i += kThreads) {
      const int4 k = t.k_ranges[b * t.k_tiles + i];
      if (k.x <= hi && k.y >= lo) {
        atomicMin(&range[0], i);
        atomicMax(&range[1], i + 1);
      }
    }
    __syncthreads();
    tb = max(tb, range[0]);
    te = min(te, range[1]);
  }
  const int n = max(te - tb, 0);

  constexpr int NB = kBuffers<DP>;
  constexpr uint32_t kO = NB * kTile;  // columns of O0; O1 follows at kO + DP
  // registers: the block starts with 5 groups x 96; the softmax threads take
  // 104 and leave the others 64 (4 x 104 + 64 = 480)
  if (warp < 16) {
    if (!SCAN) take_registers<104>();
    // ---- softmax: a thread has 64 columns of one query row
    const int w = warp >> 3, half = (warp >> 2) & 1, pair = (warp >> 3) * 4 + (warp & 3);
    const int lane_row = (warp & 3) * 32 + (tid & 31);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane 32 * (warp % 4) in bits 16 up
    const uint32_t to = tmem + lanes + kO + w * DP + half * (DP / 2);
    const int i = q0 + w * kTile + lane_row, place = info.start + i;
    const float c = p.scale * kLog2e;
    const bool raw = MODE == 0 || (SCAN && t.raw);
    const float slope2 = MODE == 2 && p.slopes ? p.slopes[h] * kLog2e : 0.f;
    int qd = -2;  // matches no document
    const int32_t* kdocs = p.k_docs ? p.k_docs + (long long)b * p.k_len : nullptr;
    int4 qr = make_int4(0, 0, 1, 0);
    if (kdocs) {
      qr = q0 + w * kTile < p.q_len ? t.q_ranges[b * t.q_tiles + q0 / kTile + w] : make_int4(0x7fffffff, -1, 0, 0);
      if (i < p.q_len) {
        const int d = p.q_docs[(long long)b * p.q_len + i];
        if (d >= 0) qd = d;
      }
    }
    // columns a row sees by length and causality: below this key
    int seen_end = info.len;
    if (p.causal) seen_end = min(seen_end, max(place + 1, info.prefix));
    // the least of the tile's rows: key tiles that end below it need no mask
    int all_end = info.len;
    if (p.causal) all_end = min(all_end, max(info.start + q0 + w * kTile + 1, info.prefix));

    float m = -INFINITY, l = 0.f;  // l: of this thread's columns
    bool ok = true;
    int buffer = w, turn = 0;  // of this tile's scores
    int scan = 0;              // scanned tiles so far, modulo 2
    int first_end = info.len;  // all_end of the first query tile
    int4 other_range = make_int4(0, 0, 1, 0);
    if (SCAN && p.causal) first_end = min(first_end, max(info.start + q0 + 1, info.prefix));
    if (SCAN && kdocs) {
      const int o = q0 / kTile + (w ^ 1);
      other_range = o < t.q_tiles ? t.q_ranges[b * t.q_tiles + o] : make_int4(0x7fffffff, -1, 0, 0);
    }
    for (int j = 0; j < n; ++j) {
      const uint32_t ts = tmem + lanes + buffer * kTile;
      const int k0 = (tb + j) * kTile, mine = k0 + half * kColumns;
      bool masked = k0 + kTile > all_end, clean = k0 + kTile > info.len && info.len < p.k_len, docs = false;
      if (kdocs) {
        const int4 kr = t.k_ranges[b * t.k_tiles + tb + j];
        if (!(qr.z && kr.z && qr.x == kr.x)) docs = masked = true;
        if (!kr.z) clean = true;
      }
      uint64_t seen = ~0ull;  // bit e: column e of this thread's is seen
      if (masked) {
        seen = column_range<kColumns>(0, seen_end - mine);
        if (docs) seen &= same_document<kColumns>(kdocs + mine, p.k_len - mine, qd);
      }
      uint64_t bad_seen = 0;
      if constexpr (SCAN) {
        // V is shared: both query tiles scan it where either has masked pairs
        bool scanned = masked || k0 + kTile > first_end;
        const int v_slot = (2 * j + 1) % L::kSlots;
        ok = true;
        if (kdocs) {
          const int4 kr = t.k_ranges[b * t.k_tiles + tb + j];
          scanned |= !(other_range.z && kr.z && other_range.x == kr.x);
        }
        if (scanned) {
          const int key = k0 + lane_row;
          ok = bar_wait(bar(kFull + v_slot), ((2 * j + 1) / L::kSlots) & 1, &dead, t.err);
          if (ok)
            clean_row<BF16, L::kBoxes>(mem + L::kRing + v_slot * L::kOperand + lane_row * 128, L::kBox, 4 * half,
                                       key >= info.len || (kdocs && kdocs[key] < 0), &bad_rows[v_slot][warp & 3],
                                       1u << (tid & 31));
          fence_async();
          __syncwarp();
          if (tid % 32 == 0) bar_arrive(bar(kScanned + w));
          ok = bar_wait(bar(kScanned + w), scan, &dead, t.err) && ok;
          const volatile uint32_t* rows = bad_rows[v_slot] + 2 * half;
          bad_seen = seen & ((uint64_t)rows[1] << 32 | rows[0]);
          scan ^= 1;
        }
        clean = false;
      }
      ok = bar_wait(bar(kSFull + buffer), turn, &dead, t.err) && (!SCAN || ok);
      fence_after();
      if (clean) {
        // rows of V that nothing may use become zeros: 0 weights times
        // whatever memory holds would not be 0
        const int it = 2 * j + 1;
        ok = bar_wait(bar(kFull + it % L::kSlots), (it / L::kSlots) & 1, &dead, t.err) && ok;
        const int key = k0 + lane_row;
        if (ok && (key >= info.len || (kdocs && kdocs[key] < 0)))
          clear_row<L::kBoxes>(mem + L::kRing + (it % L::kSlots) * L::kOperand + lane_row * 128, L::kBox, 4 * half);
        fence_async();
      }
      ok = __all_sync(0xffffffffu, ok);
      float s[kColumns], unused[1];
      uint32_t* u = (uint32_t*)s;
      tmem_ld32(ts + half * kColumns, u);
      tmem_ld32(ts + half * kColumns + 32, u + 32);
      wait_ld();
      tie32(u);
      tie32(u + 32);
      if (!raw) tile_scores<kColumns, MODE, false, false>(s, unused, p, c, bias, slope2, mine - place);
      if (masked) {
        const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
        for (int e = 0; e < kColumns; ++e) s[e] = ((e < 32 ? lo : hi) >> (e & 31) & 1) ? s[e] : -INFINITY;
      }
      if (SCAN) {
#pragma unroll
        for (int e = 0; e < kColumns; ++e) s[e] = (bad_seen >> e & 1) ? NAN : s[e];
      }
      float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int e = 4; e < kColumns; ++e) top[e & 3] = fmaxf(top[e & 3], s[e]);
      float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      row_stat[j & 1][w][half][lane_row] = mx;
      if (!pair_ok(pair, ok)) {
        ok = false;
        break;
      }
      // both warps have their scores in registers now: P may replace them
      mx = fmaxf(mx, row_stat[j & 1][w][half ^ 1][lane_row]);
      if (raw) mx *= c;  // scale > 0 here
      // each row by its own scores: what its warp's other rows see may be hidden from it
      const bool risen = mx > m + kRise || (m == -INFINITY && mx > m);
      if (__any_sync(0xffffffffu, risen)) {
        const float top_m = risen ? mx : m, f = risen ? ex2(m - mx) : 1.f;
        m = top_m;
        l *= f;
        if (j > 0) {
          // O has to hold all earlier products: two buffers' scores follow them
          // in the tensor unit's order, of three they may not
          if (NB == 3) {
            ok = bar_wait(bar(kOReady + w), (j - 1) & 1, &dead, t.err);
            fence_after();
          }
#pragma unroll 1
          for (int x = 0; x < DP / 2; x += 16) {
            uint32_t o[16];
            tmem_ld16(to + x, o);
            wait_ld();
            tie16(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(to + x, o);
          }
        }
      }
      const float m0 = (m == -INFINITY ? 0.f : m) - kLift<BF16>;
      float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 z = make_float2(s[32 * part + 2 * e], s[32 * part + 2 * e + 1]);
          const float2 a = raw ? fma2(z, both(c), both(-m0)) : add2(z, both(-m0));
          const float2 q = make_float2(ex2(a.x), ex2(a.y));
          sum[e & 1] = add2(sum[e & 1], q);
          // weights go to the product in the inputs' type: the sum keeps 32 bits
          pk[e] = pack2<BF16>(q.x, q.y);
        }
        tmem_st16(ts + 32 * half + 16 * part, pk);
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      wait_st();
      fence_before();
      __syncwarp();
      if (tid % 32 == 0) bar_arrive(bar(kPReady + buffer));
      buffer += 2;
      if (buffer >= NB) buffer -= NB, turn ^= 1;
    }
    // ---- the row's result, half of its columns a thread
    if (n > 0) ok = bar_wait(bar(kOFull + w), 0, &dead, t.err) && ok;
    // the last arrival on every barrier, before their memory serves others
    if (SCAN && NB == 3 && n > 0) ok = bar_wait(bar(kOReady + w), (n - 1) & 1, &dead, t.err) && ok;
    row_stat[n & 1][w][half][lane_row] = l;
    ok = pair_ok(pair, ok);
    if (ok) {
      fence_after();
      l += row_stat[n & 1][w][half ^ 1][lane_row];
      const float f = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse2 = l == 0.f ? -INFINITY : m - kLift<BF16> + log2f(l);
      const long long row = ((long long)b * p.heads + h) * p.q_len + i;
      const long long at = (long long)split * p.batch * p.heads * p.q_len + row;
      const long long place_out = b * p.os.b + i * p.os.t + h * p.os.h;
      const bool store = i < p.q_len;
      if (store && half == 0) {
        if (t.splits > 1) t.part_lse[at] = lse2;
        else if (p.lse) p.lse[row] = lse2 * kLn2;
      }
      // 16-bit results go through shared memory (this warp's rows and columns of
      // the query tile, which no product reads any more) to be written by lines
      constexpr int kPieces = DP / 16;  // of this thread's half row
      unsigned char* stage = mem + w * L::kOperand + (DP == 128 ? half * L::kBox : 0) + (warp & 3) * 32 * 128;
      const int first = DP == 128 ? 0 : half * kPieces, lane = tid & 31;
      const int rows_left = p.q_len - (i - lane), pieces = min(kPieces, p.dim / 8 - half * kPieces);
      float taints = 0.f;
      auto result = [&](int y, float (&v)[16]) {
        uint32_t o[16];
        if (n > 0) tmem_ld16(to + y, o);
        wait_ld();
        tie16(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          v[e] = n > 0 ? __uint_as_float(o[e]) * f : 0.f;
          taints = taint(taints, v[e]);
        }
      };
      if (t.splits > 1) {
#pragma unroll 1
        for (int y = 0; y < DP / 2; y += 16) {
          const int x = half * (DP / 2) + y;
          float v[16];
          result(y, v);
          if (store) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              if (x + e < p.dim)
                *(float4*)(t.part_o + at * p.dim + x + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
      } else {
        uint16_t* to_out = (uint16_t*)p.out + place_out - lane * p.os.t + half * (DP / 2);
        uint16_t* to_rest = (uint16_t*)p.rest + place_out - lane * p.os.t + half * (DP / 2);
#pragma unroll 1
        for (int what = 0; what < (p.rest ? 2 : 1); ++what) {
#pragma unroll 1
          for (int y = 0; y < DP / 2; y += 16) {
            float v[16];
            result(y, v);
            uint32_t r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = pack2<BF16>(v[2 * e], v[2 * e + 1]);
            if (what) {
#pragma unroll
              for (int e = 0; e < 8; ++e) r[e] = rest2<BF16>(v[2 * e], v[2 * e + 1], r[e]);
            }
            stage_piece(stage, lane, first + y / 8, make_uint4(r[0], r[1], r[2], r[3]));
            stage_piece(stage, lane, first + y / 8 + 1, make_uint4(r[4], r[5], r[6], r[7]));
          }
          __syncwarp();
          write_rows<kPieces>(stage, first, what ? to_rest : to_out, p.os.t, rows_left, pieces);
          __syncwarp();
        }
      }
      if (store && taints != 0.f) tainted = 1;  // NaN
      fence_before();
    }
  } else {
    if (!SCAN) give_registers<64>();
    const uint32_t lead = elect();
    if (warp == 16 && n > 0) {
      // ---- copies: q once, then K and V tiles in turn through the ring
      if (lead) {
        bar_expect(bar(kQFull), 2 * L::kOperand);
        for (int w = 0; w < 2; ++w)
          for (int x = 0; x < L::kBoxes; ++x)
            tma_load(base + w * L::kOperand + x * L::kBox, &t.qm, bar(kQFull), 64 * x, q0 + w * kTile, h * t.q_mh,
                     b * t.q_mb);
      }
      for (int it = 0; it < 2 * n; ++it) {
        const int s = it % L::kSlots, round = it / L::kSlots;
        const bool ok = bar_wait(bar(kEmpty + s), (round & 1) ^ 1, &dead, t.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lead) {
          if (SCAN && (it & 1)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) bad_rows[s][e] = 0;
          }
          bar_expect(bar(kFull + s), L::kOperand);
          const int row = (tb + it / 2) * kTile;
          const uint32_t to = base + L::kRing + s * L::kOperand;
#pragma unroll
          for (int x = 0; x < L::kBoxes; ++x) {
            if (it & 1) tma_load(to + x * L::kBox, &t.vm, bar(kFull + s), 64 * x, row, hk * t.v_mh, b * t.v_mb);
            else tma_load(to + x * L::kBox, &t.km, bar(kFull + s), 64 * x, row, hk * t.k_mh, b * t.k_mb);
          }
        }
        __syncwarp();
      }
      if (SCAN) {  // the last arrival on every slot's barrier
        for (int it = max(2 * n - L::kSlots, 0); it < 2 * n; ++it)
          if (!bar_wait(bar(kEmpty + it % L::kSlots), (it / L::kSlots) & 1, &dead, t.err)) break;
        __syncwarp();
      }
    } else if (warp == 17 && n > 0) {
      // ---- products
      const uint32_t id_s = instr_desc(kTile, kTile, BF16, false), id_o = instr_desc(kTile, t.dim16, BF16, true);
      const int ksteps = t.dim16 / 16;
      auto scores = [&](int w, int buffer, int slot) {
        const uint32_t a = base + w * L::kOperand, from = base + L::kRing + slot * L::kOperand;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t at = (k / 4) * L::kBox + (k % 4) * 32;
          mma_ss(k < ksteps ? lead : 0u, tmem + buffer * kTile, desc_k(a + at), desc_k(from + at), id_s, k > 0);
        }
        mma_commit(lead, bar(kSFull + buffer));
      };
      auto wait = [&](int n_bar, uint32_t parity) {
        const bool ok = bar_wait(bar(n_bar), parity, &dead, t.err);
        return __all_sync(0xffffffffu, ok) != 0;
      };
      // slot and round of the ring's next K and next V
      int sk = 0, rk = 0, sv = 1, rv = 0;
      auto advance = [&](int& s, int& r) {
        s += 2;
        if (s >= L::kSlots) s -= L::kSlots, r ^= 1;
      };
      bool ok = wait(kQFull, 0);
      int ahead = 0, fill = 0;  // the next tile to get scores, and its buffer
      auto next_scores = [&]() {
        const int w = ahead & 1;
        if (w == 0) ok = ok && wait(kFull + sk, rk);
        if (!ok) return;
        scores(w, fill, sk);
        if (w) {
          mma_commit(lead, bar(kEmpty + sk));
          advance(sk, rk);
        }
        ++ahead;
        if (++fill == NB) fill = 0;
      };
      for (int i = 0; i < NB && i < 2 * n; ++i) next_scores();
      int buffer = 0, turn = 0;
      for (int i = 0; ok && i < 2 * n; ++i) {
        const int w = i & 1;
        ok = (w || wait(kFull + sv, rv)) && wait(kPReady + buffer, turn);
        if (!ok) break;
        fence_after();
        const uint32_t from = base + L::kRing + sv * L::kOperand;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(lead, tmem + kO + w * DP, tmem + buffer * kTile + k * 8, desc_mn(from + k * 2048, L::kBox), id_o,
                 i > 1 || k > 0);
        if (w) {
          mma_commit(lead, bar(kEmpty + sv));
          advance(sv, rv);
        }
        if (NB == 3) mma_commit(lead, bar(kOReady + w));
        if (i + 2 >= 2 * n) mma_commit(lead, bar(kOFull + w));
        if (++buffer == NB) buffer = 0, turn ^= 1;
        // the tensor unit runs products in the order of issue: scores replace P
        // only after the product above has read it
        if (ahead < 2 * n) next_scores();
      }
    }
  }
  __syncthreads();
  if (!SCAN && t.flags && tid == 0) t.flags[index] = tainted;
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
  const bool well = !dead;
  if (SCAN && well) {  // another block's work may follow
    if (tid == 0) {
      for (int i = 0; i < L::kSlots; ++i) bar_free(bar(kFull + i)), bar_free(bar(kEmpty + i));
      for (int i = kQFull; i < kBarCount; ++i) bar_free(bar(i));
    }
    fence_async();
    __syncthreads();
  }
  return well;
}

template <int DP, bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1) kernel(const __grid_constant__ TcParams t) {
  block<DP, BF16, MODE, false>(t, blockIdx, (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x, 0);
}
template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) scan_kernel(const __grid_constant__ TcParams t) {
  scan_blocks(t, [&](const dim3 at, int index, uint32_t tmem) {
    return block<DP, BF16, 2, true>(t, at, index, tmem);
  });
}

template <int DP, bool BF16>
fm_status launch(TcParams t, int mode, cudaStream_t st) {
  const dim3 grid((t.p.q_len + 2 * kTile - 1) / (2 * kTile), t.p.heads, t.p.batch * t.splits);
  t.blocks[0] = grid.x, t.blocks[1] = grid.y, t.blocks[2] = grid.z;
  const size_t smem = Smem<DP>::bytes(t.p.max_distance, t.p.map != nullptr);
  auto k = mode == 0 ? kernel<DP, BF16, 0> : mode == 1 ? kernel<DP, BF16, 1> : kernel<DP, BF16, 2>;
  if (!allow_smem(k, smem)) return FM_ERR_CUDA;
  k<<<grid, kThreads, smem, st>>>(t);
  if (t.flags) {
    const long long blocks = (long long)grid.x * grid.y * grid.z;
    if (!allow_smem(scan_kernel<DP, BF16>, smem)) return FM_ERR_CUDA;
    scan_kernel<DP, BF16><<<(unsigned)(blocks < num_sms() ? blocks : num_sms()), kThreads, smem, st>>>(t);
  }
  return launch_status();
}

}  // namespace fwd
}  // namespace fm

// Attention of a few queries against a long cache of keys: one new token, or
// a handful, per stream.
//
// Bound by reading K and V once. The queries of all heads that share a key
// head make the rows of one 16-row operand (row = query * group + head), so
// that the cache crosses HBM once whatever the grouping; products run on
// mma.sync (16 rows would leave 7/8 of a tcgen05 tile empty). The key axis is
// split over blocks, and within a block over its warps, each with a ring of two
// tiles of 16 keys of its own that one lane fills by TMA: no barrier between
// warps in the loop, and the copies cost no instructions of the other lanes
// (with cp.async they took a third of 633 instructions a tile, which is what
// bound the kernel, at 38 % of the bandwidth). Warps join through shared
// memory, blocks through the join kernel. Measured, with the join: 293 MB of 64
// caches of up to 3001 frames in 63 us (0.70 of the measured bandwidth), 184 MB
// of an hour's 360001 frames in 43 (0.64), in 297 splits. What is left is the
// chain from a tile's arrival over its two products to the next: twelve warps an
// SM, as many as the registers hold, issue in 0.32 of the cycles.
#include "fm_ops_attn_tc.cuh"

namespace fm {
namespace {

using namespace tc;

constexpr int kWarps = 4, kKeys = 16, kStages = 2;

// a multiple of 1024 bytes, as TMA's swizzle wants
template <int DP>
constexpr int stage_bytes() { return 2 * kKeys * DP * 2; }
template <int DP>
constexpr size_t smem_bytes() {
  const size_t ring = (size_t)kWarps * kStages * stage_bytes<DP>() + 1024;  // and its alignment
  const size_t out = (size_t)kWarps * 16 * (DP + 2) * sizeof(float);  // warps' results, over the ring
  return ring > out ? ring : out;
}

__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

struct StepParams {
  AttnParams p;
  CUtensorMap km, vm;  // {dim, token, head, batch}, boxes of 64 x 16
  int k_mh, k_mb, v_mh, v_mb;
  ErrorWords err;
  int splits, split_keys;  // keys of one split, a multiple of kWarps * kKeys
  int row_tiles;
  float *part_o, *part_lse;
};

template <int DP, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) step(const __grid_constant__ StepParams t) {
  extern __shared__ unsigned char raw[];
  __shared__ float stat[2][kWarps][16];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ volatile int dead;
  unsigned char* mem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const AttnParams& p = t.p;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kBoxes = DP / 64, kBox = kKeys * 128, kOperand = kBoxes * kBox;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) bar_init(smem_u32(&full[warp][s]), 1);
    fence_bar_init();
    if (warp == 0) dead = 0;
  }
  __syncthreads();
  const int split = blockIdx.x / t.row_tiles, rt = blockIdx.x % t.row_tiles;
  const int hk = blockIdx.y, b = blockIdx.z;
  const RowInfo info = row_info(p, b);
  const int rows = p.q_len * p.group;
  const int quad = lane >> 2, pair = 2 * (lane & 3);
  const int k_begin = split * t.split_keys;
  int k_end = min(info.len, k_begin + t.split_keys);
  if (p.causal) k_end = min(k_end, max(info.start + p.q_len, info.prefix));

  // this thread's two rows
  int qi[2], qh[2], qd[2];
  bool row_ok[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = rt * 16 + quad + 8 * r;
    row_ok[r] = row < rows;
    qi[r] = row_ok[r] ? row / p.group : 0;
    qh[r] = hk * p.group + (row_ok[r] ? row % p.group : 0);
    qd[r] = -2;
    if (p.q_docs) {
      const int d = p.q_docs[(long long)b * p.q_len + qi[r]];
      if (d >= 0) qd[r] = d;
    }
  }
  constexpr int kSteps = DP / 16;
  uint32_t q[kSteps][4];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = e & 1, d = 16 * s + pair + 8 * (e >> 1);
      q[s][e] = row_ok[r] && d < p.dim
                    ? *(const uint32_t*)((const uint16_t*)p.q + b * p.qs.b + qi[r] * p.qs.t + qh[r] * p.qs.h + d)
                    : 0u;
    }
  float slope[2] = {0.f, 0.f}, below[2] = {0.f, 0.f}, above[2] = {0.f, 0.f};
  const int D = p.max_distance;
  const float c = p.scale * kLog2e;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (p.slopes) slope[r] = p.slopes[qh[r]] * kLog2e;
    if (p.map) {
      below[r] = kLog2e * table_value(p, (long long)p.map[0] * p.heads + qh[r], BF16);
      above[r] = kLog2e * table_value(p, (long long)p.map[2 * D] * p.heads + qh[r], BF16);
    }
  }
  const int32_t* kdocs = p.k_docs ? p.k_docs + (long long)b * p.k_len : nullptr;

  // ---- the warp's ring: tile n of the split's tiles warp, warp + 4, ...
  const uint32_t ring = smem_u32(mem) + warp * kStages * stage_bytes<DP>();
  const int tiles = k_end > k_begin ? (k_end - k_begin + kKeys - 1) / kKeys : 0;
  const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
  auto load = [&](int n) {
    if (lane == 0 && n < mine) {
      const int k0 = k_begin + (warp + n * kWarps) * kKeys;
      const uint32_t to = ring + (n % kStages) * stage_bytes<DP>(), bar = smem_u32(&full[warp][n % kStages]);
      bar_expect(bar, 2 * kOperand);
#pragma unroll
      for (int x = 0; x < kBoxes; ++x) {
        tma_load(to + x * kBox, &t.km, bar, 64 * x, k0, hk * t.k_mh, b * t.k_mb);
        tma_load(to + kOperand + x * kBox, &t.vm, bar, 64 * x, k0, hk * t.v_mh, b * t.v_mb);
      }
    }
  };
  float o[DP / 8][4];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  bool ok = true;
  const float cap_in = p.cap > 0.f ? p.scale / p.cap : 0.f, cap_out = p.cap * kLog2e;
  // this lane's places in a tile: rows of 128 bytes with TMA's swizzle, whose
  // pieces 2 st + x stand at (x ^ row % 8) ^ 2 st (64 columns further: next box)
  const int k_row = (lane & 7) + ((lane & 16) >> 1), v_row = lane & 15;
  const uint32_t k_place = k_row * 128 + ((((lane >> 3) & 1) ^ (k_row & 7)) << 4);
  const uint32_t v_place = v_row * 128 + (((lane >> 4) ^ (v_row & 7)) << 4);
  for (int n = 0; n < kStages; ++n) load(n);
  for (int n = 0; n < mine; ++n) {
    ok = bar_wait(smem_u32(&full[warp][n % kStages]), (n / kStages) & 1, &dead, t.err);
    if (!__all_sync(0xffffffffu, ok)) break;
    const int k0 = k_begin + (warp + n * kWarps) * kKeys;
    const uint32_t K = ring + (n % kStages) * stage_bytes<DP>(), V = K + kOperand;
    // columns beyond dim are zeros in q and, by the copies' fill, in K and V. Two
    // sums of every other step: half the chain of dependent products
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    float s_odd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      // four 8 x 8 pieces: keys 0-7 and 8-15, dims 16 st and 16 st + 8
      uint32_t kf[4];
      ldsm4(K + (st / 4) * kBox + (k_place ^ ((st % 4) << 5)), kf);
      mma16<BF16>(st & 1 ? s_odd[0] : s[0], q[st], kf[0], kf[1]);
      mma16<BF16>(st & 1 ? s_odd[1] : s[1], q[st], kf[2], kf[3]);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[x][e] += s_odd[x][e];
    bool masked = k0 + kKeys > k_end || kdocs;
    if (p.causal) masked = masked || k0 + kKeys > max(info.start + 1, info.prefix);
    uint32_t bad = 0;  // two bits a key: halves of its row of V that are not finite
    if (__builtin_expect(masked, 0)) {
      // rows of V that nothing may use, or that are not finite, become zeros: a
      // weight of 0 times what memory holds would not be 0
      const int row = lane >> 1, key = k0 + row;
      const bool no_use = key >= info.len || (kdocs && kdocs[key] < 0);
      bad = __ballot_sync(0xffffffffu, clean_row<BF16, kBoxes>(mem + (V - smem_u32(mem)) + row * 128, kBox,
                                                              4 * (lane & 1), no_use));
      fence_async();  // before the copy that fills this stage next
      __syncwarp();
    }
    // element e of s[x]: row quad + 8 (e / 2), key k0 + 8 x + pair + e % 2
    const bool far = !p.map || (k0 - info.start - p.q_len + 1 >= D) || (k0 + kKeys - 1 - info.start <= -D);
    // each choice outside its loop over the elements, so that they overlap
    auto each = [&](auto f) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1, key = k0 + 8 * x + pair + (e & 1);
          f(s[x][e], r, key, key - info.start - qi[r]);
        }
    };
    if (p.cap > 0.f) {
      // each score takes the form of tanh that its own size asks for
      float most = 0.f;
      each([&](float& z, int, int, int) { most = fmaxf(most, fabsf(z)); });
      const bool large = __any_sync(0xffffffffu, most * fabsf(cap_in) > kTanhSmall);
      each([&](float& z, int, int, int) {
        const float x = z * cap_in, q = x * x;
        const float t = fmaf(fmaf(fmaf(tanh_over_x(3), q, tanh_over_x(2)), q, tanh_over_x(1)), q, tanh_over_x(0)) * (z * c);
        z = large && fabsf(x) > kTanhSmall ? cap_out * tanh_from(x * (2.f * kLog2e)) : t;
      });
    } else {
      each([&](float& z, int, int, int) { z *= c; });
    }
    if (p.map && far) {
      const bool is_above = k0 > info.start;
      const float add[2] = {is_above ? above[0] : below[0], is_above ? above[1] : below[1]};
      each([&](float& z, int r, int, int) { z += add[r]; });
    } else if (p.map) {
      each([&](float& z, int r, int, int off) {
        const int at = __ldg(p.map + min(max(off, -D), D) + D);
        z += kLog2e * table_value(p, (long long)at * p.heads + qh[r], BF16);
      });
    }
    if (p.slopes) each([&](float& z, int r, int, int off) { z = fmaf(-slope[r], fabsf((float)off), z); });
    if (masked)
      each([&](float& z, int r, int key, int off) {
        bool seen = key < k_end && !(p.causal && off > 0 && key >= info.prefix);
        if (kdocs && seen) seen = __ldg(kdocs + key) == qd[r];
        z = seen ? z : -INFINITY;
      });
    if (bad != 0) {  // a query that sees such a row (its score is not -inf) returns NaN
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (s[x][e] != -INFINITY && (bad >> (2 * (8 * x + pair + (e & 1))) & 3)) s[x][e] = NAN;
    }
    // the running maximum follows only rises by 2^8, as in the tiled kernel, of
    // the row itself
    float top[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
    }
    auto risen = [&](int r) { return top[r] > m[r] + 8.f || (m[r] == -INFINITY && top[r] > m[r]); };
    if (__any_sync(0xffffffffu, risen(0) || risen(1))) {
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        f[r] = risen(r) ? ex2(m[r] - top[r]) : 1.f;
        m[r] = risen(r) ? top[r] : m[r];
        l[r] *= f[r];
      }
#pragma unroll
      for (int x = 0; x < DP / 8; ++x) {
        o[x][0] *= f[0];
        o[x][1] *= f[0];
        o[x][2] *= f[1];
        o[x][3] *= f[1];
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // f16 weights are kept 2^7 larger, so that small ones stay normal numbers
      const float zero = (m[r] == -INFINITY ? 0.f : m[r]) - kLift<BF16>;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[x][2 * r + e] = ex2(s[x][2 * r + e] - zero);
          l[r] += s[x][2 * r + e];  // this thread's columns; joined at the end
        }
    }
    // weights go to the product in the cache's type
    uint32_t pf[4] = {pack2<BF16>(s[0][0], s[0][1]), pack2<BF16>(s[0][2], s[0][3]), pack2<BF16>(s[1][0], s[1][1]),
                      pack2<BF16>(s[1][2], s[1][3])};
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      uint32_t vf[4];
      ldsm4_t(V + (st / 4) * kBox + (v_place ^ ((st % 4) << 5)), vf);
      mma16<BF16>(o[2 * st], pf, vf[0], vf[1]);
      mma16<BF16>(o[2 * st + 1], pf, vf[2], vf[3]);
    }
    __syncwarp();
    load(n + kStages);
  }
  if (!ok && lane == 0) {
    // copies still in flight land in this block's memory: give them time
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  // ---- the warps' results
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if ((lane & 3) == 0) stat[0][warp][quad + 8 * r] = m[r], stat[1][warp][quad + 8 * r] = l[r];
  }
  __syncthreads();
  float* all = (float*)mem;  // [warps][16][DP + 2]
#pragma unroll
  for (int x = 0; x < DP / 8; ++x)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *(float2*)(all + (warp * 16 + quad + 8 * r) * (DP + 2) + 8 * x + pair) = make_float2(o[x][2 * r], o[x][2 * r + 1]);
  __syncthreads();
  const int valid = min(16, rows - rt * 16);
  const int per_row = p.dim / 8;
  for (int e = tid; e < valid * per_row; e += kWarps * 32) {
    const int row = e / per_row, d = (e - row * per_row) * 8;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[0][w][row]);
    const float zero = top == -INFINITY ? 0.f : top;
    float total = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float g = ex2(stat[0][w][row] - zero);
      total = fmaf(stat[1][w][row], g, total);
      const float* from = all + (w * 16 + row) * (DP + 2) + d;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(from[k], g, acc[k]);
    }
    const float f = total == 0.f ? 0.f : 1.f / total;
    const int at_row = rt * 16 + row, i = at_row / p.group, h = hk * p.group + at_row % p.group;
    const long long stat_row = ((long long)b * p.heads + h) * p.q_len + i;
    const float lse = total == 0.f ? -INFINITY : top - kLift<BF16> + log2f(total);
    if (t.splits > 1) {
      const long long at = (long long)split * p.batch * p.heads * p.q_len + stat_row;
      if (d == 0) t.part_lse[at] = lse;
      float4* to = (float4*)(t.part_o + at * p.dim + d);
      to[0] = make_float4(acc[0] * f, acc[1] * f, acc[2] * f, acc[3] * f);
      to[1] = make_float4(acc[4] * f, acc[5] * f, acc[6] * f, acc[7] * f);
    } else {
      if (d == 0 && p.lse) p.lse[stat_row] = lse * kLn2;
      const long long at = b * p.os.b + i * p.os.t + h * p.os.h + d;
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = pack2<BF16>(acc[2 * k] * f, acc[2 * k + 1] * f);
      *(uint4*)((uint16_t*)p.out + at) = make_uint4(r[0], r[1], r[2], r[3]);
      if (p.rest) {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = rest2<BF16>(acc[2 * k] * f, acc[2 * k + 1] * f, r[k]);
        *(uint4*)((uint16_t*)p.rest + at) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
  }
}

template <int DP, bool BF16>
fm_status launch(const StepParams& t, cudaStream_t st) {
  const dim3 grid(t.splits * t.row_tiles, t.p.kv_heads, t.p.batch);
  if (!allow_smem(step<DP, BF16>, smem_bytes<DP>())) return FM_ERR_CUDA;
  step<DP, BF16><<<grid, kWarps * 32, smem_bytes<DP>(), st>>>(t);
  return launch_status();
}
}  // namespace

StepPlan step_plan(const AttnParams& p) {
  StepPlan w{};
  w.row_tiles = (p.q_len * p.group + 15) / 16;
  // Splits of at least 256 keys, as many as fill the SMs' blocks (three with
  // head size 128, four with 64: their registers) in whole waves.
  const long long slots = (long long)num_sms() * (p.dim <= 64 ? 4 : 3);
  const long long blocks = (long long)p.batch * p.kv_heads * w.row_tiles;
  const long long most = p.k_len / 256 > 1 ? p.k_len / 256 : 1;
  long long best = 1;
  double best_use = 0;
  for (long long waves = 1; waves <= 4; ++waves) {
    long long s = waves * slots / blocks;
    if (s < 1) continue;
    if (s > most) s = most;
    const long long n = s * blocks;
    const double use = (double)n / (double)((n + slots - 1) / slots * slots);
    if (use > best_use + 0.02) best = s, best_use = use;
  }
  const int unit = kWarps * kKeys;
  w.split_keys = (int)(((p.k_len + best - 1) / best + unit - 1) / unit * unit);
  if (w.split_keys < unit) w.split_keys = unit;
  w.splits = (p.k_len + w.split_keys - 1) / w.split_keys;
  if (w.splits < 1) w.splits = 1;
  return w;
}

fm_status attn_step(const AttnParams& p, int64_t dtype, const StepPlan& w, float* part_o, float* part_lse,
                    cudaStream_t st) {
  StepParams t{};
  const bool bf16 = dtype == FM_BF16;
  t.p = p;
  t.splits = w.splits;
  t.split_keys = w.split_keys;
  t.row_tiles = w.row_tiles;
  t.part_o = part_o;
  t.part_lse = part_lse;
  if (!ops_error_words(&t.err) ||
      !tc_encode(&t.km, p.k, p.ks, p.batch, p.k_len, p.kv_heads, p.dim, kKeys, bf16, &t.k_mh, &t.k_mb) ||
      !tc_encode(&t.vm, p.v, p.vs, p.batch, p.k_len, p.kv_heads, p.dim, kKeys, bf16, &t.v_mh, &t.v_mb))
    return FM_ERR_CUDA;
  return p.dim <= 64 ? (bf16 ? launch<64, true>(t, st) : launch<64, false>(t, st))
                     : (bf16 ? launch<128, true>(t, st) : launch<128, false>(t, st));
}
}  // namespace fm

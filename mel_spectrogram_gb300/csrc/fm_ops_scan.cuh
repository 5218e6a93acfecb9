// Gated linear recurrence over frames, forward and backward (fm_ops.h).
//
// One step h -> f h + b per frame and channel; steps compose as
//   (f2, b2) after (f1, b1) = (f2 f1, f2 b1 + b2),
// so that stretches of frames are walked side by side and joined afterwards. A stretch
// in which a frame starts from 0 has f = -0: its sign marks that what comes out does
// not depend on what went in, be that infinite or NaN (a product with 0 would let it
// pass).
//
// A thread walks STEPS frames of a pair of channels, LS threads side by side the
// channels of a segment, 32 / LS segments a warp; a block's four warps have a tile of
// 4 * 32 / LS * STEPS frames of 2 * LS channels, and the blocks of a cluster consecutive
// tiles of one row's time. Segments of a warp are joined by shuffles, warps through
// shared memory, blocks by asynchronous stores to one another's (distributed) shared
// memory, which count towards a barrier there (a cluster-wide barrier would wait for
// everything stored so far, the results in global memory included); each block works
// out for itself where it starts. The cluster then goes on to the next tiles until the
// row ends. Nothing is read twice, no block waits for one that is not running (a
// cluster's blocks run together), and the order of every join is fixed.
//
// Memory bound (3 items an element forward: x, gate, y; 5 backward: x, gate, dy, dx,
// dgate), but not by much: at the memory's rate an SM has 33 instructions an element.
// So channels are worked on in pairs; the segments are long (16 frames; with 8 channels
// and 4 frames a thread the joins took ten instructions an element); tiles come to
// shared memory ahead, without going through registers; and a warp whose frames are all
// used takes a path that asks nothing.
//
// Few channels in few long rows make too few clusters. Then a row is cut into stretches that
// clusters of their own take, after a first kernel has worked out what each stretch does
// to the state, which reads two of the arrays once more. 360001 frames of 80 32-bit
// channels: 52 us for the sums and 55 for the rest, 121 uncut; of 8 16-bit channels 13
// and 13 (backward 12 and 19), 114 (234) uncut.
//
// Backward: dh goes against the order of the walk with the same factors; the states
// are worked out again from those that the forward left every kMark frames.
//
// Rows that are not on 16-byte boundaries are copied word by word, 16-bit channels that
// start in the middle of a word with the word around them, and put right when they are
// read. 360001 x 511 in bf16: forward 557 us, backward 1050 (512 channels: 285 and 585);
// through registers, element by element, 1614 and 4776.
//
// Measured: 8 rows of 3001 x 1024 in bf16 forward 31 us (4.8 TB/s), backward 60 (4.1),
// with documents 35 and 63; 32 rows of 11250 x 512 forward 203 (5.4). One row of 360001 x
// 512 282 us (3.9): its blocks are few, and each waits for the others in every round.
// Blocks of eight warps, two an SM: 33, 64 and 310 us.
#pragma once

#include <cooperative_groups.h>

#include <atomic>

#include "fm_ops.cuh"
#include "fm_tc.cuh"

namespace fm {
namespace scan {
namespace cg = cooperative_groups;
using tc::add2;
using tc::fma2;
using tc::mul2;

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kMark = 16;   // frames between the states that the forward leaves
constexpr int kShort = 4;   // frames up to which a thread walks its channels alone
// frames of a segment: what a thread's registers hold
template <bool BACKWARD>
constexpr int kSteps = BACKWARD ? 8 : 16;
// Blocks of a cluster (over 8: where the device allows it). One row of 360001 x 512 in
// bf16 backward: 562 us with up to 16, 715 with up to 8.
constexpr int kMaxCluster = 16;

struct ScanParams {
  long long batch, frames;
  int channels, blocks;  // blocks of channels
  int reverse;
  long long x_s[2], g_s[2], y_s[2], dy_s[2], dx_s[2], dg_s[2];
  const void *x, *g, *dy;
  void *y, *dx, *dg;
  const float *state, *dend;
  float *end, *marks, *dstate;
  tc::ErrorWords err;
  const int32_t *lens, *docs;
  // Stretches of `length` frames that clusters of their own take, each starting from what
  // the stretches before it do: [stretches + 1][batch][channels] (A, B), where the row
  // starts and then one a stretch.
  float2* sums;
  int stretches, length;
};

// a = 1 / (1 + e^-g) and 1 - a of two channels. One step of Newton's method takes the
// approximate reciprocal's error: an error of one sign in a would add up over as many
// frames as the recurrence remembers. Below -80 a stays at 2e-35.
__device__ __forceinline__ void gates_of(float2 g, float2& a, float2& rest) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(g.x) : "f"(-80.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(g.y) : "f"(-80.f));
  g = mul2(g, tc::both(-kLog2e));
  const float2 e = make_float2(tc::ex2(g.x), tc::ex2(g.y));
  const float2 d = fma2(e, tc::both(-1.f), tc::both(-1.f));  // -(1 + e)
  a = make_float2(tc::rcp(-d.x), tc::rcp(-d.y));
  a = fma2(a, fma2(d, a, tc::both(1.f)), a);
  rest = mul2(e, a);
}

// The frames of a row in the order of the walk: frame n of the walk is frame n or, in
// reverse, frames - 1 - n; first .. last - 1 are those within the row's length.
struct Row {
  const int32_t* docs;
  int frames, first, last;
  bool reverse;
  __device__ Row(const ScanParams& p, long long b) : docs(p.docs ? p.docs + b * p.frames : nullptr), frames((int)p.frames) {
    const int used = p.lens ? min(max(p.lens[b], 0), frames) : frames;
    reverse = p.reverse;
    first = reverse ? frames - used : 0;
    last = reverse ? frames : used;
  }
  __device__ int place(int n) const { return reverse ? frames - 1 - n : n; }
  __device__ int id(int n) const { return n >= 0 && n < frames ? docs[place(n)] : 0; }
  // The document ids of a warp's frames from n on, and of those before each: a lane has
  // one frame of every 32.
  template <int N>
  struct Ids {
    int now[N], before[N];
  };
  template <int N>
  __device__ void fetch(int n, int lane, Ids<N>& ids) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = n + 32 * i + lane;
      ids.now[i] = id(f);
      ids.before[i] = id(f - 1);
    }
  }
  // Bits for the frames n0 .. n0 + STEPS - 1 of each lane's segment: used; starts from 0.
  // n: the warp's first frame, to which the ids belong.
  template <int LS, int STEPS, bool CUTS, int N>
  __device__ void look(int n, int lane, const Ids<N>& ids, unsigned& used, unsigned& fresh) const {
    constexpr unsigned kAll = (1u << STEPS) - 1;
    const int n0 = n + lane / LS * STEPS;
    if (!CUTS) {
      const int lo = max(first - n0, 0), hi = min(max(last - n0, 0), STEPS);
      used = lo < STEPS ? (kAll << lo) & ((1u << hi) - 1) : 0;
      fresh = 0;
      return;
    }
    used = fresh = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int f = n + 32 * i + lane;
      const bool u = f >= first && f < last && ids.now[i] >= 0;
      const unsigned us = __ballot_sync(0xffffffffu, u);
      const unsigned fs = __ballot_sync(0xffffffffu, u && f > 0 && ids.before[i] != ids.now[i]);
      const int mine = lane / LS * STEPS - 32 * i;  // where this lane's segment begins among these 32
      if (mine >= 0 && mine < 32) used = us >> mine & kAll, fresh = fs >> mine & kAll;
    }
  }
};

template <typename T>
__device__ __forceinline__ float2 both_of(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*(const __half2*)&w);
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// How a pair lies in the words that hold it, for the even and the odd frames of a segment
// (its first frame is an even one): 16-bit channels may start in the middle of a word.
struct Shift {
  uint32_t order[2];
  template <typename T>
  __device__ Shift(const T* frame0, long long stride) {
    const uint32_t at = (uint32_t)(uintptr_t)frame0;
    order[0] = at & 2 ? 0x5432 : 0x3210;
    order[1] = (at + (uint32_t)stride * 2) & 2 ? 0x5432 : 0x3210;
  }
};
// the pair of frame i of a segment in shared memory
template <typename T, typename S>
__device__ __forceinline__ float2 pair_of(const unsigned char* p, int i, const Shift& shift) {
  p += i * S::kRowBytes;
  if constexpr (sizeof(T) == 4) return *(const float2*)p;
  else if constexpr (S::kShifted) return both_of<T>(__byte_perm(*(const uint32_t*)p, ((const uint32_t*)p)[1], shift.order[i & 1]));
  else return both_of<T>(*(const uint32_t*)p);
}
// ALIGNED: pairs on their own boundary; otherwise where they are, `n` of two channels
template <typename T, bool ALIGNED>
__device__ __forceinline__ void leave(T* to, float2 v, int n) {
  if constexpr (sizeof(T) == 4) {
    if (ALIGNED) {
      *(float2*)to = v;
    } else {
      to[0] = v.x;
      if (n > 1) to[1] = v.y;
    }
  } else {
    const uint32_t w = tc::pack2<std::is_same<T, __nv_bfloat16>::value>(v.x, v.y);
    if (ALIGNED || (n > 1 && ((uintptr_t)to & 2) == 0)) {
      *(uint32_t*)to = w;
    } else {
      *(uint16_t*)to = (uint16_t)w;
      if (n > 1) ((uint16_t*)to)[1] = (uint16_t)(w >> 16);
    }
  }
}
// A piece of one frame, to shared memory: 16 bytes, or a word of which `bytes` are read and
// the others become 0.
template <bool ALIGNED>
__device__ __forceinline__ void fetch(unsigned char* to, const void* from, int bytes) {
  if constexpr (ALIGNED)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(to)), "l"(from), "r"(bytes) : "memory");
}
// The pieces that a thread copies: its piece of frame `at` of a tile and of those
// kFramesAtOnce further, an even number, so that all lie alike in their words.
template <typename T, typename S>
struct Source {
  const T* p;
  int bytes;  // of the piece that are the row's; none: there is nothing to copy
  // frame: the first of the block's `n` channels in this thread's first frame
  __device__ Source(const T* frame, int piece, int n) {
    constexpr int kPer = S::kPiece / (int)sizeof(T);
    const int before = S::kShifted && ((uintptr_t)frame & 2) ? 1 : 0;  // elements ahead of them in the first word
    p = frame - before + piece * kPer;
    bytes = min(max((n + before - piece * kPer) * (int)sizeof(T), 0), S::kPiece);
  }
};
// The last channel of a block's, where it lies in a word after those that Source copies.
// x: the row's first frame's first of the block's channels.
template <typename T, typename S>
__device__ __forceinline__ void fetch_last(unsigned char* tile, const T* x, long long stride, int n, int begin,
                                           int stop, int first_place, int turn) {
  if constexpr (S::kShifted) {
#pragma unroll
    for (int f = threadIdx.x; f < S::kTile; f += kThreads) {
      const T* last = x + (first_place + (long long)turn * (n + f)) * stride + S::CB - 1;
      if (n + f >= begin && n + f < stop && ((uintptr_t)last & 2) == 0)
        fetch<false>(&tile[f / S::kSteps * S::kSegBytes + f % S::kSteps * S::kRowBytes + S::CB * (int)sizeof(T)], last, 2);
    }
  }
}
__device__ __forceinline__ void fetches_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest N groups of this thread's copies are there
template <int N>
__device__ __forceinline__ void fetches_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// CUTS: whether there are frames that start from 0 at all (documents).
template <bool CUTS>
__device__ __forceinline__ bool cut(float A) {
  return CUTS && (int)__float_as_uint(A) < 0;
}
// h after the stretch (A, B), from h before it
template <bool CUTS>
__device__ __forceinline__ float2 after(float2 A, float2 h, float2 B) {
  const float2 r = fma2(A, h, B);
  return CUTS ? make_float2(cut<CUTS>(A.x) ? B.x : r.x, cut<CUTS>(A.y) ? B.y : r.y) : r;
}
// the product of two factors: a cut in either stays one, also beside a NaN
__device__ __forceinline__ float with_cut(float p, float A, float f) {
  return __uint_as_float((__float_as_uint(p) & 0x7fffffffu) | ((__float_as_uint(A) | __float_as_uint(f)) & 0x80000000u));
}
template <bool CUTS>
__device__ __forceinline__ float2 both(float2 A, float2 f) {
  const float2 p = mul2(A, f);
  return CUTS ? make_float2(with_cut(p.x, A.x, f.x), with_cut(p.y, A.y, f.y)) : p;
}
// A stretch's factor is never 0, however long the stretch: it stays at the smallest float, so
// that what came before and is infinite stays infinite.
template <bool CUTS>
__device__ __forceinline__ float2 above_zero(float2 A) {
  float2 r = A;
  if (CUTS) r = make_float2(fabsf(A.x), fabsf(A.y));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(r.x) : "f"(1.4e-45f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(r.y) : "f"(1.4e-45f));
  return CUTS ? make_float2(with_cut(r.x, A.x, 0.f), with_cut(r.y, A.y, 0.f)) : r;
}
// the factor of two stretches
template <bool CUTS>
__device__ __forceinline__ float2 joined(float2 A, float2 f) {
  return above_zero<CUTS>(both<CUTS>(A, f));
}
__device__ __forceinline__ float2 shfl_up2(float2 v, int d) {
  return make_float2(__shfl_up_sync(0xffffffffu, v.x, d), __shfl_up_sync(0xffffffffu, v.y, d));
}
__device__ __forceinline__ float2 shfl_down2(float2 v, int d) {
  return make_float2(__shfl_down_sync(0xffffffffu, v.x, d), __shfl_down_sync(0xffffffffu, v.y, d));
}

// A block's tile in shared memory: segments of kSteps rows of CB channels, padded so that
// the segments of a warp meet in no bank where a row is shorter than a line of banks.
// ALIGNED: rows come in pieces of 16 bytes; otherwise in words, of which 16-bit channels
// that start in the middle of one need one more.
template <typename T, int LS, bool BACKWARD, bool ALIGNED>
struct Shape {
  static constexpr bool kShifted = !ALIGNED && sizeof(T) == 2;
  static constexpr int kSteps = scan::kSteps<BACKWARD>, CB = 2 * LS, kSegs = kWarps * 32 / LS, kTile = kSegs * kSteps;
  static constexpr int kRowBytes = CB * (int)sizeof(T) + (kShifted ? 4 : 0);
  static constexpr int kPad = kShifted ? (LS < 32 ? (LS - kSteps * (LS + 1)) & 31 : 0) * 4 : kRowBytes < 128 ? kRowBytes : 0;
  static constexpr int kSegBytes = kSteps * kRowBytes + kPad;
  static constexpr int kPiece = ALIGNED ? 16 : 4, kPieces = CB * (int)sizeof(T) / kPiece;
  static constexpr int kFramesAtOnce = kThreads / kPieces;  // copied by all threads
  static constexpr int kTurns = kTile / kFramesAtOnce, kArrays = BACKWARD ? 3 : 2;
  // where the frame `far` turns after a thread's first lies, from that one
  static constexpr int place(int far) {
    return far * kFramesAtOnce / kSteps * kSegBytes + far * kFramesAtOnce % kSteps * kRowBytes;
  }
  static_assert(kFramesAtOnce % kSteps == 0 || kSteps % kFramesAtOnce == 0, "whole segments, or parts of one");
  static_assert(kTile % kFramesAtOnce == 0 && kFramesAtOnce % 2 == 0 && kSteps % 2 == 0, "frames in pairs");
  static_assert(kMark % kSteps == 0 && kTile % kMark == 0, "marks fall on starts of segments");
};
template <typename T, int LS, bool BACKWARD, bool ALIGNED>
struct Memory {
  using S = Shape<T, LS, BACKWARD, ALIGNED>;
  __align__(16) unsigned char tiles[2][S::kArrays][S::kSegs * S::kSegBytes];
  float4 warps[kWarps][LS];                            // (A, B) of each warp's pairs
  float4 segs[BACKWARD ? S::kSegs : 1][LS];            // (A, B) of the segments' states
  float4 blocks[2][kMaxCluster][LS];         // (A, B) of each block, two rounds in turn
  unsigned long long arrived[2];                       // barriers for them
  volatile int dead;                                   // a wait gave up
};
__device__ __forceinline__ float4 quad(float2 A, float2 B) { return make_float4(A.x, A.y, B.x, B.y); }
__device__ __forceinline__ float2 first_of(float4 q) { return make_float2(q.x, q.y); }
__device__ __forceinline__ float2 second_of(float4 q) { return make_float2(q.z, q.w); }

__device__ __forceinline__ void store_there(uint32_t to, float4 v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t in_block(uint32_t at, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
// tc::bar_wait for what other blocks stored: visible once the wait is over
__device__ __forceinline__ bool try_theirs(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ void wait_theirs(uint32_t bar, uint32_t parity, volatile int* dead, const tc::ErrorWords& err) {
#pragma unroll 1
  for (int k = 0; k < 32; ++k)
    if (try_theirs(bar, parity)) return;
  if (tc::bar_wait(bar, parity, dead, err)) try_theirs(bar, parity);
}
// The barriers, before anything arrives there; then all blocks of the cluster.
template <typename M>
__device__ __forceinline__ void meet(M& m, const cg::cluster_group& cluster, int ranks) {
  if (ranks == 1) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) tc::bar_init(tc::smem_u32(&m.arrived[i]), 1);
    tc::fence_bar_init();
    m.dead = 0;
  }
  cluster.sync();
}

// No block's memory goes while another may store there.
template <typename M>
__device__ __forceinline__ void part(M& m, const cg::cluster_group& cluster, int ranks) {
  if (ranks == 1) return;
  if (m.dead) {  // what is still under way: give it time
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  cluster.sync();
}

// The state that this block of a cluster starts from, given what its whole tile does
// (A, B), in every thread of a pair of channels; `carry`, the state that the cluster's
// first block starts from, becomes that of the next one's. A block sends its next tile
// only after all its threads have read what came of the present ones, so that two places
// for each block are enough.
template <bool CUTS, bool BACKWARD, int LS, typename M>
__device__ __forceinline__ float2 between_blocks(M& m, const ScanParams& p, int ranks, int rank, int lane, int warp,
                                                 int round, float2 A, float2 B, float2& carry) {
  float2 mine = carry;
  if (ranks == 1) {
    carry = after<CUTS>(A, carry, B);
    return mine;
  }
  const int slot = round & 1;
  const uint32_t bar = tc::smem_u32(&m.arrived[slot]);
  if (threadIdx.x == 0) tc::bar_expect(bar, (uint32_t)(ranks * LS * sizeof(float4)));
  if (lane < LS) {
    const uint32_t place = tc::smem_u32(&m.blocks[slot][rank][lane]);
    for (int r = warp; r < ranks; r += kWarps) store_there(in_block(place, r), quad(A, B), in_block(bar, r));
  }
  wait_theirs(bar, (round >> 1) & 1, &m.dead, p.err);
  for (int r = 0; r < ranks; ++r) {
    if (r == rank) mine = carry;
    const float4 s = m.blocks[slot][r][lane % LS];
    carry = after<CUTS>(first_of(s), carry, second_of(s));
  }
  return mine;
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ float2 load_pair(const T* p, int n) {
  if constexpr (!ALIGNED) return make_float2(to_f(p[0]), n > 1 ? to_f(p[1]) : 0.f);
  else if constexpr (sizeof(T) == 4) return *(const float2*)p;
  else return both_of<T>(*(const uint32_t*)p);
}
// Where a stretch of the row begins: the row's own start (in the walk's direction or, for
// dh, against it) taken through the stretches before.
template <bool CUTS, bool BACKWARD>
__device__ __forceinline__ float2 start_of(const ScanParams& p, long long b, int stretch, int c, int have) {
  float2 h = tc::both(0.f);
  if (have <= 0) return h;
  const long long row = p.batch * p.channels;
  const float2* at = p.sums + b * p.channels + c;
  const int next = have > 1 ? 1 : 0;  // a channel alone takes itself twice
  h = make_float2(at[0].y, at[next].y);
  const int count = BACKWARD ? p.stretches - 1 - stretch : stretch;
  const long long step = BACKWARD ? -row : row;
  at += BACKWARD ? p.stretches * row : row;
#pragma unroll 8
  for (int i = 0; i < count; ++i, at += step) {
    const float2 s0 = at[0], s1 = at[next];
    h = after<CUTS>(make_float2(s0.x, s1.x), h, make_float2(s0.y, s1.y));
  }
  return h;
}

template <typename T, int LS, bool CUTS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) forward(const ScanParams p) {
  using S = Shape<T, LS, false, ALIGNED>;
  constexpr int STEPS = S::kSteps, SEGW = 32 / LS;
  constexpr unsigned kAll = (1u << STEPS) - 1;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& m = *(Memory<T, LS, false, ALIGNED>*)raw;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  long long which = blockIdx.x / ranks;
  const int stretch = (int)(which % p.stretches);
  which /= p.stretches;
  const long long b = which / p.blocks;
  const int begin = stretch * p.length, stop = min(begin + p.length, (int)p.frames);
  const int first = (int)(which % p.blocks) * S::CB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seg = tid / LS, pair = tid % LS;
  const int c = first + 2 * pair, have = p.channels - c;  // of this thread's pair
  Row row(p, b);
  row.last = min(row.last, stop);
  float2 carry = make_float2(0.f, 0.f);
  if (p.stretches > 1) {
    carry = start_of<CUTS, false>(p, b, stretch, c, have);
  } else {
    if (p.state && have > 0) carry.x = p.state[b * p.channels + c];
    if (p.state && have > 1) carry.y = p.state[b * p.channels + c + 1];
  }

  const int stride = ranks * S::kTile, rounds = (stop - begin + stride - 1) / stride;
  int tile = begin + rank * S::kTile;
  const int turn = p.reverse ? -1 : 1;
  // copies: this thread's piece of frame `at`, and of those kFramesAtOnce further
  const int at = tid / S::kPieces, n_c = min(p.channels - first, S::CB), start = row.place(0);
  const long long sx = turn * p.x_s[1], sg = turn * p.g_s[1], sy = turn * p.y_s[1];
  const T* const x0 = (const T*)p.x + b * p.x_s[0] + first;
  const T* const g0 = (const T*)p.g + b * p.g_s[0] + first;
  Source<T, S> x(x0 + row.place(tile + at) * p.x_s[1], tid % S::kPieces, n_c);
  Source<T, S> g(g0 + row.place(tile + at) * p.g_s[1], tid % S::kPieces, n_c);
  const Shift shift_x(x0 + start * p.x_s[1], sx), shift_g(g0 + start * p.g_s[1], sg);
  const int to = at / STEPS * S::kSegBytes + at % STEPS * S::kRowBytes + tid % S::kPieces * S::kPiece;
  const long long far_x = S::kFramesAtOnce * sx, far_g = S::kFramesAtOnce * sg, next_x = stride * sx, next_g = stride * sg;
  auto read = [&](int n, int slot) {
    const T *px = x.p, *pg = g.p;
#pragma unroll
    for (int i = 0; i < S::kTurns; ++i) {
      if (n + at + i * S::kFramesAtOnce < stop) {
        if (x.bytes > 0) fetch<ALIGNED>(&m.tiles[slot][0][to + S::place(i)], px, x.bytes);
        if (g.bytes > 0) fetch<ALIGNED>(&m.tiles[slot][1][to + S::place(i)], pg, g.bytes);
      }
      px += far_x, pg += far_g;
    }
    if (S::kShifted && n_c == S::CB) {
      fetch_last<T, S>(m.tiles[slot][0], x0, p.x_s[1], n, begin, stop, start, turn);
      fetch_last<T, S>(m.tiles[slot][1], g0, p.g_s[1], n, begin, stop, start, turn);
    }
    fetches_end();
    x.p += next_x, g.p += next_g;
  };
  read(tile, 0);
  if (rounds > 1) read(tile + stride, 1);
  else fetches_end();
  T* y = (T*)p.y + b * p.y_s[0] + c + row.place(tile + seg * STEPS) * p.y_s[1];
  const int mine_at = seg * S::kSegBytes + 2 * pair * (int)sizeof(T);
  Row::Ids<(SEGW * STEPS + 31) / 32> ids;  // of the next tile, on their way while this one is worked on
  if (CUTS) row.fetch(tile + warp * SEGW * STEPS, lane, ids);
  meet(m, cluster, ranks);
#pragma unroll 1
  for (int round = 0; round < rounds; ++round, tile += stride) {
    const int slot = round & 1, n0 = tile + seg * STEPS;
    float2 f[STEPS], v[STEPS], A = tc::both(1.f), B = tc::both(0.f);
    unsigned used, fresh;
    row.look<LS, STEPS, CUTS>(tile + warp * SEGW * STEPS, lane, ids, used, fresh);
    const bool plain = __all_sync(0xffffffffu, used == kAll && fresh == 0);
    fetches_wait<1>();
    __syncthreads();
    {
      const unsigned char* px = &m.tiles[slot][0][mine_at];
      const unsigned char* pg = &m.tiles[slot][1][mine_at];
      if (plain) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          float2 rest;
          gates_of(pair_of<T, S>(pg, i, shift_g), f[i], rest);
          v[i] = mul2(rest, pair_of<T, S>(px, i, shift_x));
          A = mul2(A, f[i]);
          B = fma2(f[i], B, v[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          f[i] = tc::both(1.f), v[i] = tc::both(0.f);
          if (used >> i & 1) {
            float2 rest;
            gates_of(pair_of<T, S>(pg, i, shift_g), f[i], rest);
            v[i] = mul2(rest, pair_of<T, S>(px, i, shift_x));
          }
          if (CUTS && (fresh >> i & 1)) f[i] = tc::both(-0.f);
          A = both<CUTS>(A, f[i]);
          B = after<CUTS>(f[i], B, v[i]);
        }
      }
    }
    A = above_zero<CUTS>(A);
    // of the segments up to this one in the warp
#pragma unroll
    for (int d = 1; d < SEGW; d *= 2) {
      const float2 a0 = shfl_up2(A, d * LS), b0 = shfl_up2(B, d * LS);
      if (lane >= d * LS) {
        B = after<CUTS>(A, b0, B);
        A = joined<CUTS>(A, a0);
      }
    }
    if (lane >= 32 - LS) m.warps[warp][pair] = quad(A, B);
    if (SEGW > 1) {  // of those before it
      A = shfl_up2(A, LS & 31), B = shfl_up2(B, LS & 31);
      if (lane < LS) A = tc::both(1.f), B = tc::both(0.f);
    } else {
      A = tc::both(1.f), B = tc::both(0.f);
    }
    __syncthreads();
    if (round + 2 < rounds) read(tile + 2 * stride, slot);  // all have read this tile
    else fetches_end();
    if (CUTS) row.fetch(tile + stride + warp * SEGW * STEPS, lane, ids);
    float2 h;
    {
      float2 a = tc::both(1.f), s = tc::both(0.f), a1 = a, s1 = s;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) a1 = a, s1 = s;
        const float4 q = m.warps[w][pair];
        s = after<CUTS>(first_of(q), s, second_of(q));
        a = joined<CUTS>(first_of(q), a);
      }
      h = between_blocks<CUTS, false, LS>(m, p, ranks, rank, lane, warp, round, a, s, carry);
      if (warp > 0) h = after<CUTS>(a1, h, s1);
      if (SEGW > 1 && lane >= LS) h = after<CUTS>(A, h, B);
    }
    if (p.marks && have > 0 && n0 < stop) {
      float* to = p.marks + ((long long)(n0 / kMark) * p.batch + b) * p.channels + c;
      to[0] = h.x;
      if (have > 1) to[1] = h.y;
    }
    T* out = y;
    if (plain && have > 0) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        h = fma2(f[i], h, v[i]);
        leave<T, ALIGNED>(out, h, have);
        out += sy;
      }
    } else if (have > 0) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        h = after<CUTS>(f[i], h, v[i]);
        if (n0 + i < stop) leave<T, ALIGNED>(out, used >> i & 1 ? h : tc::both(0.f), have);
        out += sy;
      }
    }
    y += stride * sy;
  }
  if (rank == 0 && tid < LS && p.end && stretch == p.stretches - 1) {
    if (have > 0) p.end[b * p.channels + c] = carry.x;
    if (have > 1) p.end[b * p.channels + c + 1] = carry.y;
  }
  part(m, cluster, ranks);
}

// The blocks take the row from the walk's end: rank 0 the last tile, and so on.
template <typename T, int LS, bool CUTS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) backward(const ScanParams p) {
  using S = Shape<T, LS, true, ALIGNED>;
  constexpr int STEPS = S::kSteps, SEGW = 32 / LS;
  constexpr unsigned kAll = (1u << STEPS) - 1;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& m = *(Memory<T, LS, true, ALIGNED>*)raw;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  long long which = blockIdx.x / ranks;
  const int stretch = (int)(which % p.stretches);
  which /= p.stretches;
  const long long b = which / p.blocks;
  const int begin = stretch * p.length, stop = min(begin + p.length, (int)p.frames);
  const int first = (int)(which % p.blocks) * S::CB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seg = tid / LS, pair = tid % LS;
  const int c = first + 2 * pair, have = p.channels - c;
  Row row(p, b);
  row.first = max(row.first, begin), row.last = min(row.last, stop);
  float2 carry = make_float2(0.f, 0.f);
  if (p.stretches > 1) {
    carry = start_of<CUTS, true>(p, b, stretch, c, have);
  } else {
    if (p.dend && have > 0) carry.x = p.dend[b * p.channels + c];
    if (p.dend && have > 1) carry.y = p.dend[b * p.channels + c + 1];
  }

  const int tiles = (stop - begin + S::kTile - 1) / S::kTile, rounds = (tiles + ranks - 1) / ranks;
  const int stride = ranks * S::kTile;
  int tile = begin + (tiles - 1 - rank) * S::kTile;
  const int turn = p.reverse ? -1 : 1;
  const int at = tid / S::kPieces, n_c = min(p.channels - first, S::CB), start = row.place(0);
  const long long sx = turn * p.x_s[1], sg = turn * p.g_s[1], sd = turn * p.dy_s[1];
  const long long so = turn * p.dx_s[1], sp = turn * p.dg_s[1];
  const T* const x0 = (const T*)p.x + b * p.x_s[0] + first;
  const T* const g0 = (const T*)p.g + b * p.g_s[0] + first;
  const T* const d0 = (const T*)p.dy + b * p.dy_s[0] + first;
  Source<T, S> x(x0 + row.place(tile + at) * p.x_s[1], tid % S::kPieces, n_c);
  Source<T, S> g(g0 + row.place(tile + at) * p.g_s[1], tid % S::kPieces, n_c);
  Source<T, S> dy(d0 + row.place(tile + at) * p.dy_s[1], tid % S::kPieces, n_c);
  const Shift shift_x(x0 + start * p.x_s[1], sx), shift_g(g0 + start * p.g_s[1], sg), shift_d(d0 + start * p.dy_s[1], sd);
  const int to = at / STEPS * S::kSegBytes + at % STEPS * S::kRowBytes + tid % S::kPieces * S::kPiece;
  const long long far_x = S::kFramesAtOnce * sx, far_g = S::kFramesAtOnce * sg, far_d = S::kFramesAtOnce * sd;
  const long long next_x = stride * sx, next_g = stride * sg, next_d = stride * sd;
  auto read = [&](int n, int slot) {
    const T *px = x.p, *pg = g.p, *pd = dy.p;
#pragma unroll
    for (int i = 0; i < S::kTurns; ++i) {
      if (n + at + i * S::kFramesAtOnce >= begin && n + at + i * S::kFramesAtOnce < stop) {
        if (x.bytes > 0) fetch<ALIGNED>(&m.tiles[slot][0][to + S::place(i)], px, x.bytes);
        if (g.bytes > 0) fetch<ALIGNED>(&m.tiles[slot][1][to + S::place(i)], pg, g.bytes);
        if (dy.bytes > 0) fetch<ALIGNED>(&m.tiles[slot][2][to + S::place(i)], pd, dy.bytes);
      }
      px += far_x, pg += far_g, pd += far_d;
    }
    if (S::kShifted && n_c == S::CB) {
      fetch_last<T, S>(m.tiles[slot][0], x0, p.x_s[1], n, begin, stop, start, turn);
      fetch_last<T, S>(m.tiles[slot][1], g0, p.g_s[1], n, begin, stop, start, turn);
      fetch_last<T, S>(m.tiles[slot][2], d0, p.dy_s[1], n, begin, stop, start, turn);
    }
    fetches_end();
    x.p -= next_x, g.p -= next_g, dy.p -= next_d;
  };
  read(tile, 0);
  const int here = row.place(tile + seg * STEPS);
  T* dx = p.dx ? (T*)p.dx + b * p.dx_s[0] + c + here * p.dx_s[1] : nullptr;
  T* dg = p.dg ? (T*)p.dg + b * p.dg_s[0] + c + here * p.dg_s[1] : nullptr;
  const int mine_at = seg * S::kSegBytes + 2 * pair * (int)sizeof(T);
  Row::Ids<(SEGW * STEPS + 31) / 32> ids;  // of the next tile, on their way while this one is worked on
  if (CUTS) row.fetch(tile + warp * SEGW * STEPS, lane, ids);
  meet(m, cluster, ranks);
#pragma unroll 1
  for (int round = 0; round < rounds; ++round, tile -= stride) {
    const int slot = round & 1, n0 = tile + seg * STEPS;
    unsigned used, fresh;
    row.look<LS, STEPS, CUTS>(tile + warp * SEGW * STEPS, lane, ids, used, fresh);
    const bool plain = __all_sync(0xffffffffu, used == kAll && fresh == 0);
    // the state at the last mark: this segment's start, or that of one before it
    const int n1 = n0 / kMark * kMark;
    float2 h = tc::both(0.f);
    if (n0 >= begin && n0 < stop && have > 0) {
      const float* from = p.marks + ((long long)(n1 / kMark) * p.batch + b) * p.channels + c;
      h.x = from[0];
      if (have > 1) h.y = from[1];
    }
    fetches_wait<0>();
    __syncthreads();  // this tile is there, and all are done with the other slot
    if (round + 1 < rounds) read(tile - stride, slot ^ 1);
    if (CUTS) row.fetch(tile - stride + warp * SEGW * STEPS, lane, ids);
    const unsigned char* px = &m.tiles[slot][0][mine_at];
    const unsigned char* pg = &m.tiles[slot][1][mine_at];
    const unsigned char* pd = &m.tiles[slot][2][mine_at];

    float2 f[STEPS], rest[STEPS], A = tc::both(1.f), B = tc::both(0.f), R = B;
    if (plain) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        gates_of(pair_of<T, S>(pg, i, shift_g), f[i], rest[i]);
        A = mul2(A, f[i]);
        B = fma2(f[i], B, mul2(rest[i], pair_of<T, S>(px, i, shift_x)));
      }
#pragma unroll
      for (int i = STEPS - 1; i >= 0; --i) R = mul2(f[i], add2(R, pair_of<T, S>(pd, i, shift_d)));
    } else {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        float2 v = tc::both(0.f);
        f[i] = tc::both(1.f), rest[i] = v;
        if (used >> i & 1) {
          gates_of(pair_of<T, S>(pg, i, shift_g), f[i], rest[i]);
          v = mul2(rest[i], pair_of<T, S>(px, i, shift_x));
        }
        const float2 step = CUTS && (fresh >> i & 1) ? tc::both(-0.f) : f[i];
        A = both<CUTS>(A, step);
        B = after<CUTS>(step, B, v);
      }
#pragma unroll
      for (int i = STEPS - 1; i >= 0; --i) {
        if (used >> i & 1) R = mul2(f[i], add2(R, pair_of<T, S>(pd, i, shift_d)));
        if (CUTS && (fresh >> i & 1)) R = tc::both(0.f);
      }
    }
    A = above_zero<CUTS>(A);
    m.segs[seg][pair] = quad(A, B);
    // of the segments from this one on in the warp
#pragma unroll
    for (int d = 1; d < SEGW; d *= 2) {
      const float2 a0 = shfl_down2(A, d * LS), r0 = shfl_down2(R, d * LS);
      if (lane + d * LS < 32) {
        R = after<CUTS>(A, r0, R);
        A = joined<CUTS>(A, a0);
      }
    }
    if (lane < LS) m.warps[warp][pair] = quad(A, R);
    if (SEGW > 1) {  // of those after it
      A = shfl_down2(A, LS & 31), R = shfl_down2(R, LS & 31);
      if (lane >= 32 - LS) A = tc::both(1.f), R = tc::both(0.f);
    } else {
      A = tc::both(1.f), R = tc::both(0.f);
    }
    __syncthreads();
    {
      float2 a = tc::both(1.f), s = tc::both(0.f), a1 = a, s1 = s;
#pragma unroll
      for (int w = kWarps - 1; w >= 0; --w) {
        if (w == warp) a1 = a, s1 = s;
        const float4 q = m.warps[w][pair];
        s = after<CUTS>(first_of(q), s, second_of(q));
        a = joined<CUTS>(first_of(q), a);
      }
      float2 from = between_blocks<CUTS, true, LS>(m, p, ranks, rank, lane, warp, round, a, s, carry);
      if (warp < kWarps - 1) from = after<CUTS>(a1, from, s1);
      if (SEGW > 1 && lane < 32 - LS) from = after<CUTS>(A, from, R);
      R = from;
    }
#pragma unroll
    for (int k = kMark / STEPS - 1; k > 0; --k) {  // from the mark to this segment
      if (seg % (kMark / STEPS) >= k) {
        const float4 q = m.segs[seg - k][pair];
        h = after<CUTS>(first_of(q), h, second_of(q));
      }
    }
    float2 w[STEPS];  // a (1 - a) (h - x), h the state as the step takes it
    T *px1 = dx ? dx + (STEPS - 1) * so : nullptr, *pg1 = dg ? dg + (STEPS - 1) * sp : nullptr;
    if (plain) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const float2 xs = pair_of<T, S>(px, i, shift_x);
        w[i] = mul2(mul2(f[i], rest[i]), fma2(xs, tc::both(-1.f), h));
        h = fma2(f[i], h, mul2(rest[i], xs));
      }
#pragma unroll
      for (int i = STEPS - 1; i >= 0; --i) {
        const float2 d = add2(R, pair_of<T, S>(pd, i, shift_d));
        R = mul2(f[i], d);
        if (have > 0 && dx) leave<T, ALIGNED>(px1, mul2(d, rest[i]), have);
        if (have > 0 && dg) leave<T, ALIGNED>(pg1, mul2(d, w[i]), have);
        px1 -= so, pg1 -= sp;
      }
    } else {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        if (used >> i & 1) {
          if (CUTS && (fresh >> i & 1)) h = tc::both(0.f);
          const float2 xs = pair_of<T, S>(px, i, shift_x);
          w[i] = mul2(mul2(f[i], rest[i]), fma2(xs, tc::both(-1.f), h));
          h = fma2(f[i], h, mul2(rest[i], xs));
        }
      }
#pragma unroll
      for (int i = STEPS - 1; i >= 0; --i) {
        float2 ox = tc::both(0.f), og = ox;
        if (used >> i & 1) {
          const float2 d = add2(R, pair_of<T, S>(pd, i, shift_d));
          ox = mul2(d, rest[i]);
          og = mul2(d, w[i]);
          R = CUTS && (fresh >> i & 1) ? tc::both(0.f) : mul2(f[i], d);
        }
        if (have > 0 && n0 + i >= begin && n0 + i < stop) {
          if (dx) leave<T, ALIGNED>(px1, ox, have);
          if (dg) leave<T, ALIGNED>(pg1, og, have);
        }
        px1 -= so, pg1 -= sp;
      }
    }
    if (dx) dx -= stride * so;
    if (dg) dg -= stride * sp;
  }
  if (rank == 0 && tid < LS && p.dstate && stretch == 0) {
    if (have > 0) p.dstate[b * p.channels + c] = carry.x;
    if (have > 1) p.dstate[b * p.channels + c + 1] = carry.y;
  }
  part(m, cluster, ranks);
}

// What each stretch does to the state, or to dh: a cluster a stretch, its blocks' parts
// and their threads' runs side by side. Memory bound: nothing is kept but the sums.
template <typename T, int LS, bool CUTS, bool BACKWARD, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) stretch_sums(const ScanParams p) {
  constexpr int kSegs = kThreads / LS, kAhead = kSteps<BACKWARD>;
  __shared__ float4 segs[kSegs][LS], total[LS];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  long long which = blockIdx.x / ranks;
  const int stretch = (int)(which % p.stretches);
  which /= p.stretches;
  const long long b = which / p.blocks;
  const int tid = threadIdx.x, seg = tid / LS, pair = tid % LS;
  const int c = (int)(which % p.blocks) * 2 * LS + 2 * pair, have = p.channels - c;
  const long long at = b * p.channels + c;
  if (stretch == (BACKWARD ? 0 : p.stretches - 1) && p.stretches > 1) return;  // none starts from it
  if (stretch == (BACKWARD ? p.stretches - 1 : 0) && rank == 0 && seg == 0) {
    const float* from = BACKWARD ? p.dend : p.state;
    if (have > 0) p.sums[at] = make_float2(0.f, from ? from[at] : 0.f);
    if (have > 1) p.sums[at + 1] = make_float2(0.f, from ? from[at + 1] : 0.f);
  }
  Row row(p, b);
  const int run = p.length / ranks / kSegs, n = stretch * p.length + (rank * kSegs + seg) * run;
  const long long* vs = BACKWARD ? p.dy_s : p.x_s;
  const T* v = (const T*)(BACKWARD ? p.dy : p.x) + b * vs[0] + c;
  const T* g = (const T*)p.g + b * p.g_s[0] + c;
  float2 A = tc::both(1.f), B = tc::both(0.f);
  for (int f0 = 0; f0 < run && have > 0; f0 += kAhead) {
    float2 in[kAhead], gate[kAhead];
    unsigned used = 0, fresh = 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int f = BACKWARD ? n + run - 1 - f0 - i : n + f0 + i;
      bool u = f >= row.first && f < row.last;
      if (CUTS && u) {
        const int id = row.id(f);
        u = id >= 0;
        if (u && f > 0 && row.id(f - 1) != id) fresh |= 1u << i;
      }
      if (u) {
        used |= 1u << i;
        in[i] = load_pair<T, ALIGNED>(v + row.place(f) * vs[1], have);
        gate[i] = load_pair<T, ALIGNED>(g + row.place(f) * p.g_s[1], have);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!(used >> i & 1)) continue;
      float2 f, rest;
      gates_of(gate[i], f, rest);
      const bool cuts = CUTS && (fresh >> i & 1);
      if (BACKWARD) {
        B = cuts ? tc::both(0.f) : mul2(f, add2(B, in[i]));
        A = both<CUTS>(A, cuts ? tc::both(-0.f) : f);
      } else {
        if (cuts) f = tc::both(-0.f);
        A = both<CUTS>(A, f);
        B = after<CUTS>(f, B, mul2(rest, in[i]));
      }
    }
  }
  segs[seg][pair] = quad(above_zero<CUTS>(A), B);
  __syncthreads();
  A = tc::both(1.f), B = tc::both(0.f);
  if (seg == 0) {
#pragma unroll 4
    for (int i = 0; i < kSegs; ++i) {
      const float4 q = segs[BACKWARD ? kSegs - 1 - i : i][pair];
      B = after<CUTS>(first_of(q), B, second_of(q));
      A = joined<CUTS>(first_of(q), A);
    }
    total[pair] = quad(A, B);
  }
  cluster.sync();
  if (rank == 0 && seg == 0) {
    A = tc::both(1.f), B = tc::both(0.f);
    for (int i = 0; i < ranks; ++i) {
      const float4 q = *cluster.map_shared_rank(&total[pair], BACKWARD ? ranks - 1 - i : i);
      B = after<CUTS>(first_of(q), B, second_of(q));
      A = joined<CUTS>(first_of(q), A);
    }
    float2* to = p.sums + (stretch + 1) * p.batch * p.channels + at;
    if (have > 0) to[0] = make_float2(A.x, B.x);
    if (have > 1) to[1] = make_float2(A.y, B.y);
  }
  cluster.sync();  // no block's memory goes while it is read
}

// A few frames: a thread walks its channels alone.
template <typename T, int VC>
__global__ void __launch_bounds__(128) scan_short(const ScanParams p) {
  const long long at = (long long)blockIdx.x * 128 + threadIdx.x;
  const int packs = p.channels / VC;
  const long long b = at / packs;
  if (b >= p.batch) return;
  const int c = (int)(at % packs) * VC;
  const Row row(p, b);
  const T* x = (const T*)p.x + b * p.x_s[0] + c;
  const T* g = (const T*)p.g + b * p.g_s[0] + c;
  T* y = (T*)p.y + b * p.y_s[0] + c;
  float h[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) h[k] = p.state ? p.state[b * p.channels + c + k] : 0.f;
  if (p.marks && p.frames > 0) {
#pragma unroll
    for (int k = 0; k < VC; ++k) p.marks[b * p.channels + c + k] = h[k];
  }
  int before = 0;
  for (int n = 0; n < (int)p.frames; ++n) {
    bool u = n >= row.first && n < row.last, go = true;
    if (row.docs) {
      const int id = row.id(n);
      u = u && id >= 0;
      go = n == 0 || id == before;
      before = id;
    }
    Pack<T, VC> q;
#pragma unroll
    for (int k = 0; k < VC; ++k) q.v[k] = from_f<T>(0.f);
    if (u) {
      const Pack<T, VC> qx = *(const Pack<T, VC>*)(x + row.place(n) * p.x_s[1]);
      const Pack<T, VC> qg = *(const Pack<T, VC>*)(g + row.place(n) * p.g_s[1]);
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        float2 a, rest;
        gates_of(tc::both(to_f(qg.v[k])), a, rest);
        h[k] = fmaf(a.x, go ? h[k] : 0.f, rest.x * to_f(qx.v[k]));
        q.v[k] = from_f<T>(h[k]);
      }
    }
    *(Pack<T, VC>*)(y + row.place(n) * p.y_s[1]) = q;
  }
  if (p.end) {
#pragma unroll
    for (int k = 0; k < VC; ++k) p.end[b * p.channels + c + k] = h[k];
  }
}

struct Split {
  int ranks;
  long long rounds;  // or what the stretches' first kernel costs besides, in such rounds
  int stretches = 1;
  long long length = 0;  // frames of each; 0: all
};
constexpr int kMaxStretches = 64;

// One set of kernels, over channels (2 * LS) and by alignment.
template <typename T, int LS, bool BACKWARD, bool ALIGNED>
struct Kernels {
  using S = Shape<T, LS, BACKWARD, ALIGNED>;
  static constexpr size_t kBytes = sizeof(Memory<T, LS, BACKWARD, ALIGNED>);
  static void (*kernel(bool docs))(ScanParams) {
    if constexpr (BACKWARD) return docs ? backward<T, LS, true, ALIGNED> : backward<T, LS, false, ALIGNED>;
    else return docs ? forward<T, LS, true, ALIGNED> : forward<T, LS, false, ALIGNED>;
  }
  static long long groups(const ScanParams& p) { return p.batch * ((p.channels + S::CB - 1) / S::CB); }
  // Clusters of n blocks that the device runs at once, 0 where it takes none of this
  // size: asked for once. A question that fails is none of its answers: the next call asks
  // again.
  static int at_once(int n) {
    static std::atomic<int> known[64][kMaxCluster + 1];  // 1 more than the answer
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int v = known[dev][n].load(std::memory_order_relaxed);
    if (v > 0) return v - 1;
    auto k = kernel(false);
    cudaLaunchAttribute attr{};
    const cudaLaunchConfig_t cfg = config(n, n, &attr, nullptr);
    if (!ready(k, n) || cudaOccupancyMaxActiveClusters(&v, k, &cfg) != cudaSuccess || v < 0) {
      cudaGetLastError();
      return 0;
    }
    known[dev][n].store(v + 1, std::memory_order_relaxed);
    return v;
  }
  static bool wide_enough(void (*k)(ScanParams), int ranks) {
    return ranks <= 8 ||
           cudaFuncSetAttribute((const void*)k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  }
  static bool ready(void (*k)(ScanParams), int ranks) { return allow_smem(k, kBytes) && wide_enough(k, ranks); }
  // Blocks of a cluster, and the rounds that all rows then take one after another: every
  // block of a launch takes equally long, so that the number of waves counts. Of equal
  // ones the smallest, whose blocks wait for fewest.
  // Stretches, as many as fill the device: their first kernel reads two arrays of three (two
  // of five backward), at about the memory's rate, and is another launch: half the rounds
  // and two. Elements one by one take it longer than the rounds: 360001 x 341 in bf16 834
  // us with stretches, 538 without.
  static Split split(const ScanParams& p) {
    const long long tiles = (p.frames + S::kTile - 1) / S::kTile;
    Split best{1, 1LL << 58};  // consider() takes six times this
    for (int n = 1; n <= kMaxCluster && n <= tiles; ++n) {
      const int slots = at_once(n);
      if (slots == 0) continue;
      const long long rounds = (groups(p) + slots - 1) / slots * ((tiles + n - 1) / n);
      if (rounds < best.rounds) best = Split{n, rounds};
      const long long most = p.sums ? std::min<long long>(slots / groups(p), kMaxStretches) : 0;
      if (most < 2) continue;
      const long long each = ((tiles + most - 1) / most + n - 1) / n, cost = each + (ALIGNED ? each / 2 : 2 * each) + 2;
      if (cost < best.rounds && each * n < tiles)
        best = Split{n, cost, (int)((tiles + each * n - 1) / (each * n)), each * n * S::kTile};
    }
    return best;
  }
  static cudaLaunchConfig_t config(long long blocks, int ranks, cudaLaunchAttribute* attr, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = st;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)ranks;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
  }
  static fm_status launch(ScanParams p, const Split& s, cudaStream_t st) {
    auto k = kernel(p.docs != nullptr);
    if (!ready(k, s.ranks)) return FM_ERR_CUDA;
    p.blocks = (p.channels + S::CB - 1) / S::CB;
    p.stretches = s.stretches;
    p.length = (int)(s.length ? s.length : p.frames);
    const long long blocks = groups(p) * s.stretches * s.ranks;
    if (blocks > 0x7fffffffLL) return FM_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr{};
    cudaLaunchConfig_t cfg = config(blocks, s.ranks, &attr, st);
    if (s.stretches > 1) {
      auto first = p.docs ? stretch_sums<T, LS, true, BACKWARD, ALIGNED> : stretch_sums<T, LS, false, BACKWARD, ALIGNED>;
      if (!wide_enough(first, s.ranks)) return FM_ERR_CUDA;
      cudaLaunchConfig_t small = cfg;
      small.dynamicSmemBytes = 0;
      if (cudaLaunchKernelEx(&small, first, p) != cudaSuccess) {
        cudaGetLastError();
        return FM_ERR_CUDA;
      }
    }
    if (cudaLaunchKernelEx(&cfg, k, p) != cudaSuccess) {
      cudaGetLastError();
      return FM_ERR_CUDA;
    }
    return launch_status();
  }
};

// Rows of 128, 64 or 32 bytes of a segment: the widest, unless a narrower one has a fifth
// fewer rounds. Few channels in few rows make too few blocks of the widest, even with the
// largest clusters; narrower ones have more segments to join, and shorter pieces to read.
// 100000 frames of 512 channels in bf16: 95 us with 16 pairs across, 90 with 8 (in blocks
// of eight warps); eight rows of 3001 x 1024 backward, where 8 would save one round of 15:
// 64 us with 32, 86 with 8. 16 bytes: 100000 frames of 80 32-bit channels 49 us for 38.
template <typename T, bool BACKWARD, bool ALIGNED, int LS>
void consider(const ScanParams& p, Split& best, fm_status (**launch)(ScanParams, const Split&, cudaStream_t)) {
  using K = Kernels<T, LS, BACKWARD, ALIGNED>;
  const Split s = K::split(p);
  if (*launch && 6 * s.rounds >= 5 * best.rounds) return;
  best = s;
  *launch = K::launch;
}
template <typename T, bool BACKWARD, bool ALIGNED>
fm_status sized(const ScanParams& p, cudaStream_t st) {
  constexpr int kWide = 128 / 2 / (int)sizeof(T);
  Split best{1, 0};
  fm_status (*launch)(ScanParams, const Split&, cudaStream_t) = nullptr;
  consider<T, BACKWARD, ALIGNED, kWide>(p, best, &launch);
  consider<T, BACKWARD, ALIGNED, kWide / 2>(p, best, &launch);
  consider<T, BACKWARD, ALIGNED, kWide / 4>(p, best, &launch);
  return launch(p, best, st);
}

template <typename T>
fm_status typed(const ScanParams& p, bool back, cudaStream_t st) {
  // 16-byte accesses where every frame of every array starts on such a boundary
  constexpr int V = 16 / (int)sizeof(T);
  auto ok = [&](const void* q, const long long (&s)[2]) {
    return q == nullptr || (((uintptr_t)q & 15) == 0 && s[0] % V == 0 && s[1] % V == 0);
  };
  const bool aligned = p.channels % V == 0 && ok(p.x, p.x_s) && ok(p.g, p.g_s) && ok(p.y, p.y_s) && ok(p.dy, p.dy_s) &&
                       ok(p.dx, p.dx_s) && ok(p.dg, p.dg_s);
  if (!back && p.frames <= kShort) {
    const long long blocks = (p.batch * (aligned ? p.channels / V : p.channels) + 127) / 128;
    if (blocks > 0x7fffffffLL) return FM_ERR_UNSUPPORTED;
    if (aligned) scan_short<T, V><<<(unsigned)blocks, 128, 0, st>>>(p);
    else scan_short<T, 1><<<(unsigned)blocks, 128, 0, st>>>(p);
    return launch_status();
  }
  if (back) return aligned ? sized<T, true, true>(p, st) : sized<T, true, false>(p, st);
  return aligned ? sized<T, false, true>(p, st) : sized<T, false, false>(p, st);
}

}  // namespace scan
}  // namespace fm

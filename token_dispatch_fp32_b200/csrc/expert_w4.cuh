// expert_w4.cuh -- the experts' products on 4-bit weights with group scales,
// for batches of few tokens (Kimi K2 "Add shared output" page, moe_infer:
// sorted_tokens = x[idxs // k], expert(sorted_tokens[start_idx:end_idx])).
//
//   out[j][n] = sum_G scale[e][n][G] * sum_{c in G} (q[e][n][c] - 8) * x[perm[j]/k][c]
//
// for the sorted row j of expert e, groups G of 32, 64 or 128 columns.  A few
// rows per expert make this a stream of the hit experts' weights from HBM
// (n_out * d / 2 bytes each plus the scales): the kernel's work per weight
// should stay below what the SMs issue while those bytes arrive, about 50 cycles
// of an SM for 16 x 128 weights.  So
//  * weights meet x in tensor-core MMAs with the weights as the 16-row operand
//    and 8 rows of x as the columns (mma.sync m16n8k16: at this shape the
//    tensor pipe is nearly idle, and its operands come from registers; a
//    128-row tcgen05 tile would first have to pass the widened weights, four
//    times the bytes, through shared or tensor memory);
//  * a nibble u becomes the bf16 value 16 + u by one AND-OR of two weights (its
//    four bits are the upper mantissa bits of 16.0), rotated into place by one
//    shift; nothing is subtracted per weight: the sums start from -24 * sum x
//    of the group's columns, which one more MMA pair with a constant operand
//    forms for all rows at once.
// Measured: 62 cycles per 16 x 128 weights (about 140 instructions, half of them
// on the half-rate integer pipe); a decode batch of 64 tokens takes 405 to 445 us
// from box to box, 63 to 69 % of the HBM rate: 355 us where no warp waits for
// weights, 272 us for the stream without the arithmetic; the rest (x through L1,
// the ends of items) is not measured apart.  Subtracting per weight instead took
// 557 us; 8-bit MMAs, whose e4m3 codes 0 .. 15 are the nibbles themselves, run as
// two 16-bit ones with unpacking on this GPU (639 us); a ring shared by the CTA
// with a producer warp 643 us.
// Every product is exact in fp32.  A group's sum runs through at most 55 * sum
// |x| (24 + 31) where |q - 8| alone would reach 8 * sum |x|, in fp32; it is
// then scaled and added in fp32, and the result rounded to bf16 once.
//
// Packed layout (written once by w4_pack_kernel): units of 64 output rows x 128
// columns, unit (e, tile, kb) at index (e * tiles + tile) * KB + kb.  A unit is
// read in four steps i of 32 columns.  With lane l of a warp standing for the
// rows 16 m + l / 4 and 16 m + 8 + l / 4 (m = 0..3) and the columns 32 i + 8 (l
// % 4) .. + 7 -- what it feeds to two steps of an m16n8k16 MMA, so that the
// lane's share of x is 16 contiguous bytes -- its weights of step i are four
// words (m = 0..3) for the first rows at 1024 i + 16 l and four for the second
// at 1024 i + 512 + 16 l.  In a word, column 2 p of the eight is the nibble at
// bit 3 + 4 p, column 2 p + 1 the one at bit 19 + 4 p (modulo 32).  The unit's
// scales follow in their own type as [128 / group][8 rows l / 4][4 m][2], so
// that a lane reads its eight scales of a step at once.  Padded rows and columns
// hold the value 0 (nibble 8) and scale 0.
//
// The kernel is persistent, two CTAs per SM.  An item is 64 output rows of one
// expert against up to 16 of its sorted rows; a team of `ks` of the CTA's
// eight warps (chosen from the number of items) takes it, splits its columns
// (member m takes units m, m + ks, ..) and meets in shared memory at the item's
// end, adding in member order.  Each warp has its own ring of units in shared
// memory, filled by one bulk copy each, and requests a unit as soon as it has
// finished the one whose place it takes, through the ends of items, so that the
// stream from HBM does not pause; no warp waits for another but its team at an
// item's end.  x comes through L1.  Every mbarrier wait is bounded.
// Segments of many rows may go to expert_w4_tile.cuh's kernel (long_to_tile).
#pragma once

#include <type_traits>

#include "expert_gemm.cuh"
#include "mr_common.cuh"

namespace mr {
namespace w4 {

using namespace mr::tc;

constexpr int kTile = 64;      // output rows per unit and item
constexpr int kCols = 128;     // columns per unit
constexpr int kWeightBytes = kTile * kCols / 2;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;     // units per warp's ring
constexpr int kRowsPerPass = 16;  // sorted rows per item (two column tiles of the MMA)

struct Layout {
  int tiles, KB;         // tiles of n_out, units along d
  int unit_bytes;
  size_t total;
};

inline Layout make_layout(int N_r, int n_out, int d, int group, int scale_bytes) {
  Layout l;
  l.tiles = (n_out + kTile - 1) / kTile;
  l.KB = (d + kCols - 1) / kCols;
  l.unit_bytes = kWeightBytes + kTile * (kCols / group) * scale_bytes;
  l.total = (size_t)N_r * l.tiles * l.KB * l.unit_bytes;
  return l;
}

// q [N_r, n_out, d / 2] (column 2 i in the low nibble of byte i), scales
// [N_r, n_out, ceil(d / group)] -> the packed layout.  One CTA per unit.
template <typename S>
__global__ void __launch_bounds__(128)
    w4_pack_kernel(const uint8_t* __restrict__ q, const S* __restrict__ scales, int n_out, int d,
                   int group, int tiles, int KB, int unit_bytes, uint8_t* __restrict__ packed) {
  const int lane = threadIdx.x & 31, i = threadIdx.x >> 5;
  const long b = blockIdx.x;
  const int kb = (int)(b % KB);
  const int tile = (int)((b / KB) % tiles);
  const long e = b / ((long)KB * tiles);
  uint8_t* unit = packed + b * unit_bytes;
  const int c0 = kb * kCols + 32 * i + 8 * (lane % 4);
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4];
    for (int m = 0; m < 4; ++m) {
      const int n = tile * kTile + m * 16 + 8 * h + lane / 4;
      uint32_t v = 0x44444444u;  // nibbles of 8, rotated; the eight columns are all in or all out
      if (n < n_out && c0 < d) {
        const uint8_t* src = q + ((e * n_out + n) * (long)d + c0) / 2;
        v = 0;
        for (int p = 0; p < 4; ++p) {
          const uint32_t byte = src[p];
          v |= (byte & 15u) << (4 * p);
          v |= (byte >> 4) << (16 + 4 * p);
        }
        v = __funnelshift_l(v, v, 3);
      }
      w[m] = v;
    }
    *reinterpret_cast<uint4*>(unit + 1024 * i + 512 * h + 16 * lane) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int ng = kCols / group, groups = (d + group - 1) / group;
  S* sp = reinterpret_cast<S*>(unit + kWeightBytes);
  for (int o = threadIdx.x; o < kTile * ng; o += 128) {
    const int h = o & 1, m = (o >> 1) & 3, r = (o >> 3) & 7;
    const int n = tile * kTile + m * 16 + 8 * h + r, g = kb * ng + (o >> 6);
    S v{};
    if (n < n_out && g < groups) v = scales[(e * n_out + n) * (long)groups + g];
    sp[o] = v;
  }
}

// 16 + u of the weight pair p of w, as two bf16 values.
__device__ __forceinline__ uint32_t widen2(uint32_t w, int p) {
  const uint32_t v = p ? __funnelshift_r(w, w, 4 * p) : w;
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00780078, %2, 0xea;" : "=r"(r) : "r"(v), "r"(0x41804180u));
  return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}

struct Params {
  const uint16_t* x;
  const int32_t* perm;  // null: x holds the sorted rows
  const int32_t* offsets;
  const uint8_t* wp;
  uint16_t* out;
  int T, d, k, N_r, n_out, tiles, KB, unit_bytes;
  int tile_rows;  // segments of more rows may go to expert_w4_tile.cuh's kernel (0: never)
  int sms;
};

// The scales of step i: s[2 m + h] for the row 16 m + 8 h + lane / 4.
template <int GROUP>
__device__ __forceinline__ void load_scales(const uint8_t* sc, int i, int lane, float (&s)[8],
                                            uint16_t) {
  const uint4 v = *reinterpret_cast<const uint4*>(sc + (i * 32 / GROUP) * 128 + (lane / 4) * 16);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    s[2 * m] = __uint_as_float(w[m] << 16);
    s[2 * m + 1] = __uint_as_float(w[m] & 0xffff0000u);
  }
}
template <int GROUP>
__device__ __forceinline__ void load_scales(const uint8_t* sc, int i, int lane, float (&s)[8],
                                            float) {
  const float4* p =
      reinterpret_cast<const float4*>(sc + (i * 32 / GROUP) * 256 + (lane / 4) * 32);
  const float4 a = p[0], b = p[1];
  s[0] = a.x, s[1] = a.y, s[2] = a.z, s[3] = a.w;
  s[4] = b.x, s[5] = b.y, s[6] = b.z, s[7] = b.w;
}

// The lane's x of step i of a unit: x4[t] the lane's row of tile t at the
// unit's first column + 8 (lane % 4); n8: 16-byte pieces of a row from the
// unit's first column to d (columns past d are 0: their weights are 0, but 0
// times what lies there need not be).
template <int NT>
__device__ __forceinline__ void load_x(const uint4* const (&x4)[NT], int i, int n8, int lane,
                                       uint4 (&xv)[NT]) {
  if (n8 >= kCols / 8) {
#pragma unroll
    for (int t = 0; t < NT; ++t) xv[t] = __ldg(x4[t] + 4 * i);
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      xv[t] = 4 * i + lane % 4 < n8 ? __ldg(x4[t] + 4 * i) : make_uint4(0, 0, 0, 0);
  }
}

// 32 columns (step i) of one unit (at w) times NT * 8 rows of x.
template <int GROUP, typename S, int NT>
__device__ __forceinline__ void step(const uint8_t* w, int i, int lane, const uint4 (&xv)[NT],
                                     float (&acc)[4][NT][4]) {
  const uint4 w0 = *reinterpret_cast<const uint4*>(w + 1024 * i + 16 * lane);
  const uint4 w1 = *reinterpret_cast<const uint4*>(w + 1024 * i + 512 + 16 * lane);
  float s[8];
  load_scales<GROUP>(w + kWeightBytes, i, lane, s, S{});
  const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w}, wb[4] = {w1.x, w1.y, w1.z, w1.w};
  const uint32_t off = 0xc1c0c1c0u;  // -24
  const uint32_t o4[4] = {off, off, off, off};
  float z[NT][4];  // -24 * sum of x over the step's columns
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    mma16816(z[t], o4, xv[t].x, xv[t].y, 0.f, 0.f, 0.f, 0.f);
    mma16816(z[t], o4, xv[t].z, xv[t].w, z[t][0], z[t][1], z[t][2], z[t][3]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint32_t a[4] = {widen2(wa[m], 0), widen2(wb[m], 0), widen2(wa[m], 1),
                           widen2(wb[m], 1)};
    const uint32_t b[4] = {widen2(wa[m], 2), widen2(wb[m], 2), widen2(wa[m], 3),
                           widen2(wb[m], 3)};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float c[4];
      mma16816(c, a, xv[t].x, xv[t].y, z[t][0], z[t][1], z[t][2], z[t][3]);
      mma16816(c, b, xv[t].z, xv[t].w, c[0], c[1], c[2], c[3]);
      acc[m][t][0] = fmaf(s[2 * m], c[0], acc[m][t][0]);
      acc[m][t][1] = fmaf(s[2 * m], c[1], acc[m][t][1]);
      acc[m][t][2] = fmaf(s[2 * m + 1], c[2], acc[m][t][2]);
      acc[m][t][3] = fmaf(s[2 * m + 1], c[3], acc[m][t][3]);
    }
  }
}

// Whether the segments of more than kLongRows rows go to the many-row kernel
// (expert_w4_tile.cuh), decided alike by both kernels from the segments:
// `passes` passes of kRowsPerPass of their rows here, or `blocks` blocks there.  There a
// 128-row tile of n_out takes an SM 1.0 to 1.4 us for 128 columns, however few the
// rows of its block; here a unit and pass takes the whole GPU 1.4 to 2 ns.
// Measured (d = 7168, n_out = 2048, groups of 32, bf16 scales), here / there: 4 x 64
// rows (512 units and passes per wave of items) 64 / 71 us, 8 x 33 rows (768) 89 / 71,
// 32 x 40 rows (768) 248 / 245, 64 x 40 rows (878) 456 / 419, 4 x 128 rows (1024) 113 /
// 89, 256 x 128 rows 4.9 / 2.2 ms; groups of 128 with fp32 scales, 8 x 48 rows 87 / 71;
// d = 1408, n_out = 512, 40 x 64 rows (640) 53 / 42.
constexpr int kLongRows = 32;
__device__ __forceinline__ int passes_of(int rows) {
  return (rows + kRowsPerPass - 1) / kRowsPerPass;
}
constexpr int kTileRows = 128;     // rows per block there
constexpr int kTilePasses = 700;   // units and passes that take as long as a wave there
__device__ __forceinline__ bool long_to_tile(long passes, long blocks, int n_out, int sms) {
  const long items = blocks * ((n_out + 127) / 128);
  return passes * ((n_out + kTile - 1) / kTile) > kTilePasses * ((items + sms - 1) / sms);
}
// The sums over the CTA's threads of (passes, blocks) of their long segments
// (every thread calls it; tmp: two ints per warp).
__device__ __forceinline__ void sum_pair(int& a, int& b, int* tmp, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((threadIdx.x & 31) == 0) {
    tmp[2 * (threadIdx.x >> 5)] = a;
    tmp[2 * (threadIdx.x >> 5) + 1] = b;
  }
  __syncthreads();
  a = b = 0;
  for (int w = 0; w < warps; ++w) {
    a += tmp[2 * w];
    b += tmp[2 * w + 1];
  }
}

// What the CTA shares.
constexpr int kRedLane = 17;  // floats per lane (one more than 16: no bank conflicts)
constexpr int kRed = kWarps * 32 * kRedLane;
struct Shared {
  uint64_t bars[kWarps][kStages];
  int wsum[kWarps], pair[2 * kWarps];
  int abort;
  int* first;  // [N_r + 1] passes before expert e
  int* off;    // [N_r + 1] the experts' segments
  float* red;  // [2][kRed]
};
// Dynamic shared memory: the rings, the sums, the two arrays.
inline int smem_bytes(int unit_bytes, int N_r) {
  return kWarps * kStages * unit_bytes + 2 * kRed * 4 + 2 * (N_r + 1) * 4;
}

// A warp's walk over its units: item after item, its columns of each.
struct Walk {
  long item;
  int e, row0, rows, tile, kb;
};

// Item -> expert (the last e with first[e] <= pass), rows, tile.
__device__ __forceinline__ void find(const Params& P, const Shared& sh, Walk& k) {
  const int pass = (int)(k.item / P.tiles);
  k.tile = (int)(k.item % P.tiles);
  int lo = 0, hi = P.N_r - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh.first[mid] <= pass) lo = mid;
    else hi = mid - 1;
  }
  k.e = lo;
  k.row0 = sh.off[lo] + (pass - sh.first[lo]) * kRowsPerPass;
  k.rows = min(sh.off[lo + 1] - k.row0, kRowsPerPass);
}

template <int GROUP, typename S>
__global__ void __launch_bounds__(kThreads, 2) expert_w4_kernel(const Params P) {
  extern __shared__ __align__(128) uint8_t ring[];  // [kWarps][kStages][unit_bytes]
  __shared__ Shared sh;
  volatile int* abort = &sh.abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = P.T * P.k;
  if (tid < kWarps * kStages) mbar_init(smem_u32(&sh.bars[0][0] + tid), 1);
  if (tid == 0) {
    sh.abort = 0;
    sh.red = reinterpret_cast<float*>(ring + kWarps * kStages * P.unit_bytes);
    sh.first = reinterpret_cast<int*>(sh.red + 2 * kRed);
    sh.off = sh.first + P.N_r + 1;
  }
  __syncthreads();
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  for (int e = tid; e <= P.N_r; e += kThreads) sh.off[e] = min(max(P.offsets[e], 0), n);
  __syncthreads();
  {  // exclusive scan of the experts' passes (thread i owns experts [i c, i c + c))
    const int c = (P.N_r + kThreads - 1) / kThreads;
    const int e0 = tid * c, e1 = e0 + c < P.N_r ? e0 + c : P.N_r;
    bool without_long = false;
    if (P.tile_rows > 0) {
      int lp = 0, lb = 0;
      for (int e = e0; e < e1; ++e) {
        const int rows = sh.off[e + 1] - sh.off[e];
        if (rows > P.tile_rows) {
          lp += passes_of(rows);
          lb += (rows + kTileRows - 1) / kTileRows;
        }
      }
      sum_pair(lp, lb, sh.pair, kWarps);
      without_long = long_to_tile(lp, lb, P.n_out, P.sms);
    }
    auto passes = [&](int e) {
      const int rows = sh.off[e + 1] - sh.off[e];
      if (rows <= 0 || (without_long && rows > P.tile_rows)) return 0;
      return passes_of(rows);
    };
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += passes(e);
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.wsum[warp] = x;
    __syncthreads();
    int before = x - mine;
    for (int w = 0; w < warp; ++w) before += sh.wsum[w];
    for (int e = e0; e < e1; ++e) {
      sh.first[e] = before;
      before += passes(e);
    }
    if (e0 < P.N_r && e1 == P.N_r) sh.first[P.N_r] = before;
  }
  __syncthreads();
  const long items = (long)sh.first[P.N_r] * P.tiles;

  // Team size: a team spends about KB / ks units and two units' time of its own
  // (finding the item, the rows' first loads, the meeting) on each item, and
  // half an item is lost at the end.  Measured, ks = 8 / 4 / 2 / 1: decode batch
  // of 64 tokens (256 experts, d = 7168, 7104 items) 441 / 412 / 398 / 397 us,
  // 8 tokens (1820 items) 129 / 118 / 134 / 131 us, one token (256 items) 26 /
  // 27 / 45 / 81 us, 200 tokens on 8 experts (d = 1408, 2640 items) 88 / 71 / 66
  // / 72 us.
  int ks = kWarps;
  float best = INFINITY;
  for (int c = kWarps; c >= 1; c /= 2) {
    const float item_cost = (float)((P.KB + c - 1) / c + 2);
    const float cost = ((float)items / (float)(gridDim.x * (kWarps / c)) + 0.5f) * item_cost;
    if (cost < best) {
      best = cost;
      ks = c;
    }
  }
  const int team = warp / ks, member = warp % ks;
  const long stride = (long)gridDim.x * (kWarps / ks);
  const long item0 = (long)blockIdx.x * (kWarps / ks) + team;

  // ---- the warp's ring ---------------------------------------------------------
  uint8_t* slots = ring + warp * kStages * P.unit_bytes;
  Walk ahead;  // the next unit to request
  ahead.item = member < P.KB ? item0 : items;
  ahead.kb = member;
  const uint8_t* src = nullptr;
  const long step_bytes = (long)ks * P.unit_bytes;
  auto start = [&]() {
    if (ahead.item >= items) return;
    find(P, sh, ahead);
    src = P.wp + (((long)ahead.e * P.tiles + ahead.tile) * P.KB + member) * (long)P.unit_bytes;
  };
  start();
  int requested = 0, used = 0;
  auto request = [&]() {  // whole warp
    if (ahead.item >= items) return;
    const int s = requested % kStages;
    if (lane == 0) {
      const uint32_t bar = smem_u32(&sh.bars[warp][s]);
      mbar_arrive_expect_tx(bar, (uint32_t)P.unit_bytes);
      eg::bulk_load(smem_u32(slots + s * P.unit_bytes), src, (uint32_t)P.unit_bytes, bar);
    }
    ++requested;
    ahead.kb += ks;
    src += step_bytes;
    if (ahead.kb >= P.KB) {
      ahead.kb = member;
      ahead.item += stride;
      start();
    }
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) request();

  bool go = true;
  int par = 0;
  auto run = [&](auto nt, const Walk& k) {
    constexpr int NT = decltype(nt)::value;
    const uint4* x4[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // a lane without a row reads the item's first one; its results are dropped
      const int r = t * 8 + lane / 4;
      int tok = k.row0 + (r < k.rows ? r : 0);
      if (P.perm) {
        const int p = P.perm[tok];
        tok = p >= 0 && p < n ? p / P.k : 0;
        if (p < 0 || p >= n) mr_raise(MR_FLAG_BAD_INDEX);
      }
      x4[t] = reinterpret_cast<const uint4*>(P.x + (long)tok * P.d) + lane % 4 +
              member * (kCols / 8);
    }
    float acc[4][NT][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;
    uint4 xn[4][NT];
    if constexpr (NT == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        load_x<NT>(x4, i, member < P.KB ? P.d / 8 - member * (kCols / 8) : 0, lane, xn[i]);
    }
    for (int kb = member; kb < P.KB; kb += ks) {
      const int s = used % kStages, n8 = P.d / 8 - kb * (kCols / 8);
      const uint8_t* w = slots + s * P.unit_bytes;
      const uint32_t bar = smem_u32(&sh.bars[warp][s]), ph = (uint32_t)(used / kStages) & 1u;
      if constexpr (NT == 1) {  // x runs one unit ahead
        uint4 xc[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) xc[i][0] = xn[i][0];
        if (kb + ks < P.KB) {
          x4[0] += ks * (kCols / 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) load_x<NT>(x4, i, n8 - ks * (kCols / 8), lane, xn[i]);
        }
        go = go && __all_sync(0xffffffffu, mbar_wait(bar, ph, abort));
        if (!go) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) step<GROUP, S, NT>(w, i, lane, xc[i], acc);
      } else {  // the unit's x is on its way while the weights arrive
        uint4 xv[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_x<NT>(x4, i, n8, lane, xv[i]);
        go = go && __all_sync(0xffffffffu, mbar_wait(bar, ph, abort));
        if (!go) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) step<GROUP, S, NT>(w, i, lane, xv[i], acc);
      }
      __syncwarp();
      ++used;
      request();
      if constexpr (NT > 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          x4[t] += ks * (kCols / 8);
      }
    }
    // the team's sums meet, one tile of 8 rows of x at a time: acc 0, 1 are rows
    // 2 (lane % 4), + 1 of x against output row 16 m + lane / 4; acc 2, 3 the
    // same against 16 m + 8 + lane / 4
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float* red = sh.red + par * kRed;  // the other half is still being read
      par ^= 1;
      float* mine = red + (warp * 32 + lane) * kRedLane;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[4 * m + i] = acc[m][t][i];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * ks) : "memory");
      for (int o = member * 32 + lane; o < 8 * kTile; o += 32 * ks) {
        const int c = o / kTile, r = o % kTile;
        const float* src = red + team * ks * 32 * kRedLane + ((r % 8) * 4 + c / 2) * kRedLane + 4 * (r / 16) + (c & 1) +
                           2 * ((r / 8) & 1);
        float v = 0.0f;
        for (int w = 0; w < ks; ++w) v += src[w * 32 * kRedLane];
        const int row = t * 8 + c, col = k.tile * kTile + r;
        if (row < k.rows && col < P.n_out && !*abort) {
          const __nv_bfloat16 b = __float2bfloat16_rn(v);
          P.out[(long)(k.row0 + row) * P.n_out + col] =
              *reinterpret_cast<const uint16_t*>(&b);
        }
      }
    }
  };
  for (long it = item0; it < items; it += stride) {
    Walk k;
    k.item = it;
    find(P, sh, k);
    if (k.rows <= 8) run(std::integral_constant<int, 1>{}, k);
    else run(std::integral_constant<int, 2>{}, k);
  }
  // after a give-up: every requested copy lands before the CTA exits
  if (lane == 0)
    for (; used < requested; ++used)
      mbar_wait(smem_u32(&sh.bars[warp][used % kStages]), (uint32_t)(used / kStages) & 1u, abort,
                true);
  // a programmatic dependent of the many-row kernel, when that runs too: this
  // one's end comes after both (they share nothing but their inputs)
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace w4
}  // namespace mr

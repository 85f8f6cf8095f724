// expert_w4_tile.cuh -- the experts' products on 4-bit weights for segments of
// many rows (expert_w4.cuh has the few-row kernel, the definition and the packed
// layout).
//
// With more rows per expert the widening of the weights is worth sharing: here
// a CTA widens 128 output rows x 128 columns at a time into shared memory and
// tcgen05 multiplies them with up to 128 of the expert's rows.  Each group of
// columns has an accumulation of its own: u - 8 is exact in bf16 and so is its
// product with x in fp32, the tensor core adds a group's 2 to 8 steps of 16
// products (rounding toward zero), and the group's sum, times the scale of its
// output row, is added to fp32 registers (to nearest); the result is rounded to
// bf16 once.  One accumulation over all of d, with the scales multiplied into the
// weights, drifts toward zero with every step: 150 rows x 8 experts (d = 1408)
// differed by 1.5e-4 (2-norm of the bf16 results) from fp32 sums, 6e-5 so.
//
// tcgen05 kind::f16, M = 128 (output rows), N = 16 .. 128 (rows of x, rounded up
// to 16), stages of 128 columns (two halves of 128-byte swizzled rows), TMEM holds
// four accumulations; groups of 32 and 64 are handed over two at a time (each wait
// costs the threads that take turns about 150 cycles).
//   warp 0       TMEM owner and MMA issuer (one elected thread)
//   warp 1       packed units into a ring (bulk copies)
//   warps 2-3    rows of x, 16 bytes a copy (cp.async)
//   warps 4-7    weights: each lane widens 16 x 8 of a stage
//   warps 8-15   the groups' sums, 32 output rows and up to four times 16 rows of
//                x each; at the end -> bf16 -> out.  A lane is an output row, so a
//                group's scale is one register.
// An item is a block of up to 128 rows of a segment of more than kMinRows rows
// and a 128-row tile of n_out (none when long_to_tile says that the few-row
// kernel is faster); one CTA per SM takes items blockIdx.x, + gridDim.x,
// .. (only the device knows how many there are).  Every mbarrier wait is bounded.
//
// Measured (d = 7168, n_out = 2048): 128 rows x 256 experts 2.16 ms with groups of
// 32 (2.28 with scaled weights in two planes and one accumulation), 1.71 with
// groups of 128 (2.28); 150 rows x 8 experts (d = 1408, n_out = 2056, groups of 128,
// fp32 scales: three planes before) 32.8 us (36.9); segments of 129 to 192
// rows are two blocks here and were one, 160 rows x 64 experts 933 us (616), since
// the sums of 192 rows do not fit the registers.  With groups of 32 a stage of 128
// columns of 128 rows takes about 2250 cycles, bound by the sums' way out of TMEM: 256
// KB, two warps a lane quarter at 128 bytes a cycle in all; more warps for them
// were 1 to 7 % slower, loads of 32 columns 10 %, loads under the additions of the
// one before 5 %.  With groups of 128 it takes about 1600, bound by the two warps
// that copy x (1180 to issue, 250 for the copies to land); its MMAs take 600.
#pragma once

#include "expert_w4.cuh"

namespace mr {
namespace w4t {

using namespace mr::tc;

constexpr int kRows = w4::kTileRows;  // 128 rows of x per CTA (MMA N at most)
constexpr int kAccs = 4;              // accumulations in TMEM
constexpr int kTmem = kAccs * kRows;  // columns allocated (a power of two)
constexpr int kOut = 128;             // output rows per CTA (MMA M): two packed units
constexpr int kK = 64;                // columns of a 128-byte row
// Rings of stages of 128 columns (a packed unit): rows of x and widened weights,
// packed units (two per stage).
constexpr int kStages = 3, kUnitStages = 3;
constexpr int kCopyWarps = 2, kWidenWarps = 4, kSumWarps = 8;
constexpr int kThreads = 32 * (2 + kCopyWarps + kWidenWarps + kSumWarps);
constexpr uint32_t kWHalf = kOut * kK * 2, kWBytes = 2 * kWHalf;
constexpr uint32_t kXHalf = kRows * kK * 2, kXBytes = 2 * kXHalf;
inline uint32_t smem_bytes(int unit_bytes) {
  return kStages * (kXBytes + kWBytes) + kUnitStages * 2 * (uint32_t)unit_bytes + 1024;
}
// Segments of up to this many rows go to the few-row kernel in any case.
constexpr int kMinRows = w4::kLongRows;

struct Params {
  const uint16_t* x;
  const int32_t* perm;  // null: x holds the sorted rows
  const int32_t* offsets;
  const uint8_t* wp;
  uint16_t* out;
  int T, d, k, N_r, n_out, tiles, KB, unit_bytes, sms;
};

// Place in a ring of N stages and its parity, from the count g of stages before;
// kept incrementally (divisions in every warp and stage would cost more than
// they look).
template <int N>
struct Place {
  int s;
  uint32_t ph;
  __device__ __forceinline__ explicit Place(int g) : s(g % N), ph((uint32_t)(g / N) & 1u) {}
  __device__ __forceinline__ void step() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// u - 8 of the weight pair p of w as two bf16 values.
__device__ __forceinline__ uint32_t weight2(uint32_t w, int p) {
  const uint32_t v = w4::widen2(w, p);  // 16 + u
  const uint32_t k24 = 0x41c041c0u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&k24));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float to_f32(uint16_t s) { return mr_bf16_to_f32(s); }
__device__ __forceinline__ float to_f32(float s) { return s; }

template <int GROUP, typename S>
__global__ void __launch_bounds__(kThreads, 1) expert_w4_tile_kernel(const Params P) {
  constexpr int kUnitGroups = w4::kCols / GROUP;
  // accumulations handed over at once, such turns per stage, turns that TMEM holds
  constexpr int kBatch = GROUP == w4::kCols ? 1 : 2;
  constexpr int kTurns = kUnitGroups / kBatch, kParts = kAccs / kBatch;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t bars[2 * (kStages + kUnitStages + kParts) + 1];
  __shared__ int tok_s[kRows];
  __shared__ int wsum[kThreads / 32], pair[2 * (kThreads / 32)];
  __shared__ int found[3];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  volatile int* abort = &abort_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = P.T * P.k;
  const uint32_t smem0 = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int B_FULL = 0, B_EMPTY = kStages, B_ACCF = 2 * kStages, B_ACCE = B_ACCF + kParts,
            B_UFULL = B_ACCE + kParts, B_UEMPTY = B_UFULL + kUnitStages,
            B_DRAIN = B_UEMPTY + kUnitStages;
  // the rings: rows of x, widened weights, packed units (two per 128 columns)
  constexpr uint32_t kWAt = kStages * kXBytes, kUAt = kWAt + kStages * kWBytes;
  const uint32_t x0 = smem0, w0 = smem0 + kWAt, u0 = smem0 + kUAt;

  // ---- which segment and which block of it ---------------------------------------
  auto segment = [&](int e, int& a) {
    a = min(max(P.offsets[e], 0), n);
    const int rows = min(max(P.offsets[e + 1], 0), n) - a;
    return rows > kMinRows ? rows : 0;
  };
  // blocks of the experts [e0, e1) of this thread come after `first` others
  const int c = (P.N_r + kThreads - 1) / kThreads;
  const int e0 = min(tid * c, P.N_r), e1 = min(e0 + c, P.N_r);
  int mine = 0, first = 0, blocks_all = 0;
  {
    int a;
    int lp = 0;
    for (int e = e0; e < e1; ++e) {
      const int rows = segment(e, a);
      lp += w4::passes_of(rows);
      mine += (rows + kRows - 1) / kRows;
    }
    int lb = mine;
    w4::sum_pair(lp, lb, pair, kThreads / 32);
    if (!w4::long_to_tile(lp, lb, P.n_out, P.sms)) {
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      return;  // every thread leaves together: the few-row kernel takes them
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    first = x - mine;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) first += wsum[w];
      blocks_all += wsum[w];
    }
  }
  const int gy = (P.n_out + kOut - 1) / kOut;
  const long items = (long)blocks_all * gy;
  if ((long)blockIdx.x >= items) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    return;  // every thread leaves together
  }
  const int KB = P.KB;  // stages per item
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(B_FULL + s), 2 * kCopyWarps + kWidenWarps);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int b = 0; b < kParts; ++b) {
      mbar_init(bar(B_ACCF + b), 1);
      mbar_init(bar(B_ACCE + b), kSumWarps);
    }
    for (int s = 0; s < kUnitStages; ++s) {
      mbar_init(bar(B_UFULL + s), 1);
      mbar_init(bar(B_UEMPTY + s), kWidenWarps + kSumWarps);
    }
    mbar_init(bar(B_DRAIN), 1);
    abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int done = 0;  // items of this CTA so far: the stages run on through them
  for (long it = blockIdx.x; it < items; it += gridDim.x, ++done) {
    const int blk = (int)(it / gy), out0 = (int)(it % gy) * kOut;
    if (blk >= first && blk < first + mine) {
      int at = first, a;
      for (int e = e0; e < e1; ++e) {
        const int rows = segment(e, a), blocks = (rows + kRows - 1) / kRows;
        if (blk < at + blocks) {
          // blocks of equal size, a multiple of 16 rows
          const int i = blk - at, per = ((rows + blocks - 1) / blocks + 15) / 16 * 16;
          found[0] = e;
          found[1] = a + i * per;
          found[2] = min(rows - i * per, per);
          break;
        }
        at += blocks;
      }
    }
    __syncthreads();
    const int e = found[0], row0 = found[1], rows = found[2];
    if (tid < kRows) {
      // places past the rows load the block's first row; their results are dropped
      int tok = row0 + (tid < rows ? tid : 0);
      if (P.perm) {
        const int p = P.perm[tok];
        tok = p >= 0 && p < n ? p / P.k : 0;
        if (p < 0 || p >= n) mr_raise(MR_FLAG_BAD_INDEX);
      }
      tok_s[tid] = tok;
    }
    __syncthreads();
    const int g0 = done * KB;  // stages and pairs of units before this item's
    const int tile = out0 / w4::kTile;
    const int tiles_here = min(2, P.tiles - tile);

    if (warp == 0) {
      if (lane == 0) {
        const uint32_t idesc = make_idesc_bf16((rows + 15) / 16 * 16, kOut);
        Place<kStages> sp(g0);
        uint32_t j = (uint32_t)g0 * kTurns;  // turns before this one
        bool go = true;
        for (int kb = 0; kb < KB && go; ++kb, sp.step()) {
          if (!mbar_wait(bar(B_FULL + sp.s), sp.ph, abort)) break;
          const uint64_t da = make_desc(w0 + sp.s * kWBytes), db = make_desc(x0 + sp.s * kXBytes);
#pragma unroll
          for (int v = 0; v < kTurns; ++v, ++j) {
            const uint32_t part = j % kParts;
            // (passes at once for the first kParts)
            go = mbar_wait(bar(B_ACCE + (int)part), ((j / kParts) & 1u) ^ 1u, abort);
            if (!go) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kBatch * GROUP / 16; ++i) {
              const int kk = v * (kBatch * GROUP / 16) + i;  // 16 columns, 32 bytes of a row
              const uint32_t at = (kk / 4) * (kWHalf >> 4) + (kk % 4) * 2;
              static_assert(kWHalf == kXHalf, "one offset for both operands");
              mma_bf16(tmem_base + (part * kBatch + i / (GROUP / 16)) * kRows, da + at, db + at,
                       idesc, i % (GROUP / 16) > 0 ? 1u : 0u);
            }
            mma_commit(bar(B_ACCF + (int)part));
          }
          if (!go) break;
          mma_commit(bar(B_EMPTY + sp.s));
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---- packed units, as they lie ------------------------------------------------
      if (lane == 0) {
        const uint8_t* src = P.wp + ((long)e * P.tiles + tile) * P.KB * (long)P.unit_bytes;
        Place<kUnitStages> up(g0), last(g0);
        int issued = 0;
        for (; issued < KB; ++issued, up.step()) {
          if (!mbar_wait(bar(B_UEMPTY + up.s), up.ph ^ 1u, abort)) break;
          const uint32_t full = bar(B_UFULL + up.s);
          mbar_arrive_expect_tx(full, (uint32_t)(tiles_here * P.unit_bytes));
          for (int u = 0; u < tiles_here; ++u)
            eg::bulk_load(u0 + (uint32_t)((2 * up.s + u) * P.unit_bytes),
                          src + ((long)u * P.KB + issued) * P.unit_bytes, (uint32_t)P.unit_bytes,
                          full);
        }
        // after a give-up: every copy lands before the CTA exits
        for (int i = 0; i < issued; ++i, last.step())
          if (i >= issued - kUnitStages) mbar_wait(bar(B_UFULL + last.s), last.ph, abort, true);
      }
      __syncwarp();
    } else if (warp < 2 + kCopyWarps) {
      // ---- rows of x: copy i of half a stage (ct + 64 u): row i / 8, chunk i % 8 -----
      const int ct = tid - 64;
      constexpr int kLag = 2;  // halves of a stage on their way
      auto hand_over = [&](int st) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLag - 1) : "memory");
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_FULL + st));
      };
      bool go = true;
      // this thread's copies: rows r0 + 8 u, 16-byte chunk c
      const int r0 = ct >> 3, c = ct & 7, n_rows = (rows + 15) / 16 * 16;
      const uint32_t dst0 = (uint32_t)r0 * 128u + ((uint32_t)(c ^ (r0 & 7)) << 4);
      constexpr int kCopies = kRows / 8;  // 8 rows of 8 chunks per round
      static_assert(32 * kCopyWarps == 8 * 8, "a round copies 8 rows");
      const uint16_t* from[kCopies];
#pragma unroll
      for (int u = 0; u < kCopies; ++u) from[u] = P.x + (long)tok_s[r0 + 8 * u] * P.d + c * 8;
      Place<kStages> xp(g0), lag(g0);
      for (int kc = 0; kc < 2 * KB; ++kc) {
        if (kc >= kLag) {
          hand_over(lag.s);
          if (kc & 1) lag.step();
        }
        if (!(kc & 1)) {
          if (kc > 0) xp.step();
          go = __all_sync(0xffffffffu, mbar_wait(bar(B_EMPTY + xp.s), xp.ph ^ 1u, abort));
          if (!go) break;
        }
        const uint32_t base = x0 + xp.s * kXBytes + (kc & 1) * kXHalf + dst0;
        const int col = kc * kK + c * 8;
        // columns past d: zeros (nothing is read)
        const uint32_t bytes = col < P.d ? 16u : 0u;
        const int at = col < P.d ? kc * kK : 0;
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          if (8 * u >= n_rows) break;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + u * 1024),
                       "l"(from[u] + at), "r"(bytes)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async();
      __syncwarp();
      static_assert(kLag == 2, "the last stage's halves are left");
      if (go && lane == 0) {
        mbar_arrive(bar(B_FULL + lag.s));
        mbar_arrive(bar(B_FULL + lag.s));
      }
    } else if (warp < 2 + kCopyWarps + kWidenWarps) {
      // ---- weights: unit u2 of the two, half h, every m and step ---------------------
      const int wd = warp - 2 - kCopyWarps;
      const int u2 = wd >> 1, h = wd & 1;
      const bool here = u2 < tiles_here;
      // Rows of even and odd l / 4 store the two steps in opposite order, so that a
      // quarter warp's 16-byte stores (two rows) fall on distinct banks.
      const int odd = (lane / 4) & 1;
      const uint32_t row = (uint32_t)(u2 * 64 + 8 * h + lane / 4);
      Place<kStages> wp(g0);
      Place<kUnitStages> up(g0);
      bool go;
      for (int kb = 0; kb < KB; ++kb, wp.step(), up.step()) {
        go = __all_sync(0xffffffffu, mbar_wait(bar(B_UFULL + up.s), up.ph, abort)) &&
             __all_sync(0xffffffffu, mbar_wait(bar(B_EMPTY + wp.s), wp.ph ^ 1u, abort));
        if (!go) break;
        if (here) {
          const uint8_t* unit =
              smem + kUAt + (uint32_t)((2 * up.s + u2) * P.unit_bytes) + 512 * h + 16 * lane;
          uint8_t* a = smem + kWAt + wp.s * kWBytes + row * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // half i / 2 of the stage
            const int step = i ^ odd;
            const uint4 w = *reinterpret_cast<const uint4*>(unit + 1024 * step);
            const uint32_t c = (uint32_t)((step & 1) * 4 + lane % 4) ^ (row & 7);
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int m = 0; m < 4; ++m)  // output rows row + 16 m, r % 8 the same
              *reinterpret_cast<uint4*>(a + (i / 2) * kWHalf + m * 2048 + (c << 4)) =
                  make_uint4(weight2(words[m], 0), weight2(words[m], 1), weight2(words[m], 2),
                             weight2(words[m], 3));
          }
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_FULL + wp.s));
          mbar_arrive(bar(B_UEMPTY + up.s));
        }
      }
    } else {
      // ---- sums: TMEM lane = output row, column = row of x; this warp's columns are
      // 16 at a time, chunk wj + kStep i of them -----------------------------------------
      constexpr int kStep = kSumWarps / 4, kChunks = kRows / 16 / kStep;
      const int q = warp & 3, wj = (warp - 2 - kCopyWarps - kWidenWarps) >> 2;
      const int n16 = (rows + 15) / 16;
      const uint32_t lane_off = (uint32_t)(q * 32) << 16;
      const bool here = (q >> 1) < tiles_here;
      const int ru = (q & 1) * 32 + lane;  // row of the unit
      const uint8_t* scales = smem + kUAt + (uint32_t)((q >> 1) * P.unit_bytes) +
                              w4::kWeightBytes +
                              ((ru & 7) * 8 + (ru >> 4) * 2 + ((ru >> 3) & 1)) * (int)sizeof(S);
      float acc[kChunks][16];
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[i][c] = 0.0f;
      uint32_t j = (uint32_t)g0 * kTurns;
      // the scales of the next unit: its place in the ring is free early
      Place<kUnitStages> up(g0);
      S next[kUnitGroups];
      bool go;
      auto fetch = [&]() {
        go = __all_sync(0xffffffffu, mbar_wait(bar(B_UFULL + up.s), up.ph, abort));
#pragma unroll
        for (int i = 0; i < kUnitGroups; ++i)
          next[i] = here && go ? *reinterpret_cast<const S*>(scales + 2 * up.s * P.unit_bytes +
                                                             64 * i * sizeof(S))
                               : S{};
        __syncwarp();
        if (go && lane == 0) mbar_arrive(bar(B_UEMPTY + up.s));
        up.step();
        return go;
      };
      fetch();
      for (int kb = 0; kb < KB && go; ++kb) {
        float s[kUnitGroups];
#pragma unroll
        for (int i = 0; i < kUnitGroups; ++i) s[i] = to_f32(next[i]);
        if (kb + 1 < KB && !fetch()) break;
#pragma unroll
        for (int v = 0; v < kTurns; ++v, ++j) {
          const uint32_t part = j % kParts;
          go = __all_sync(0xffffffffu,
                          mbar_wait(bar(B_ACCF + (int)part), (j / kParts) & 1u, abort));
          if (!go) break;
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
              if (wj + kStep * i >= n16) break;
              float t[16];
              tmem_ld16(tmem_base + lane_off + (part * kBatch + b) * kRows + (wj + kStep * i) * 16,
                        t);
#pragma unroll
              for (int c = 0; c < 16; c += 2)
                fma2(acc[i][c], acc[i][c + 1], s[v * kBatch + b], t[c], t[c + 1]);
            }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_ACCE + (int)part));
        }
        if (!go) break;
      }
      const int col = out0 + q * 32 + lane;
      if (go && col < P.n_out) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int r = (wj + kStep * i) * 16 + c;
            if (r >= rows) break;
            const __nv_bfloat16 b = __float2bfloat16_rn(acc[i][c]);
            P.out[(long)(row0 + r) * P.n_out + col] = *reinterpret_cast<const uint16_t*>(&b);
          }
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();  // the sums are done, every stage consumed
    tc_fence_after();
    if (*abort) break;
  }
  if (warp == 0) {
    if (lane == 0) {  // after a give-up: every MMA issued is done before TMEM is released
      mma_commit(bar(B_DRAIN));
      mbar_wait(bar(B_DRAIN), 0, abort, true);
    }
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmem)
                 : "memory");
  }
}

}  // namespace w4t
}  // namespace mr

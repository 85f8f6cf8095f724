// expert_w4_tile.cuh -- the experts' products on 4-bit weights for segments of
// many rows (expert_w4.cuh has the few-row kernel, the definition and the packed
// layout).
//
// With more rows per expert the widening of the weights is worth sharing: here
// a CTA widens 128 output rows x 64 columns at a time into shared memory and
// tcgen05 multiplies them with up to 192 of the expert's rows.  The group scale
// is applied to the weight, without loss: a bf16 scale (8 significant bits)
// times an integer in [-8, 7] has at most 12, so the product is the sum of two
// bf16 planes, hi = bf16(s q) and lo = s q - hi (one multiply and one fused
// multiply-add per pair); with fp32 scales the fp32 product is split into three.
// Each plane times bf16 x is exact in fp32, the tensor core adds in fp32, and
// the result is rounded to bf16 once.
//
// tcgen05 kind::f16, M = 128 (output rows), N = 16 .. 192 (rows of x, rounded up
// to 16), K staged 64 at a time (128-byte swizzled rows).  The rows of x and the
// widened weights have rings of their own.
//   warp 0       TMEM owner and MMA issuer (one elected thread)
//   warps 1-4    rows of x, 16 bytes a copy (cp.async); at the end TMEM -> bf16
//                -> out
//   warps 5-20   weights: two sets of eight warps take the stages in turn; each
//                lane widens 4 x 8 weights, the words and scales of its set's
//                next three stages already on their way
// An item is a block of up to 192 rows of a segment of more than kMinRows rows
// and a 128-row tile of n_out (none when long_to_tile says that the few-row
// kernel is faster); one CTA per SM takes items blockIdx.x, + gridDim.x,
// .. (only the device knows how many there are).  Every mbarrier wait is bounded.
//
// Shared memory bounds it: at 128 rows a stage writes 32 KB of widened weights
// (two planes) and 16 KB of x, and its MMAs read 64 KB, about 900 of the 1150
// cycles it takes; the widening itself is hidden (sixteen warps).  One block for
// a segment where blocks of 128 rows would widen its weights twice.  Measured:
// 150 rows x 8 experts (d = 1408, n_out = 2056, fp32 scales) 67 us with blocks of
// 128 rows, eight warps and a CTA for every block there might be, 37 us so; 128
// rows x 256 experts (d = 7168, n_out = 2048) 2.6 ms with the rows' addresses
// formed for every copy, 2.3 ms so; eight or twelve copy warps 2.4 and 2.6 ms.
#pragma once

#include <type_traits>

#include "expert_w4.cuh"

namespace mr {
namespace w4t {

using namespace mr::tc;

constexpr int kRows = w4::kTileRows;  // 192 rows of x per CTA (MMA N at most)
constexpr int kTmem = 256;       // columns allocated (a power of two)
constexpr int kOut = 128;        // output rows per CTA (MMA M): two packed units
constexpr int kK = 64;           // columns per stage
constexpr int kXStages = 5;      // stages of x
constexpr int kCopyWarps = 4, kWidenWarps = 8, kWidenSets = 2;
constexpr int kThreads = 32 * (1 + kCopyWarps + kWidenSets * kWidenWarps);
constexpr uint32_t kPlane = kOut * kK * 2;
constexpr uint32_t kXBytes = kRows * kK * 2;
// Segments of up to this many rows go to the few-row kernel in any case.
constexpr int kMinRows = w4::kLongRows;

// Stages of widened weights: what the x ring leaves, three of two planes or two
// of three.
__host__ __device__ constexpr int w_stages(int planes) { return planes == 2 ? 3 : 2; }
__host__ __device__ constexpr uint32_t smem_bytes(int planes) {
  return kXStages * kXBytes + w_stages(planes) * planes * kPlane + 1024;
}

struct Params {
  const uint16_t* x;
  const int32_t* perm;  // null: x holds the sorted rows
  const int32_t* offsets;
  const uint8_t* wp;
  uint16_t* out;
  int T, d, k, N_r, n_out, tiles, KB, unit_bytes, sms;
};

// Place in a ring of N stages and its parity, from the count g of stages before;
// kept incrementally (divisions in every warp and stage cost as much as the
// widening).
template <int N>
struct Place {
  int s;
  uint32_t ph;
  __device__ __forceinline__ explicit Place(int g) : s(g % N), ph((uint32_t)(g / N) & 1u) {}
  __device__ __forceinline__ void step(int by = 1) {
    s += by;
    if (s >= N) {
      s -= N;
      ph ^= 1u;
    }
  }
};

// (u - 8) of the weight pair p of w as two bf16 values.
__device__ __forceinline__ __nv_bfloat162 weight2(uint32_t w, int p) {
  const uint32_t v = w4::widen2(w, p);  // 16 + u
  const uint32_t k24 = 0x41c041c0u;
  return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                 *reinterpret_cast<const __nv_bfloat162*>(&k24));
}
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}

// Planes of s times a weight pair.
__device__ __forceinline__ void planes2(__nv_bfloat162 q, uint16_t s, uint32_t (&o)[2]) {
  const uint32_t d = (uint32_t)s | ((uint32_t)s << 16);
  const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&d);
  const __nv_bfloat162 hi = __hmul2(q, s2);
  o[0] = bits(hi);
  o[1] = bits(__hfma2(q, s2, __hneg2(hi)));
}
__device__ __forceinline__ void planes2(__nv_bfloat162 q, float s, uint32_t (&o)[3]) {
  const uint32_t u = bits(q);
  float a = s * __uint_as_float(u << 16), b = s * __uint_as_float(u & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < 3; ++i) {  // pairs at a time: packed conversions
    o[i] = bits(__floats2bfloat162_rn(a, b));
    a -= __uint_as_float(o[i] << 16);
    b -= __uint_as_float(o[i] & 0xffff0000u);
  }
}

template <int GROUP, typename S>
__global__ void __launch_bounds__(kThreads, 1) expert_w4_tile_kernel(const Params P) {
  constexpr int NP = sizeof(S) == 2 ? 2 : 3;
  constexpr int kWStages = w_stages(NP);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t bars[2 * kXStages + 2 * kWStages + 1];
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
  const int B_XFULL = 0, B_XEMPTY = kXStages, B_WFULL = 2 * kXStages,
            B_WEMPTY = 2 * kXStages + kWStages, B_ACC = 2 * kXStages + 2 * kWStages;
  const uint32_t x0 = smem0, w0 = smem0 + kXStages * kXBytes;  // the rings

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
      lp += (rows + 15) / 16;
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
  const int KC = (P.d + kK - 1) / kK;
  if (tid == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(bar(B_XFULL + s), kCopyWarps);
      mbar_init(bar(B_XEMPTY + s), 1);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(bar(B_WFULL + s), kWidenWarps);
      mbar_init(bar(B_WEMPTY + s), 1);
    }
    mbar_init(bar(B_ACC), 1);
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
    const int g0 = done * KC;  // stages before this item's

    if (warp == 0) {
      if (lane == 0) {
        const uint32_t idesc = make_idesc_bf16((rows + 15) / 16 * 16, kOut);
        Place<kXStages> xp(g0);
        Place<kWStages> wp(g0);
        for (int kc = 0; kc < KC; ++kc, xp.step(), wp.step()) {
          if (!mbar_wait(bar(B_XFULL + xp.s), xp.ph, abort)) break;
          if (!mbar_wait(bar(B_WFULL + wp.s), wp.ph, abort)) break;
          tc_fence_after();
          const uint32_t a = w0 + wp.s * NP * kPlane, b = x0 + xp.s * kXBytes;
#pragma unroll
          for (int kk = 0; kk < kK / 16; ++kk)
#pragma unroll
            for (int p = NP - 1; p >= 0; --p)  // the small plane first
              mma_bf16(tmem_base, make_desc(a + p * kPlane + kk * 32), make_desc(b + kk * 32),
                       idesc, (kc > 0 || kk > 0 || p < NP - 1) ? 1u : 0u);
          mma_commit(bar(B_XEMPTY + xp.s));
          mma_commit(bar(B_WEMPTY + wp.s));
        }
        // also after an abort: every MMA is done before TMEM is read or freed
        mma_commit(bar(B_ACC));
      }
      __syncwarp();
    } else if (warp <= kCopyWarps) {
      // ---- rows of x: copy i of a stage (ct + 128 u): row i / 8, 16-byte chunk i % 8 --
      const int ct = tid - 32;
      constexpr int kLag = kXStages - 1;
      auto hand_over = [&](int st) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLag - 1) : "memory");
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_XFULL + st));
      };
      bool go = true;
      // this thread's copies of a stage: rows r0 + 16 u, 16-byte chunk c
      const int r0 = ct >> 3, c = ct & 7, n_rows = (rows + 15) / 16 * 16;
      const uint32_t dst0 = (uint32_t)r0 * 128u + ((uint32_t)(c ^ (r0 & 7)) << 4);
      constexpr int kCopies = kRows / 16;  // 16 rows of 8 chunks per round
      static_assert(32 * kCopyWarps == 16 * 8, "a round copies 16 rows");
      const uint16_t* from[kCopies];
#pragma unroll
      for (int u = 0; u < kCopies; ++u) from[u] = P.x + (long)tok_s[r0 + 16 * u] * P.d + c * 8;
      Place<kXStages> xp(g0), lag(g0);
      for (int kc = 0; kc < KC; ++kc, xp.step()) {
        if (kc >= kLag) {
          hand_over(lag.s);
          lag.step();
        }
        if (g0 + kc >= kXStages) {
          go = __all_sync(0xffffffffu, mbar_wait(bar(B_XEMPTY + xp.s), xp.ph ^ 1u, abort));
          if (!go) break;
        }
        const uint32_t base = x0 + xp.s * kXBytes + dst0;
        const int col = kc * kK + c * 8;
        // columns past d: zeros (nothing is read)
        const uint32_t bytes = col < P.d ? 16u : 0u;
        const int at = col < P.d ? kc * kK : 0;
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          if (16 * u >= n_rows) break;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + u * 2048),
                       "l"(from[u] + at), "r"(bytes)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async();
      __syncwarp();
      if (go && lane == 0)
        for (int kc = KC - kLag < 0 ? 0 : KC - kLag; kc < KC; ++kc, lag.step())
          mbar_arrive(bar(B_XFULL + lag.s));
      // ---- TMEM lane = output row, column = row of x ------------------------------
      const int q = warp & 3;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(B_ACC), (uint32_t)done & 1u, abort, true)) &&
                      !*abort;
      tc_fence_after();
      const int col = out0 + q * 32 + lane;
      for (int c0 = 0; c0 < rows; c0 += 16) {
        float v[16];
        __syncwarp();
        tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);  // whole warp
        if (ok && col < P.n_out) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c0 + i >= rows) break;
            const __nv_bfloat16 b = __float2bfloat16_rn(v[i]);
            P.out[(long)(row0 + c0 + i) * P.n_out + col] =
                *reinterpret_cast<const uint16_t*>(&b);
          }
        }
      }
    } else {
      // ---- weights: unit u2 of the two, half h, m = 2 mh and 2 mh + 1, both steps --
      const int wd = (warp - 1 - kCopyWarps) % kWidenWarps;
      const int set = (warp - 1 - kCopyWarps) / kWidenWarps;
      const int u2 = wd >> 2, h = (wd >> 1) & 1, mh = wd & 1;
      const int tile = out0 / w4::kTile + u2;
      const bool here = tile < P.tiles;
      const uint8_t* src =
          P.wp + ((long)e * P.tiles + (here ? tile : 0)) * P.KB * (long)P.unit_bytes;
      // the words and the scales (m, then h; as loaded) of the next kAhead stages;
      // each buffer is loaded again as soon as it has been read (moving them up
      // would wait for the newest)
      using Sc = typename std::conditional<sizeof(S) == 2, uint2, uint4>::type;
      constexpr int kAhead = 3;
      uint2 w[kAhead][2];
      Sc sc[kAhead][2];
      auto fetch = [&](int kc, int b) {
        if (!here || kc >= KC) return;
        const uint8_t* unit = src + (long)(kc >> 1) * P.unit_bytes;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = (kc & 1) * 2 + j;
          w[b][j] =
              __ldg(reinterpret_cast<const uint2*>(unit + 1024 * i + 512 * h + 16 * lane) + mh);
          sc[b][j] = __ldg(reinterpret_cast<const Sc*>(unit + w4::kWeightBytes) +
                           ((i * 32 / GROUP) * 8 + lane / 4) * 2 + mh);
        }
      };
      // Rows of even and odd l / 4 store the two steps in opposite order, so that a
      // quarter warp's 16-byte stores (two rows) fall on distinct banks.
      const bool odd = (lane / 4) & 1;
      const uint32_t row = (uint32_t)(u2 * 64 + mh * 32 + 8 * h + lane / 4);
#pragma unroll
      for (int b = 0; b < kAhead; ++b) fetch(set + b * kWidenSets, b);
      Place<kWStages> wp(g0 + set);
      auto widen = [&](int kc, int b) {  // false: a wait gave up
        uint2 wc[2];
        Sc scc[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          wc[j] = odd ? w[b][1 - j] : w[b][j];
          scc[j] = odd ? sc[b][1 - j] : sc[b][j];
        }
        fetch(kc + kAhead * kWidenSets, b);
        if (g0 + kc >= kWStages &&
            !__all_sync(0xffffffffu, mbar_wait(bar(B_WEMPTY + wp.s), wp.ph ^ 1u, abort)))
          return false;
        if (here) {
          uint8_t* a = smem + kXStages * kXBytes + wp.s * NP * kPlane + row * 128;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t c = (uint32_t)((j ^ (int)odd) * 4 + lane % 4);
#pragma unroll
            for (int m = 0; m < 2; ++m) {  // output rows row + 16 m, r % 8 the same
              S sv;
              if constexpr (sizeof(S) == 2)
                sv = (uint16_t)(h ? (m ? scc[j].y : scc[j].x) >> 16
                                  : (m ? scc[j].y : scc[j].x) & 0xffffu);
              else
                sv = __uint_as_float(h ? (m ? scc[j].w : scc[j].y) : (m ? scc[j].z : scc[j].x));
              uint32_t o[4][NP];
#pragma unroll
              for (int p = 0; p < 4; ++p)
                planes2(weight2(m ? wc[j].y : wc[j].x, p), sv, o[p]);
#pragma unroll
              for (int pl = 0; pl < NP; ++pl)
                *reinterpret_cast<uint4*>(a + pl * kPlane + m * 2048 + ((c ^ (row & 7)) << 4)) =
                    make_uint4(o[0][pl], o[1][pl], o[2][pl], o[3][pl]);
            }
          }
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_WFULL + wp.s));
        wp.step(kWidenSets);
        return true;
      };
      bool go = true;
      for (int kc = set; kc < KC && go; kc += kAhead * kWidenSets) {
#pragma unroll
        for (int b = 0; b < kAhead; ++b)
          if (go && kc + b * kWidenSets < KC) go = widen(kc + b * kWidenSets, b);
      }
    }
    tc_fence_before();
    __syncthreads();  // the accumulator has been read, every stage consumed
    tc_fence_after();
    if (*abort) break;
  }
  if (warp == 0) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmem)
                 : "memory");
  }
}

}  // namespace w4t
}  // namespace mr

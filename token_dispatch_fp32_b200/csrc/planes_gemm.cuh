// planes_gemm.cuh -- the gate gradient's dense products on the 5th-generation
// tensor cores, with fp32 operands given as bf16 planes.
//
//   dx = dL . W   [T, d],   K = N_r:  A = dL [T, N_r], B = W [N_r, d]
//   dW = dL^T . x [N_r, d], K = T:    A = dL [T, N_r], B = x [T, d]
//
// An fp32 value is the sum of three bf16 planes (split3), a bf16 one its own
// plane.  Products of planes are exact in fp32; those of order 2^-27 and below
// are left out: planes (pa, pb) with pa + pb <= 2, i.e. six products for dx
// with fp32 W, three for bf16 W and for dW of bf16 rows.
//
// tcgen05 kind::f16, M = 128, N = 256, K staged 32 at a time by TMA.  B lies in
// memory with its columns contiguous, so it is an MN-major operand (64-column
// boxes, 128-byte swizzle); so is A for dW (its rows are dL's columns), while
// for dx A is K-major (64-byte swizzle).  No operand is transposed in memory.
//   warp 0      TMA producer
//   warp 1      TMEM owner and MMA issuer (one elected thread)
//   warps 2..9  workers: after every 128 K they add the finished accumulator to
//               fp32 registers (the tensor core rounds toward zero; two TMEM
//               buffers alternate), and write the tile at its end.
// Persistent: CTA i takes the tiles i, i + gridDim.x, ..; the producer and the
// MMA run on into the next tile while the workers write one.  dW may split K
// (P.splits slices, summed in order afterwards).  Every mbarrier wait is
// bounded.  Measured at T = 4096, d = 7168, N_r = 256: dx 86 us (six products, 1.05
// PFLOP/s issued), dW 53 us (three, 0.85 PFLOP/s: 53 bytes a cycle and SM of
// operands through L2); fp32 on the CUDA cores took 547 and 643 us.
#pragma once

#include "router_tc.cuh"

namespace mr {
namespace pg {

using namespace mr::tc;

constexpr int kBN = 256;       // columns per tile
constexpr int kBK = 32;        // K per stage
constexpr int kInterval = 4;   // stages per accumulation interval (128 K)
constexpr uint32_t kABytes = 3 * BM * kBK * 2;
constexpr uint32_t kPlaneBytes = kBN * kBK * 2;

__host__ __device__ constexpr uint32_t stage_bytes(int npb) { return kABytes + npb * kPlaneBytes; }
__host__ __device__ constexpr int num_stages(int npb) {
  return (int)((kSmemBudget - 2048) / stage_bytes(npb));
}
__host__ __device__ constexpr uint32_t smem_bytes(int npb) {
  return num_stages(npb) * stage_bytes(npb) + 1024;
}

struct GemmParams {
  int M, N, K;             // rows and columns of the result, reduction length
  int m_tiles, n_tiles, splits;
  const void* add;         // dx: [M, N] of the output's type, or null (may be out)
  void* out;               // dx: bf16 or fp32 [M, N]; dW: fp32 [splits][M][N]
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// MN-major operand, 128-byte swizzle: 64 elements along M or N are 128
// contiguous bytes, one K per 128-byte row; the next 8 K are 1024 bytes on
// (stride offset), the next 64 elements kBK rows on (leading offset).
__device__ __forceinline__ uint64_t make_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((kBK * 128u) >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// DW: dW = dL^T . x (A MN-major), else dx = dL . W (A K-major).  NPB: planes of B.
template <bool DW, int NPB, bool OBF16>
__global__ void __launch_bounds__(kThreads, 1)
    planes_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const GemmParams P) {
  constexpr int STAGES = num_stages(NPB);
  constexpr uint32_t kStage = stage_bytes(NPB);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t bars[2 * STAGES + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  volatile int* abort = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem0 = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int B_FULL = 0, B_EMPTY = STAGES, B_ACCF = 2 * STAGES, B_ACCE = 2 * STAGES + 2,
            B_DRAIN = 2 * STAGES + 4;
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B_ACCF + b), 1);
      mbar_init(bar(B_ACCE + b), kWorkers);
    }
    mbar_init(bar(B_DRAIN), 1);
    abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(2 * kBN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  // a programmatic dependent of the kernel before it: the set-up above runs
  // while that one ends
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int KC = (P.K + kBK - 1) / kBK;
  const int items = P.m_tiles * P.n_tiles * P.splits;
  // tiles that share B run at the same time (m fastest)
  auto locate = [&](int it, int& m0, int& n0, int& z, int& k0, int& k1) {
    m0 = it % P.m_tiles * BM;
    const int r = it / P.m_tiles;
    n0 = r % P.n_tiles * kBN;
    z = r / P.n_tiles;
    k0 = (int)((long)KC * z / P.splits);
    k1 = (int)((long)KC * (z + 1) / P.splits);
  };

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long issued = 0;
      bool go = true;
      for (int it = blockIdx.x; it < items && go; it += gridDim.x) {
        int m0, n0, z, k0, k1;
        locate(it, m0, n0, z, k0, k1);
        for (int kc = k0; kc < k1; ++kc, (++s == STAGES ? (s = 0, ph ^= 1u) : 0u)) {
          if (issued >= STAGES && !mbar_wait(bar(B_EMPTY + s), ph ^ 1u, abort)) {
            go = false;
            break;
          }
          const uint32_t a = smem0 + s * kStage, b = a + kABytes, full = bar(B_FULL + s);
          mbar_arrive_expect_tx(full, kStage);
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            if constexpr (DW) {
              tma_load_3d(a + p * (BM * kBK * 2), &map_a, full, m0, kc * kBK, p);
              tma_load_3d(a + p * (BM * kBK * 2) + kBK * 128, &map_a, full, m0 + 64, kc * kBK, p);
            } else {
              tma_load_3d(a + p * (BM * kBK * 2), &map_a, full, kc * kBK, m0, p);
            }
          }
#pragma unroll
          for (int p = 0; p < NPB; ++p)
#pragma unroll
            for (int g = 0; g < kBN / 64; ++g)
              tma_load_3d(b + p * kPlaneBytes + g * kBK * 128, &map_b, full, n0 + 64 * g,
                          kc * kBK, p);
          ++issued;
        }
      }
      // every copy this CTA issued lands before the CTA may exit
      for (long i = issued - STAGES < 0 ? 0 : issued - STAGES; i < issued; ++i)
        mbar_wait(bar(B_FULL + (int)(i % STAGES)), (uint32_t)((i / STAGES) & 1), abort, true);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // A K-major or MN-major (bit 15), B MN-major (bit 16)
      const uint32_t idesc = make_idesc_bf16(kBN, BM) | (DW ? 1u << 15 : 0u) | (1u << 16);
      int s = 0;
      uint32_t ph = 0;
      long j = 0;
      bool go = true;
      for (int it = blockIdx.x; it < items && go; it += gridDim.x) {
        int m0, n0, z, k0, k1;
        locate(it, m0, n0, z, k0, k1);
        for (int kc = k0; kc < k1; ++kc, (++s == STAGES ? (s = 0, ph ^= 1u) : 0u)) {
          const bool first = (kc - k0) % kInterval == 0;
          const int buf = (int)(j & 1);
          if (first && j >= 2 &&
              !mbar_wait(bar(B_ACCE + buf), (uint32_t)(((j >> 1) - 1) & 1), abort)) {
            go = false;
            break;
          }
          if (!mbar_wait(bar(B_FULL + s), ph, abort)) {
            go = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem0 + s * kStage, b = a + kABytes;
          const uint32_t dt = tmem_base + (uint32_t)(buf * kBN);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
#pragma unroll
            for (int pa = 2; pa >= 0; --pa)  // the small products first
#pragma unroll
              for (int pb = 0; pb < NPB; ++pb) {
                if (pa + pb > 2) continue;
                const uint32_t ap = a + pa * (BM * kBK * 2);
                const uint64_t da =
                    DW ? make_desc_mn(ap + kk * 2048) : make_desc_sw64(ap + kk * 32);
                const uint64_t db = make_desc_mn(b + pb * kPlaneBytes + kk * 2048);
                mma_bf16(dt, da, db, idesc, (!first || kk > 0 || pa < 2) ? 1u : 0u);
              }
          mma_commit(bar(B_EMPTY + s));
          if ((kc - k0) % kInterval == kInterval - 1 || kc == k1 - 1) {
            mma_commit(bar(B_ACCF + buf));
            ++j;
          }
        }
      }
      // every MMA issued so far has completed before TMEM is released
      mma_commit(bar(B_DRAIN));
      mbar_wait(bar(B_DRAIN), 0, abort, true);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    long j = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      int m0, n0, z, k0, k1;
      locate(it, m0, n0, z, k0, k1);
      float acc[8][16];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[i][c] = 0.0f;
      const int intervals = (k1 - k0 + kInterval - 1) / kInterval;
      for (int v = 0; v < intervals; ++v, ++j) {
        const int buf = (int)(j & 1);
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_ACCF + buf), (uint32_t)((j >> 1) & 1), abort));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float v0[16], v1[16];
          const uint32_t ta = tmem_base + lane_off + (uint32_t)(buf * kBN + h * 128 + i * 16);
          tmem_ld16x2(ta, ta + 16, v0, v1);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            acc[i][c] += v0[c];
            acc[i + 1][c] += v1[c];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_ACCE + buf));
      }
      const int row = m0 + q * 32 + lane;
      if (!ok || row >= P.M) continue;
      const long base = ((DW ? (long)z * P.M : 0) + row) * P.N;
#pragma unroll
      for (int i = 0; i < 16; ++i) {  // eight columns at a time (N is a multiple of 8)
        const int col = n0 + h * 128 + i * 8;
        if (col >= P.N) break;
        float f[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = acc[i / 2][(i % 2) * 8 + c];
        if constexpr (OBF16) {
          if (P.add) {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.add) +
                                                            base + col);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              f[2 * c] += __uint_as_float(w[c] << 16);
              f[2 * c + 1] += __uint_as_float(w[c] & 0xffff0000u);
            }
          }
          uint32_t o[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * c], f[2 * c + 1]);
            o[c] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + base + col) =
              make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          if (P.add) {
            const float* a = static_cast<const float*>(P.add) + base + col;
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] += a[c];
          }
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(P.out) + base + col);
          o[0] = make_float4(f[0], f[1], f[2], f[3]);
          o[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(2 * kBN)
                 : "memory");
  }
}

}  // namespace pg
}  // namespace mr

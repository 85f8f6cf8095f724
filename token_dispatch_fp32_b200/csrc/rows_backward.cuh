// rows_backward.cuh -- gradients of the row movers (gather.cuh, combine.cuh).
//
// combine, forward: y[t] = sum_j w[t,j] * E[r] + shared[t], r = inv[t*k + j]
// (Kimi K2 "Add shared output" page: new_x[idxs] = outs, weighted sum over k,
// y + shared).  The two roundings of y pass a gradient through unchanged:
//   dE[r]   = w[t,j] * dy[t]          (rounded once to the row dtype)
//   dw[t,j] = sum_c dy[t,c] * E[r,c]  (fp32)
//   dshared = dy.
// gather, forward: xs[r] = x[t] for the k rows r of token t, hence
//   dx[t] = sum_j dxs[inv[t*k + j]] (+ add[t])   (fp32, rounded once).
//
// Both are bound by HBM (at most 3 flops per element moved): combine_backward
// reads dy once and each expert row once and writes each expert row's gradient
// once.  One CTA per token, so dy stays in registers for the k rows and the k
// dot products meet inside the CTA in a fixed order: no atomics, the result
// does not change from run to run.  Measured on the full DeepSeek-V3 batch (16384
// tokens, d = 7168, k = 8, bf16, skewed): combine_backward 595 us, 6.7 TB/s;
// gather_backward with add 339 us, 6.9 TB/s (the copy rate of the GPU is 6.57).
#pragma once

#include "combine.cuh"
#include "rows_common.cuh"

namespace mr {

// A vector of a row as fp32 values: bf16 pairs per word (BF16) or one fp32
// per word.
template <typename V, bool BF16>
struct RowVec {
  static constexpr int kWords = (int)(sizeof(V) / 4);
  static constexpr int kElems = BF16 ? 2 * kWords : kWords;
  static __device__ __forceinline__ void unpack(const V& v, float (&f)[kElems]) {
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
      if constexpr (BF16) bf16x2_unpack(word(v, q), f[2 * q], f[2 * q + 1]);
      else f[q] = __uint_as_float(word(v, q));
    }
  }
  static __device__ __forceinline__ V pack(const float (&f)[kElems]) {
    V v;
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
      if constexpr (BF16) set_word(v, q, bf16x2_pack_rn(f[2 * q], f[2 * q + 1]));
      else set_word(v, q, __float_as_uint(f[q]));
    }
    return v;
  }
};
// One element per step, for rows that no vector width fits.
template <>
struct RowVec<uint16_t, true> {
  static constexpr int kElems = 1;
  static __device__ __forceinline__ void unpack(const uint16_t& v, float (&f)[1]) {
    f[0] = mr_bf16_to_f32(v);
  }
  static __device__ __forceinline__ uint16_t pack(const float (&f)[1]) {
    const __nv_bfloat16 b = __float2bfloat16_rn(f[0]);
    return *reinterpret_cast<const uint16_t*>(&b);
  }
};
template <>
struct RowVec<float, false> {
  static constexpr int kElems = 1;
  static __device__ __forceinline__ void unpack(const float& v, float (&f)[1]) { f[0] = v; }
  static __device__ __forceinline__ float pack(const float (&f)[1]) { return f[0]; }
};

// A load of memory that this kernel may also write (add may be dx): not
// through the read-only path.
template <typename V>
__device__ __forceinline__ V ld_plain(const V* p) {
  return *reinterpret_cast<const volatile V*>(p);
}
template <>
__device__ __forceinline__ uint4 ld_plain<uint4>(const uint4* p) {
  return __ldcs(p);
}
template <>
__device__ __forceinline__ Vec32 ld_plain<Vec32>(const Vec32* p) {
  Vec32 r;
  asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                 "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p));
  return r;
}

// Slots whose rows are in flight at once: 8, or 4 for single elements.
template <typename V>
__host__ __device__ constexpr int bwd_group() {
  return sizeof(V) >= 16 ? 8 : 4;
}

// Vectors of a row in flight per thread and slot: one 16- or 32-byte vector,
// four single elements (with one, the element path of 1999 tokens x 3 slots of
// 1001 bf16 took 23.6 us, a chain of load latencies).
template <typename V>
__host__ __device__ constexpr int bwd_unroll() {
  return sizeof(V) >= 16 ? 1 : 4;
}

// Rows of up to two vectors per thread of a small CTA go to CTAs of that size:
// more tokens in flight, fewer idle threads.  combine / gather gradient of 16384
// x 8 bf16 rows of 1024 118 / 68 us with kRowThreads, 88 / 50 so; 8192 x 6 of 2048
// 70 / 42 and 68 / 39; 15452 x 2 of 384 47 / 28 and 28 / 22.
constexpr int kRowSmall = 64;
template <typename V>
bool small_rows(long nvec) {
  return nvec <= 2 * kRowSmall * bwd_unroll<V>();
}

// Sorted row of slot i of T * k, -1 for none: a dropped slot, or (flagged) an
// entry past the rows.
__device__ __forceinline__ long slot_row(const int32_t* inv, long i, long rows) {
  const long r = inv[i];
  if (r >= rows) mr_raise(MR_FLAG_BAD_INDEX);
  return r >= 0 && r < rows ? r : -1;
}

// E may be null (no dw wanted), dE may be null (frozen experts).
template <typename V, bool BF16, int kThreads>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const V* __restrict__ dy, const V* __restrict__ E,
                            const float* __restrict__ w, const int32_t* __restrict__ inv,
                            V* __restrict__ dE, float* __restrict__ dw, long nvec, int k) {
  using R = RowVec<V, BF16>;
  constexpr int NE = R::kElems;
  constexpr int VU = bwd_unroll<V>();
  constexpr int kBwdGroup = bwd_group<V>();
  constexpr int kWarps = kThreads / 32;
  __shared__ long row_s[kRowMaxK];
  __shared__ float w_s[kRowMaxK];
  __shared__ float red[kWarps][kBwdGroup];
  const long t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j = threadIdx.x; j < k; j += kThreads) {
    row_s[j] = slot_row(inv, t * k + j, (long)gridDim.x * k);
    w_s[j] = w[t * k + j];
  }
  __syncthreads();
  const V* g = dy + t * nvec;
  for (int j0 = 0; j0 < k; j0 += kBwdGroup) {
    long row[kBwdGroup];
    float dot[kBwdGroup];
#pragma unroll
    for (int u = 0; u < kBwdGroup; ++u) {
      row[u] = j0 + u < k ? row_s[j0 + u] : -1;
      dot[u] = 0.0f;
    }
    for (long v0 = threadIdx.x; v0 < nvec; v0 += VU * kThreads) {
      V gv[VU], e[VU][kBwdGroup];
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const long v = v0 + i * kThreads;
        const bool in = VU == 1 || v < nvec;
        gv[i] = in ? ld_stream(g + v) : V{};
        if (E) {
#pragma unroll
          for (int u = 0; u < kBwdGroup; ++u)
            e[i][u] = in && row[u] >= 0 ? ld_stream(E + row[u] * nvec + v) : V{};
        }
      }
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const long v = v0 + i * kThreads;
        if (VU > 1 && v >= nvec) break;
        float gf[NE];
        R::unpack(gv[i], gf);
#pragma unroll
        for (int u = 0; u < kBwdGroup; ++u) {
          if (row[u] < 0) continue;
          if (E) {
            float ef[NE];
            R::unpack(e[i][u], ef);
#pragma unroll
            for (int c = 0; c < NE; ++c) dot[u] = fmaf(gf[c], ef[c], dot[u]);
          }
          if (dE) {
            const float wj = w_s[j0 + u];
            float o[NE];
#pragma unroll
            for (int c = 0; c < NE; ++c) o[c] = wj * gf[c];
            st_stream(dE + row[u] * nvec + v, R::pack(o));
          }
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int u = 0; u < kBwdGroup; ++u) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
          dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], off);
        if (lane == 0) red[warp][u] = dot[u];
      }
      __syncthreads();
      if (threadIdx.x < kBwdGroup && j0 + threadIdx.x < k) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) s += red[q][threadIdx.x];
        dw[t * k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

template <typename V, bool BF16, int kThreads>
__global__ void __launch_bounds__(kThreads)
    gather_backward_kernel(const V* __restrict__ dxs, const int32_t* __restrict__ inv,
                           const V* add, V* dx, long T, long nvec,
                           int k) {
  using R = RowVec<V, BF16>;
  constexpr int NE = R::kElems;
  constexpr int VU = bwd_unroll<V>();
  constexpr int kBwdGroup = bwd_group<V>();
  __shared__ long row_s[kRowMaxK];
  for (long t = blockIdx.x; t < T; t += gridDim.x) {
    for (int j = threadIdx.x; j < k; j += kThreads) row_s[j] = slot_row(inv, t * k + j, T * k);
    __syncthreads();
    for (long v0 = threadIdx.x; v0 < nvec; v0 += VU * kThreads) {
      V av[VU];
      float acc[VU][NE];
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const long v = v0 + i * kThreads;
        av[i] = add && v < nvec ? ld_plain(add + t * nvec + v) : V{};
#pragma unroll
        for (int c = 0; c < NE; ++c) acc[i][c] = 0.0f;
      }
      for (int j0 = 0; j0 < k; j0 += kBwdGroup) {
        V e[VU][kBwdGroup];
#pragma unroll
        for (int u = 0; u < kBwdGroup; ++u) {
          const long r = j0 + u < k ? row_s[j0 + u] : -1;
#pragma unroll
          for (int i = 0; i < VU; ++i) {
            const long v = v0 + i * kThreads;
            e[i][u] = r >= 0 && v < nvec ? ld_stream(dxs + r * nvec + v) : V{};
          }
        }
#pragma unroll
        for (int u = 0; u < kBwdGroup; ++u)  // V{} of a missing slot adds 0
#pragma unroll
          for (int i = 0; i < VU; ++i) {
            float ef[NE];
            R::unpack(e[i][u], ef);
#pragma unroll
            for (int c = 0; c < NE; ++c) acc[i][c] += ef[c];
          }
      }
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const long v = v0 + i * kThreads;
        if (v >= nvec) break;
        if (add) {
          float af[NE];
          R::unpack(av[i], af);
#pragma unroll
          for (int c = 0; c < NE; ++c) acc[i][c] += af[c];
        }
        st_stream(dx + t * nvec + v, R::pack(acc[i]));
      }
    }
    __syncthreads();
  }
}

}  // namespace mr

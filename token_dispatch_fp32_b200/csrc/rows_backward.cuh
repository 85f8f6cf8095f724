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
// four single elements (one would be a chain of load latencies).
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

// ---- gather: rows of bf16 that no vector fits -----------------------------------
//
// Read as whole words all the same.  A row that starts on a word has columns
// 2w, 2w + 1 in its word w, one that starts inside a word (o = 1) has 2w - 1, 2w
// there.  The first and the last row are read by elements: their outer words may
// lie outside the buffer.  8192 x 6 rows of 2049 take 81 us, 137 by elements.
// combine's gradient keeps to elements (142 us): by words it needs dy at both
// offsets and writes rows of either kind too, and took 200 to 340 us.
constexpr int kWordUnroll = 4, kWordGroup = 4;

__device__ __forceinline__ int starts_inside(const uint16_t* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) >> 1) & 1;
}
// Columns c, c + 1 of a row of d by elements, 0 outside.
__device__ __forceinline__ uint32_t two_elements(const uint16_t* row, long c, long d) {
  uint32_t v = 0;
  if (c >= 0 && c < d) v = row[c];
  if (c + 1 >= 0 && c + 1 < d) v |= (uint32_t)row[c + 1] << 16;
  return v;
}

// Rows of either kind have sums of their own, which meet at the end: the lower
// half of the second kind belongs to the word before, so the last word of a
// span serves only that one.  A half outside the row goes to a sum that no
// column uses.
template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    gather_backward_words_kernel(const uint16_t* __restrict__ dxs,
                                 const int32_t* __restrict__ inv, const uint16_t* add,
                                 uint16_t* dx, long T, long d, int k) {
  constexpr int VU = kWordUnroll, G = kWordGroup;
  constexpr int kSpan = VU * kThreads - 1;
  __shared__ long row_s[kRowMaxK];
  __shared__ float next[VU * kThreads];
  for (long t = blockIdx.x; t < T; t += gridDim.x) {
    for (int j = threadIdx.x; j < k; j += kThreads) row_s[j] = slot_row(inv, t * k + j, T * k);
    __syncthreads();
    for (long base = 0; base < (d + 1) / 2; base += kSpan) {
      const long w0 = base + threadIdx.x;
      float even[VU][2], odd[VU][2], av[VU][2];
      bool in[VU];  // a half of this word, or of the row's end, is in the row
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const long c = 2 * (w0 + i * kThreads);
        even[i][0] = even[i][1] = odd[i][0] = odd[i][1] = 0.0f;
        in[i] = c <= d;
        av[i][0] = add && c < d ? mr_bf16_to_f32(ld_plain(add + t * d + c)) : 0.0f;
        av[i][1] = add && c + 1 < d ? mr_bf16_to_f32(ld_plain(add + t * d + c + 1)) : 0.0f;
      }
      for (int j0 = 0; j0 < k; j0 += G) {
        uint32_t x[G][VU];
        long row[G];
        bool edge = false;
#pragma unroll
        for (int u = 0; u < G; ++u) {
          row[u] = j0 + u < k ? row_s[j0 + u] : -1;
          edge |= row[u] == 0 || row[u] == T * k - 1;
        }
        if (!edge) {
#pragma unroll
          for (int u = 0; u < G; ++u) {
            const uint16_t* r = dxs + row[u] * d;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(r - starts_inside(r)) + w0;
#pragma unroll
            for (int i = 0; i < VU; ++i)
              x[u][i] = row[u] >= 0 && in[i] ? ld_stream(q + i * kThreads) : 0u;
          }
        } else {
#pragma unroll
          for (int u = 0; u < G; ++u) {
            const uint16_t* r = dxs + row[u] * d;
#pragma unroll
            for (int i = 0; i < VU; ++i)
              x[u][i] = row[u] >= 0
                            ? two_elements(r, 2 * (w0 + i * kThreads) - starts_inside(r), d)
                            : 0u;
          }
        }
#pragma unroll
        for (int u = 0; u < G; ++u) {
          if (row[u] < 0) continue;
          const bool o = starts_inside(dxs + row[u] * d);
#pragma unroll
          for (int i = 0; i < VU; ++i) {
            float lo, hi;
            bf16x2_unpack(x[u][i], lo, hi);
            if (o) {
              odd[i][0] += lo;
              odd[i][1] += hi;
            } else {
              even[i][0] += lo;
              even[i][1] += hi;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < VU; ++i) next[i * kThreads + threadIdx.x] = odd[i][0];
      __syncthreads();
      const bool inside = starts_inside(dx + t * d);
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const int l = i * kThreads + threadIdx.x;
        const long c = 2 * (w0 + i * kThreads);
        if (l >= kSpan || c >= d) continue;
        uint16_t* out = dx + t * d + c;
        const uint32_t v = bf16x2_pack_rn(even[i][0] + odd[i][1] + av[i][0],
                                          even[i][1] + next[l + 1] + av[i][1]);
        if (!inside && c + 1 < d) {
          st_stream(reinterpret_cast<uint32_t*>(out), v);
        } else {
          out[0] = (uint16_t)v;
          if (c + 1 < d) out[1] = (uint16_t)(v >> 16);
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace mr

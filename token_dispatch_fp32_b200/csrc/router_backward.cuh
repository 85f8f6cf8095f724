// router_backward.cuh -- gradient of the gate (router_tc.cuh, route.cuh,
// router_splitk.cuh): from the router weights' gradient g = dw [T,k] to the
// hidden states and the gate weight.
//
// Forward of token t (Kimi K2 "Normalize weights" page, MoEGate.forward;
// DeepSeek-V3.2-Exp "Normalize weights" page, Gate.forward): L = x . W^T,
// s = sigmoid(L) or softmax(L), w_j = scale * s_j / (S + eps), S = sum_j s_j
// (softmax: w_j = scale * s_j).  The choice of experts is piecewise constant
// and the bias only enters the choice, so neither has a gradient:
//   sigmoid: dl_j = scale/(S+eps) * (g_j - sum_i g_i s_i / (S+eps)) * s_j (1 - s_j)
//            on the k chosen logits, 0 elsewhere;
//   softmax: dL_i = scale * s_i * ([i chosen] g_i - sum_j g_j s_j), every i.
//   dx = dL . W (+ add),  dW = dL^T . x.
// With sigmoid scores dL has k of N_r entries per token: dx sums k rows of W,
// dW[e] sums the rows of the tokens that chose e, which mr_dispatch's
// permutation lists.  Softmax makes both dense products.
#pragma once

#include "combine.cuh"
#include "mr_common.cuh"
#include "planes_gemm.cuh"
#include "rows_backward.cuh"

namespace mr {
namespace rb {

constexpr float kEps = 1e-20f;
constexpr int kMaxK = 32;
constexpr int kMaxN = 512;

// sigmoid(L) and 1 - sigmoid(L), each to full relative accuracy.
__device__ __forceinline__ void sigmoid_pair(float L, float& s, float& c) {
  const float q = expf(-fabsf(L));
  const float r = 1.0f / (1.0f + q);
  s = L >= 0.0f ? r : q * r;
  c = L >= 0.0f ? q * r : r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// One warp per token.  Sigmoid: slot[t*k + j] = dl_j (0 for an id outside
// [0, N_r)); `dense` (optional) gets the whole row dL[t].  Softmax: slot is not
// written; `dense` gets the row and `planes` its three bf16 planes [3][T][Np]
// (Np = N_r rounded up to 8, the padding 0), either may be null.
constexpr int kDlWarps = 4;
template <bool SOFTMAX>
__global__ void __launch_bounds__(32 * kDlWarps)
    dlogits_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                   const float* __restrict__ g, int T, int N_r, int k, float scale, float eps,
                   float* __restrict__ slot, float* __restrict__ dense,
                   __nv_bfloat16* __restrict__ planes) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long t = (long)blockIdx.x * kDlWarps + warp;
  if (t >= T) return;
  const float* L = logits + t * N_r;
  const int e = lane < k ? idx[t * k + lane] : -1;
  const bool ok = e >= 0 && e < N_r;
  if (lane < k && !ok) mr_raise(MR_FLAG_BAD_INDEX);
  const float gj = ok ? g[t * k + lane] : 0.0f;
  if constexpr (!SOFTMAX) {
    float s = 0.0f, c = 0.0f;
    if (ok) sigmoid_pair(L[e], s, c);
    const float inv = 1.0f / (warp_sum(s) + eps);
    const float mean = warp_sum(gj * s) * inv;
    const float dl = ok ? scale * inv * (gj - mean) * (s * c) : 0.0f;
    if (lane < k) slot[t * k + lane] = dl;
    if (dense) {
      for (int i = lane; i < N_r; i += 32) dense[t * N_r + i] = 0.0f;
      float sum = 0.0f;  // an id may repeat: its slots' sum, the same in each of their lanes
      for (int j = 0; j < k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j);
        const float dj = __shfl_sync(0xffffffffu, dl, j);
        if (ej == e) sum += dj;
      }
      __syncwarp();
      if (ok) dense[t * N_r + e] = sum;
    }
  } else {
    float mx = -INFINITY;
    for (int i = lane; i < N_r; i += 32) mx = fmaxf(mx, L[i]);
    mx = warp_max(mx);
    float sum = 0.0f;
    for (int i = lane; i < N_r; i += 32) sum += expf(L[i] - mx);
    const float inv = 1.0f / warp_sum(sum);
    const float pj = ok ? expf(L[e] - mx) * inv : 0.0f;
    const float mean = warp_sum(gj * pj);
    // a chosen entry is scale * p * (sum of its slots' g - mean); its own sum
    // first, in slot order in each of an id's lanes, then the difference, so no
    // two large terms cancel late
    float gs = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl_sync(0xffffffffu, e, j);
      const float gg = __shfl_sync(0xffffffffu, gj, j);
      if (ej == e) gs += gg;
    }
    const int Np = (N_r + 7) & ~7;
    auto put = [&](int i, float v) {
      if (dense && i < N_r) dense[t * N_r + i] = v;
      if (planes) {
        __nv_bfloat16 p[3];
        tc::split3(v, p[0], p[1], p[2]);
#pragma unroll
        for (int q = 0; q < 3; ++q) planes[((long)q * T + t) * Np + i] = p[q];
      }
    };
    for (int i = lane; i < Np; i += 32)
      put(i, i < N_r ? -scale * (expf(L[i] - mx) * inv) * mean : 0.0f);
    __syncwarp();
    if (ok) put(e, scale * pj * (gs - mean));  // equal ids write equal values
  }
}

// ---- sigmoid: dx[t] = sum_j dl[t,j] * W[idx[t,j]] (+ add[t]) ------------------
//
// A CTA keeps CW = 32 * CPL columns of every expert's row of W (fp32, plus one
// row of zeros for ids out of range) in shared memory and walks a range of
// tokens: each slot is one conflict-free read of its expert's CW columns and
// CPL fused multiply-adds per lane.  The k * d reads of W per token then come
// from shared memory (128 bytes a cycle and SM), which is what bounds the
// kernel, instead of L2.  The grid is one wave: the (column chunk, block of
// tokens) pairs are dealt out evenly, so a CTA loads its columns of W once or
// twice.  A warp takes kDxTokens tokens at a time (independent reads in flight)
// and stages their (row, dl) pairs in its own piece of shared memory, the next
// tokens' already on their way (addv may be dxv: neither is __restrict__).
// slot is not __restrict__ here nor in dw_slots_kernel: dlogits_kernel may still
// be writing it when these start, so it is read by ordinary loads behind the wait.
//
// The kernel is a programmatic dependent of dlogits_kernel: W is loaded while
// that runs.  Measured on the full DeepSeek-V3 batch (16384 tokens, 256
// experts, with add): 167 us with dlogits_kernel, against 118 us for the reads of
// shared memory alone; without the paired multiply-adds 180 us; 1024 threads of
// 64 registers 205 us (spills), one token per warp at a time 435 us.  It lets
// dw_slots_kernel start as its CTAs finish (10 us less for the whole call than
// one after the other); making room for both on an SM (80 registers a thread)
// gained nothing, the spills cost what the overlap saved.
constexpr int kDxThreads = 512;
constexpr int kDxTokens = 4;
// (row, dl) pairs per lane of a warp's tokens: one for k <= 8, else up to four
constexpr int kDxSmall = (kDxTokens * 8 + 31) / 32, kDxLarge = kDxTokens * kMaxK / 32;

__host__ __device__ constexpr size_t dx_smem_bytes(int N_r, int cw, int k) {
  // two buffers per warp of kDxTokens rows of pairs, each padded to an even count
  return ((size_t)N_r + 1) * cw * 4 +
         (size_t)(kDxThreads / 32) * 2 * kDxTokens * ((k + 1) & ~1) * 8;
}

template <int CPL, bool VEC, bool BF16, int kRegs>
__global__ void __launch_bounds__(kDxThreads)
    dx_slots_kernel(const void* __restrict__ Wv, bool wbf16, const int32_t* __restrict__ idx,
                    const float* slot, const void* addv, void* dxv, int T, int d,
                    int N_r, int k) {
  constexpr int CW = 32 * CPL;
  constexpr int U = kDxTokens;
  constexpr int kWarps = kDxThreads / 32;
  extern __shared__ __align__(16) float sm[];
  float* Ws = sm;  // [N_r + 1][CW]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kp = (k + 1) & ~1;
  int2* pairs = reinterpret_cast<int2*>(sm + (N_r + 1) * CW) + warp * 2 * U * kp;  // [2][U][kp]
  // the pairs of tokens t .. t + U - 1: id and dl; pair i of a lane belongs to
  // token tk[i] (U for none) and goes to place at[i] of the buffer
  int er[kRegs], tk[kRegs], at[kRegs];
  float gr[kRegs];
#pragma unroll
  for (int r = 0; r < kRegs; ++r) {
    const int i = lane + 32 * r;
    tk[r] = i < U * k ? i / k : U;
    at[r] = tk[r] * kp + i % k;
  }
  auto fetch = [&](long t, long t_end) {
#pragma unroll
    for (int r = 0; r < kRegs; ++r) {
      const bool in = tk[r] < U && t + tk[r] < t_end;
      er[r] = in ? idx[t * k + lane + 32 * r] : -1;
      gr[r] = in ? slot[t * k + lane + 32 * r] : 0.0f;
    }
  };
  for (int i = lane; i < 2 * U * kp; i += 32) pairs[i] = make_int2(N_r * CW, 0);  // odd k: padding
  // columns of this lane: CPL consecutive ones (VEC) or every 32nd
  auto col = [&](int i) { return VEC ? lane * CPL + i : lane + 32 * i; };
  constexpr int kBlock = kWarps * U;  // tokens per step of the CTA
  const long blocks = ((long)T + kBlock - 1) / kBlock;
  const long units = blocks * ((d + CW - 1) / CW);
  const long u_end = units * (blockIdx.x + 1) / gridDim.x;
  bool waited = false;
  for (long unit = units * blockIdx.x / gridDim.x; unit < u_end;) {
    const int c0 = (int)(unit / blocks) * CW;
    const long b0 = unit % blocks;
    const long b1 = b0 + (u_end - unit) < blocks ? b0 + (u_end - unit) : blocks;
    unit += b1 - b0;
    const long t_end = b1 * kBlock < T ? b1 * kBlock : T;
    __syncthreads();  // the last chunk's columns have been read
    if (VEC && !wbf16) {  // d is a multiple of 4, W 16-byte aligned
      constexpr int Q = CW / 4;
#pragma unroll 4
      for (int i = threadIdx.x; i < (N_r + 1) * Q; i += kDxThreads) {
        const int e = i / Q, c = c0 + 4 * (i % Q);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < N_r && c < d)
          v = __ldg(
              reinterpret_cast<const float4*>(static_cast<const float*>(Wv) + (long)e * d + c));
        *reinterpret_cast<float4*>(Ws + 4 * i) = v;
      }
    } else {
#pragma unroll 4
      for (int i = threadIdx.x; i < (N_r + 1) * CW; i += kDxThreads) {
        const int e = i / CW, c = c0 + i % CW;
        float v = 0.0f;
        if (e < N_r && c < d)
          v = wbf16 ? mr_bf16_to_f32(static_cast<const uint16_t*>(Wv)[(long)e * d + c])
                    : static_cast<const float*>(Wv)[(long)e * d + c];
        Ws[i] = v;
      }
    }
    if (!waited) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // dlogits_kernel's slots
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      waited = true;
    }
    __syncthreads();
    long t = b0 * kBlock + warp * U;
    fetch(t, t_end);
    const bool mine = c0 + lane * CPL < d;  // VEC: d is a multiple of CPL
    for (int par = 0; t < t_end; t += kWarps * U, par ^= 1) {
      int2* buf = pairs + par * U * kp;
#pragma unroll
      for (int r = 0; r < kRegs; ++r) {
        const bool ok = er[r] >= 0 && er[r] < N_r;
        if (tk[r] < U)
          buf[at[r]] = make_int2((ok ? er[r] : N_r) * CW, ok ? __float_as_int(gr[r]) : 0);
      }
      __syncwarp();
      fetch(t + kWarps * U, t_end);
      float acc[U][CPL];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[u][i] = 0.0f;
      // add, on its way while the slots are summed
      uint32_t ab[U][CPL / 2];
      float af[U][CPL];
      if (VEC && addv) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (t + u >= t_end || !mine) continue;
          const long o = (t + u) * d + c0 + lane * CPL;
          if constexpr (BF16) {
            const uint16_t* a = static_cast<const uint16_t*>(addv) + o;
            if constexpr (CPL == 4)
              *reinterpret_cast<uint2*>(ab[u]) = *reinterpret_cast<const uint2*>(a);
            else ab[u][0] = *reinterpret_cast<const uint32_t*>(a);
          } else {
            const float* a = static_cast<const float*>(addv) + o;
            if constexpr (CPL == 4)
              *reinterpret_cast<float4*>(af[u]) = *reinterpret_cast<const float4*>(a);
            else *reinterpret_cast<float2*>(af[u]) = *reinterpret_cast<const float2*>(a);
          }
        }
      }
#pragma unroll 4
      for (int j = 0; j < kp; j += 2) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int4 pr = *reinterpret_cast<const int4*>(buf + u * kp + j);
          const float a0 = __int_as_float(pr.y), a1 = __int_as_float(pr.w);
          const float *w0 = Ws + pr.x, *w1 = Ws + pr.z;
          if constexpr (VEC && CPL == 4) {
            const float4 v0 = *reinterpret_cast<const float4*>(w0 + lane * 4);
            const float4 v1 = *reinterpret_cast<const float4*>(w1 + lane * 4);
            fma2(acc[u][0], acc[u][1], a0, v0.x, v0.y);
            fma2(acc[u][2], acc[u][3], a0, v0.z, v0.w);
            fma2(acc[u][0], acc[u][1], a1, v1.x, v1.y);
            fma2(acc[u][2], acc[u][3], a1, v1.z, v1.w);
          } else {
#pragma unroll
            for (int i = 0; i < CPL; ++i)
              acc[u][i] = fmaf(a1, w1[col(i)], fmaf(a0, w0[col(i)], acc[u][i]));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= t_end) break;
        const long base = (t + u) * d + c0;
        if constexpr (VEC) {
          if (!mine) continue;
          if constexpr (BF16) {
            uint32_t o[CPL / 2];
#pragma unroll
            for (int i = 0; i < CPL / 2; ++i) {
              float lo = 0.0f, hi = 0.0f;
              if (addv) bf16x2_unpack(ab[u][i], lo, hi);
              o[i] = bf16x2_pack_rn(acc[u][2 * i] + lo, acc[u][2 * i + 1] + hi);
            }
            uint16_t* out = static_cast<uint16_t*>(dxv) + base + lane * CPL;
            if constexpr (CPL == 4) __stcs(reinterpret_cast<uint2*>(out), make_uint2(o[0], o[1]));
            else __stcs(reinterpret_cast<uint32_t*>(out), o[0]);
          } else {
            float* out = static_cast<float*>(dxv) + base + lane * CPL;
            if (addv) {
#pragma unroll
              for (int i = 0; i < CPL; ++i) acc[u][i] += af[u][i];
            }
            if constexpr (CPL == 4)
              __stcs(reinterpret_cast<float4*>(out),
                     make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]));
            else __stcs(reinterpret_cast<float2*>(out), make_float2(acc[u][0], acc[u][1]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < CPL; ++i) {
            const int c = col(i);
            if (c0 + c >= d) continue;
            float v = acc[u][i];
            if constexpr (BF16) {
              if (addv) v += mr_bf16_to_f32(static_cast<const uint16_t*>(addv)[base + c]);
              const __nv_bfloat16 b = __float2bfloat16_rn(v);
              static_cast<uint16_t*>(dxv)[base + c] = *reinterpret_cast<const uint16_t*>(&b);
            } else {
              if (addv) v += static_cast<const float*>(addv)[base + c];
              static_cast<float*>(dxv)[base + c] = v;
            }
          }
        }
      }
    }
  }
}

// ---- sigmoid: dW[e] = sum over the sorted rows r of e of dl[perm[r]] * x[perm[r]/k]
//
// Each expert's segment is cut into pieces of 1 << sh sorted rows (at least one
// piece, so that an expert without rows gets its zeros); a CTA takes one piece
// and one slab of columns (consecutive CTAs share the slab, so its columns of x
// stay in L2 while every expert reads them).  An expert's first piece goes to
// dW, the others to `part`, and dw_join_kernel adds them in order: no atomics, a
// long segment is spread over many SMs.  Bound by L2: T * k rows of x pass from
// there to the SMs, 12 TB/s on the full DeepSeek-V3 batch (the call 314 us of GPU
// time, of which dx 150; pieces of 512 rows make it 14 us longer).
constexpr int kDwMaxShift = 8;
constexpr int kDwRows = 1 << kDwMaxShift;  // at most; dw_piece_shift
constexpr int kDwThreads = 128;
constexpr int kDwWide = 4;  // columns or words per thread where no 16-byte vector fits

// log2 of the rows of a piece, for n sorted rows of d columns.  A piece is a
// chain of loads (eight rows at a time), so fewer of them than the GPU holds CTAs
// leave it waiting: halved until there are 512.  Pieces of 256 / 128 / 64 / 32
// rows, dW alone: 2048 x 2 rows of 4096 38 / 27 / 19 / 16 us, 1577 x 8 of 1088
// 44 / 29 / 20 / 18, 4096 x 8 of 7168 on 256 experts 51 / 59 / 60 / 67, 16384 x 8
// 166 / 171 / 197 / 254 (the partial sums cost more than the balance gains).  Up to 256 rows in
// all stay one piece per expert, without the launch that joins them.
inline int dw_piece_shift(long n, long d) {
  int sh = kDwMaxShift;
  if (n <= kDwRows) return sh;
  while (sh > 5 && (n >> sh) * ((d + 1023) / 1024) < 512) --sh;
  return sh;
}

// Extra pieces (beyond an expert's first) of all experts before expert e are
// numbered consecutively; there are at most n >> sh of them (1 << sh rows a piece).
struct Piece {
  int e, row0, rows, extra;  // extra: index in `part`, -1 for an expert's first piece
};

// (pieces hold 1 << sh rows)
__device__ __forceinline__ int pieces(int rows, int sh) {
  return rows > (1 << sh) ? (rows + (1 << sh) - 1) >> sh : 1;
}

// Finds piece `b` (all threads of the CTA call it; e = -1 past the last one).
__device__ __forceinline__ Piece find_piece(const int32_t* __restrict__ offsets, int N_r, int n,
                                            int sh, int b) {
  __shared__ Piece found;
  __shared__ int wsum[2][kDwThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = (N_r + kDwThreads - 1) / kDwThreads;
  const int e0 = tid * c, e1 = e0 + c < N_r ? e0 + c : N_r;
  auto rows_of = [&](int e, int& lo) {
    lo = offsets[e];
    int hi = offsets[e + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > n ? n : hi;
    return hi > lo ? hi - lo : 0;
  };
  int mine = 0, extra = 0;
  for (int e = e0; e < e1; ++e) {
    int lo;
    const int p = pieces(rows_of(e, lo), sh);
    mine += p;
    extra += p - 1;
  }
  int a = mine, x = extra;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int ya = __shfl_up_sync(0xffffffffu, a, off), yx = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) {
      a += ya;
      x += yx;
    }
  }
  if (lane == 31) {
    wsum[0][warp] = a;
    wsum[1][warp] = x;
  }
  if (tid == 0) found.e = -1;
  __syncthreads();
  int before = a - mine, xb = x - extra;
  for (int w = 0; w < warp; ++w) {
    before += wsum[0][w];
    xb += wsum[1][w];
  }
  if (b >= before && b < before + mine) {
    for (int e = e0; e < e1; ++e) {
      int lo;
      const int cnt = rows_of(e, lo), p = pieces(cnt, sh);
      if (b < before + p) {
        const int i = b - before;
        found.e = e;
        found.row0 = lo + (i << sh);
        found.rows = cnt - (i << sh) < (1 << sh) ? cnt - (i << sh) : 1 << sh;
        found.extra = i == 0 ? -1 : xb + i - 1;
        // more extra pieces than `part` holds: offsets that overlap (flagged)
        if (found.extra >= n >> sh) found.e = -1;
        break;
      }
      before += p;
      xb += p - 1;
    }
  }
  __syncthreads();
  return found;
}

// V: uint4 (8 bf16 or 4 fp32 columns per thread), or for rows that no vector
// fits kDwWide columns per thread (float) or words (uint16_t: pairs of bf16).
//
// Rows of bf16 at odd addresses are read as whole words all the same.  A row that
// starts on a word has columns 2w, 2w + 1 in its word w, one that starts inside a
// word has 2w - 1, 2w there; each kind has sums of its own, which meet at the end
// (the lower half of the second kind belongs to the word before, so a CTA's last
// word serves only that one).  With one element per load, 16384 rows of 7105
// took 864 us.
template <typename V, bool BF16>
struct DwShape {
  static constexpr bool kPairs = sizeof(V) == 2;
  static constexpr int kElems = (int)sizeof(V) / (BF16 ? 2 : 4);  // columns of a V
  static constexpr int VU = sizeof(V) == 16 ? 1 : kDwWide;
  // vectors, columns or words per CTA
  static constexpr int kSpan = VU * kDwThreads - (kPairs ? 1 : 0);
  static unsigned slabs(long nvec) {
    const long units = kPairs ? (nvec + 1) / 2 : nvec;
    return (unsigned)((units + kSpan - 1) / kSpan);
  }
};

template <typename V, bool BF16>
__global__ void __launch_bounds__(kDwThreads)
    dw_slots_kernel(const V* __restrict__ x, const int32_t* __restrict__ perm,
                    const int32_t* __restrict__ offsets, const float* slot, int n,
                    int N_r, int k, int sh, long nvec, float* __restrict__ dW,
                    float* __restrict__ part, bool wait_first) {
  using S = DwShape<V, BF16>;
  constexpr int NE = S::kElems;
  constexpr int VU = S::VU;
  constexpr int U = 8;
  // Programmatic dependent of dlogits_kernel (wait_first), or of dx_slots_kernel,
  // every CTA of which (one wave) has seen dlogits_kernel complete before this
  // kernel starts; then only this kernel's end waits for that one's, so that
  // whatever follows on the stream comes after both.
  if (wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0)  // one CTA: the segments lie in order, inside the rows
    for (int e = threadIdx.x; e <= N_r; e += kDwThreads)
      if (offsets[e] < 0 || offsets[e] > n || (e < N_r && offsets[e + 1] < offsets[e]))
        mr_raise(MR_FLAG_BAD_INDEX);
  const Piece pc = find_piece(offsets, N_r, n, sh, blockIdx.x);
  if (pc.e < 0) {
    if (!wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  __shared__ int tok[kDwRows];
  __shared__ float gs[kDwRows];
  for (int i = threadIdx.x; i < pc.rows; i += kDwThreads) {
    const int p = perm[pc.row0 + i];
    const bool ok = p >= 0 && p < n;
    if (!ok) mr_raise(MR_FLAG_BAD_INDEX);
    tok[i] = ok ? p / k : -1;
    gs[i] = ok ? slot[p] : 0.0f;
  }
  if constexpr (S::kPairs) {  // whole groups: the piece's first row again, not added
    const int i = pc.rows + threadIdx.x;
    if (i < (pc.rows + U - 1) / U * U) {
      const int p = perm[pc.row0];
      tok[i] = p >= 0 && p < n ? p / k : -1;
    }
  }
  __syncthreads();
  const long v0 = (long)blockIdx.y * S::kSpan + threadIdx.x;
  const long d = nvec * NE;
  float* out = pc.extra < 0 ? dW + (long)pc.e * d : part + (long)pc.extra * d;
  if constexpr (S::kPairs) {
    float even[VU][2], odd[VU][2];
    bool in[VU];  // a half of this word, or of the row's end, is in the row
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      even[i][0] = even[i][1] = odd[i][0] = odd[i][1] = 0.0f;
      in[i] = 2 * (v0 + i * kDwThreads) <= d;
    }
    const int last = n / k - 1;
    for (int r = 0; r < pc.rows; r += U) {
      uint32_t xv[U][VU];
      // The halves a word has outside its row go to sums that no column uses, so
      // they may be read: all but those of the first and the last row, which
      // may lie outside x.
      bool edge = false;
#pragma unroll
      for (int u = 0; u < U; ++u) edge |= tok[r + u] <= 0 || tok[r + u] >= last;
      if (!edge) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const V* row = x + (long)tok[r + u] * d;
          const uint32_t* q = reinterpret_cast<const uint32_t*>(row - starts_inside(row)) + v0;
#pragma unroll
          for (int i = 0; i < VU; ++i) xv[u][i] = in[i] ? ld_stream(q + i * kDwThreads) : 0u;
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int t = tok[r + u];
          const V* row = x + (long)t * d;
#pragma unroll
          for (int i = 0; i < VU; ++i) {
            const long c = 2 * (v0 + i * kDwThreads) - starts_inside(row);
            xv[u][i] = t >= 0 ? two_elements(row, c, d) : 0u;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u >= pc.rows || tok[r + u] < 0) continue;
        const float g = gs[r + u];
        float lo, hi;
        if (starts_inside(x + (long)tok[r + u] * d)) {
#pragma unroll
          for (int i = 0; i < VU; ++i) {
            bf16x2_unpack(xv[u][i], lo, hi);
            fma2(odd[i][0], odd[i][1], g, lo, hi);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VU; ++i) {
            bf16x2_unpack(xv[u][i], lo, hi);
            fma2(even[i][0], even[i][1], g, lo, hi);
          }
        }
      }
    }
    __shared__ float next[VU * kDwThreads];
#pragma unroll
    for (int i = 0; i < VU; ++i) next[i * kDwThreads + threadIdx.x] = odd[i][0];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const int l = i * kDwThreads + threadIdx.x;
      const long c = 2 * (v0 + i * kDwThreads);
      if (l >= S::kSpan) continue;
      if (c < d) out[c] = even[i][0] + odd[i][1];
      if (c + 1 < d) out[c + 1] = even[i][1] + next[l + 1];
    }
  } else if (v0 < nvec) {
    float acc[VU][NE];
#pragma unroll
    for (int j = 0; j < VU; ++j)
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[j][i] = 0.0f;
    for (int r = 0; r < pc.rows; r += U) {
      V xv[U][VU];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = r + u < pc.rows ? tok[r + u] : -1;
#pragma unroll
        for (int j = 0; j < VU; ++j) {
          const long v = v0 + j * kDwThreads;
          xv[u][j] = t >= 0 && (VU == 1 || v < nvec) ? ld_stream(x + (long)t * nvec + v) : V{};
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float g = r + u < pc.rows ? gs[r + u] : 0.0f;
#pragma unroll
        for (int j = 0; j < VU; ++j) {
          float xf[NE];
          RowVec<V, BF16>::unpack(xv[u][j], xf);
          if constexpr (NE % 2 == 0) {
#pragma unroll
            for (int i = 0; i < NE; i += 2)
              fma2(acc[j][i], acc[j][i + 1], g, xf[i], xf[i + 1]);
          } else {
            acc[j][0] = fmaf(g, xf[0], acc[j][0]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < VU; ++j) {
      const long v = v0 + j * kDwThreads;
      if (VU > 1 && v >= nvec) break;
#pragma unroll
      for (int i = 0; i < NE; ++i) out[v * NE + i] = acc[j][i];
    }
  }
  if (!wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// dW[e] += the extra pieces of e, in order.
__global__ void __launch_bounds__(256)
    dw_join_kernel(const int32_t* __restrict__ offsets, int n, int N_r, int d, int sh,
                   const float* __restrict__ part, float* __restrict__ dW) {
  const int e = blockIdx.x;
  __shared__ int first_s, count_s;
  {  // no extra piece: nothing to add
    const int lo = offsets[e], hi = offsets[e + 1];
    if ((hi > n ? n : hi) - (lo < 0 ? 0 : lo) <= 1 << sh) return;
  }
  if (threadIdx.x < 32) {
    int x = 0, mine = 0;
    for (int i = threadIdx.x; i <= e; i += 32) {
      int lo = offsets[i], hi = offsets[i + 1];
      lo = lo < 0 ? 0 : lo;
      hi = hi > n ? n : hi;
      const int p = pieces(hi - lo, sh);
      if (i == e) mine = p;
      else x += p - 1;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, off);
      mine += __shfl_xor_sync(0xffffffffu, mine, off);
    }
    if (threadIdx.x == 0) {
      first_s = x;
      count_s = mine;
    }
  }
  __syncthreads();
  const int first = first_s, count = count_s;
  if (count <= 1 || first + count - 1 > n >> sh) return;
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < d; c += gridDim.y * blockDim.x) {
    float s = dW[(long)e * d + c];
    for (int i = 0; i + 1 < count; i += 8) {  // eight loads in flight, added in order
      float p[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        p[u] = i + u + 1 < count ? part[(long)(first + i + u) * d + c] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u + 1 < count) s += p[u];
    }
    dW[(long)e * d + c] = s;
  }
}

// ---- softmax: dense fp32 products on the CUDA cores -----------------------------
//
// For rows that TMA does not take (d no multiple of 8, unaligned buffers) and for
// dW of fp32 rows; planes_gemm.cuh has the others.
// C [M, N] = A . B, fp32 fused multiply-adds: 128 x 128 tiles, K in steps of
// 16, 256 threads of 8 x 8 elements each.  TA: A is stored [K, M] (dL for dW),
// else [M, K] (dL for dx).  B [K, N] row-major, fp32 or bf16.  K may be split
// over gridDim.z; slice z of C then goes to C + z * M * N (fp32) and
// sum_slices_kernel adds them in order.
constexpr int kGemmT = 128, kGemmK = 16;

template <bool TA, bool BBF16, bool OBF16>
__global__ void __launch_bounds__(256)
    dense_kernel(const float* __restrict__ A, const void* __restrict__ Bv,
                 const void* addv, void* Cv, int M, int N, int K) {
  __shared__ float As[kGemmK][kGemmT + 4];
  __shared__ float Bs[kGemmK][kGemmT + 4];
  const int tid = threadIdx.x;
  const long m0 = (long)blockIdx.y * kGemmT, n0 = (long)blockIdx.x * kGemmT;
  const int steps = (K + kGemmK - 1) / kGemmK;
  const int s_begin = (int)((long)steps * blockIdx.z / gridDim.z);
  const int s_end = (int)((long)steps * (blockIdx.z + 1) / gridDim.z);
  const int tm = tid / 16, tn = tid % 16;
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  float ra[8], rb[8];
  auto fetch = [&](int step) {
    const long k0 = (long)step * kGemmK;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = tid + 256 * i;
      const int kk = TA ? q / kGemmT : q % kGemmK, mm = TA ? q % kGemmT : q / kGemmK;
      const long kg = k0 + kk, mg = m0 + mm;
      ra[i] = kg < K && mg < M ? A[TA ? kg * M + mg : mg * K + kg] : 0.0f;
      const long kb = k0 + q / kGemmT, ng = n0 + q % kGemmT;
      rb[i] = 0.0f;
      if (kb < K && ng < N) {
        if constexpr (BBF16) rb[i] = mr_bf16_to_f32(static_cast<const uint16_t*>(Bv)[kb * N + ng]);
        else rb[i] = static_cast<const float*>(Bv)[kb * N + ng];
      }
    }
  };
  if (s_begin < s_end) fetch(s_begin);
  for (int s = s_begin; s < s_end; ++s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = tid + 256 * i;
      if constexpr (TA) As[q / kGemmT][q % kGemmT] = ra[i];
      else As[q % kGemmK][q / kGemmK] = ra[i];
      Bs[q / kGemmT][q % kGemmT] = rb[i];
    }
    __syncthreads();
    if (s + 1 < s_end) fetch(s + 1);
#pragma unroll
    for (int kk = 0; kk < kGemmK; ++kk) {
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(a + i) =
            *reinterpret_cast<const float4*>(&As[kk][tm * 4 + (i / 4) * 64]);
        *reinterpret_cast<float4*>(b + i) =
            *reinterpret_cast<const float4*>(&Bs[kk][tn * 4 + (i / 4) * 64]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long m = m0 + tm * 4 + (i / 4) * 64 + i % 4;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long c = n0 + tn * 4 + (j / 4) * 64 + j % 4;
      if (c >= N) continue;
      float v = acc[i][j];
      const long o = m * N + c;
      if constexpr (OBF16) {
        if (addv) v += mr_bf16_to_f32(static_cast<const uint16_t*>(addv)[o]);
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        static_cast<uint16_t*>(Cv)[o] = *reinterpret_cast<const uint16_t*>(&b);
      } else {
        if (addv) v += static_cast<const float*>(addv)[o];
        static_cast<float*>(Cv)[(long)blockIdx.z * M * N + o] = v;
      }
    }
  }
}

__global__ void __launch_bounds__(256)
    sum_slices_kernel(const float* __restrict__ part, int slices, long n, float* __restrict__ out) {
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long)gridDim.x * blockDim.x) {
    float s = 0.0f;
    for (int z = 0; z < slices; ++z) s += part[z * n + i];
    out[i] = s;
  }
}

}  // namespace rb
}  // namespace mr

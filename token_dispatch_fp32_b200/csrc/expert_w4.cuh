// expert_w4.cuh -- the experts' products on 4-bit weights with group scales,
// for batches of few tokens (Kimi K2 "Add shared output" page, moe_infer:
// sorted_tokens = x[idxs // k], expert(sorted_tokens[start_idx:end_idx])).
//
//   out[j][n] = sum_G scale[e][n][G] * sum_{c in G} (q[e][n][c] - 8) * x[perm[j]/k][c]
//
// for the sorted row j of expert e, groups G of 32, 64 or 128 columns.  A few
// rows per expert make this a stream of the hit experts' weights from HBM
// (n_out * d / 2 bytes each plus the scales): the kernel's work per weight has
// to stay below what the SMs issue while those bytes arrive, about three
// instructions per weight.  So a weight is widened once, two at a time, by an
// integer trick (nibble u in the low mantissa bits of 128.0 is 128 + u in
// bf16; subtracting 136 is exact), and multiplied by tensor-core MMAs with the
// weights as the 16-row operand and up to 8 rows of x as the 8 columns
// (mma.sync m16n8k16: at this shape the tensor pipe is nearly idle; a 128-row
// tcgen05 tile would first have to pass the widened weights, four times the
// bytes, through shared or tensor memory).  Products of bf16 x by integers in
// [-8, 7] are exact in fp32; each group's fp32 sum is scaled and added in
// fp32, so the only rounding to fewer bits is the output's.
//
// Packed layout (written once by w4_pack_kernel): the weights are cut into
// blocks of 16 output rows x 128 columns, block (e, mt, kb) at index
// (e * MT + mt) * KB + kb, 1024 bytes: 512 for rows 0-7 and 512 for rows 8-15
// of the block, lane l's 16 bytes at 16 * l.  They are four words, word i for
// the columns 32 i + 8 (l % 4) .. + 7 of row l / 4 (+ 8): the columns the lane
// feeds to two MMA steps, so that a warp's load is 512 contiguous bytes, the
// lane's share of x is 16 contiguous bytes, and one MMA never spans two
// groups.  In a word, column 2 p of the eight is the nibble at bit 4 p, column
// 2 p + 1 the one at bit 16 + 4 p.  Scales follow as [block][16 rows][128 /
// group] in their own type.  Padded rows and columns hold the value 0 (nibble
// 8) and scale 0.
#pragma once

#include "mr_common.cuh"

namespace mr {
namespace w4 {

constexpr int kRows = 16;      // output rows per block (MMA M)
constexpr int kCols = 128;     // columns per block
constexpr int kBlockBytes = 1024;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMT = 2;         // row blocks per CTA

struct Layout {
  int MT, KB;            // blocks along n_out and d
  long blocks;           // N_r * MT * KB
  size_t scale_off;      // bytes of the weight part
  size_t total;
};

inline Layout make_layout(int N_r, int n_out, int d, int group, int scale_bytes) {
  Layout l;
  l.MT = (n_out + kRows - 1) / kRows;
  l.KB = (d + kCols - 1) / kCols;
  l.blocks = (long)N_r * l.MT * l.KB;
  l.scale_off = (size_t)l.blocks * kBlockBytes;
  l.total = l.scale_off + (size_t)l.blocks * kRows * (kCols / group) * scale_bytes;
  return l;
}

// q [N_r, n_out, d / 2] (column 2 i in the low nibble of byte i), scales
// [N_r, n_out, ceil(d / group)] -> the packed layout.  One warp per block.
template <typename S>
__global__ void __launch_bounds__(256)
    w4_pack_kernel(const uint8_t* __restrict__ q, const S* __restrict__ scales, int n_out, int d,
                   int group, int MT, int KB, long blocks, uint4* __restrict__ wp,
                   S* __restrict__ sp) {
  const int lane = threadIdx.x & 31;
  const long b = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (b >= blocks) return;
  const int kb = (int)(b % KB);
  const int mt = (int)((b / KB) % MT);
  const long e = b / ((long)KB * MT);
  for (int h = 0; h < 2; ++h) {
    const int n = mt * kRows + 8 * h + lane / 4;
    uint32_t w[4];
    for (int i = 0; i < 4; ++i) {
      const int c0 = kb * kCols + 32 * i + 8 * (lane % 4);
      uint32_t v = 0x88888888u;  // d % 8 == 0: the eight columns are all in or all out
      if (n < n_out && c0 < d) {
        const uint8_t* src = q + ((e * n_out + n) * (long)d + c0) / 2;
        v = 0;
        for (int p = 0; p < 4; ++p) {
          const uint32_t byte = src[p];
          v |= (byte & 15u) << (4 * p);
          v |= (byte >> 4) << (16 + 4 * p);
        }
      }
      w[i] = v;
    }
    wp[b * (kBlockBytes / 16) + 32 * h + lane] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int ng = kCols / group, groups = (d + group - 1) / group;
  for (int i = lane; i < kRows * ng; i += 32) {
    const int n = mt * kRows + i / ng, g = kb * ng + i % ng;
    S v{};
    if (n < n_out && g < groups) v = scales[(e * n_out + n) * (long)groups + g];
    sp[b * (kRows * ng) + i] = v;
  }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return mr_bf16_to_f32(v); }

// Nibbles at bits s and 16 + s of w as two bf16 values minus 8 (low half: the
// nibble at bit s).
__device__ __forceinline__ uint32_t widen2(uint32_t w, int s) {
  const uint32_t m = ((w >> s) & 0x000f000fu) | 0x43004300u;  // 128 + u
  const uint32_t k136 = 0x43084308u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                   *reinterpret_cast<const __nv_bfloat162*>(&k136));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct Params {
  const uint16_t* x;
  const int32_t* perm;     // null: x holds the sorted rows
  const int32_t* offsets;
  const uint4* wp;
  const void* sp;
  uint16_t* out;
  int T, d, k, N_r, n_out, MT, KB;
  int rows_mode;  // gridDim.y counts sorted rows (a row that opens its segment works), else experts
};

// One block of 128 columns of kMT row blocks against NT * 8 rows of x.
template <int GROUP, typename S>
struct Frag {
  static constexpr int kNg = kCols / GROUP;
  uint4 w[kMT][2];
  S s[kMT][2][kNg];

  __device__ __forceinline__ void load(const Params& P, long blk0, int KB, int n_mt, int lane) {
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      if (m >= n_mt) continue;
      const long b = blk0 + (long)m * KB;
      w[m][0] = __ldcs(P.wp + b * (kBlockBytes / 16) + lane);
      w[m][1] = __ldcs(P.wp + b * (kBlockBytes / 16) + 32 + lane);
      const S* sp = static_cast<const S*>(P.sp) + b * (kRows * kNg) + (lane / 4) * kNg;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (sizeof(S) * kNg == 16)
          *reinterpret_cast<uint4*>(s[m][h]) =
              __ldg(reinterpret_cast<const uint4*>(sp + 8 * h * kNg));
        else if constexpr (sizeof(S) * kNg == 8)
          *reinterpret_cast<uint2*>(s[m][h]) =
              __ldg(reinterpret_cast<const uint2*>(sp + 8 * h * kNg));
        else if constexpr (sizeof(S) * kNg == 4)
          *reinterpret_cast<uint32_t*>(s[m][h]) =
              __ldg(reinterpret_cast<const uint32_t*>(sp + 8 * h * kNg));
        else
          s[m][h][0] = __ldg(sp + 8 * h * kNg);
      }
    }
  }
};

// A CTA owns kMT * 16 output rows of one expert; its warps split the columns
// (warp w takes blocks w, w + 8, ..) and their partial sums meet in shared
// memory in warp order.  NT * 8 sorted rows per pass.
template <int GROUP, typename S, int NT>
__device__ __forceinline__ void pass(const Params& P, int e, int mt0, int n_mt, int row0, int rows,
                                     const int* tok, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kNg = kCols / GROUP;
  const uint4* xr[NT];  // this lane's row of x in each column tile (null: no row)
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = t * 8 + lane / 4;
    const int tk = r < rows ? tok[r] : -1;
    xr[t] = tk >= 0 ? reinterpret_cast<const uint4*>(P.x + (long)tk * P.d) + lane % 4 : nullptr;
  }
  float acc[kMT][NT][4];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;

  const long blk0 = ((long)e * P.MT + mt0) * P.KB;
  const int d8 = P.d / 8;
  for (int kb = warp; kb < P.KB; kb += kWarps) {
    Frag<GROUP, S> cur;
    uint4 xc[NT][4];
    cur.load(P, blk0 + kb, P.KB, n_mt, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = kb * 16 + 4 * i;  // 16-byte units of x; + lane % 4 is in xr
        xc[t][i] = xr[t] && c + lane % 4 < d8 ? __ldg(xr[t] + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      if (m >= n_mt) continue;
#pragma unroll
      for (int g = 0; g < kNg; ++g) {
        float c[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[t][i] = 0.0f;
#pragma unroll
        for (int ii = 0; ii < GROUP / 32; ++ii) {
          const int i = g * (GROUP / 32) + ii;
          const uint32_t w0 = reinterpret_cast<const uint32_t*>(&cur.w[m][0])[i];
          const uint32_t w1 = reinterpret_cast<const uint32_t*>(&cur.w[m][1])[i];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t a[4] = {widen2(w0, 8 * s), widen2(w1, 8 * s), widen2(w0, 8 * s + 4),
                                   widen2(w1, 8 * s + 4)};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t b0 = s ? xc[t][i].z : xc[t][i].x;
              const uint32_t b1 = s ? xc[t][i].w : xc[t][i].y;
              mma16816(c[t], a, b0, b1);
            }
          }
        }
        const float s0 = to_f32(cur.s[m][0][g]), s1 = to_f32(cur.s[m][1][g]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[m][t][0] = fmaf(s0, c[t][0], acc[m][t][0]);
          acc[m][t][1] = fmaf(s0, c[t][1], acc[m][t][1]);
          acc[m][t][2] = fmaf(s1, c[t][2], acc[m][t][2]);
          acc[m][t][3] = fmaf(s1, c[t][3], acc[m][t][3]);
        }
      }
    }
  }
  // red[warp][row of x][output row]: acc 0, 1 are columns 2 (l % 4), + 1 of
  // output row l / 4; acc 2, 3 the same columns of output row l / 4 + 8
  constexpr int kN = kMT * kRows;
  float* mine = red + warp * (NT * 8 * kN);
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mine[(t * 8 + 2 * (lane % 4) + (i & 1)) * kN + m * kRows + lane / 4 + 8 * (i >> 1)] =
            acc[m][t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * kN; i += kThreads) {
    const int r = i / kN, n = mt0 * kRows + i % kN;
    if (n >= P.n_out) continue;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w * (NT * 8 * kN) + i];
    const __nv_bfloat16 b = __float2bfloat16_rn(s);
    P.out[(long)(row0 + r) * P.n_out + n] = *reinterpret_cast<const uint16_t*>(&b);
  }
  __syncthreads();
}

constexpr int kMaxNT = 2;  // 16 sorted rows per pass over the expert's weights

template <int GROUP, typename S>
__global__ void __launch_bounds__(kThreads, 2) expert_w4_kernel(const Params P) {
  __shared__ int found[3];
  __shared__ int tok[8 * kMaxNT];
  __shared__ __align__(16) float red[kWarps * kMaxNT * 8 * kMT * kRows];
  const int tid = threadIdx.x;
  const int n = P.T * P.k;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  if (P.rows_mode) {
    const int j = blockIdx.y;
    for (int e = tid; e < P.N_r; e += kThreads) {
      const int a = P.offsets[e], b = P.offsets[e + 1];
      if (a == j && b > a) {
        found[0] = e;
        found[1] = a;
        found[2] = b < n ? b : n;
      }
    }
  } else if (tid == 0) {
    const int e = blockIdx.y;
    const int a = P.offsets[e], b = P.offsets[e + 1];
    if (b > a && a >= 0) {
      found[0] = e;
      found[1] = a;
      found[2] = b < n ? b : n;
    }
  }
  __syncthreads();
  const int e = found[0];
  if (e < 0) return;
  const int begin = found[1], end = found[2];
  const int mt0 = blockIdx.x * kMT;
  const int n_mt = P.MT - mt0 < kMT ? P.MT - mt0 : kMT;
  for (int row0 = begin; row0 < end; row0 += 8 * kMaxNT) {
    const int rows = end - row0 < 8 * kMaxNT ? end - row0 : 8 * kMaxNT;
    __syncthreads();
    if (tid < rows) {
      int t = row0 + tid;
      if (P.perm) {
        const int p = P.perm[row0 + tid];
        t = p >= 0 && p < n ? p / P.k : -1;
        if (t < 0) mr_raise(MR_FLAG_BAD_INDEX);
      }
      tok[tid] = t;
    }
    __syncthreads();
    if (rows <= 8) pass<GROUP, S, 1>(P, e, mt0, n_mt, row0, rows, tok, red);
    else pass<GROUP, S, 2>(P, e, mt0, n_mt, row0, rows, tok, red);
  }
}

}  // namespace w4
}  // namespace mr

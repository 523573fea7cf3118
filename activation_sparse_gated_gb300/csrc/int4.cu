// int4.cu -- 4-bit weights without a handle: codes and scales of a bf16 matrix
// and back, the product of bf16 tokens by 4-bit weights, and the gated block
// h = A(x W1^T) .* (x W3^T) of 4-bit weights.
//
// A code is an integer in -7 .. 7; a group of columns of a row (64, 128, .. or
// the whole row) shares one fp32 scale s = max|w| / 7, and w stands for code * s.
// Byte b of a row holds code 2 b in its low nibble and 2 b + 1 in its high one,
// two's complement: the layout of the handles' int4 weights.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

constexpr int I4_GROUP = 64;    // groups are multiples of this many columns
constexpr int I4_WARPS = 8;     // warps of a block
constexpr int I4_UNIT = 1024;   // columns of a row that a warp of the element kernels takes: 32 a lane

// index of the group that 64-column chunk c (< 2^10) lies in: c / d by a product, exact for c, d < 2^10
__host__ __device__ inline uint32_t group_magic(int chunks_per_group) { return ((1u << 20) + chunks_per_group - 1) / chunks_per_group; }
__device__ __forceinline__ int group_of(int c, uint32_t magic) { return (int)(((uint32_t)c * magic) >> 20); }

// ------------------------------------------------------------------ codes

// The codes of eight packed bf16 values, a nibble each.  1.5 * 2^23 + v / s rounds to an integer, to even, whose low
// nibble is the code; the product with 1 / s is off by a few units in the last place, so it decides as the correctly
// rounded quotient does unless it lies near a half, and only then is that taken.
__device__ __forceinline__ uint32_t codes8(const uint4& c, float s, float inv) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const float2 round = make_float2(12582912.f, 12582912.f), minus = make_float2(-1.f, -1.f), iv = make_float2(inv, inv);
  uint32_t out = 0;
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    float2 t = round, d = round;
    ffma2(t, v, iv);
    ffma2(d, t, minus);  // the code, negated
    ffma2(d, v, iv);
    far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
    out |= (__float_as_uint(t.x) & 15u) << (8 * i) | (__float_as_uint(t.y) & 15u) << (8 * i + 4);
  }
  if (far < 0.4999f && s > 1e-30f && s < 1e30f) return out;
  out = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    const int q = min(max(__float2int_rn(__fdiv_rn(v, s)), -7), 7);
    out |= ((uint32_t)q & 15u) << (4 * i);
  }
  return out;
}

// the largest |value| of eight, as bits (ordered like the values, NaN above infinity)
__device__ __forceinline__ uint32_t max8(const uint4& c) {
  uint32_t m = 0;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) asm("max.s16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j] & 0x7fff7fffu));
  return max(m << 16, m & 0xffff0000u);
}

// The group's scale from its largest magnitude.  A group that holds a NaN or an infinity: scale NaN, codes 0, so that
// whatever is computed from it is NaN.  A group of zeros: scale 0, codes 0.
__device__ __forceinline__ float scale_of(uint32_t m) {
  return m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(m), 7.f);
}

struct QuantArgs {
  const uint16_t* w;
  long long ldw;
  uint8_t* q;
  float* s;
  int N, K, group, G;
  uint32_t magic;
};

// Groups of 64, 128 or 256 columns: LPG = group / 8 lanes hold a group, so a shuffle finds its maximum and the weights
// are read once.  A warp takes 1024 columns of one row, 16 bytes a lane four times.
template <int LPG>
__global__ void __launch_bounds__(32 * I4_WARPS) quantize_int4_kernel(const QuantArgs a) {
  const int lane = threadIdx.x & 31, c0 = blockIdx.y * I4_UNIT + lane * 8;
  const long long n = (long long)blockIdx.x * I4_WARPS + (threadIdx.x >> 5);
  pdl_launch_dependents();
  pdl_wait();
  if (n >= a.N) return;
  const uint16_t* row = a.w + n * a.ldw;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + 256 * i;
    v[i] = c < a.K ? __ldcs(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + 256 * i;
    uint32_t m = max8(v[i]);
#pragma unroll
    for (int o = 1; o < LPG; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (c >= a.K) continue;
    const float s = scale_of(m);
    if ((lane & (LPG - 1)) == 0) a.s[n * a.G + c / (8 * LPG)] = s;
    const bool zero = m == 0 || m >= 0x7f800000u || s == 0.f;
    *reinterpret_cast<uint32_t*>(a.q + n * (a.K / 2) + c / 2) = zero ? 0u : codes8(v[i], s, __fdiv_rn(1.f, s));
  }
}

// Any other group, whole rows among them: a block a group.  Up to V pieces of eight values a thread stay in registers
// between the maximum and the codes; longer groups (V = 0) are read twice.
template <int V>
__global__ void __launch_bounds__(32 * I4_WARPS) quantize_int4_wide_kernel(const QuantArgs a) {
  __shared__ uint32_t s_max[I4_WARPS];
  constexpr int NT = 32 * I4_WARPS;
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const long long n = blockIdx.x;
  const int c0 = blockIdx.y * a.group, pieces = min(a.group, a.K - c0) / 8;
  const uint4* row = reinterpret_cast<const uint4*>(a.w + n * a.ldw + c0);
  uint32_t* out = reinterpret_cast<uint32_t*>(a.q + n * (a.K / 2) + c0 / 2);
  uint4 v[V > 0 ? V : 1];
  uint32_t m = 0;
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = tid + i * NT < pieces ? __ldcs(row + tid + i * NT) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, max8(v[i]));
  } else {
    for (int i = tid; i < pieces; i += NT) m = max(m, max8(row[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, s_max[tid & (I4_WARPS - 1)]);
  const float s = scale_of(m);
  if (tid == 0) a.s[n * a.G + blockIdx.y] = s;
  const bool zero = m == 0 || m >= 0x7f800000u || s == 0.f;
  const float inv = __fdiv_rn(1.f, s);
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + i * NT < pieces) out[tid + i * NT] = zero ? 0u : codes8(v[i], s, inv);
  } else {
    for (int i = tid; i < pieces; i += NT) out[i] = zero ? 0u : codes8(row[i], s, inv);
  }
}

// ------------------------------------------------------------------ values

enum { I4_BF16, I4_F32, I4_SPLIT };

struct ValueArgs {
  const uint8_t* q[2];  // blockIdx.z: which matrix
  const float* s[2];
  void* y[2];
  long long ldy;
  int N, K, G, half;  // I4_SPLIT: columns of a part
  uint32_t magic;
};

// y = code * scale, eight codes (four bytes) a lane, 1024 columns of a row a warp.  The product is rounded to fp32, then
// to y's type.  I4_SPLIT: two bf16 matrices side by side whose sum is the value to 2^-16, [high | low], each filled up
// with zeros to `half` columns.
template <int MODE>
__global__ void __launch_bounds__(32 * I4_WARPS) dequantize_int4_kernel(const ValueArgs a) {
  const int lane = threadIdx.x & 31, c0 = blockIdx.y * I4_UNIT + lane * 8, z = blockIdx.z;
  const long long n = (long long)blockIdx.x * I4_WARPS + (threadIdx.x >> 5);
  pdl_launch_dependents();
  pdl_wait();
  if (n >= a.N) return;
  const uint8_t* row = (z ? a.q[1] : a.q[0]) + n * (a.K / 2);
  const float* srow = (z ? a.s[1] : a.s[0]) + n * a.G;
  void* y = z ? a.y[1] : a.y[0];
  uint32_t w[4];
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + 256 * i;
    w[i] = 0x88888888u;
    s[i] = 0.f;
    if (c < a.K) {
      w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + c / 2)) ^ 0x88888888u;
      s[i] = __ldg(srow + group_of(c / I4_GROUP, a.magic));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + 256 * i;
    if (c >= (MODE == I4_SPLIT ? a.half : a.K)) continue;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)  // a code plus 8 is a nibble u; the float with bits 0x4b000000 | u is 2^23 + u
      f[j] = (__uint_as_float((w[i] >> (4 * j) & 15u) | 0x4b000000u) - 8388616.f) * s[i];
    if constexpr (MODE == I4_F32) {
      float4* to = reinterpret_cast<float4*>(static_cast<float*>(y) + n * a.ldy + c);
      to[0] = make_float4(f[0], f[1], f[2], f[3]);
      to[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = pack_bf16x2_rn(f[2 * j], f[2 * j + 1]);
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + n * a.ldy + c);
      *to = make_uint4(h[0], h[1], h[2], h[3]);
      if constexpr (MODE == I4_SPLIT) {
        uint32_t l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float d0 = f[2 * j] - __uint_as_float(h[j] << 16), d1 = f[2 * j + 1] - __uint_as_float(h[j] & 0xffff0000u);
          if (!(fabsf(d0) < 1e38f)) d0 = 0.f;  // the high part is no number, or has all there is
          if (!(fabsf(d1) < 1e38f)) d1 = 0.f;
          l[j] = pack_bf16x2_rn(d0, d1);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + n * a.ldy + a.half + c) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
}

// ------------------------------------------------------------------ products of few tokens
//
// With few tokens the product is a read of the codes, so what counts is bytes in flight and few instructions a code.
// The multiply-adds go to mma.sync, which takes sixteen rows of w and eight tokens: sixteen weights a lane-instruction
// where the CUDA cores take one, and its idle columns cost nothing that the memory would not wait for.  A code becomes
// an exact bf16 in two instructions a pair (the nibble's two's complement plus 8 is u, the bf16 with bits 0x4300 | u is
// 128 + u, and 128 + u - 136 is the code), the sums of a 64-column chunk are exact products in fp32, and the scale
// multiplies the chunk's sum: nothing is rounded before the result.
//
// A lane's 16 codes of a chunk are 8 consecutive bytes of its row and their x's 32 consecutive bytes: the order of K
// inside a chunk is the MMA's to choose, as long as both operands agree.  Step i of a chunk takes columns (i, i + 4) and
// (i + 8, i + 12) of each lane's sixteen, which are nibbles i and i + 4 of its two words.
//
// A block takes 16 MR rows of w (of both matrices, GATED) and its warps cut K; their sums meet in shared memory and are
// added in the warps' order.

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// codes i and i + 4 of a word as a pair of bf16
__device__ __forceinline__ uint32_t pair4(uint32_t w, int i) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(v) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43084308u));  // (w & m) ^ c
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));
  return r;
}

struct RowsArgs {
  const uint16_t* x;
  long long ldx;
  const uint8_t* w[2];
  const float* s[2];
  void* y;
  long long ldy;
  int T, N, K, G, y_f32, act;
  uint32_t magic;
};

template <int NT, int MR, bool GATED, int U>
__global__ void __launch_bounds__(32 * I4_WARPS) int4_rows_kernel(const RowsArgs a) {
  constexpr int M = GATED ? 2 * MR : MR, P = 16 * M + 4;  // row tiles; pitch of a token's sums (no bank conflict)
  extern __shared__ float s_sum[];                        // [warps][8 NT tokens][P]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16 * MR, t0 = blockIdx.y * 8 * NT;
  pdl_launch_dependents();
  pdl_wait();
  const int nc = (a.K + 63) / 64, c0 = nc * warp / I4_WARPS, c1 = nc * (warp + 1) / I4_WARPS;
  const uint8_t* wr[M][2];
  const float* sr[M][2];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(n0 + 16 * (m % MR) + 8 * h + g, a.N - 1);
      wr[m][h] = a.w[m / MR] + (size_t)r * (a.K / 2) + 8 * t;
      sr[m][h] = a.s[m / MR] + (size_t)r * a.G;
    }
  const uint16_t* xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xr[j] = a.x + (long long)min(t0 + 8 * j + g, a.T - 1) * a.ldx + 16 * t;
  float acc[M][NT][4] = {};
  for (int c = c0; c < c1; c += U) {
    uint2 w[U][M][2];
    float s[U][M][2];
    uint4 x[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = c + u < c1 && (c + u) * 64 + 16 * t < a.K;
      const int gi = group_of(c + u, a.magic);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[u][m][h] = in ? __ldg(reinterpret_cast<const uint2*>(wr[m][h] + (c + u) * 32)) : make_uint2(0, 0);
          s[u][m][h] = c + u < c1 ? __ldg(sr[m][h] + gi) : 0.f;
        }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const bool on = in && t0 + 8 * j + g < a.T;
        const uint4* p = reinterpret_cast<const uint4*>(xr[j] + (c + u) * 64);
        x[u][j][0] = on ? __ldg(p) : make_uint4(0, 0, 0, 0);
        x[u][j][1] = on ? __ldg(p + 1) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= c1) break;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float sum[NT][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f[4] = {pair4(w[u][m][0].x, i), pair4(w[u][m][1].x, i), pair4(w[u][m][0].y, i),
                                 pair4(w[u][m][1].y, i)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 lo = x[u][j][0], hi = x[u][j][1];
            const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
            const uint32_t b0 = i < 2 ? __byte_perm(lo.x, lo.z, sel) : __byte_perm(lo.y, lo.w, sel);
            const uint32_t b1 = i < 2 ? __byte_perm(hi.x, hi.z, sel) : __byte_perm(hi.y, hi.w, sel);
            mma16816(sum[j], f, b0, b1);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[m][j][0] = fmaf(s[u][m][0], sum[j][0], acc[m][j][0]);
          acc[m][j][1] = fmaf(s[u][m][0], sum[j][1], acc[m][j][1]);
          acc[m][j][2] = fmaf(s[u][m][1], sum[j][2], acc[m][j][2]);
          acc[m][j][3] = fmaf(s[u][m][1], sum[j][3], acc[m][j][3]);
        }
      }
    }
  }
  float* mine = s_sum + warp * (8 * NT * P);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[(8 * j + 2 * t + (q & 1)) * P + 16 * m + g + 8 * (q >> 1)] = acc[m][j][q];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * NT * 16 * MR; i += 32 * I4_WARPS) {
    const int tok = i / (16 * MR), r = i % (16 * MR);
    if (t0 + tok >= a.T || n0 + r >= a.N) continue;
    float v = 0.f, up = 0.f;
#pragma unroll
    for (int q = 0; q < I4_WARPS; ++q) {
      v += s_sum[q * (8 * NT * P) + tok * P + r];
      if (GATED) up += s_sum[q * (8 * NT * P) + tok * P + 16 * MR + r];
    }
    if (GATED) {
      const float gate = v != v ? v : activation(a.act, v);  // a NaN gate is live
      v = gate != 0.f ? gate * up : 0.f;                     // a dead unit is exactly 0
    }
    const size_t at = (size_t)(t0 + tok) * a.ldy + n0 + r;
    if (a.y_f32)
      static_cast<float*>(a.y)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  }
}

template <int NT, int MR, bool GATED, int U>
cudaError_t rows_go(const RowsArgs& r, cudaStream_t s) {
  constexpr size_t smem = sizeof(float) * I4_WARPS * 8 * NT * (16 * (GATED ? 2 * MR : MR) + 4);
  static_assert(smem <= 48 * 1024, "more than a block has without asking");
  const dim3 grid((unsigned)((r.N + 16 * MR - 1) / (16 * MR)), (unsigned)((r.T + 8 * NT - 1) / (8 * NT)));
  return ops_launch(int4_rows_kernel<NT, MR, GATED, U>, grid, 32 * I4_WARPS, smem, s, 1, r);
}

constexpr int I4_ROWS = 32;  // most tokens of the form above

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Columns of a copy's row.  A product in fp32, and the gated block, whose gate is a small difference of sums that a
// weight's rounding to bf16 would reach, take the weights as two bf16 parts each (2^-16); a bf16 product takes one: its
// rounding, 2^-8 at most a weight and independent, adds to y's own as a second one would.
size_t copy_row(int K, int split) { return split ? 2 * round_up(K, 64) : (size_t)K; }

int groups(int K, int group) { return group > 0 && group < K ? (K - 1) / group + 1 : 1; }

uint32_t magic_of(int K, int group) { return group_magic(group > 0 && group < K ? group / I4_GROUP : 1 << 10); }

}  // namespace

cudaError_t launch_quantize_int4(const void* w, long long ldw, uint8_t* q, float* sc, int N, int K, int group,
                                 cudaStream_t s) {
  QuantArgs a = {static_cast<const uint16_t*>(w), ldw, q, sc, N, K, group > 0 && group < K ? group : K,
                 groups(K, group), 0};
  if (a.group == 64 || a.group == 128 || a.group == 256) {
    const dim3 grid((unsigned)((N + I4_WARPS - 1) / I4_WARPS), (unsigned)((K + I4_UNIT - 1) / I4_UNIT));
    auto kernel = a.group == 64 ? quantize_int4_kernel<8> : a.group == 128 ? quantize_int4_kernel<16> : quantize_int4_kernel<32>;
    return ops_launch(kernel, grid, 32 * I4_WARPS, 0, s, 1, a);
  }
  const dim3 grid((unsigned)N, (unsigned)a.G);
  const int per = (a.group / 8 + 32 * I4_WARPS - 1) / (32 * I4_WARPS);
  auto kernel = per <= 2 ? quantize_int4_wide_kernel<2> : per <= 8 ? quantize_int4_wide_kernel<8> : quantize_int4_wide_kernel<0>;
  return ops_launch(kernel, grid, 32 * I4_WARPS, 0, s, 1, a);
}

cudaError_t launch_dequantize_int4(const uint8_t* q, const float* sc, void* y, long long ldy, int N, int K, int group,
                                   int y_f32, cudaStream_t s) {
  ValueArgs a = {{q, q}, {sc, sc}, {y, y}, ldy, N, K, groups(K, group), 0, magic_of(K, group)};
  const dim3 grid((unsigned)((N + I4_WARPS - 1) / I4_WARPS), (unsigned)((K + I4_UNIT - 1) / I4_UNIT));
  return ops_launch(y_f32 ? dequantize_int4_kernel<I4_F32> : dequantize_int4_kernel<I4_BF16>, grid, 32 * I4_WARPS, 0, s, 1, a);
}

size_t int4_workspace(int T, int N, int K, int split, int gated) {
  return T <= I4_ROWS ? 0 : (gated ? 2 : 1) * round_up(2 * (size_t)N * copy_row(K, split), 256);
}

cudaError_t launch_matmul_int4(const Int4Args& a, cudaStream_t s) {
  const bool gated = a.w3 != nullptr;
  if (a.T <= I4_ROWS) {
    const RowsArgs r = {static_cast<const uint16_t*>(a.x), a.ldx, {a.w, a.w3}, {a.sw, a.s3}, a.y, a.ldy, a.T, a.N, a.K,
                        groups(a.K, a.group), a.y_f32, a.act, magic_of(a.K, a.group)};
    if (gated) {
      if (a.T <= 8) return rows_go<1, 1, true, 4>(r, s);
      if (a.T <= 16) return rows_go<2, 1, true, 2>(r, s);
      return rows_go<4, 1, true, 1>(r, s);
    }
    if (a.T <= 8) return rows_go<1, 1, false, 4>(r, s);
    if (a.T <= 16) return rows_go<2, 1, false, 2>(r, s);
    return rows_go<4, 2, false, 1>(r, s);
  }
  // more tokens: the weights as bf16 copies, then the products on the tensor cores
  const int split = a.y_f32 || gated;
  const size_t row = copy_row(a.K, split), one = round_up(2 * (size_t)a.N * row, 256);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  ValueArgs v = {{a.w, gated ? a.w3 : a.w}, {a.sw, gated ? a.s3 : a.sw}, {ws, ws + one}, (long long)row, a.N, a.K,
                 groups(a.K, a.group), split ? (int)(row / 2) : 0, magic_of(a.K, a.group)};
  const dim3 grid((unsigned)((a.N + I4_WARPS - 1) / I4_WARPS), (unsigned)((a.K + I4_UNIT - 1) / I4_UNIT), gated ? 2u : 1u);
  cudaError_t e = ops_launch(split ? dequantize_int4_kernel<I4_SPLIT> : dequantize_int4_kernel<I4_BF16>, grid, 32 * I4_WARPS,
                             0, s, 1, v);
  if (e != cudaSuccess) return e;
  GmmArgs p;
  p.x = a.x;
  p.ldx = a.ldx;
  p.w = ws;
  p.w3 = gated ? ws + one : nullptr;
  p.y = a.y;
  p.ldy = a.ldy;
  p.R = p.XR = a.T;
  p.N = a.N;
  p.K = a.K;
  p.split = split;
  p.y_f32 = a.y_f32;
  p.act = a.act;
  return launch_gmm(p, s);
}

}  // namespace sffn

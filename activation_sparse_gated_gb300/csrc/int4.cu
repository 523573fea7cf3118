// int4.cu -- 4-bit weights without a handle: codes and scales of a bf16 matrix
// and back, the product of bf16 tokens by 4-bit weights, and the gated block
// h = A(x W1^T) .* (x W3^T) of 4-bit weights.
//
// A code is an integer in -7 .. 7; a group of columns of a row (64, 128, .. or
// the whole row) shares one fp32 scale s = max|w| / 7, and w stands for code * s.
// Byte b of a row holds code 2 b in its low nibble and 2 b + 1 in its high one,
// two's complement: the layout of the handles' int4 weights.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "ops.h"
#include "tc.cuh"

namespace sffn {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // ffn_tc.cu

namespace {

constexpr int I4_GROUP = 64;    // groups are multiples of this many columns
constexpr int I4_WARPS = 8;     // warps of a block
constexpr int I4_UNIT = 1024;   // columns of a row that a warp of the element kernels takes: 32 a lane

// index of the group that 64-column chunk c (< 2^10) lies in: c / d by a product, exact for c, d < 2^10
__host__ __device__ inline uint32_t group_magic(int chunks_per_group) { return ((1u << 20) + chunks_per_group - 1) / chunks_per_group; }
__device__ __forceinline__ int group_of(int c, uint32_t magic) { return (int)(((uint32_t)c * magic) >> 20); }

// ------------------------------------------------------------------ codes

// The codes of eight packed bf16 values, a nibble each; inv is 1 / s, correctly rounded.  A code is decided by the correctly
// rounded quotient, which here comes from inv by Markstein's theorem (1990): q = v inv is within a unit in the last place of v
// / s, r = v - q s is exact in a fused multiply-add, and q + r inv then rounds to the quotient, ties and all (s = max / 7 of a
// bf16 value is never just below a power of two, the theorem's exception).  1.5 * 2^23 + quotient rounds to an integer, to
// even, whose low nibble is the code.  (Ties are common: half a group's maximum is 3.5 scales.  Deciding by v inv alone and
// dividing what lies near a half took 40.5 us for 14336 x 4096 weights, so often did some lane divide; this, with nothing else
// changed, 28.9.)
__device__ __forceinline__ uint32_t codes8(const uint4& c, float s, float inv) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  if (!(s > 1e-30f && s < 1e30f)) {  // out of the theorem's range: the residual or inv may underflow
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
      out |= ((uint32_t)min(max(__float2int_rn(__fdiv_rn(v, s)), -7), 7) & 15u) << (4 * i);
    }
    return out;
  }
  const float2 iv = make_float2(inv, inv), minus = make_float2(-s, -s), round = make_float2(12582912.f, 12582912.f);
  uint32_t pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    float2 q = make_float2(0.f, 0.f), r = v;
    ffma2(q, v, iv);
    ffma2(r, q, minus);
    ffma2(q, r, iv);
    const float2 t = fadd2(q, round);
    pair[i] = (__float_as_uint(t.x) & 15u) | (__float_as_uint(t.y) << 4 & ~15u);  // the low byte
  }
  return __byte_perm(__byte_perm(pair[0], pair[1], 0x0040), __byte_perm(pair[2], pair[3], 0x0040), 0x5410);
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
};

// Groups of 64, 128, .. 1024 columns: a lane takes 32 columns and LPG = group / 32 lanes hold a group, so a shuffle or a few
// find its maximum, the scale is computed once for 32 values and the weights are read once.  A warp takes 1024 columns of one
// row.  (Eight columns a lane four times, each with its scale: 28.9 us for 14336 x 4096 in groups of 64; so
// 24.1, 90 % of the copy rate.)
template <int LPG>
__global__ void __launch_bounds__(32 * I4_WARPS) quantize_int4_kernel(const QuantArgs a) {
  const int lane = threadIdx.x & 31, c0 = blockIdx.y * I4_UNIT + lane * 32;
  const long long n = (long long)blockIdx.x * I4_WARPS + (threadIdx.x >> 5);
  pdl_launch_dependents();
  pdl_wait();
  if (n >= a.N) return;
  const uint4* row = reinterpret_cast<const uint4*>(a.w + n * a.ldw + c0);
  uint4 v[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = c0 + 8 * i < a.K ? __ldg(row + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max8(v[i]));
#pragma unroll
  for (int o = 1; o < LPG; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (c0 >= a.K) return;
  const float s = scale_of(m);
  if ((lane & (LPG - 1)) == 0) a.s[n * a.G + c0 / (32 * LPG)] = s;
  const bool zero = m == 0 || m >= 0x7f800000u || s == 0.f;
  const float inv = __frcp_rn(s);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = zero ? 0u : codes8(v[i], s, inv);
  // (K is a multiple of 16: a row's codes are 8-byte aligned, and its last lane has all of its 32 columns or half of them)
  uint2* out = reinterpret_cast<uint2*>(a.q + n * (a.K / 2) + c0 / 2);
  if (a.K % 32 == 0) {
    *reinterpret_cast<uint4*>(out) = make_uint4(q[0], q[1], q[2], q[3]);
  } else {
    out[0] = make_uint2(q[0], q[1]);
    if (c0 + 16 < a.K) out[1] = make_uint2(q[2], q[3]);
  }
}

// Other groups of up to 2048 columns: a warp a group, up to eight pieces of eight values a lane.
__global__ void __launch_bounds__(32 * I4_WARPS) quantize_int4_warp_kernel(const QuantArgs a) {
  const int lane = threadIdx.x & 31, gi = blockIdx.y * I4_WARPS + (threadIdx.x >> 5);
  pdl_launch_dependents();
  pdl_wait();
  if (gi >= a.G) return;
  const long long n = blockIdx.x;
  const int c0 = gi * a.group, pieces = min(a.group, a.K - c0) / 8;
  const uint4* row = reinterpret_cast<const uint4*>(a.w + n * a.ldw + c0);
  uint32_t* out = reinterpret_cast<uint32_t*>(a.q + n * (a.K / 2) + c0 / 2);
  uint4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (32 * i < pieces) v[i] = lane + 32 * i < pieces ? __ldcs(row + lane + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (32 * i < pieces) m = max(m, max8(v[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  const float s = scale_of(m);
  if (lane == 0) a.s[n * a.G + gi] = s;
  const bool zero = m == 0 || m >= 0x7f800000u || s == 0.f;
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 32 * i < pieces) out[lane + 32 * i] = zero ? 0u : codes8(v[i], s, inv);
}

// Longer groups, whole rows among them: a block a group.  Up to V pieces of eight values a thread stay in registers
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
  const float inv = __frcp_rn(s);
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

// The code in the low nibble: plus 8 (the caller's XOR) it is u, and the float with bits 0x4b000000 | u is 2^23 + u.
__device__ __forceinline__ float value_of(uint32_t u) { return __uint_as_float((u & 15u) | 0x4b000000u) - 8388616.f; }

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
  if constexpr (MODE == I4_F32) {  // four codes a lane eight times, so that a store is 16 bytes of consecutive ones
    uint32_t v[8];
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = blockIdx.y * I4_UNIT + 128 * i + 4 * lane;
      v[i] = 0;
      f[i] = 0.f;
      if (c < a.K) {
        v[i] = __ldg(reinterpret_cast<const uint16_t*>(row + c / 2)) ^ 0x8888u;
        f[i] = __ldg(srow + group_of(c / I4_GROUP, a.magic));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = blockIdx.y * I4_UNIT + 128 * i + 4 * lane;
      if (c < a.K)
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(y) + n * a.ldy + c),
               make_float4(value_of(v[i]) * f[i], value_of(v[i] >> 4) * f[i], value_of(v[i] >> 8) * f[i], value_of(v[i] >> 12) * f[i]));
    }
  } else {
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
      for (int j = 0; j < 8; ++j) f[j] = value_of(w[i] >> (4 * j)) * s[i];
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = pack_bf16x2_rn(f[2 * j], f[2 * j + 1]);
      uint16_t* to = static_cast<uint16_t*>(y) + n * a.ldy + c;
      *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
      if constexpr (MODE == I4_SPLIT) {
        uint32_t l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float d0 = f[2 * j] - __uint_as_float(h[j] << 16), d1 = f[2 * j + 1] - __uint_as_float(h[j] & 0xffff0000u);
          if (!(fabsf(d0) < 1e38f)) d0 = 0.f;  // the high part is no number, or has all there is
          if (!(fabsf(d1) < 1e38f)) d1 = 0.f;
          l[j] = pack_bf16x2_rn(d0, d1);
        }
        *reinterpret_cast<uint4*>(to + a.half) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
}

// ------------------------------------------------------------------ products of few tokens
//
// With few tokens the product is a read of the codes, so what counts is bytes in flight and few instructions a code.
// The multiply-adds go to mma.sync, which takes sixteen rows of w and eight tokens: an instruction for eight weights a lane
// and all the tokens, where the CUDA cores take one or two weights and one token; columns without a token cost nothing that
// the codes would not wait for.  A code becomes
// an exact bf16 in two instructions a pair (the nibble's two's complement plus 8 is u, the bf16 with bits 0x4300 | u is
// 128 + u, and 128 + u - 136 is the code), the sums of a 64-column chunk are exact products in fp32, and the scale
// multiplies the chunk's sum: nothing is rounded before the result.
//
// A lane's 16 codes of a chunk are 8 consecutive bytes of its row and their x's 32 consecutive bytes: the order of K
// inside a chunk is the MMA's to choose, as long as both operands agree.  Step i of a chunk takes columns (i, i + 4) and
// (i + 8, i + 12) of each lane's sixteen, which are nibbles i and i + 4 of its two words.
//
// Up to eight tokens (int4_rows_kernel; up to sixteen with two tiles of tokens, NT): a block takes 16 rows of w (of both
// matrices, GATED), its W warps take pairs of chunks in turn, and their sums meet in shared memory and are added in the warps'
// order.  Measured (us a call in a graph, the same codes again, from L2; one token): 7168 x 2560 4.5 (2.1 of it a launch), 14336 x
// 4096 9.0, 2560 x 7168 5.5, 13 tokens 7.7; gated, two 7168 x 2560 5.7; codes from memory: 14336 x 4096 11.0 (3.0 TB/s).  What
// bounds it is instructions and their latency: some 70 a chunk of 16 rows, 44 of them the codes.  Loads that no condition
// guards (a token past T reads the last one's x, missing columns are the last pair's alone) took a third of them out (gated,
// codes from memory, 10.3 -> 7.9).  Not faster: sixteen bytes of codes a lane and halves traded between lanes, one pair at a time,
// a warp's codes and x through a TMA ring (7168 x 2560 6.6).

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same from zero
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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

// A(z) u: a NaN gate is live, a dead unit exactly 0.
__device__ __forceinline__ float gated(int act, float z, float u) {
  const float gate = z != z ? z : activation(act, z);
  return gate != 0.f ? gate * u : 0.f;
}

template <bool GATED, int NT, int W>
__global__ void __launch_bounds__(32 * W) int4_rows_kernel(const RowsArgs a) {
  constexpr int M = GATED ? 2 : 1, P = 16 * M + 4;  // matrices; pitch of a token's sums (no bank conflict)
  __shared__ float s_sum[W * 8 * NT * P];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 8 * NT;
  pdl_launch_dependents();
  pdl_wait();
  const uint8_t* wr[M][2];
  const float* sr[M][2];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(n0 + 8 * h + g, a.N - 1);
      wr[m][h] = a.w[m] + (size_t)r * (a.K / 2) + warp * 64 + 8 * t;
      sr[m][h] = a.s[m] + (size_t)r * a.G;
    }
  // tokens past T are computed on the last one and not stored
  const uint16_t* xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xr[j] = a.x + (long long)min(t0 + 8 * j + g, a.T - 1) * a.ldx + warp * 128 + 16 * t;
  float acc[M][NT][4] = {};
  // U pairs of 64-column chunks, W pairs apart, from pair c on.  CUT: the last pair, of which columns may be missing.
  auto step = [&](auto pairs, auto cut, int c) {
    constexpr int U = decltype(pairs)::value;
    constexpr bool CUT = decltype(cut)::value;
    uint2 w[U][2][M][2];
    float s[M][2];
    uint4 x[U][2][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = !CUT || c * 128 + 64 * q + 16 * t < a.K;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            w[u][q][m][h] = in ? __ldg(reinterpret_cast<const uint2*>(wr[m][h] + u * (64 * W) + 32 * q)) : make_uint2(0, 0);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4* p = reinterpret_cast<const uint4*>(xr[j] + u * (128 * W) + 64 * q);
          x[u][q][j][0] = in ? __ldg(p) : make_uint4(0, 0, 0, 0);
          x[u][q][j][1] = in ? __ldg(p + 1) : make_uint4(0, 0, 0, 0);
        }
      }
    {  // lane t of four holds the scale of the t-th of the 2 U chunks
      const int ch = 2 * (c + (U == 2 ? (t >> 1) * W : 0)) + (t & 1);
      const bool in = !CUT || ch * 64 < a.K;
      const int gi = group_of(in ? ch : 0, a.magic);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[m][h] = in ? __ldg(sr[m][h] + gi) : 0.f;
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) wr[m][h] += U * 64 * W;
#pragma unroll
    for (int j = 0; j < NT; ++j) xr[j] += U * 128 * W;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float sum[M][NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
          uint32_t b[NT][2];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 lo = x[u][q][j][0], hi = x[u][q][j][1];
            b[j][0] = i < 2 ? __byte_perm(lo.x, lo.z, sel) : __byte_perm(lo.y, lo.w, sel);
            b[j][1] = i < 2 ? __byte_perm(hi.x, hi.z, sel) : __byte_perm(hi.y, hi.w, sel);
          }
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const uint2 (&v)[2] = w[u][q][m];
            const uint32_t f[4] = {pair4(v[0].x, i), pair4(v[1].x, i), pair4(v[0].y, i), pair4(v[1].y, i)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              if (i == 0)
                mma16816_first(sum[m][j], f, b[j][0], b[j][1]);
              else
                mma16816(sum[m][j], f, b[j][0], b[j][1]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float sc = __shfl_sync(0xffffffffu, s[m][h], 2 * u + q, 4);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[m][j][2 * h] = fmaf(sc, sum[m][j][2 * h], acc[m][j][2 * h]);
              acc[m][j][2 * h + 1] = fmaf(sc, sum[m][j][2 * h + 1], acc[m][j][2 * h + 1]);
            }
          }
      }
  };
  const int whole = a.K / 128;  // pairs without a missing column; the warps take them in turn, so that they read rows together
  int c = warp;
  if constexpr (NT * M <= 2)
    for (; c + W < whole; c += 2 * W) step(std::integral_constant<int, 2>(), std::false_type(), c);
  for (; c < whole; c += W) step(std::integral_constant<int, 1>(), std::false_type(), c);
  if (c == whole && a.K % 128 != 0) step(std::integral_constant<int, 1>(), std::true_type(), c);
  float* mine = s_sum + warp * (8 * NT * P);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[(8 * j + 2 * t + (q & 1)) * P + 16 * m + g + 8 * (q >> 1)] = acc[m][j][q];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * NT * 16; i += 32 * W) {
    const int tok = i / 16, r = i % 16;
    if (t0 + tok >= a.T || n0 + r >= a.N) continue;
    float v = 0.f, up = 0.f;
#pragma unroll
    for (int q = 0; q < W; ++q) {  // in the warps' order
      v += s_sum[q * (8 * NT * P) + tok * P + r];
      if (GATED) up += s_sum[q * (8 * NT * P) + tok * P + 16 + r];
    }
    if (GATED) v = gated(a.act, v, up);
    const size_t at = (size_t)(t0 + tok) * a.ldy + n0 + r;
    if (a.y_f32)
      static_cast<float*>(a.y)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  }
}

template <bool GATED, int NT>
cudaError_t rows_go(const RowsArgs& r, cudaStream_t s) {
  const dim3 grid((unsigned)((r.N + 15) / 16), (unsigned)((r.T + 8 * NT - 1) / (8 * NT)));
  // More warps a block, as many as leave room for two blocks an SM, where that is all blocks at once (us, eight warps / as
  // here: one token, 2560 x 7168 7.0 / 5.7, 4096 x 4096 5.7 / 4.1, gated 3000 x 2560 5.7 / 4.6; 13 tokens, 2560 x 7168 9.7 / 8.0, 3000
  // x 2560 4.7 / 3.9; and else: one token, 7168 x 2560 4.9 / 5.6, gated 7.8 / 9.8).  Two tiles of tokens and two matrices have no room.
  constexpr int many = GATED && NT > 1 ? 8 : GATED || NT > 1 ? 12 : 16;
  if ((long long)grid.x * grid.y <= 2 * ops_num_sms())
    return ops_launch(int4_rows_kernel<GATED, NT, many>, grid, 32 * many, 0, s, 1, r);
  return ops_launch(int4_rows_kernel<GATED, NT, 8>, grid, 32 * 8, 0, s, 1, r);
}

constexpr int I4_STAGES = 3;
constexpr uint64_t I4_TIMEOUT_NS = 250000000ull;
constexpr uint32_t I4_BOX = 16 * 64;  // bytes of a tile's part of a warp's stage

// The weight row that row g of a tile's MMA stands for: rows g = 0 .. 3 lie in different banks of the 64-byte-swizzled box.
__device__ __forceinline__ int row_of(int g) { return (g & 1) | (g & 2) << 1 | (g & 4) >> 1; }

bool encode_codes(CUtensorMap* m, const uint8_t* w, int N, int K) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)N}, strides[1] = {(cuuint64_t)K / 2};
  const cuuint32_t box[2] = {64u, 16u}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's dynamic shared memory beyond what a block has without asking, allowed once on each device.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::once_flag (&once)[64], cudaError_t (&attr)[64]) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] { attr[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
  return attr[dev];
}

// More than sixteen tokens (int4_tile_kernel, K a multiple of 32): x is what repeats, so a block takes 128 rows of w a tile (M
// tiles; both matrices, GATED), keeps its share of x in shared memory for all of them, already in the order of the MMA's
// operands, and lets every warp walk K over its own 16 rows.  A warp's codes come by TMA, boxes of 16 rows by 128 columns
// (64 bytes), into a ring of its own.  K is cut over the blocks of a cluster, whose sums are added through distributed shared
// memory in the blocks' order.  Measured (us in a graph): 32 tokens, 7168 x 2560 9.3, 2560 x 7168 12.6; 24, 14336 x 4096
// 19.2; gated, two 14336 x 4096, 24 tokens 35.5 (each warp with x of its own from L2: 52).
constexpr int x_chunks(int NT) { return NT == 3 ? 14 : 12; }  // of x that shared memory holds at a time
constexpr size_t tile_smem(int NT, int M) {
  return 1024 + std::max<size_t>(I4_WARPS * I4_STAGES * M * I4_BOX + x_chunks(NT) * NT * 1024, sizeof(float) * 8 * NT * (16 * I4_WARPS * M + 4));
}

template <int NT, int M, bool GATED>
__global__ void __launch_bounds__(32 * I4_WARPS, 2)
    int4_tile_kernel(const __grid_constant__ CUtensorMap m0, const __grid_constant__ CUtensorMap m1, const RowsArgs a, int cut,
                     int* err) {
  constexpr int MR = GATED ? M / 2 : M, ROWS = 16 * I4_WARPS * MR;  // rows of a matrix
  constexpr int P = 16 * I4_WARPS * M + 4;                          // pitch of a token's sums
  constexpr int XC = x_chunks(NT);
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t bars[I4_WARPS][I4_STAGES];
  __shared__ int abort_flag;
  uint8_t* sm = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);  // the rings, then x [XC][NT][2][lane]; then the sums
  uint4* s_x = reinterpret_cast<uint4*>(sm + I4_WARPS * I4_STAGES * M * I4_BOX);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kr = blockIdx.x % cut, n0 = blockIdx.x / cut * ROWS, t0 = blockIdx.y * 8 * NT;
  const int nd = (a.K + 127) / 128, d0 = nd * kr / cut, d1 = nd * (kr + 1) / cut;  // this block's pairs of chunks
  uint64_t* full = bars[warp];
  if (lane == 0) {
    for (int i = 0; i < I4_STAGES; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    tma_prefetch_map(&m0);
    if (GATED) tma_prefetch_map(&m1);
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  float acc[M][NT][4] = {};
  {
    uint8_t* ring = sm + warp * (I4_STAGES * M) * I4_BOX;
    auto fetch = [&](int d, int stage) {
      if (d >= d1 || lane != 0) return;
      mbar_arrive_expect_tx(&full[stage], M * I4_BOX);
#pragma unroll
      for (int m = 0; m < M; ++m)
        tma_tile_2d(ring + (stage * M + m) * I4_BOX, m / MR ? &m1 : &m0, d * 64, n0 + 16 * (I4_WARPS * (m % MR) + warp), &full[stage]);
    };
#pragma unroll
    for (int i = 0; i < I4_STAGES; ++i) fetch(d0 + i, i);
    const float* sr[M][2];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        sr[m][h] = a.s[m / MR] + (size_t)min(n0 + 16 * (I4_WARPS * (m % MR) + warp) + 8 * h + row_of(g), a.N - 1) * a.G;
    float s[M][2];  // of the next pair of chunks: lanes with t odd the second one's
    auto scales = [&](int d) {
      const bool in = d < d1 && (2 * d + (t & 1)) * 64 < a.K;
      const int gi = group_of(2 * d + (t & 1), a.magic);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[m][h] = in ? __ldg(sr[m][h] + gi) : 0.f;
    };
    scales(d0);
    // where the lane's eight bytes of the box's two chunks are: 16-byte piece p of row r sits at p ^ (r >> 1 & 3)
    const int r0 = row_of(g), x3 = r0 >> 1 & 3;
    const uint32_t at0 = smem_u32(ring) + (uint32_t)(r0 * 64 + (((t >> 1) ^ x3) << 4) + 8 * (t & 1));
    const uint32_t at1 = smem_u32(ring) + (uint32_t)(r0 * 64 + ((((t >> 1) + 2) ^ x3) << 4) + 8 * (t & 1));
    int stage = 0;
    uint32_t par = 0;
    int done = 0;  // stages multiplied
    bool ok = true;
    for (int x0 = d0; x0 < d1; x0 += XC / 2) {
      const int xn = min(XC / 2, d1 - x0);
      if (x0 != d0) named_barrier(1, 32 * I4_WARPS);  // the chunks before have been multiplied
      for (int i = threadIdx.x; i < 2 * xn * NT * 32; i += 32 * I4_WARPS) {
        const int c = 2 * x0 + i / (NT * 32), tok = t0 + 8 * (i / 32 % NT) + (i & 31) / 4, k = c * 64 + 16 * (i & 3);
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        if (tok < a.T && k < a.K) {
          const uint4* p = reinterpret_cast<const uint4*>(a.x + (long long)tok * a.ldx + k);
          lo = __ldg(p);
          hi = __ldg(p + 1);
        }
        // step i of a chunk takes columns (i, i + 4) and (i + 8, i + 12) of a lane's sixteen
        uint4* to = s_x + (i / 32) * 64 + (i & 31);
        to[0] = make_uint4(__byte_perm(lo.x, lo.z, 0x5410), __byte_perm(hi.x, hi.z, 0x5410), __byte_perm(lo.x, lo.z, 0x7632),
                           __byte_perm(hi.x, hi.z, 0x7632));
        to[32] = make_uint4(__byte_perm(lo.y, lo.w, 0x5410), __byte_perm(hi.y, hi.w, 0x5410), __byte_perm(lo.y, lo.w, 0x7632),
                            __byte_perm(hi.y, hi.w, 0x7632));
      }
      named_barrier(1, 32 * I4_WARPS);
      for (int d = x0; d < x0 + xn; ++d) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], par, &abort_flag, err, I4_TIMEOUT_NS));
        if (!ok) break;  // (the other copies in flight are waited for below)
        const uint32_t st = (uint32_t)(stage * M) * I4_BOX;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint2 w[M][2];
          float sc[M][2];
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                           : "=r"(w[m][h].x), "=r"(w[m][h].y)
                           : "r"((q ? at1 : at0) + st + (uint32_t)m * I4_BOX + 512u * h));
              sc[m][h] = __shfl_sync(0xffffffffu, s[m][h], q, 4);
            }
          if (q == 1) {
            __syncwarp();  // the stage is read
            fetch(d + I4_STAGES, stage);
            scales(d + 1);
          }
          // a chunk's four steps over all the tiles: an MMA follows one that it doesn't wait for
          float sum[M][NT][4];
          const uint4* from = s_x + (2 * (d - x0) + q) * NT * 64 + lane;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 b[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) b[j] = from[j * 64 + h * 32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t f[M][4];
#pragma unroll
              for (int m = 0; m < M; ++m) {
                f[m][0] = pair4(w[m][0].x, 2 * h + i);
                f[m][1] = pair4(w[m][1].x, 2 * h + i);
                f[m][2] = pair4(w[m][0].y, 2 * h + i);
                f[m][3] = pair4(w[m][1].y, 2 * h + i);
              }
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                  if (h == 0 && i == 0)
                    mma16816_first(sum[m][j], f[m], b[j].x, b[j].y);
                  else
                    mma16816(sum[m][j], f[m], i ? b[j].z : b[j].x, i ? b[j].w : b[j].y);
                }
            }
          }
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[m][j][e] = fmaf(sc[m][e >> 1], sum[m][j][e], acc[m][j][e]);
        }
        if (++stage == I4_STAGES) {
          stage = 0;
          par ^= 1;
        }
        ++done;
      }
    }
    if (!ok && lane == 0)  // after a failed wait, copies in flight land before the block goes on
      for (int d = done; d < min(done + I4_STAGES, d1 - d0); ++d)
        mbar_wait_drain(&full[d % I4_STAGES], d / I4_STAGES & 1, I4_TIMEOUT_NS);
    __syncwarp();
  }
  __syncthreads();  // the rings' and x's place becomes the sums'
  float* sums = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sums[(8 * j + 2 * t + (q & 1)) * P + 16 * (I4_WARPS * m + warp) + row_of(g) + 8 * (q >> 1)] = acc[m][j][q];
  if (cut > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // four rows of a token a thread, a block of the cluster its share of them
  const uint32_t base = smem_u32(sums);
  const int live = min(8 * NT, a.T - t0);
  const int end = live * (ROWS / 4) * (kr + 1) / cut;
  for (int i = live * (ROWS / 4) * kr / cut + threadIdx.x; i < end; i += blockDim.x) {
    const int tok = i / (ROWS / 4), r = i % (ROWS / 4) * 4;
    if (n0 + r >= a.N) continue;
    float v[4] = {}, up[4] = {};
    for (int k = 0; k < cut; ++k) {
      const uint32_t at = base + (uint32_t)(tok * P + r) * 4u;
      const float4 p = cut > 1 ? ld_cluster_f4(cluster_map(at, (uint32_t)k)) : *reinterpret_cast<const float4*>(sums + tok * P + r);
      v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
      if (GATED) {
        const float4 q = cut > 1 ? ld_cluster_f4(cluster_map(at + ROWS * 4u, (uint32_t)k))
                                 : *reinterpret_cast<const float4*>(sums + tok * P + ROWS + r);
        up[0] += q.x, up[1] += q.y, up[2] += q.z, up[3] += q.w;
      }
    }
    const size_t at = (size_t)(t0 + tok) * a.ldy + n0 + r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (n0 + r + q >= a.N) break;
      if (GATED) v[q] = gated(a.act, v[q], up[q]);
      if (a.y_f32)
        static_cast<float*>(a.y)[at + q] = v[q];
      else
        static_cast<__nv_bfloat16*>(a.y)[at + q] = __float2bfloat16_rn(v[q]);
    }
  }
  if (cut > 1) cluster_sync_all();  // the sums stay until every block has read them
}

template <int NT, int M, bool GATED>
cudaError_t tile_go(const RowsArgs& r, cudaStream_t s) {
  auto kernel = int4_tile_kernel<NT, M, GATED>;
  constexpr size_t smem = tile_smem(NT, M);
  static std::once_flag once[64];
  static cudaError_t attr[64];
  cudaError_t e = allow_smem(kernel, smem, once, attr);
  if (e != cudaSuccess) return e;
  constexpr int rows = 16 * I4_WARPS * (GATED ? M / 2 : M);
  const int nb = (r.N + rows - 1) / rows, tb = (r.T + 8 * NT - 1) / (8 * NT), nc = (r.K + 127) / 128;
  // as many blocks as run at once, two an SM (24 tokens, 14336 x 4096, cut 2 / 3 / 4 / 5 / 8: 29.2 / 24.2 / 19.8 / 19.2 / 25.7 us)
  const int cut = (int)std::max<long long>(1, std::min<long long>({8, nc / 2, 2ll * ops_num_sms() / ((long long)nb * tb)}));
  int* err = nullptr;
  if ((e = ops_error_word(&err)) != cudaSuccess) return e;
  CUtensorMap m0, m1;
  if (!encode_codes(&m0, r.w[0], r.N, r.K) || !encode_codes(&m1, GATED ? r.w[1] : r.w[0], r.N, r.K)) return cudaErrorInvalidValue;
  return ops_launch(kernel, dim3((unsigned)(nb * cut), (unsigned)tb), 32 * I4_WARPS, smem, s, cut, m0, m1, r, cut, err);
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Whether the codes themselves are multiplied, or bf16 copies of them.  (us, codes / copies, N = 7168, K = 2560: bf16 48
// tokens 15.7 / 17.9, 128 26.7 / 19.6; fp32 64 tokens 15.9 / 26.9; gated 64 tokens 29.2 / 57.5, 128 50.6 / 60.6; N = 14336, K
// = 4096, bf16, 64 tokens 39.9 / 50.6.)  Rows of codes that TMA does not take go eight tokens at a time.
bool codes_themselves(int T, int K, int split) { return T <= (K % 32 != 0 ? 32 : split ? 128 : 64); }

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
                 groups(K, group)};
  auto kernel = a.group == 64 ? quantize_int4_kernel<2> : a.group == 128 ? quantize_int4_kernel<4>
              : a.group == 256 ? quantize_int4_kernel<8> : a.group == 512 ? quantize_int4_kernel<16>
              : a.group == 1024 ? quantize_int4_kernel<32> : nullptr;
  if (kernel) {
    const dim3 grid((unsigned)((N + I4_WARPS - 1) / I4_WARPS), (unsigned)((K + I4_UNIT - 1) / I4_UNIT));
    return ops_launch(kernel, grid, 32 * I4_WARPS, 0, s, 1, a);
  }
  // (4096 x 14336 in groups of 512 this way, a block / a warp each: 131 / 42 us)
  if (a.group <= 2048 && a.G > 1)
    return ops_launch(quantize_int4_warp_kernel, dim3((unsigned)N, (unsigned)((a.G + I4_WARPS - 1) / I4_WARPS)), 32 * I4_WARPS, 0, s,
                      1, a);
  const dim3 grid((unsigned)N, (unsigned)a.G);
  const int per = (a.group / 8 + 32 * I4_WARPS - 1) / (32 * I4_WARPS);
  auto wide = per <= 2 ? quantize_int4_wide_kernel<2> : per <= 8 ? quantize_int4_wide_kernel<8> : quantize_int4_wide_kernel<0>;
  return ops_launch(wide, grid, 32 * I4_WARPS, 0, s, 1, a);
}

cudaError_t launch_dequantize_int4(const uint8_t* q, const float* sc, void* y, long long ldy, int N, int K, int group,
                                   int y_f32, cudaStream_t s) {
  ValueArgs a = {{q, q}, {sc, sc}, {y, y}, ldy, N, K, groups(K, group), 0, magic_of(K, group)};
  const dim3 grid((unsigned)((N + I4_WARPS - 1) / I4_WARPS), (unsigned)((K + I4_UNIT - 1) / I4_UNIT));
  return ops_launch(y_f32 ? dequantize_int4_kernel<I4_F32> : dequantize_int4_kernel<I4_BF16>, grid, 32 * I4_WARPS, 0, s, 1, a);
}

size_t int4_workspace(int T, int N, int K, int split, int gated) {
  return codes_themselves(T, K, split) ? 0 : (gated ? 2 : 1) * round_up(2 * (size_t)N * copy_row(K, split), 256);
}

cudaError_t launch_matmul_int4(const Int4Args& a, cudaStream_t s) {
  const bool gated = a.w3 != nullptr;
  const int split = a.y_f32 || gated;
  if (codes_themselves(a.T, a.K, split)) {
    const RowsArgs r = {static_cast<const uint16_t*>(a.x), a.ldx, {a.w, a.w3}, {a.sw, a.s3}, a.y, a.ldy, a.T, a.N, a.K,
                        groups(a.K, a.group), a.y_f32, a.act, magic_of(a.K, a.group)};
    if (a.T <= 8) return gated ? rows_go<true, 1>(r, s) : rows_go<false, 1>(r, s);
    // Up to sixteen tokens, and where TMA does not take the rows of codes, the same with two tiles of tokens (us, this / the tiles
    // below, 13 tokens: 7168 x 2560 5.4 / 8.0, 14336 x 4096 14.9 / 15.7, 2560 x 7168 8.0 / 8.7, 4096 x 14336 16.7 / 15.4; gated
    // 3000 x 2560 6.4 / 9.2, 14336 x 4096 26.7 / 27.4).
    if (a.T <= 16 || a.K % 32 != 0) return gated ? rows_go<true, 2>(r, s) : rows_go<false, 2>(r, s);
    if (gated) return a.T <= 24 ? tile_go<3, 2, true>(r, s) : tile_go<4, 2, true>(r, s);
    // two tiles a block where the cut of K, eight at most, still fills the SMs (us, one / two tiles: 24 tokens, 14336 x 4096
    // 20.2 / 19.2; 32 tokens, 7168 x 2560 9.3 / 13.0)
    if ((a.N + 255) / 256 < 2 * ops_num_sms() / 8) return a.T <= 24 ? tile_go<3, 1, false>(r, s) : tile_go<4, 1, false>(r, s);
    return a.T <= 24 ? tile_go<3, 2, false>(r, s) : tile_go<4, 2, false>(r, s);
  }
  // more tokens: the weights as bf16 copies, then the products on the tensor cores
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

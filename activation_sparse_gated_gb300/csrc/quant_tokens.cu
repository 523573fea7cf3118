// quant_tokens.cu -- symmetric int8 codes of activations, one fp32 scale per
// token: s = max|x| / 127, code = round-half-to-even(x / s), both decided in
// binary32 (the convention of the library's weight codes).  An all-zero token
// gets s = 0 and codes 0; a token that holds a NaN or an infinity gets s = NaN
// and codes 0, so that whatever is computed from it is NaN.
//
// Bound by memory: 2 bytes read and 1 written per value.  One block per token
// keeps the token in registers between the maximum and the codes, so it is
// read once.  The code of a value is decided by the correctly rounded quotient,
// which costs more than the memory; a product with 1 / s is off by at most a
// few units in the last place, below 1e-4 for quotients up to 127, so it gives
// the same code unless it lies that near a half, and only then is the quotient
// taken.  (8192 tokens of 14336: 60 us, 86 % of the copy rate; 69 before the
// products were packed two to an instruction, 77 before the next token's pieces
// were requested ahead, 90 with quotients throughout.)
#include <algorithm>

#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

__device__ __forceinline__ int code_of(float v, float s) {
  const int q = __float2int_rn(__fdiv_rn(v, s));
  return q > 127 ? 127 : q < -127 ? -127 : q;
}

// The codes of four packed bf16 values by the product with 1 / s: 1.5 * 2^23 + v / s rounds to an integer, to even,
// whose low byte is the code.  *far is raised to the largest distance of a product from its code.
__device__ __forceinline__ uint32_t fast_codes(uint32_t w0, uint32_t w1, float2 inv, float* far) {
  const float2 round = make_float2(12582912.f, 12582912.f), minus = make_float2(-1.f, -1.f);
  uint32_t pair[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? w1 : w0;
    const float2 v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    float2 t = round, d = round;
    ffma2(t, v, inv);
    ffma2(d, t, minus);  // the code, negated
    ffma2(d, v, inv);
    *far = fmaxf(*far, fmaxf(fabsf(d.x), fabsf(d.y)));
    pair[i] = __byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040);
  }
  return __byte_perm(pair[0], pair[1], 0x5410);
}

// NT threads, V 16-byte pieces a thread in registers, or (V = 0) one value at a
// time from memory twice (strides that align with nothing, or longer rows).  A
// block walks tokens gridDim.x apart and requests the next one's pieces before
// it works on this one's.
//
// SHIFT: rows that start anywhere, K odd for instance, where x and q are aligned
// as wholes and x's and q's rows start at the same place in a piece of eight.
// Pieces are those of the whole tensors; a row's first and last one may belong
// to its neighbours in part: their values count as zeros and their codes are
// not written.  (4346 tokens of 9668: 37 us, one value at a time 64; 9672 28.)
template <int NT, int V, bool SHIFT>
__global__ void __launch_bounds__(NT) quantize_tokens_kernel(const uint16_t* __restrict__ x, long long ld,
                                                             int8_t* __restrict__ q, float* __restrict__ sc, int T,
                                                             int K) {
  __shared__ uint32_t s_max[2][NT / 32];
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  uint4 c[V > 0 ? V : 1], next[V > 0 ? V : 1];
  auto load = [&](uint32_t t, uint4* to) {
    const size_t start = (size_t)t * ld;
    const int ph = SHIFT ? (int)(start & 7) : 0, n = SHIFT ? (ph + K + 7) / 8 : K / 8;
    const uint4* row = reinterpret_cast<const uint4*>(x + (start - ph));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = tid + i * NT, lo = 8 * at - ph;  // lo: the piece's first value in the row
      if (SHIFT && at < n && (lo < 0 || lo + 8 > K)) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (lo + j >= 0 && lo + j < K) w[j >> 1] |= (uint32_t)x[start + lo + j] << (16 * (j & 1));
        to[i] = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        to[i] = at < n ? __ldcs(row + at) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  if constexpr (V > 0) load(blockIdx.x, next);
  int turn = 0;
  for (uint32_t t = blockIdx.x; t < (uint32_t)T; t += gridDim.x, turn ^= 1) {  // (unsigned: t may pass 2^31 at the end)
    const uint16_t* row = x + (size_t)t * ld;
    int8_t* out = q + (size_t)t * K;
    const int ph = SHIFT ? (int)((size_t)t * K & 7) : 0, n = SHIFT ? (ph + K + 7) / 8 : K / 8;
    uint32_t m = 0;  // the largest |x| as bits: ordered like the values, NaN above infinity
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = next[i];
      if (t + gridDim.x < (uint32_t)T) load(t + gridDim.x, next);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("max.s16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j] & 0x7fff7fffu));  // halves without signs are ordered ints
      }
      m = max(m << 16, m & 0xffff0000u);
    } else {
      for (int i = tid; i < K; i += NT) m = max(m, ((uint32_t)row[i] << 16) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) s_max[turn][tid >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, (tid & 31) < NT / 32 ? s_max[turn][tid & 31] : 0u);
    const bool bad = m >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(m), 127.f);
    if (tid == 0) sc[t] = s;
    const bool zero = bad || s == 0.f;
    const float inv = __fdiv_rn(1.f, s);
    const float2 inv2 = make_float2(inv, inv);
    const bool tiny = !zero && !(s > 1e-30f && s < 1e30f);
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int at = tid + i * NT;
        if (at >= n) continue;
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t o[2] = {0, 0};
        float far = 0.f;
        if (!zero) {
          o[0] = fast_codes(w[0], w[1], inv2, &far);
          o[1] = fast_codes(w[2], w[3], inv2, &far);
        }
        if (!(far < 0.4999f) || tiny) {  // near a half (or 1 / s is no number): by the quotients
          o[0] = o[1] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = (uint32_t)code_of(__uint_as_float(w[j] << 16), s) & 0xffu;
            const uint32_t hi = (uint32_t)code_of(__uint_as_float(w[j] & 0xffff0000u), s) & 0xffu;
            o[j >> 1] |= (lo | (hi << 8)) << (16 * (j & 1));
          }
        }
        const int lo = 8 * at - ph;
        if (SHIFT && (lo < 0 || lo + 8 > K)) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (lo + j >= 0 && lo + j < K) out[lo + j] = (int8_t)(o[j >> 2] >> (8 * (j & 3)));
        } else {
          __stcs(reinterpret_cast<uint2*>(out + lo), make_uint2(o[0], o[1]));
        }
      }
    } else {
      for (int i = tid; i < K; i += NT)
        out[i] = zero ? 0 : (int8_t)code_of(__uint_as_float((uint32_t)row[i] << 16), s);
    }
  }
}

template <int NT, int V, bool SHIFT = false>
cudaError_t go(const void* x, long long ld, int8_t* q, float* sc, int T, int K, cudaStream_t s) {
  return ops_launch(quantize_tokens_kernel<NT, V, SHIFT>, dim3((unsigned)std::min(T, 2048 / NT * ops_num_sms())), NT, 0, s, 1, (const uint16_t*)x, ld, q, sc, T, K);
}

}  // namespace

cudaError_t launch_quantize_tokens(const void* x, long long ld, int8_t* q, float* sc, int T, int K, cudaStream_t s) {
  const bool aligned = ((uintptr_t)x & 15) == 0 && ((uintptr_t)q & 7) == 0;
  const int most = K % 8 ? (K + 14) / 8 : K / 8;  // pieces of a row
  if (!aligned || (T > 1 && (ld - K) % 8 != 0) || most > 512 * 4) return go<256, 0>(x, ld, q, sc, T, K, s);
  if (K % 8 != 0) {
    const int n = most;
    if (n <= 128) return go<128, 1, true>(x, ld, q, sc, T, K, s);
    if (n <= 256) return go<256, 1, true>(x, ld, q, sc, T, K, s);
    if (n <= 512) return go<256, 2, true>(x, ld, q, sc, T, K, s);
    if (n <= 1024) return go<256, 4, true>(x, ld, q, sc, T, K, s);
    return go<512, 4, true>(x, ld, q, sc, T, K, s);
  }
  const int n = K / 8;
  if (n <= 128) return go<128, 1>(x, ld, q, sc, T, K, s);
  if (n <= 256) return go<256, 1>(x, ld, q, sc, T, K, s);
  if (n <= 512) return go<256, 2>(x, ld, q, sc, T, K, s);
  if (n <= 1024) return go<256, 4>(x, ld, q, sc, T, K, s);
  return go<512, 4>(x, ld, q, sc, T, K, s);
}

}  // namespace sffn

// quant_tokens.cu -- symmetric int8 codes of activations, one fp32 scale per
// token: s = max|x| / 127, code = round-half-to-even(x / s), both decided in
// binary32 (the convention of the library's weight codes).  An all-zero token
// gets s = 0 and codes 0; a token that holds a NaN or an infinity gets s = NaN
// and codes 0, so that whatever is computed from it is NaN.
//
// Bound by memory: 2 bytes read and 1 written per value.  One block per token
// keeps the token in registers between the maximum and the codes, so it is
// read once; the quotient is the correctly rounded division, which a product
// with 1 / s is not.
#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

__device__ __forceinline__ int code_of(float v, float s) {
  const int q = __float2int_rn(__fdiv_rn(v, s));
  return q > 127 ? 127 : q < -127 ? -127 : q;
}

// NT threads, V 16-byte pieces a thread in registers, or (V = 0) one value at a
// time from memory twice (rows that are not 16-byte aligned, or longer).
template <int NT, int V>
__global__ void __launch_bounds__(NT) quantize_tokens_kernel(const uint16_t* __restrict__ x, long long ld,
                                                             int8_t* __restrict__ q, float* __restrict__ sc, int T,
                                                             int K) {
  __shared__ uint32_t s_max[NT / 32];
  const int tid = threadIdx.x, t = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const uint16_t* row = x + (size_t)t * ld;
  int8_t* out = q + (size_t)t * K;
  uint4 c[V > 0 ? V : 1];
  uint32_t m = 0;  // the largest |x| as bits: ordered like the values, NaN above infinity
  if constexpr (V > 0) {
    const int n = K / 8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = tid + i * NT;
      c[i] = at < n ? reinterpret_cast<const uint4*>(row)[at] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
    }
  } else {
    for (int i = tid; i < K; i += NT) m = max(m, ((uint32_t)row[i] << 16) & 0x7fffffffu);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) m = max(m, s_max[w]);
  const bool bad = m >= 0x7f800000u;
  const float s = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(m), 127.f);
  if (tid == 0) sc[t] = s;
  const bool zero = bad || s == 0.f;
  if constexpr (V > 0) {
    const int n = K / 8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = tid + i * NT;
      if (at >= n) continue;
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
      uint32_t o[2] = {0, 0};
      if (!zero) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = (uint32_t)code_of(__uint_as_float(w[j] << 16), s) & 0xffu;
          const uint32_t hi = (uint32_t)code_of(__uint_as_float(w[j] & 0xffff0000u), s) & 0xffu;
          o[j >> 1] |= (lo | (hi << 8)) << (16 * (j & 1));
        }
      }
      reinterpret_cast<uint2*>(out)[at] = make_uint2(o[0], o[1]);
    }
  } else {
    for (int i = tid; i < K; i += NT)
      out[i] = zero ? 0 : (int8_t)code_of(__uint_as_float((uint32_t)row[i] << 16), s);
  }
}

template <int NT, int V>
cudaError_t go(const void* x, long long ld, int8_t* q, float* sc, int T, int K, cudaStream_t s) {
  return ops_launch(quantize_tokens_kernel<NT, V>, dim3((unsigned)T), NT, 0, s, 1, (const uint16_t*)x, ld, q, sc, T, K);
}

}  // namespace

cudaError_t launch_quantize_tokens(const void* x, long long ld, int8_t* q, float* sc, int T, int K, cudaStream_t s) {
  const bool vec = K % 8 == 0 && ld % 8 == 0 && ((uintptr_t)x & 15) == 0 && ((uintptr_t)q & 7) == 0;
  if (!vec || K > 256 * 8 * 8) return go<256, 0>(x, ld, q, sc, T, K, s);
  const int n = K / 8;
  if (n <= 128) return go<128, 1>(x, ld, q, sc, T, K, s);
  if (n <= 256) return go<256, 1>(x, ld, q, sc, T, K, s);
  if (n <= 512) return go<256, 2>(x, ld, q, sc, T, K, s);
  if (n <= 1024) return go<256, 4>(x, ld, q, sc, T, K, s);
  return go<256, 8>(x, ld, q, sc, T, K, s);
}

}  // namespace sffn

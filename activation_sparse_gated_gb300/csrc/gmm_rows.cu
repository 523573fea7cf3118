// gmm_rows.cu -- products grouped by expert for groups of few rows, on the CUDA
// cores: y[r, n] = sum_k x[r, k] w[e, n, k] for the rows r of expert e.
//
// With one to a few rows per expert the product is a read of the weights, so
// what counts is bytes in flight and an even share per SM.  A warp takes RW
// rows of w and up to TM rows of x: lanes stride along K in 16-byte pieces, a
// piece of w serves every x row, and the sums end in one warp reduction.  The
// work is cut along N only, so any N and any group size keep the whole GPU
// streaming and the result does not depend on timing.  bf16: fp32 sums in
// packed FMAs; int8: exact int32 dot products of four.
#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

constexpr int GR_WARPS = 4;

__device__ __forceinline__ void group_bounds(const GmmArgs& a, int e, int* r0, int* r1) {
  if (!a.offsets) {
    *r0 = 0;
    *r1 = a.R;
    return;
  }
  const int b = a.offsets[e], c = a.offsets[e + 1];
  *r0 = min(max(b, 0), a.R);
  *r1 = min(max(c, *r0), a.R);
}

__device__ __forceinline__ int source_row(const GmmArgs& a, int r) {
  const int i = a.index ? a.index[r] : r;
  const int s = a.index ? i / a.index_div : i;
  return i >= 0 && s < a.XR ? s : -1;
}

template <bool I8, int RW, int TM>
__global__ void __launch_bounds__(32 * GR_WARPS) gmm_rows_kernel(const GmmArgs a) {
  constexpr int VPC = I8 ? 16 : 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  int r0, r1;
  group_bounds(a, e, &r0, &r1);
  const int n0 = (blockIdx.x * GR_WARPS + warp) * RW;
  if (r0 >= r1 || n0 >= a.N) return;
  const int nk = a.K / VPC;
  const size_t pitch = (size_t)a.K * (I8 ? 1 : 2);
  const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w) + (size_t)e * a.N * pitch;
  const uint4* wr[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) wr[i] = reinterpret_cast<const uint4*>(w + (size_t)min(n0 + i, a.N - 1) * pitch);
  for (int c0 = r0; c0 < r1; c0 += TM) {
    const uint4* xr[TM];
    int src[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      src[t] = c0 + t < r1 ? source_row(a, c0 + t) : -1;
      xr[t] = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.x) +
                                             (size_t)max(src[t], 0) * a.ldx * (I8 ? 1 : 2));
    }
    float out[RW][TM];
    if constexpr (I8) {
      int acc[RW][TM] = {};
#pragma unroll 4
      for (int k = lane; k < nk; k += 32) {
        uint4 wv[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) wv[i] = __ldg(wr[i] + k);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          const uint4 xv = src[t] >= 0 ? __ldg(xr[t] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            acc[i][t] = __dp4a((int)wv[i].x, (int)xv.x, acc[i][t]);
            acc[i][t] = __dp4a((int)wv[i].y, (int)xv.y, acc[i][t]);
            acc[i][t] = __dp4a((int)wv[i].z, (int)xv.z, acc[i][t]);
            acc[i][t] = __dp4a((int)wv[i].w, (int)xv.w, acc[i][t]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int t = 0; t < TM; ++t) out[i][t] = (float)__reduce_add_sync(0xffffffffu, acc[i][t]);
    } else {
      float2 acc[RW][TM] = {};
#pragma unroll 4
      for (int k = lane; k < nk; k += 32) {
        float2 wf[RW][4];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          float v[8];
          Elt<bf16_tag>::unpack(__ldg(wr[i] + k), v);
#pragma unroll
          for (int j = 0; j < 4; ++j) wf[i][j] = make_float2(v[2 * j], v[2 * j + 1]);
        }
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          float v[8];
          Elt<bf16_tag>::unpack(src[t] >= 0 ? __ldg(xr[t] + k) : make_uint4(0, 0, 0, 0), v);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RW; ++i) ffma2(acc[i][t], wf[i][j], make_float2(v[2 * j], v[2 * j + 1]));
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int t = 0; t < TM; ++t) out[i][t] = warp_sum(acc[i][t].x + acc[i][t].y);
    }
    // lane i * TM + t stores one result
    float v = 0.f;
    int row = -1, n = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int t = 0; t < TM; ++t)
        if (lane == i * TM + t && n0 + i < a.N && c0 + t < r1) {
          n = n0 + i;
          row = c0 + t;
          v = out[i][t];
          if (I8) v = v * (src[t] >= 0 ? a.sx[src[t]] : 0.f) * a.sw[(size_t)e * a.N + n];
        }
    if (row >= 0) {
      const size_t at = (size_t)row * a.ldy + n;
      if (a.y_f32)
        reinterpret_cast<float*>(a.y)[at] = v;
      else
        reinterpret_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    }
  }
}

template <bool I8, int RW, int TM>
cudaError_t go(const GmmArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.N + GR_WARPS * RW - 1) / (GR_WARPS * RW)), (unsigned)a.E);
  return ops_launch(gmm_rows_kernel<I8, RW, TM>, grid, 32 * GR_WARPS, 0, s, 1, a);
}

// [E, K, N] weights (kn): thread = 8 neighbouring columns n, the block's warps split K.
constexpr int GK_WARPS = 8;
__global__ void __launch_bounds__(32 * GK_WARPS) gmm_rows_kn_kernel(const GmmArgs a) {
  __shared__ float s_sum[GK_WARPS][32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  int r0, r1;
  group_bounds(a, e, &r0, &r1);
  const int n = (blockIdx.x * 32 + lane) * 8;
  const uint16_t* w = reinterpret_cast<const uint16_t*>(a.w) + (size_t)e * a.N * a.K;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x);
  for (int r = r0; r < r1; ++r) {
    const int src = source_row(a, r);
    float2 acc[4] = {};
    if (src >= 0 && n < a.N) {
#pragma unroll 4
      for (int k = warp; k < a.K; k += GK_WARPS) {
        const float xv = __uint_as_float((uint32_t)x[(size_t)src * a.ldx + k] << 16);
        float v[8];
        Elt<bf16_tag>::unpack(__ldg(reinterpret_cast<const uint4*>(w + (size_t)k * a.N + n)), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) ffma2(acc[j], make_float2(v[2 * j], v[2 * j + 1]), make_float2(xv, xv));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s_sum[warp][lane][2 * j] = acc[j].x;
      s_sum[warp][lane][2 * j + 1] = acc[j].y;
    }
    __syncthreads();
    const int l = threadIdx.x >> 3, j = threadIdx.x & 7, nn = (blockIdx.x * 32 + l) * 8 + j;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < GK_WARPS; ++q) v += s_sum[q][l][j];
    if (nn < a.N) {
      const size_t at = (size_t)r * a.ldy + nn;
      if (a.y_f32)
        reinterpret_cast<float*>(a.y)[at] = v;
      else
        reinterpret_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_gmm_rows(const GmmArgs& a, cudaStream_t s) {
  if (a.kn)
    return ops_launch(gmm_rows_kn_kernel, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.E), 32 * GK_WARPS, 0, s, 1, a);
  // rows of w per warp: 4 share a piece of x, unless that leaves the SMs short of warps
  const long long rows = (long long)a.N * (a.E < a.R ? a.E : a.R);
  const bool wide = rows >= 4ll * 16 * ops_num_sms();
  const bool one = a.R <= a.E || a.R == 1;
  if (a.i8) {
    if (one) return wide ? go<true, 4, 1>(a, s) : go<true, 1, 1>(a, s);
    return wide ? go<true, 4, 8>(a, s) : go<true, 1, 8>(a, s);
  }
  if (one) return wide ? go<false, 4, 1>(a, s) : go<false, 1, 1>(a, s);
  return wide ? go<false, 4, 8>(a, s) : go<false, 1, 8>(a, s);
}

}  // namespace sffn

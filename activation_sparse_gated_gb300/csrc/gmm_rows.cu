// gmm_rows.cu -- int8 products grouped by expert for groups of one to a few
// rows, on the CUDA cores: y[r, n] = sx sw sum_k x[r, k] w[e, n, k].
//
// With so few rows the product is a read of the codes, so what counts is bytes
// in flight and an even share per SM.  A warp takes RW rows of w and up to TM
// rows of x: lanes stride along K in 16-byte pieces, a piece of w serves every
// x row, and the exact int32 sums of dot products of four end in one warp
// reduction.  The work is cut along N only, so any N keeps the whole GPU
// streaming.  (The tensor cores walk 128 rows of w an MMA however few rows of x
// there are, and widen the codes first: they win from a few rows on.)
//
// Measured: one row, 7168 x 2560: 3.8 us, 4.8 TB/s (71 % of the copy rate).
#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

constexpr int GR_WARPS = 4;

template <int RW, int TM>
__global__ void __launch_bounds__(32 * GR_WARPS) gmm_rows_kernel(const GmmArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  int r0 = 0, r1 = a.R;
  if (a.offsets) {
    const int b = a.offsets[e], c = a.offsets[e + 1];
    r0 = min(max(b, 0), a.R);
    r1 = min(max(c, r0), a.R);
  }
  const int n0 = (blockIdx.x * GR_WARPS + warp) * RW;
  if (r0 >= r1 || n0 >= a.N) return;
  const int nk = a.K / 16;
  const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w) + (size_t)e * a.N * a.K;
  const uint4* wr[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) wr[i] = reinterpret_cast<const uint4*>(w + (size_t)min(n0 + i, a.N - 1) * a.K);
  for (int c0 = r0; c0 < r1; c0 += TM) {
    const uint4* xr[TM];
    int src[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      src[t] = -1;
      if (c0 + t < r1) {
        const int i = a.index ? a.index[c0 + t] : c0 + t;
        const int s = a.index ? i / a.index_div : i;
        if (i >= 0 && s < a.XR) src[t] = s;
      }
      xr[t] = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.x) + (size_t)max(src[t], 0) * a.ldx);
    }
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
    // lane i * TM + t stores one result
    float v = 0.f;
    int row = -1, n = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const float sum = (float)__reduce_add_sync(0xffffffffu, acc[i][t]);
        if (lane == i * TM + t && n0 + i < a.N && c0 + t < r1) {
          n = n0 + i;
          row = c0 + t;
          v = sum * (src[t] >= 0 ? a.sx[src[t]] : 0.f) * a.sw[(size_t)e * a.N + n];
        }
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

template <int RW, int TM>
cudaError_t go(const GmmArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.N + GR_WARPS * RW - 1) / (GR_WARPS * RW)), (unsigned)a.E);
  return ops_launch(gmm_rows_kernel<RW, TM>, grid, 32 * GR_WARPS, 0, s, 1, a);
}

}  // namespace

// Four rows of w a warp, unless that leaves the SMs fewer than eight warps each (us, one / four rows a warp: N = 2560,
// K = 7168, one row of x 6.7 / 10.6; 8 experts of N = 1024, K = 2560 17.3 / 6.0); four rows of x together where there
// are several (N = 14336, K = 4096, four rows of x, one / four together: 21.1 / 15.4).
// The host knows how many rows there are, not whose: up to as many as experts are taken for one each, and where they lie
// in one group after all, every row reads that expert's codes again (128 experts of N = 1024, K = 2560: 128 rows of
// 128 experts 52 us, 128 rows of one 178; the tensor cores take 129 rows of one in 17).
cudaError_t launch_gmm_rows(const GmmArgs& a, cudaStream_t s) {
  const int busy = a.E < a.R ? a.E : a.R;
  const bool wide = (long long)a.N * busy >= 32ll * ops_num_sms();
  if (a.R <= busy) return wide ? go<4, 1>(a, s) : go<1, 1>(a, s);
  return wide ? go<4, 4>(a, s) : go<1, 4>(a, s);
}

}  // namespace sffn

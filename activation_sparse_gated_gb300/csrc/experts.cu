// experts.cu -- the gated experts' forward behind the router, for few tokens:
//
//   y_t = sum_j w_tj  W2_e (A(W1_e x_t) .* (W3_e x_t)),   e = ids[t, j]
//
// with the gate first, as everywhere in this library: a warp computes a hidden
// unit's gate z = W1_e[i] . x_t, and only a live unit's row of W3_e is read;
// the down product then gathers the live units' rows of W2_e^T.  Both passes
// are reads of weight rows (bf16, fp32 sums; h stays fp32).
#include <cstdlib>

#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

constexpr int EG_WARPS = 8;

__global__ void __launch_bounds__(32 * EG_WARPS) experts_gate_kernel(const ExpertsArgs a, float* __restrict__ h) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p = blockIdx.y, t = p / a.k;
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x * EG_WARPS + warp;
  if (i >= a.H) return;
  const int e = a.ids[p];
  float out = 0.f;
  if (e >= 0 && e < a.E) {
    const size_t off = ((size_t)e * a.H + i) * a.D;
    const uint4* w1 = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.W1) + off);
    const uint4* w3 = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.W3) + off);
    const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + (size_t)t * a.ldx);
    const int n = a.D / 8;
    auto dot = [&](const uint4* w) {
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int k = lane; k < n; k += 32) {
        float u[8], v[8];
        Elt<bf16_tag>::unpack(__ldg(w + k), u);
        Elt<bf16_tag>::unpack(__ldg(x + k), v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ffma2(acc, make_float2(u[2 * j], u[2 * j + 1]), make_float2(v[2 * j], v[2 * j + 1]));
      }
      return warp_sum(acc.x + acc.y);
    };
    const float g = activation(a.act, dot(w1));
    if (g != 0.f) out = g * dot(w3);
  }
  if (lane == 0) h[(size_t)p * a.H + i] = out;
}

// y[t, 8 columns a lane] = sum over the token's choices and live units.
constexpr int ED_WARPS = 8;
__global__ void __launch_bounds__(32 * ED_WARPS) experts_down_kernel(const ExpertsArgs a, const float* __restrict__ h) {
  __shared__ float s_sum[ED_WARPS][32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  const int n = (blockIdx.x * 32 + lane) * 8;
  float2 acc[4] = {};
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j, e = a.ids[p];
    const float w = a.weights[p];
    if (e < 0 || e >= a.E || w == 0.f) continue;
    const uint16_t* w2 = reinterpret_cast<const uint16_t*>(a.W2t) + (size_t)e * a.H * a.D;
    for (int i0 = warp * 32; i0 < a.H; i0 += 32 * ED_WARPS) {
      const float hv = i0 + lane < a.H ? h[(size_t)p * a.H + i0 + lane] * w : 0.f;
      uint32_t live = __ballot_sync(0xffffffffu, hv != 0.f);
      while (live) {
        const int b = __ffs(live) - 1;
        live &= live - 1;
        const float c = __shfl_sync(0xffffffffu, hv, b);
        if (n < a.D) {
          float v[8];
          Elt<bf16_tag>::unpack(__ldg(reinterpret_cast<const uint4*>(w2 + (size_t)(i0 + b) * a.D + n)), v);
#pragma unroll
          for (int q = 0; q < 4; ++q) ffma2(acc[q], make_float2(v[2 * q], v[2 * q + 1]), make_float2(c, c));
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    s_sum[warp][lane][2 * q] = acc[q].x;
    s_sum[warp][lane][2 * q + 1] = acc[q].y;
  }
  __syncthreads();
  const int l = threadIdx.x >> 3, j = threadIdx.x & 7, nn = (blockIdx.x * 32 + l) * 8 + j;
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < ED_WARPS; ++q) v += s_sum[q][l][j];
  if (nn < a.D) reinterpret_cast<__nv_bfloat16*>(a.y)[(size_t)t * a.D + nn] = __float2bfloat16_rn(v);
}

// y[t] = sum_j weights[t, j] o[t k + j] in the order of the places; a place
// without an expert or of weight 0 is not read (its row of o was not written).
// Bound by reading o; 16-byte pieces, one thread per four columns and token.
constexpr int EC_THREADS = 256;
__global__ void __launch_bounds__(EC_THREADS) experts_combine_kernel(const ExpertsArgs a, const float* __restrict__ o) {
  const int t = blockIdx.y, c = (blockIdx.x * EC_THREADS + threadIdx.x) * 4;
  pdl_launch_dependents();
  pdl_wait();
  if (c >= a.D) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j;
    const float w = a.ids[p] >= 0 ? a.weights[p] : 0.f;
    if (w != 0.f) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(o + (size_t)p * a.D + c));
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
      sum.z = fmaf(w, v.z, sum.z);
      sum.w = fmaf(w, v.w, sum.w);
    }
  }
  *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + (size_t)t * a.D + c) =
      make_uint2(pack_bf16x2_rn(sum.x, sum.y), pack_bf16x2_rn(sum.z, sum.w));
}

// xg[r] = x[rows[r] / k]: a grouped copy of the tokens, one block a row.
__global__ void __launch_bounds__(128) experts_gather_kernel(const ExpertsArgs a, uint16_t* __restrict__ xg) {
  const int r = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int i = a.rows[r];
  if (i < 0 || i / a.k >= a.T) return;
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + (size_t)(i / a.k) * a.ldx);
  uint4* dst = reinterpret_cast<uint4*>(xg + (size_t)r * a.D);
  for (int c = threadIdx.x; c < a.D / 8; c += 128) dst[c] = __ldg(src + c);
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Few choices: the gate-first passes above; more: the grouped products on the tensor cores.
bool few(int T, int k) { return (long long)T * k <= 64; }

}  // namespace

size_t experts_workspace(int T, int k, int D, int H) {
  const size_t R = (size_t)T * k;
  if (few(T, k)) return sizeof(float) * R * H;
  // h, then the choices' products (and before them, in the same place, the grouped tokens)
  return round_up(2 * R * round_up(H, 8), 256) + sizeof(float) * R * D;
}

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (few(a.T, a.k)) {
    float* h = static_cast<float*>(a.workspace);
    if ((e = ops_launch(experts_gate_kernel, dim3((a.H + EG_WARPS - 1) / EG_WARPS, a.T * a.k), 32 * EG_WARPS, 0, s, 1, a,
                        h)) != cudaSuccess)
      return e;
    return ops_launch(experts_down_kernel, dim3((a.D + 255) / 256, a.T), 32 * ED_WARPS, 0, s, 1, a, (const float*)h);
  }
  const int R = a.T * a.k, Hp = (int)round_up(a.H, 8);
  float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + round_up(2 * (size_t)R * Hp, 256));
  GmmArgs up;
  up.x = a.x;
  up.ldx = a.ldx;
  up.w = a.W1;
  up.w3 = a.W3;
  up.offsets = a.offsets;
  up.index = a.rows;
  up.index_div = a.k;
  up.y = a.workspace;
  up.ldy = Hp;
  up.R = R;
  up.XR = a.T;
  up.N = a.H;
  up.K = a.D;
  up.E = a.E;
  up.act = a.act;
  if (!std::getenv("SFFN_GATHER4")) {
    uint16_t* xg = reinterpret_cast<uint16_t*>(o);
    if ((e = ops_launch(experts_gather_kernel, dim3((unsigned)R), 128, 0, s, 1, a, xg)) != cudaSuccess) return e;
    up.x = xg;
    up.ldx = a.D;
    up.index = nullptr;
    up.XR = R;
  }
  if ((e = launch_gmm(up, s)) != cudaSuccess) return e;
  GmmArgs down;
  down.x = a.workspace;
  down.ldx = Hp;
  down.w = a.W2t;
  down.kn = 1;
  down.offsets = a.offsets;
  down.out_index = a.rows;
  down.y = o;
  down.y_f32 = 1;
  down.ldy = a.D;
  down.R = R;
  down.XR = R;
  down.N = a.D;
  down.K = a.H;
  down.E = a.E;
  if ((e = launch_gmm(down, s)) != cudaSuccess) return e;
  return ops_launch(experts_combine_kernel, dim3((a.D + 4 * EC_THREADS - 1) / (4 * EC_THREADS), a.T), EC_THREADS, 0, s, 1,
                    a, (const float*)o);
}

}  // namespace sffn

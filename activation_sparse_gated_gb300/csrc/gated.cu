// gated.cu -- the first half of a gated FFN as an operator of its own,
//
//   h = A(z) .* u,   z = x W1^T,  u = x W3^T            (x [T, D], W1, W3 [H, D])
//
// and its backward pass: with dz = dh .* u .* A'(z) and du = dh .* A(z),
//
//   dx = dz W1 + du W3,   dW1 = dz^T x,   dW3 = du^T x.
//
// A few tokens are a read of the weights, gate first (gated_rows_kernel); more
// are one product on the tensor cores that computes z and u together and
// multiplies them in its epilogue (gmm_tc.cu).  For training that product also
// stores z and u, in fp32: dz and du are rounded to bf16 once, as the operands of
// an MMA have to be, and rounding what they are made of as well would nearly
// double the gradients' error.
#include <algorithm>

#include "common.cuh"
#include "ops.h"

namespace sffn {
namespace {

constexpr int GU_WARPS = 8;
constexpr int GU_TOKENS = 4;             // most tokens of the gate-first form
constexpr int GU_U = 5;                   // pieces of a weight row requested before the first is used
constexpr size_t GU_STAGE = 40 * 1024;   // most bytes of x in shared memory

// A warp takes UN hidden units and the TM tokens together: the units' rows of W1 are read once for them, GU_U pieces of each
// requested before the first is used, and a unit's row of W3 only where a token keeps it.  Bound by memory latency: the rows of
// W1, then those of W3.  (One token, D = 2560, H = 7168, 10 % of the units live: 9.9 us for 40 MB, 60 % of the copy rate; D =
// 4096, H = 14336 25 us, 76 %.  Eight or ten pieces ahead: 12.2 and 10.9, 23.7 both.)
template <int TM, int UN, bool STAGED>
__global__ void __launch_bounds__(32 * GU_WARPS) gated_rows_kernel(const GatedArgs a) {
  extern __shared__ uint4 s_x[];  // [TM][D / 8]
  const int lane = threadIdx.x & 31, i0 = (blockIdx.x * GU_WARPS + (threadIdx.x >> 5)) * UN, n = a.D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const uint4* x[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t)  // tokens past T are computed on the last one and not stored
    x[t] = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + (long long)min(t, a.T - 1) * a.ldx);
  const uint4 *w1[UN], *w3[UN];
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    const size_t off = (size_t)min(i0 + i, a.H - 1) * a.D;
    w1[i] = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.W1) + off);
    w3[i] = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.W3) + off);
  }
  uint4 w[UN][GU_U];
  auto request = [&](const uint4* const (&p)[UN], const bool (&on)[UN], int k0) {
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
      for (int q = 0; q < GU_U; ++q)
        w[i][q] = on[i] && k0 + 32 * q < n ? __ldg(p[i] + k0 + 32 * q) : make_uint4(0, 0, 0, 0);
  };
  bool on[UN];
#pragma unroll
  for (int i = 0; i < UN; ++i) on[i] = true;
  request(w1, on, lane);  // the first pieces of W1 travel while x is staged
  if (STAGED) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
      for (int k = threadIdx.x; k < n; k += 32 * GU_WARPS) s_x[t * n + k] = __ldg(x[t] + k);
    __syncthreads();
  }
  if (i0 >= a.H) return;
  auto dots = [&](const uint4* const (&p)[UN], bool loaded, float (&out)[UN][TM]) {
    float2 acc[UN][TM] = {};
    for (int k0 = lane; k0 < n; k0 += 32 * GU_U) {
      if (!loaded || k0 != lane) request(p, on, k0);
#pragma unroll
      for (int q = 0; q < GU_U; ++q) {
        const int k = k0 + 32 * q;
        if (k < n) {
          float v[TM][8];
#pragma unroll
          for (int t = 0; t < TM; ++t) Elt<bf16_tag>::unpack(STAGED ? lds16(s_x + t * n + k) : __ldg(x[t] + k), v[t]);
#pragma unroll
          for (int i = 0; i < UN; ++i) {
            float u[8];
            Elt<bf16_tag>::unpack(w[i][q], u);
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                ffma2(acc[i][t], make_float2(u[2 * j], u[2 * j + 1]), make_float2(v[t][2 * j], v[t][2 * j + 1]));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
      for (int t = 0; t < TM; ++t) out[i][t] = on[i] ? warp_sum(acc[i][t].x + acc[i][t].y) : 0.f;
  };
  float g[UN][TM], u[UN][TM] = {};
  dots(w1, true, g);
  bool any = false;
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    on[i] = false;
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      g[i][t] = g[i][t] != g[i][t] ? g[i][t] : activation(a.act, g[i][t]);  // a NaN gate is live
      on[i] = on[i] || (g[i][t] != 0.f && i0 + i < a.H);
    }
    any = any || on[i];
  }
  if (any) dots(w3, false, u);
#pragma unroll
  for (int i = 0; i < UN; ++i)
#pragma unroll
    for (int t = 0; t < TM; ++t)
      if (lane == i * TM + t && t < a.T && i0 + i < a.H)
        reinterpret_cast<__nv_bfloat16*>(a.h)[(long long)t * a.ldh + i0 + i] =
            __float2bfloat16_rn(g[i][t] != 0.f ? g[i][t] * u[i][t] : 0.f);
}

template <int TM, int UN>
cudaError_t rows_go(const GatedArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.H + GU_WARPS * UN - 1) / (GU_WARPS * UN)));
  const size_t bytes = TM * 2 * (size_t)a.D;
  return bytes <= GU_STAGE ? ops_launch(gated_rows_kernel<TM, UN, true>, grid, 32 * GU_WARPS, bytes, s, 1, a)
                           : ops_launch(gated_rows_kernel<TM, UN, false>, grid, 32 * GU_WARPS, 0, s, 1, a);
}

// The 2-norm of a row, or a little more, by a warp; norms past 2^63 count as that (a product of two stays in fp32), those of
// rows that hold an infinity or a NaN, whose sums no second sum betters, as 0.
__device__ __forceinline__ float row_norm(const uint16_t* row, int D) {
  const uint4* p = reinterpret_cast<const uint4*>(row);
  const int lane = threadIdx.x & 31, n = D / 8;
  float scale = 1.f;
  for (;;) {
    float2 acc[4] = {};
    float top = 0.f;
    for (int k0 = lane; k0 < n; k0 += 320) {
      uint4 c[10];
#pragma unroll
      for (int q = 0; q < 10; ++q) c[q] = k0 + 32 * q < n ? __ldg(p + k0 + 32 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 10; ++q) {
        float v[8];
        Elt<bf16_tag>::unpack(c[q], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          top = fmaxf(top, fabsf(v[j]));
          v[j] *= scale;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = make_float2(v[2 * j], v[2 * j + 1]);
          ffma2(acc[j], f, f);
        }
      }
    }
    const float sum = warp_sum((acc[0].x + acc[0].y + acc[1].x + acc[1].y) + (acc[2].x + acc[2].y + acc[3].x + acc[3].y));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (sum != sum || !(top < 3.4e38f) || top == 0.f) return 0.f;
    if (scale != 1.f || (sum > 0x1p-80f && sum < 0x1p120f)) return fminf(1.001f * sqrtf(sum) / scale, 0x1p63f);
    scale = top < 1.f ? 0x1p100f : 0x1p-100f;  // squares that left fp32: once more, of values that do not
  }
}

// |x| of every token and c |w| of every unit of W1, for the signs of the gates (gate_near in gmm_tc.cu).  A caller of the block
// gives no scratch, so they wait in z and u themselves, where the warp that stores a piece of a tile reads them first: each 32
// columns of z hold the norms of the GATE_ROWS tokens from their row on (narrower, a column holds the largest of those
// that share it), and the rows of u that a tile's two halves of the epilogue's warps begin with (tiles of `per` rows) their
// units'.  Bound by memory: x and W1 in, which the product then finds in L2, and 1 / 32 of z out.  A block takes GATE_ROWS
// tokens, or as many units, a warp a row of them.
struct NormArgs {
  const uint16_t *x, *W1;
  long long ldx, ldz;
  float *z, *u;
  int T, D, H, per, tokens;  // tokens: blocks of them
  float c;
};
__global__ void __launch_bounds__(32 * GATE_ROWS, 2) gate_norms_kernel(const NormArgs a) {
  __shared__ float s_norm[GATE_ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = threadIdx.x & (GATE_ROWS - 1), slot = threadIdx.x / GATE_ROWS;
  const bool of_x = blockIdx.x < (unsigned)a.tokens;
  const int r0 = (of_x ? blockIdx.x : blockIdx.x - a.tokens) * GATE_ROWS;
  pdl_launch_dependents();
  pdl_wait();
  float v = 0.f;
  if (of_x && r0 + warp < a.T) v = row_norm(a.x + (long long)(r0 + warp) * a.ldx, a.D);
  if (!of_x && r0 + warp < a.H) v = a.c * row_norm(a.W1 + (size_t)(r0 + warp) * a.D, a.D);
  if (lane == 0) s_norm[warp] = v;
  __syncthreads();
  if (of_x) {
    float* z = a.z + (long long)r0 * a.ldz;
    for (int c = slot * 32; c < a.H; c += 32 * 32) {
      const int cols = min(32, a.H - c);
      v = s_norm[l];
      for (int i = l + cols; i < GATE_ROWS; i += cols) v = fmaxf(v, s_norm[i]);
      if (l < cols) z[c + l] = v;
    }
  } else if (r0 + l < a.H) {
    for (long long i = slot; (i >> 1) * a.per < a.T; i += 32) {
      const long long r = (i >> 1) * a.per + 32 * (i & 1);
      if (r < a.T) a.u[r * a.ldz + r0 + l] = s_norm[l];
    }
  }
}

// dz = dh u A'(z) and du = dh A(z) of one element.  A gate that is closed passes nothing, whatever dh and the other factor
// are: both are 0 where z <= 0 (ReLU, R-S+), and SiLU's are where its value or its slope is 0 in fp32.
__device__ __forceinline__ float2 gate_grad(int act, float z, float u, float dh) {
  if (act != ACT_SILU && z <= 0.f) return make_float2(0.f, 0.f);
  if (act == 0) return make_float2(dh * u, dh * z);
  // A(z) = z p and A'(z) = p (1 + z (1 - p)) with p = 1 / (1 + e^-z) and 1 - p = e^-z p; past |z| = 88, where e^-z leaves
  // fp32, A is z or 0 and A' is 1 or 0 to below 1e-30
  const bool wide = fabsf(z) > 88.f;
  const float e = __expf(-z), p = __fdividef(1.f, 1.f + e);
  const float v = wide ? (z > 0.f ? z : 0.f) : z * p;
  const float d = wide ? (z > 0.f ? 1.f : 0.f) : p * (1.f + z * (e * p));
  return make_float2(d == 0.f ? 0.f : dh * u * d, v == 0.f ? 0.f : dh * v);
}

// The two gradients of the gate's inputs side by side, [dz | du], each filled up with zeros to Hp = round_up(H, 64)
// columns: the x side of both products of the backward pass.  Bound by memory: fp32 z and u and bf16 dh in, two bf16 out,
// 14 bytes an element; a thread takes eight columns of a row.
struct GradArgs {
  const uint16_t* dh;
  long long lddh;
  const float *z, *u;
  long long ldz;
  uint16_t* g;
  int T, H, Hp, act;
};
template <bool VEC>
__global__ void __launch_bounds__(256) gate_grad_kernel(const GradArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (c >= a.Hp) return;
  for (long long t = (long long)blockIdx.y * blockDim.y + threadIdx.y; t < a.T; t += (long long)gridDim.y * blockDim.y) {
    float dh[8], z[8], u[8];
    if (VEC && c + 8 <= a.H) {
      Elt<bf16_tag>::unpack(__ldcs(reinterpret_cast<const uint4*>(a.dh + t * a.lddh + c)), dh);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(a.z + t * a.ldz + c) + q);
        const float4 w = __ldcs(reinterpret_cast<const float4*>(a.u + t * a.ldz + c) + q);
        z[4 * q] = v.x, z[4 * q + 1] = v.y, z[4 * q + 2] = v.z, z[4 * q + 3] = v.w;
        u[4 * q] = w.x, u[4 * q + 1] = w.y, u[4 * q + 2] = w.z, u[4 * q + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = c + j < a.H;
        dh[j] = in ? __uint_as_float((uint32_t)a.dh[t * a.lddh + c + j] << 16) : 0.f;
        z[j] = in ? a.z[t * a.ldz + c + j] : 0.f;
        u[j] = in ? a.u[t * a.ldz + c + j] : 0.f;
      }
    }
    uint32_t dz[4], du[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = gate_grad(a.act, z[2 * j], u[2 * j], dh[2 * j]);
      const float2 q = gate_grad(a.act, z[2 * j + 1], u[2 * j + 1], dh[2 * j + 1]);
      dz[j] = pack_bf16x2_rn(p.x, q.x);
      du[j] = pack_bf16x2_rn(p.y, q.y);
    }
    uint16_t* to = a.g + t * 2 * a.Hp + c;
    *reinterpret_cast<uint4*>(to) = make_uint4(dz[0], dz[1], dz[2], dz[3]);
    *reinterpret_cast<uint4*>(to + a.Hp) = make_uint4(du[0], du[1], du[2], du[3]);
  }
}

int padded(int H) { return (H + 63) / 64 * 64; }

}  // namespace

cudaError_t launch_gated_up(const GatedArgs& a, cudaStream_t s) {
  // Gate first for one or two tokens, and for up to four where the products' launch is most of their time (us, gate first /
  // products, ReLU: 2 tokens, D = 4096, H = 14336 31 / 40; 4 tokens, D = 1024, H = 1000 4.1 / 7.3, D = 2560, H = 7168 19.0 /
  // 16.9).  Two units a warp where one each is more warps than run at once (one token, D = 2560, one / two: H = 7168 ReLU
  // 10.7 / 9.9, SiLU 15.2 / 13.0, H = 1024 3.9 / 4.4).
  if (!a.z && a.T <= GU_TOKENS && (a.T <= 2 || (long long)a.H * a.D <= 8 << 20)) {
    if (a.T == 1) return a.H > 40 * ops_num_sms() ? rows_go<1, 2>(a, s) : rows_go<1, 1>(a, s);
    return a.T == 2 ? rows_go<2, 1>(a, s) : rows_go<GU_TOKENS, 1>(a, s);
  }
  GmmArgs p;
  p.x = a.x;
  p.ldx = a.ldx;
  p.w = a.W1;
  p.w3 = a.W3;
  p.y = a.h;
  p.ldy = a.ldh;
  p.R = p.XR = a.T;
  p.N = a.H;
  p.K = a.D;
  p.act = a.act;
  p.z = a.z;
  p.u = a.u;
  p.ldz = a.ldz;
  return launch_gmm(p, s);
}

cudaError_t launch_gate_norms(const GmmArgs& a, int per, cudaStream_t s) {
  const NormArgs n = {static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.w), a.ldx, a.ldz, a.z, a.u, a.R, a.K, a.N,
                      per, (a.R + GATE_ROWS - 1) / GATE_ROWS,
                      // what the MMAs' steps of 16 cut off of the running sums, and the join of a cut K, see gate_near
                      (float)(2 * ((a.K + 63) / 64) + 8) * 0x1p-24f};
  return ops_launch(gate_norms_kernel, dim3((unsigned)(n.tokens + (a.N + GATE_ROWS - 1) / GATE_ROWS)), 32 * GATE_ROWS, 0, s, 1, n);
}

size_t gated_grad_workspace(int T, int H) { return sizeof(uint16_t) * 2 * (size_t)T * padded(H); }

cudaError_t launch_gated_grad(const GatedGradArgs& a, cudaStream_t s) {
  const int Hp = padded(a.H);
  uint16_t* g = static_cast<uint16_t*>(a.workspace);
  const GradArgs r = {static_cast<const uint16_t*>(a.dh), a.lddh, a.z, a.u, a.ldz, g, a.T, a.H, Hp, a.act};
  const bool vec = ((uintptr_t)a.dh & 15) == 0 && a.lddh % 8 == 0 && ((uintptr_t)a.z & 15) == 0 &&
                   ((uintptr_t)a.u & 15) == 0 && a.ldz % 4 == 0;
  int bx = 8;  // threads along a row
  while (bx < 256 && bx * 8 < Hp) bx *= 2;
  const int by = 256 / bx;
  const dim3 grid((unsigned)((Hp / 8 + bx - 1) / bx), (unsigned)std::min((a.T + by - 1) / by, 65535));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)bx, (unsigned)by);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, vec ? gate_grad_kernel<true> : gate_grad_kernel<false>, r);
  if (e != cudaSuccess) return e;
  if (a.dx) {  // [dz | du] by W1 below W3
    GmmArgs p;
    p.x = g;
    p.ldx = 2 * Hp;
    p.w = a.W1;
    p.w3 = a.W3;
    p.kn = 1;
    p.K1 = a.H;
    p.K = 2 * Hp;
    p.y = a.dx;
    p.ldy = a.D;
    p.R = p.XR = a.T;
    p.N = a.D;
    if ((e = launch_gmm(p, s)) != cudaSuccess) return e;
  }
  if (a.dW1 || a.dW3) {  // their rows are dz's and du's columns, the sum runs over the tokens
    GmmArgs p;
    p.x = a.dW1 ? g : g + Hp;
    p.ldx = 2 * Hp;
    p.xt = 1;
    p.w = a.x;
    p.ldw = a.ldx;
    p.kn = 1;
    p.K = a.T;
    p.E = a.dW1 && a.dW3 ? 2 : 1;
    p.per = a.H;
    p.xper = Hp;
    p.R = p.XR = p.E * a.H;
    p.y = a.dW1 ? a.dW1 : a.dW3;
    p.y2 = a.dW3;
    p.ldy = a.D;
    p.N = a.D;
    if ((e = launch_gmm(p, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sffn

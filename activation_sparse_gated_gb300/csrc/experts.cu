// experts.cu -- the gated experts' forward behind the router, for few tokens:
//
//   y_t = sum_j w_tj  W2_e (A(W1_e x_t) .* (W3_e x_t)),   e = ids[t, j]
//
// with the gate first, as everywhere in this library: a warp computes a hidden
// unit's gate z = W1_e[i] . x_t, and only a live unit's row of W3_e is read;
// the down product then gathers the live units' rows of W2_e^T.  Both passes
// are reads of weight rows (bf16, fp32 sums; h stays fp32).
//
// Measured: one token, 8 of 64 experts, D = 2560, H = 1024, ReLU at 90 %: 20 us
// with its router (50 MB, 37 % of the copy rate): loads that wait for the
// choice, for the gate, for the live units, one after the other.  Many tokens
// are products on the tensor cores (4096 tokens 480 to 499 us by the board): gate and up 227, down
// 148 (its fp32 rows are 335 MB; 127 with rows of bf16), combination 62, the
// grouped copy of x 31, the router 15.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "tc.cuh"

namespace sffn {
namespace {

// Gate and up of few tokens: h[p, i] = A(W1_e[i] . x_t) (W3_e[i] . x_t) for the
// choices p = (t, j) of expert e.  blockIdx.y is a choice (one token: its
// choices are its experts) or the y-th busy expert; a warp takes one hidden
// unit and up to EG_ROWS of the expert's rows together, so W1 is read once for them and
// W3 only where a row keeps the unit.  EG_U pieces of a weight row are
// requested before the first is used; the rows of x sit in shared memory
// (STAGED) unless they are too long for it.
// Five pieces are whole rounds where D is a multiple of 1280, and the best of 4,
// 5 and 8 there (one token, 4 of 16 experts, us: D = 1280, H = 2048 13.8 / 12.7 /
// 13.6; 2560, 1024 12.8 / 12.3 / 14.3; 5120, 1536 28.0 / 27.6 / 27.5); at multiples
// of 1024 four are a little better (1024, 2048 11.3 / 11.5 / 12.6; 2048, 1024
// 10.5 / 10.9 / 11.1; 4096, 2048 25.9 / 27.2 / 26.2): one count for all.
constexpr int EG_WARPS = 8;
constexpr int EG_U = 5;
constexpr int EG_ROWS = 4;
constexpr size_t EG_STAGE = 40 * 1024;  // most bytes of staged x a block

// The unit's TM rows from c0 on: rows past r1 are computed on row c0's token and not stored.
template <int TM, bool STAGED>
__device__ __forceinline__ void gate_rows(const ExpertsArgs& a, float* __restrict__ h, uint4* s_x, const uint4* w1,
                                          const uint4* w3, int i, int c0, int r1, bool by_choice) {
  const int lane = threadIdx.x & 31, P = a.T * a.k, n = a.D / 8;
  int p[TM];
  const uint4* x[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    p[t] = by_choice ? c0 : c0 + t < r1 ? a.rows[c0 + t] : -1;
    if (p[t] >= P) p[t] = -1;
    x[t] = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + (size_t)(max(p[t], 0) / a.k) * a.ldx);
  }
  uint4 w[EG_U];
#pragma unroll
  for (int q = 0; q < EG_U; ++q)  // the first pieces of W1 travel while x is staged
    w[q] = lane + 32 * q < n ? __ldg(w1 + lane + 32 * q) : make_uint4(0, 0, 0, 0);
  if (STAGED) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TM; ++t)
      for (int k = threadIdx.x; k < n; k += 32 * EG_WARPS) s_x[t * n + k] = __ldg(x[t] + k);
    __syncthreads();
  }
  auto dot = [&](const uint4* wp, bool loaded, float (&out)[TM]) {
    float2 acc[TM] = {};
    for (int k0 = lane; k0 < n; k0 += 32 * EG_U) {
      if (!loaded || k0 != lane) {
#pragma unroll
        for (int q = 0; q < EG_U; ++q) w[q] = k0 + 32 * q < n ? __ldg(wp + k0 + 32 * q) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < EG_U; ++q) {
        const int k = k0 + 32 * q;
        if (k < n) {
          float u[8];
          Elt<bf16_tag>::unpack(w[q], u);
#pragma unroll
          for (int t = 0; t < TM; ++t) {
            float v[8];
            Elt<bf16_tag>::unpack(STAGED ? lds16(s_x + t * n + k) : __ldg(x[t] + k), v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              ffma2(acc[t], make_float2(u[2 * j], u[2 * j + 1]), make_float2(v[2 * j], v[2 * j + 1]));
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) out[t] = warp_sum(acc[t].x + acc[t].y);
  };
  float g[TM], u[TM];
  dot(w1, true, g);
  bool live = false;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    g[t] = g[t] != g[t] ? g[t] : activation(a.act, g[t]);  // a NaN gate is live: its token must come out as NaN
    u[t] = 0.f;
    live = live || (p[t] >= 0 && g[t] != 0.f);
  }
  if (live && i < a.H) dot(w3, false, u);
#pragma unroll
  for (int t = 0; t < TM; ++t)
    if (lane == t && p[t] >= 0 && i < a.H) h[(size_t)p[t] * a.H + i] = g[t] != 0.f ? g[t] * u[t] : 0.f;
}

template <bool ONE, bool STAGED>
__global__ void __launch_bounds__(32 * EG_WARPS) experts_gate_kernel(const ExpertsArgs a, float* __restrict__ h) {
  extern __shared__ uint4 s_x[];  // [ONE ? 1 : EG_ROWS][D / 8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * EG_WARPS + warp;
  const int P = a.T * a.k;
  pdl_launch_dependents();
  pdl_wait();
  int e = -1, r0 = 0, r1 = 0;
  if (ONE) {
    e = a.ids[blockIdx.y];
    if (e >= a.E) e = -1;
  } else {
    int left = blockIdx.y;
    for (int e0 = 0; e0 < a.E && e < 0; e0 += 32) {
      int b = 0, c = 0;
      if (e0 + lane < a.E) {
        b = min(max(a.offsets[e0 + lane], 0), P);
        c = min(max(a.offsets[e0 + lane + 1], b), P);
      }
      const uint32_t busy = __ballot_sync(0xffffffffu, c > b);
      const int m = __popc(busy);
      if (left < m) {
        const int at = __fns(busy, 0, left + 1);
        e = e0 + at;
        r0 = __shfl_sync(0xffffffffu, b, at);
        r1 = __shfl_sync(0xffffffffu, c, at);
      }
      left -= m;
    }
  }
  if (e < 0) return;  // the whole block
  const size_t off = ((size_t)e * a.H + min(i, a.H - 1)) * a.D;
  const uint4* w1 = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.W1) + off);
  const uint4* w3 = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.W3) + off);
  if (ONE) {
    gate_rows<1, STAGED>(a, h, s_x, w1, w3, i, (int)blockIdx.y, 0, true);
  } else {
    for (int c0 = r0; c0 < r1; c0 += EG_ROWS) {
      if (r1 - c0 == 1) gate_rows<1, STAGED>(a, h, s_x, w1, w3, i, c0, r1, false);
      else if (r1 - c0 == 2) gate_rows<2, STAGED>(a, h, s_x, w1, w3, i, c0, r1, false);
      else gate_rows<EG_ROWS, STAGED>(a, h, s_x, w1, w3, i, c0, r1, false);
    }
  }
}

// y[t, 256 columns] = sum over the token's choices and their live units of
// (w h) W2^T[unit].  A cluster of ED_SPLIT blocks cuts the k H units; a warp
// lists the live ones of its share (ballots), then gathers their row segments
// eight at a time, 16 bytes a lane; sums go over the warps in shared memory and
// over the blocks through distributed shared memory, in a fixed order.
constexpr int ED_WARPS = 16;
constexpr int ED_SPLIT = 8;
constexpr int ED_ROWS = 8;    // row segments in flight a lane
constexpr int ED_LIST = 128;  // units a warp lists before it gathers
__global__ void __launch_bounds__(32 * ED_WARPS) experts_down_kernel(const ExpertsArgs a, const float* __restrict__ h) {
  __shared__ float s_sum[ED_WARPS][256 + 4];
  __shared__ float s_c[ED_WARPS][ED_LIST];
  __shared__ int s_u[ED_WARPS][ED_LIST];  // row of W2^T: expert * H + unit (in rows, checked against 31 bits)
  __shared__ float s_part[256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y;
  const int rank = blockIdx.x % ED_SPLIT, n = (blockIdx.x / ED_SPLIT) * 256 + lane * 8;
  pdl_launch_dependents();
  pdl_wait();
  float2 acc[4] = {};
  const uint16_t* w2 = reinterpret_cast<const uint16_t*>(a.W2t) + n;
  const int seg = (a.H + 31) / 32, segs = seg * a.k;  // 32-unit pieces of the token's choices
  const int s0 = (int)((long long)segs * (rank * ED_WARPS + warp) / (ED_SPLIT * ED_WARPS));
  const int s1 = (int)((long long)segs * (rank * ED_WARPS + warp + 1) / (ED_SPLIT * ED_WARPS));
  int count = 0;
  auto gather = [&] {
    __syncwarp();
    if (n < a.D) {
      for (int i = 0; i < count; i += ED_ROWS) {
        uint4 v[ED_ROWS];
#pragma unroll
        for (int q = 0; q < ED_ROWS; ++q)
          if (i + q < count) v[q] = __ldg(reinterpret_cast<const uint4*>(w2 + (size_t)s_u[warp][i + q] * a.D));
#pragma unroll
        for (int q = 0; q < ED_ROWS; ++q)
          if (i + q < count) {
            float f[8];
            Elt<bf16_tag>::unpack(v[q], f);
            const float c = s_c[warp][i + q];
#pragma unroll
            for (int j = 0; j < 4; ++j) ffma2(acc[j], make_float2(f[2 * j], f[2 * j + 1]), make_float2(c, c));
          }
      }
    }
    __syncwarp();
    count = 0;
  };
  constexpr int AHEAD = 2;  // pieces whose expert, weight and units are loaded together
  for (int s = s0; s < s1; s += AHEAD) {
    int e[AHEAD], u[AHEAD];
    float w[AHEAD], hv[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int at = min(s + q, s1 - 1), j = at / seg, p = t * a.k + j;
      u[q] = (at - j * seg) * 32 + lane;
      e[q] = a.ids[p];
      w[q] = a.weights[p];
      hv[q] = u[q] < a.H ? h[(size_t)p * a.H + u[q]] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      // (a choice that is not taken has no h: what was read for it is not used)
      const bool on = s + q < s1 && e[q] >= 0 && e[q] < a.E && w[q] != 0.f && u[q] < a.H;
      const float c = on ? hv[q] * w[q] : 0.f;
      const uint32_t live = __ballot_sync(0xffffffffu, c != 0.f);
      if (count + __popc(live) > ED_LIST) gather();
      if (c != 0.f) {
        const int at = count + __popc(live & ((1u << lane) - 1));
        s_c[warp][at] = c;
        s_u[warp][at] = e[q] * a.H + u[q];
      }
      count += __popc(live);
    }
  }
  gather();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    s_sum[warp][lane * 8 + 2 * q] = acc[q].x;
    s_sum[warp][lane * 8 + 2 * q + 1] = acc[q].y;
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < ED_WARPS; ++q) v += s_sum[q][threadIdx.x];
    s_part[threadIdx.x] = v;
  }
  cluster_sync_all();
  constexpr int SHARE = 256 / ED_SPLIT;
  const int c = rank * SHARE + (int)threadIdx.x, col = (blockIdx.x / ED_SPLIT) * 256 + c;
  if (threadIdx.x < SHARE && col < a.D) {
    const uint32_t at = smem_u32(&s_part[c]);
    float v[ED_SPLIT], sum = 0.f;
#pragma unroll
    for (int q = 0; q < ED_SPLIT; ++q)
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[q]) : "r"(cluster_map(at, (uint32_t)q)) : "memory");
#pragma unroll
    for (int q = 0; q < ED_SPLIT; ++q) sum += v[q];
    reinterpret_cast<__nv_bfloat16*>(a.y)[(size_t)t * a.D + col] = __float2bfloat16_rn(sum);
  }
  cluster_sync_all();  // the partial sums stay until every block has read them
}

// y[t] = sum_j weights[t, j] o[slot[t k + j]] in the order of the places; a
// place without an expert or of weight 0 is not read (o has no row for it).
// Bound by reading o; 16-byte pieces, one thread per four columns and token.
constexpr int EC_THREADS = 256;
__global__ void __launch_bounds__(EC_THREADS) experts_combine_kernel(const ExpertsArgs a, const float* __restrict__ o,
                                                                     const int* __restrict__ slot) {
  const int t = blockIdx.x, c = (blockIdx.y * EC_THREADS + threadIdx.x) * 4;
  pdl_launch_dependents();
  pdl_wait();
  if (c >= a.D) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j;
    const float w = a.ids[p] >= 0 ? a.weights[p] : 0.f;
    const int r = slot[p];
    if (w != 0.f && r >= 0 && r < a.T * a.k) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(o + (size_t)r * a.D + c));
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
      sum.z = fmaf(w, v.z, sum.z);
      sum.w = fmaf(w, v.w, sum.w);
    }
  }
  *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + (size_t)t * a.D + c) =
      make_uint2(pack_bf16x2_rn(sum.x, sum.y), pack_bf16x2_rn(sum.z, sum.w));
}

// xg[r] = x[rows[r] / k]: a grouped copy of the tokens, and slot[rows[r]] = r; a warp a row, four
// pieces of 16 bytes a lane in flight.
constexpr int EX_WARPS = 8;
__global__ void __launch_bounds__(32 * EX_WARPS) experts_gather_kernel(const ExpertsArgs a, uint16_t* __restrict__ xg,
                                                                       int* __restrict__ slot) {
  const int lane = threadIdx.x & 31, n = a.D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const int r = blockIdx.x * EX_WARPS + (threadIdx.x >> 5);
  if (r >= a.T * a.k) return;
  const int i = a.rows[r];
  if (i < 0 || i >= a.T * a.k) return;
  if (lane == 0) slot[i] = r;
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + (size_t)(i / a.k) * a.ldx);
  uint4* dst = reinterpret_cast<uint4*>(xg + (size_t)r * a.D);
  for (int c = lane; c < n; c += 128) {
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + 32 * q < n) v[q] = __ldg(src + c + 32 * q);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + 32 * q < n) dst[c + 32 * q] = v[q];
  }
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Up to two choices an expert: the gate-first passes above; more: the grouped products on the tensor cores (us, passes
// / products, ReLU at 90 %, D = 2560, H = 1024: 8 of 64 experts 50 / 83 at 4 tokens, 79 / 101 at 8, 134 / 129 at 16; 2 of
// 8 experts 31 / 38 at 8 tokens, 51 / 40 at 16; D = H = 4096, 4 of 16 experts 192 / 213 at 8, 328 / 256 at 16).
//
// The passes cost by the unit, the products by the byte: with SiLU, where every unit is live, products from 12288 units of
// all choices on (H = 1500, D = 320: 16 choices 38 / 32, 8 23 / 23; D = 4096, H = 2048: 5 choices 68 / 69, 8 92 / 85), and
// else from 100 D units on (ReLU, H = 1500, D = 320: 32 choices 34 / 34, 80 65 / 39; D = 640: 37 / 42, 68 / 54; D = 1024:
// 44 / 56, 79 / 71; D = 2560: 73 / 113, 140 / 143).
bool few(const ExpertsArgs& a) {
  const long long choices = (long long)a.T * a.k, units = choices * a.H;
  if (choices > 2ll * a.E) return false;
  return units <= (a.act == ACT_SILU ? 12288 : 100ll * a.D);
}

}  // namespace

size_t experts_workspace(int T, int k, int D, int H) {
  const size_t R = (size_t)T * k;
  // h, the rows' products (before them, in the same place, the grouped tokens), and the choices' rows
  const size_t products = round_up(2 * R * round_up(H, 8), 256) + round_up(sizeof(float) * R * D, 256) + sizeof(int) * R;
  return std::max(products, sizeof(float) * R * H);  // the gate-first passes: h in fp32
}

cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (few(a)) {
    float* h = static_cast<float*>(a.workspace);
    const dim3 grid((unsigned)((a.H + EG_WARPS - 1) / EG_WARPS), (unsigned)(a.T == 1 ? a.k : std::min(a.E, a.T * a.k)));
    const size_t row = 2 * (size_t)a.D;
    if (a.T == 1)
      e = row <= EG_STAGE ? ops_launch(experts_gate_kernel<true, true>, grid, 32 * EG_WARPS, row, s, 1, a, h)
                          : ops_launch(experts_gate_kernel<true, false>, grid, 32 * EG_WARPS, 0, s, 1, a, h);
    else
      e = EG_ROWS * row <= EG_STAGE ? ops_launch(experts_gate_kernel<false, true>, grid, 32 * EG_WARPS, EG_ROWS * row, s, 1, a, h)
                              : ops_launch(experts_gate_kernel<false, false>, grid, 32 * EG_WARPS, 0, s, 1, a, h);
    if (e != cudaSuccess) return e;
    return ops_launch(experts_down_kernel, dim3((unsigned)((a.D + 255) / 256 * ED_SPLIT), (unsigned)a.T), 32 * ED_WARPS, 0,
                      s, ED_SPLIT, a, (const float*)h);
  }
  const int R = a.T * a.k, Hp = (int)round_up(a.H, 8);
  float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + round_up(2 * (size_t)R * Hp, 256));
  int* slot = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(o) + round_up(sizeof(float) * (size_t)R * a.D, 256));
  // A copy of the tokens in the rows' order: reading them through gather4 instead costs the gate and up product more
  // than the copy from 256 tokens on (at 4096 tokens, 8 choices, D = 2560: 735 against 606 us); below neither form is
  // faster, so there is this one.
  uint16_t* xg = reinterpret_cast<uint16_t*>(o);
  e = ops_launch(experts_gather_kernel, dim3((unsigned)((R + EX_WARPS - 1) / EX_WARPS)), 32 * EX_WARPS, 0, s, 1, a, xg,
                 slot);
  if (e != cudaSuccess) return e;
  // h is rounded to bf16 here, as the intermediate of a dense bf16 FFN is: an MMA's operands have 16 bits.  (Relative error
  // against 64 bits at 4096 tokens 0.0024, of the few-token form with h in fp32 0.0017: that of y's own rounding.)
  GmmArgs up;
  up.x = xg;
  up.ldx = a.D;
  up.w = a.W1;
  up.w3 = a.W3;
  up.offsets = a.offsets;
  up.y = a.workspace;
  up.ldy = Hp;
  up.R = R;
  up.XR = R;
  up.N = a.H;
  up.K = a.D;
  up.NY = Hp;
  up.E = a.E;
  up.act = a.act;
  if ((e = launch_gmm(up, s)) != cudaSuccess) return e;
  GmmArgs down;
  down.x = a.workspace;
  down.ldx = Hp;
  down.w = a.W2t;
  down.kn = 1;
  down.offsets = a.offsets;
  down.y = o;
  down.y_f32 = 1;
  down.ldy = a.D;
  down.R = R;
  down.XR = R;
  down.N = a.D;
  down.K = a.H;
  down.E = a.E;
  if ((e = launch_gmm(down, s)) != cudaSuccess) return e;
  return ops_launch(experts_combine_kernel, dim3((unsigned)a.T, (unsigned)((a.D + 4 * EC_THREADS - 1) / (4 * EC_THREADS))),
                    EC_THREADS, 0, s, 1, a, (const float*)o, (const int*)slot);
}

}  // namespace sffn

// route.cu -- the router's choice and the grouping of its choices by expert.
//
// Per token the k largest of E logits (ties to the lowest index; -inf and NaN
// are closed experts and are never chosen), their weights
//   softmax   w_j = exp(z_j - m) / sum_i exp(z_i - m), i over the chosen
//             (normalised) or over all E
//   sigmoid   w_j = 1 / (1 + exp(-z_j)), over their sum when normalised (where
//             the largest z_j, m, is below 0, both times 1 + exp(-m): fp32 holds
//             no sigmoid below about -88, but their ratios it does),
// and a stable counting sort of the T k choices by expert: offsets[E + 1] and,
// for every grouped row, the choice token * k + place that it serves.
//
// One warp takes a token: the logits sit in registers (E / 32 a lane) as
// order-preserving integer keys that each lane sorts, and a choice is one or
// two warp-wide maxima over the lanes' firsts (redux, no shuffle trees).
// The sort is exact integer work, so its result does not depend on timing: a
// cluster of blocks owns a chunk of consecutive tokens (a token or two a warp:
// the choice is a chain of dependent steps, so it wants warps) and counts its
// choices per expert, and a second kernel adds the counts of the chunks before
// its own.  A few choices are one block's work altogether.
//
// Measured (us): one token, 8 of 64 experts, 6.4 a call, 2.9 in a graph (a chain
// of dependent steps, next to nothing is read); 16384 tokens, 8 of 256 experts,
// bf16 logits, 25.5 against 1.5 for their bytes: the choice is bound by its
// instructions (17; 68 % of the issue slots are used), the sort by latency.
#include "common.cuh"
#include "ops.h"
#include "tc.cuh"

namespace sffn {
namespace {

constexpr int ROUTE_WARPS = 16;
constexpr int ROUTE_THREADS = 32 * ROUTE_WARPS;
// Choices that one block sorts by itself, of so many tokens at most (us, one block / two kernels, 2 of 8 experts: 64 tokens
// 6.7 / 9.4, 128 8.8 / 9.3, 256 15.2 / 9.4; 8 of 64: 64 tokens 7.4 / 9.3; 8 of 256: 48 8.6 / 9.8, 64 10.6 / 9.6).
constexpr int ROUTE_ONE = 512, ROUTE_ONE_TOKENS = 128;
constexpr int ROUTE_CHUNKS = 128; // most chunks of the two-kernel form

// Larger float <-> larger key; NaN and -inf share the key 0 (closed).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 ties with 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Below this a sigmoid is 0 in binary64 as well (exp(-745.2) rounds to 0): a token whose largest logit lies there, at a
// mask of the type's lowest value say, keeps weights of 0.
constexpr float SIGMOID_LOWEST = -745.f;

// exp(v - m) for v <= m, with equal infinities counting as equal
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.f : expf(v - m); }

// A lane's logits as keys, sorted once (up to 8 of them); then a round looks at the lanes' firsts alone and the
// winner's list moves up.  hi orders, lo says which: the larger lo is the lower index.
//   bf16 (and E <= 65535): value and index fit one word, so a round is one redux;
//   fp32: the value, then the index among the lanes that hold it.
template <int L, bool BF16>
struct Keys {
  uint32_t hi[L], lo[BF16 ? 1 : L];

  // A lane holds V neighbouring logits at a time, one load of them where rows are aligned to it (a.vec).
  static constexpr int V = L < (BF16 ? 8 : 4) ? L : (BF16 ? 8 : 4);

  __device__ __forceinline__ void load(const RouteArgs& a, size_t base, int lane) {
    constexpr int EB = BF16 ? 2 : 4;
    const uint8_t* row = reinterpret_cast<const uint8_t*>(a.logits) + base * EB;
#pragma unroll
    for (int c = 0; c < L / V; ++c) {
      const int e0 = (c * 32 + lane) * V;
      uint32_t raw[V * EB >= 4 ? V * EB / 4 : 1] = {};
      const bool one = a.vec && e0 + V <= a.E;
      if (one) {
        if constexpr (V * EB == 16) {
          const uint4 v = *reinterpret_cast<const uint4*>(row + (size_t)e0 * EB);
          raw[0] = v.x;
          raw[1] = v.y;
          raw[2] = v.z;
          raw[3] = v.w;
        } else if constexpr (V * EB == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(row + (size_t)e0 * EB);
          raw[0] = v.x;
          raw[1] = v.y;
        } else if constexpr (V * EB == 4) {
          raw[0] = *reinterpret_cast<const uint32_t*>(row + (size_t)e0 * EB);
        } else {
          raw[0] = *reinterpret_cast<const uint16_t*>(row + (size_t)e0 * EB);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = c * V + j, e = e0 + j;
        float v = -INFINITY;
        if (one)
          v = BF16 ? __uint_as_float((j & 1) ? raw[j / 2] & 0xffff0000u : raw[j / 2] << 16) : __uint_as_float(raw[BF16 ? 0 : j]);
        else if (e < a.E)
          v = BF16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(row)[e] << 16)
                   : reinterpret_cast<const float*>(row)[e];
        hi[i] = order_key(v);
        if (BF16) {
          if (hi[i]) hi[i] = (hi[i] & 0xffff0000u) | (uint32_t)(0xffff - e);  // a bf16 value's low half is all ones or zeros
        } else {
          lo[i] = ~(uint32_t)e;
        }
      }
    }
  }
  __device__ __forceinline__ void order(int i, int j) {  // the larger first
    if (BF16) {
      const uint32_t x = max(hi[i], hi[j]);
      hi[j] = min(hi[i], hi[j]);
      hi[i] = x;
    } else {
      const bool sw = hi[j] > hi[i] || (hi[j] == hi[i] && lo[j] > lo[i]);
      const uint32_t h = hi[i], l = lo[i];
      hi[i] = sw ? hi[j] : h;
      lo[i] = sw ? lo[j] : l;
      hi[j] = sw ? h : hi[j];
      lo[j] = sw ? l : lo[j];
    }
  }
  static constexpr bool SORTED = L <= 8;  // longer lists look for their first in every round
  __device__ __forceinline__ void sort() {  // odd-even transposition
    if (!SORTED) return;
#pragma unroll
    for (int r = 0; r < L; ++r)
#pragma unroll
      for (int i = 0; i + 1 < L; ++i)
        if (((i ^ r) & 1) == 0) order(i, i + 1);
  }
  __device__ __forceinline__ void pop() {
#pragma unroll
    for (int i = 0; i + 1 < L; ++i) {
      hi[i] = hi[i + 1];
      if (!BF16) lo[i] = lo[i + 1];
    }
    hi[L - 1] = 0;
  }
  // The largest key of the warp (0: none is open) and, for fp32, the low word that says whose it is; the lane that
  // holds it drops it.
  __device__ __forceinline__ uint32_t next(uint32_t* low) {
    uint32_t top = hi[0];
    if (!SORTED) {
#pragma unroll
      for (int i = 1; i < L; ++i) top = max(top, hi[i]);
    }
    const uint32_t best = __reduce_max_sync(0xffffffffu, top);
    if (BF16) {
      if (SORTED) {
        if (top == best) pop();
      } else {
#pragma unroll
        for (int i = 0; i < L; ++i) hi[i] = hi[i] == best ? 0u : hi[i];
      }
      return best;
    }
    uint32_t mine = top == best ? lo[0] : 0u;
    if (!SORTED) {
      mine = 0;
#pragma unroll
      for (int i = L - 1; i >= 0; --i)
        if (hi[i] == best) mine = max(mine, lo[i]);
    }
    const uint32_t at = __reduce_max_sync(0xffffffffu, mine);
    if (SORTED) {
      if (top == best && mine == at) pop();
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) hi[i] = lo[i] == at ? 0u : hi[i];
    }
    *low = at;
    return best;
  }
  // a bf16 key's low half holds the index: the value's was zeros, or ones where the key is complemented (negative)
  static __device__ __forceinline__ float value(uint32_t key) {
    return key_value(!BF16 ? key : (key & 0x80000000u) ? key & 0xffff0000u : key | 0xffffu);
  }
  static __device__ __forceinline__ int index(uint32_t key, uint32_t low) {
    return BF16 ? 0xffff - (int)(key & 0xffffu) : (int)~low;
  }
};

// One token by one warp: lane j < k ends up with choice j, and returns it.  L: logits a lane.
template <int L, bool BF16>
__device__ __forceinline__ int choose(const RouteArgs& a, int t, int lane) {
  Keys<L, BF16> keys;
  keys.load(a, (size_t)t * a.ld, lane);
  float all = 0.f;
  if (!a.sigmoid && !a.normalize) {  // the sum over every open expert
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) top = max(top, keys.hi[i]);
    const float mx = keys.value(__reduce_max_sync(0xffffffffu, top));
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (keys.hi[i]) all += exp_below(keys.value(keys.hi[i]), mx);
    all = warp_sum(all);
  }
  keys.sort();
  uint32_t ck = 0, cl = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t low = 0;
    const uint32_t best = keys.next(&low);
    if (best == 0) break;  // no open expert is left
    if (lane == j) {
      ck = best;
      cl = low;
    }
  }
  const int ce = ck ? keys.index(ck, cl) : -1;
  const float m = keys.value(__shfl_sync(0xffffffffu, ck, 0)), v = keys.value(ck);
  float w = 0.f;
  if (ce >= 0) {
    if (!a.sigmoid)
      w = exp_below(v, m);
    else if (a.normalize && m < 0.f && m > SIGMOID_LOWEST)
      w = exp_below(v, m) * (1.f + expf(m)) / (1.f + expf(v));
    else
      w = 1.f / (1.f + expf(-v));
  }
  float total = 1.f;
  if (a.normalize) total = warp_sum(w);
  else if (!a.sigmoid) total = all;
  if (lane < a.k) {
    a.weights[(size_t)t * a.k + lane] = total > 0.f ? w / total : 0.f;
    a.ids[(size_t)t * a.k + lane] = ce;
  }
  return ce;
}

// Tokens [t0, t1) of this block: choices, then counts per expert in s_hist.
template <int L, bool BF16>
__device__ __forceinline__ void choose_block(const RouteArgs& a, int t0, int t1, int* s_hist) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) s_hist[e] = 0;
  __syncthreads();
  for (int t = t0 + warp; t < t1; t += ROUTE_WARPS) {
    const int e = choose<L, BF16>(a, t, lane);
    if (lane < a.k && e >= 0) atomicAdd(&s_hist[e], 1);
  }
  __syncthreads();
}

// Grouped rows of this block's choices, given s_base[e] = the row of its first
// choice of expert e.  Warps take consecutive spans of choices; s_cnt[w][e]
// (zero before) counts span w, and the spans before a warp's own give its first
// row.
__device__ __forceinline__ void scatter_block(const RouteArgs& a, int t0, int t1, const int* s_base, int* s_cnt,
                                              int warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p0 = t0 * a.k, n = (t1 - t0) * a.k;
  const int span = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int b = min(n, warp * span), c = warp < warps ? min(n, b + span) : b;
  constexpr int KEEP = 4;  // the span's first choices stay in registers
  int kept[KEEP];
#pragma unroll
  for (int q = 0; q < KEEP; ++q) kept[q] = b + 32 * q + lane < c ? a.ids[p0 + b + 32 * q + lane] : -1;
#pragma unroll
  for (int q = 0; q < KEEP; ++q)
    if (kept[q] >= 0) atomicAdd(&s_cnt[warp * a.E + kept[q]], 1);
  for (int i = b + 32 * KEEP + lane; i < c; i += 32) {
    const int e = a.ids[p0 + i];
    if (e >= 0) atomicAdd(&s_cnt[warp * a.E + e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) {
    int at = s_base[e];
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
      const int v = s_cnt[w * a.E + e];
      s_cnt[w * a.E + e] = at;
      at += v;
    }
  }
  __syncthreads();
  auto place = [&](int i0, int e) {
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) a.rows[s_cnt[warp * a.E + e] + __popc(same & ((1u << lane) - 1))] = p0 + i0 + lane;
    __syncwarp();
    if (e >= 0 && (same >> lane) == 1u) s_cnt[warp * a.E + e] += __popc(same);  // the last lane of its expert
    __syncwarp();
  };
#pragma unroll
  for (int q = 0; q < KEEP; ++q)
    if (b + 32 * q < c) place(b + 32 * q, kept[q]);
  for (int i0 = b + 32 * KEEP; i0 < c; i0 += 32) place(i0, i0 + lane < c ? a.ids[p0 + i0 + lane] : -1);
}

// Exclusive sums of s_v[0 .. E) into s_v, the total in s_v[E] (whole block).
__device__ __forceinline__ void exclusive_scan(int* s_v, int E, int* s_w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += ROUTE_THREADS) {
    const int e = e0 + tid;
    const int v = e < E ? s_v[e] : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    int before = carry, total = carry;
    for (int w = 0; w < ROUTE_WARPS; ++w) {
      if (w < warp) before += s_w[w];
      total += s_w[w];
    }
    if (e < E) s_v[e] = before + x - v;
    carry = total;
    __syncthreads();
  }
  if (tid == 0) s_v[E] = carry;
  __syncthreads();
}

template <int L, bool BF16>
__global__ void __launch_bounds__(ROUTE_THREADS) route_one_kernel(const RouteArgs a, int warps) {
  extern __shared__ int sm[];
  int* s_base = sm;               // [E + 1]
  int* s_w = s_base + a.E + 1;    // [ROUTE_WARPS]
  int* s_cnt = s_w + ROUTE_WARPS; // [warps][E]
  for (int i = threadIdx.x; i < warps * a.E; i += ROUTE_THREADS) s_cnt[i] = 0;
  pdl_launch_dependents();
  pdl_wait();
  choose_block<L, BF16>(a, 0, a.T, s_base);
  exclusive_scan(s_base, a.E, s_w);
  for (int e = threadIdx.x; e <= a.E; e += ROUTE_THREADS) a.offsets[e] = s_base[e];
  const int total = s_base[a.E];
  for (int i = total + threadIdx.x; i < a.T * a.k; i += ROUTE_THREADS) a.rows[i] = -1;
  scatter_block(a, 0, a.T, s_base, s_cnt, warps);
}

// One token by one warp, with no shared memory and no barrier: its choices are
// different experts, so a choice's row is the number of choices below it.
template <int L, bool BF16>
__global__ void __launch_bounds__(32) route_token_kernel(const RouteArgs a) {
  const int lane = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int mine = choose<L, BF16>(a, 0, lane);  // lane j < k: choice j, or -1
  int rank = 0;
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(0xffffffffu, mine, j);
    rank += e >= 0 && e < mine;
  }
  if (lane < a.k) a.rows[mine >= 0 ? rank : lane] = mine >= 0 ? lane : -1;  // places without an expert are the last
  for (int e0 = 0; e0 <= a.E; e0 += 32) {
    const int e = e0 + lane;
    int below = 0;
    for (int j = 0; j < a.k; ++j) {
      const int c = __shfl_sync(0xffffffffu, mine, j);
      below += c >= 0 && c < e;
    }
    if (e <= a.E) a.offsets[e] = below;
  }
}

template <int L, bool BF16>
__global__ void __launch_bounds__(ROUTE_THREADS) route_choose_kernel(const RouteArgs a, int per, int split) {
  extern __shared__ int sm[];
  pdl_launch_dependents();
  pdl_wait();
  const int chunk = blockIdx.x / split, rank = blockIdx.x % split, sub = (per + split - 1) / split;
  const int c1 = min(a.T, chunk * per + per), t0 = min(c1, chunk * per + rank * sub), t1 = min(c1, t0 + sub);
  choose_block<L, BF16>(a, t0, t1, sm);
  if (split > 1) cluster_sync_all();
  for (int e = rank * ROUTE_THREADS + threadIdx.x; e < a.E; e += split * ROUTE_THREADS) {
    int v = sm[e];
    if (split > 1) {
      v = 0;
      const uint32_t at = smem_u32(sm + e);
      for (int q = 0; q < split; ++q) {
        int w;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w) : "r"(cluster_map(at, (uint32_t)q)) : "memory");
        v += w;
      }
    }
    a.hist[(size_t)chunk * a.E + e] = v;
  }
  if (split > 1) cluster_sync_all();  // the counts stay until every block has read them
}

__global__ void __launch_bounds__(ROUTE_THREADS) route_group_kernel(const RouteArgs a, int per, int nb, int warps) {
  extern __shared__ int sm[];
  int* s_base = sm;
  int* s_w = s_base + a.E + 1;
  int* s_mine = s_w + ROUTE_WARPS;  // [E] choices of the chunks before this one
  int* s_cnt = s_mine + a.E;
  for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) s_mine[e] = s_base[e] = 0;
  for (int i = threadIdx.x; i < warps * a.E; i += ROUTE_THREADS) s_cnt[i] = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  // several threads an expert where there are few: each sums every `stride`-th chunk
  const int cols = min((a.E + 31) / 32 * 32, ROUTE_THREADS), stride = ROUTE_THREADS / cols, from = threadIdx.x / cols;
  for (int e = threadIdx.x % cols; e < a.E && from < stride; e += cols) {
    int before = 0, total = 0;
    constexpr int B = 32;  // counts in flight
    for (int b0 = from; b0 < nb; b0 += B * stride) {
      int v[B];
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = b0 + i * stride < nb ? a.hist[(size_t)(b0 + i * stride) * a.E + e] : 0;
#pragma unroll
      for (int i = 0; i < B; ++i) {
        if (b0 + i * stride < (int)blockIdx.x) before += v[i];
        total += v[i];
      }
    }
    atomicAdd(&s_mine[e], before);
    atomicAdd(&s_base[e], total);
  }
  __syncthreads();
  exclusive_scan(s_base, a.E, s_w);
  const int total = s_base[a.E], t0 = min(a.T, (int)blockIdx.x * per), t1 = min(a.T, t0 + per);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= a.E; e += ROUTE_THREADS) a.offsets[e] = s_base[e];
  }
  for (int i = total + blockIdx.x * ROUTE_THREADS + threadIdx.x; i < a.T * a.k; i += gridDim.x * ROUTE_THREADS)
    a.rows[i] = -1;
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) s_base[e] += s_mine[e];
  __syncthreads();
  scatter_block(a, t0, t1, s_base, s_cnt, warps);
}

// warps that take part in the scatter: as many as 48 KB of shared counts have room for
int scatter_warps(int E, int fixed_ints) {
  const int w = (48 * 1024 / 4 - fixed_ints) / E;
  return w < 1 ? 1 : w > ROUTE_WARPS ? ROUTE_WARPS : w;
}

bool one_block(int T, int k) { return T <= ROUTE_ONE_TOKENS && (long long)T * k <= ROUTE_ONE; }

int route_chunks(int T, int* per) {
  *per = (T + ROUTE_CHUNKS - 1) / ROUTE_CHUNKS;
  if (*per < ROUTE_WARPS) *per = ROUTE_WARPS;
  return (T + *per - 1) / *per;
}

template <int L, bool BF16>
cudaError_t route_lt(const RouteArgs& a, cudaStream_t s) {
  if (a.T == 1) return ops_launch(route_token_kernel<L, BF16>, dim3(1), 32, 0, s, 1, a);
  if (one_block(a.T, a.k)) {
    const int fixed = a.E + 1 + ROUTE_WARPS, warps = scatter_warps(a.E, fixed);
    return ops_launch(route_one_kernel<L, BF16>, dim3(1), ROUTE_THREADS, sizeof(int) * (fixed + warps * a.E), s, 1, a, warps);
  }
  int per;
  const int nb = route_chunks(a.T, &per);
  const int split = per > 8 * ROUTE_WARPS ? 8 : per > 4 * ROUTE_WARPS ? 4 : per > 2 * ROUTE_WARPS ? 2 : 1;
  cudaError_t e = ops_launch(route_choose_kernel<L, BF16>, dim3(nb * split), ROUTE_THREADS, sizeof(int) * a.E, s, split, a, per,
                             split);
  if (e != cudaSuccess) return e;
  const int fixed = 2 * a.E + 1 + ROUTE_WARPS, warps = scatter_warps(a.E, fixed);
  return ops_launch(route_group_kernel, dim3(nb), ROUTE_THREADS, sizeof(int) * (fixed + warps * a.E), s, 1, a, per, nb,
                    warps);
}

template <int L>
cudaError_t route_l(const RouteArgs& a, cudaStream_t s) {
  return a.bf16 ? route_lt<L, true>(a, s) : route_lt<L, false>(a, s);
}

}  // namespace

size_t route_workspace(int T, int E, int k) {
  if (one_block(T, k)) return 0;
  int per;
  return sizeof(int) * (size_t)route_chunks(T, &per) * E;
}

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  const int l = (a.E + 31) / 32;
  if (l <= 1) return route_l<1>(a, s);
  if (l <= 2) return route_l<2>(a, s);
  if (l <= 4) return route_l<4>(a, s);
  if (l <= 8) return route_l<8>(a, s);
  if (l <= 16) return route_l<16>(a, s);
  return route_l<32>(a, s);
}

}  // namespace sffn

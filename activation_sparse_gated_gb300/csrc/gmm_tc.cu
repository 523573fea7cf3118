// gmm_tc.cu -- products grouped by expert on the tensor cores (tcgen05), for
// groups of more than a few rows:
//
//   plain   y[r, n] = sum_k x[s(r), k] w[e, n, k]
//   gated   h[r, n] = A(sum_k x w1) * (sum_k x w3)      (two products, one pass over x)
//   int8    y[r, n] = sx sw sum_k xq wq
//
// The weights are the M side of the MMA (128 rows of w a block, 256 a pair of
// blocks with cta_group::2) and the rows of x the N side, whose width is any
// multiple of 16 (32 for a pair) up to 256, so a ragged tile's MMAs are as wide
// as its rows.  (Its copies are not: without an index x comes in boxes of 32 rows
// or of a whole tile, through one in fours.)  An MMA of 16 K values takes N / 2 cycles from 96 columns on and 49
// below (measured, one block, operands in shared memory): full tensor rate from
// 128 columns on, 256 halve the traffic of w; and 128 x 16 weights per 49 cycles
// and SM are above the memory's rate, which is what bounds short groups.
//
// A block walks the tiles of all groups (persistent, tile ids strided by the
// grid); the tile list is a prefix sum over the groups that every block makes
// for itself from the device's offsets, so the host never waits for them.  Two
// warps feed a ring of shared stages by TMA (one the weights, one the rows of x:
// a single one is too slow for 128-wide tiles), one warp issues the MMAs, and
// eight empty one TMEM accumulator while the MMAs fill the other.  Tiles are
// taken eight weight tiles at a time over a group's rows (1, 2 and 4 or 32 and
// 64 are up to 5 and 15 % slower at 8192 x 14336 x 4096: L2).
//
// Rows of x come as 2D tiles, or, through an index, by gather4 (four rows a
// copy), so a grouped copy of x need not be made.
//
// int8: this part's int8 MMA rate is far below its 16-bit rate, and int8 codes are
// exact in fp16 with exact products and fp32 sums that are exact below 2^24.  So
// the raw codes arrive by TMA, 128 a row, and sixteen warps widen them: half the
// memory traffic of 16-bit weights.  The widened w goes to TMEM (an MMA takes its
// A operand from there), the widened x to shared memory, which at 128 x 128 is
// busy with copies, loads, stores and the MMAs' reads of x for four cycles in
// five.  64 codes of a 128 x 128 tile take 0.28 us, 0.19 without the widening,
// 0.13 the MMAs.  Where groups are long the codes are widened once into fp16
// copies instead (widen_kernel).
//
// Few tiles and a long sum: the blocks of a cluster cut K and add their partial
// tiles through distributed shared memory in a fixed order.
//
// Measured (us; share of the copy rate / of cuBLAS's burst rate; long ones by the
// board): bf16, 128 rows over 64 experts of 1024 x 2560 44.1 (97 % / 1 %); 16384
// ragged rows over 64 experts of 7168 x 2560 502 to 550 (72 % / 57 % at 543); one
// group 8192 x 14336 x 4096 499 (- / 99 %); int8 8192 x 14336 x 4096 531 to 556 (-
// / 90 % at 550, 40 us of it the copies), 77 x 2560 x 7168 14.6 (20 % / 10 %:
// latency of the chunks' chain and of the launch),
// 4093 rows over 16 experts of 1000 x 2560 43 to 45 (20 % / 25 %: widening; 50 with
// w widened in shared memory, a value a store and 64 codes a stage).
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "ops.h"
#include "sffn.h"
#include "tc.cuh"

namespace sffn {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // ffn_tc.cu

namespace {

constexpr int TG_EPI_WARP0 = 4;   // warps 4..11 (int8: 4..7): epilogue (TMEM lane quarter = warp % 4)
constexpr int TG_CONV_WARP0 = 8;  // warps 8..23: int8 -> fp16
constexpr int TG_CONV_WARPS = 16, TG_CONV_GROUPS = 2;
constexpr int TG_THREADS = 384, TG_THREADS_I8 = 32 * (TG_CONV_WARP0 + TG_CONV_WARPS);
constexpr uint64_t TG_TIMEOUT_NS = 250000000ull;
constexpr size_t TG_SMEM = 227 * 1024;
constexpr int TG_DEVICES = 64;
// what a kernel multiplies: bf16; bf16 gate and up together; int8 codes widened in flight; fp16 copies of codes
enum { TG_BF16, TG_GATED, TG_I8, TG_F16 };
// the epilogue's shared scratch of a warp: 16 rows of 32 words, 4 words apart (no bank conflicts either way)
constexpr int TG_EPI_PITCH = 36;
constexpr int TG_PART = 132;  // words between the rows of a partial tile
constexpr uint32_t TG_EPI_BYTES = 16 * TG_EPI_PITCH * 4;
constexpr int TG_G = 8;           // weight tiles of one raster group

struct TgArgs {
  GmmArgs g;
  int NT;      // most rows of x a tile
  int bxr;     // rows of a small x box (no index); the large one has NT / CTAS
  int MT;      // weight tiles: ceil(N / (128 CTAS))
  int KC;      // 64-wide K chunks
  int S;       // operand stages (int8: of widened codes)
  int SR;      // raw stages (int8)
  int wcol;    // int8: first TMEM column of the widened weights
  int ks;      // blocks of a cluster that cut K between them (1: no cut)
  int cols;    // TMEM columns allocated
  int vec;     // rows of y take 16-byte stores: y, ldy and N are multiples of that
  int nacc;    // accumulators: 2, or 1 where one takes all of TMEM (the epilogue is not hidden then)
  int* err;
};

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait; PAIR: it also sees what threads of the pair's other block released.
template <bool PAIR>
__device__ __forceinline__ bool tg_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  uint64_t t0 = 0;  // the clock is read only after many tries: reading it costs more than most waits
  for (uint32_t i = 1;; ++i) {
    if (PAIR ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > TG_TIMEOUT_NS) {
        *abort = 1;
        atomicOr(err, DEV_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tma_w3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tma_x2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// four rows y[0..3] of the map (box one row high), 128 bytes each
template <int CTAS>
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&y)[4],
                                            uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar)
        : "memory");
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(v));
  return v != 0;
}

// Operand descriptors travel as their low words: the high words are the same for every stage.
template <int CTAS>
__device__ __forceinline__ void tg_mma(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                       uint32_t idesc, uint32_t acc) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
}

// The same with A in TMEM: lane = row, a column = two values of K.
__device__ __forceinline__ void tg_mma_t(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
      : "memory");
}

// Arrive on `bar` (in both blocks of a pair) when the MMAs this thread issued so far are done.
template <int CTAS>
__device__ __forceinline__ void tg_commit(uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tg_alloc(uint32_t* slot, uint32_t ncols) {
  if constexpr (CTAS == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, ncols);
  }
}
template <int CTAS>
__device__ __forceinline__ void tg_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}

// 16 consecutive columns of this thread's lane, written; not waited for.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 32 consecutive fp32 columns of this thread's lane, not waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 16 int8 codes -> 16 fp16 values, exactly: a code plus 128 is a byte u, the
// half with bits 0x6400 | u is 1024 + u, and 1024 + u - 1152 is the code.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t* out) {
  const uint32_t u = v ^ 0x80808080u;
  uint32_t lo, hi;
  asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(lo) : "r"(u), "r"(0x64646464u));
  asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(hi) : "r"(u), "r"(0x64646464u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[0]) : "r"(lo), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[1]) : "r"(hi), "r"(0x64806480u));
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts4(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 lds16a(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// One tile: expert, weight tile, rows [r0, r1) of x and the MMA width n.
struct Tile {
  int e, mt, r0, r1, n;
};

template <int CTAS>
__device__ __forceinline__ Tile tile_at(const TgArgs& p, const int* s_off, const int* s_pre, int t) {
  int lo = 0, hi = p.g.E;  // the last expert whose first tile is <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_pre[mid] <= t) lo = mid;
    else hi = mid;
  }
  Tile q;
  q.e = lo;
  const int m = s_off[lo + 1] - s_off[lo];
  const int tt = (m + p.NT - 1) / p.NT;
  constexpr int Q = 16 * CTAS;
  const int per = ((m + tt - 1) / tt + Q - 1) / Q * Q;
  const int i = t - s_pre[lo];
  const int g = i / (TG_G * tt), rest = i - g * TG_G * tt, gm = min(TG_G, p.MT - g * TG_G);
  q.mt = g * TG_G + rest % gm;
  q.r0 = s_off[lo] + (rest / gm) * per;
  q.r1 = min(s_off[lo + 1], q.r0 + per);
  q.n = (q.r1 - q.r0 + Q - 1) / Q * Q;
  return q;
}

// activation() with the device's fast exponential and quotient.  Gate and up leave no room for a second accumulator, so
// this stands between two tiles' MMAs (4096 tokens, 8 of 64 experts, D = 2560, H = 1024, R-S+ 540 us with the
// precise ones, 521 so; SiLU 531 / 523).  Its relative error is below 2^-15 for z above -87.3; below that, where 1 + exp(-z)
// passes 2^126, SiLU is 0 instead of something less than 1e-36 from it.  The product with the up value is then rounded to
// bf16 (2^-8).
//
// The product h = A(z) u of a unit whose gate is 0 is exactly 0 whatever its up value, as in the gate-first passes, which
// do not read it; a NaN gate is not below 0 and stays one.  (The activation's own branch and this one in a single
// choice a value: R-S+ 513 -> 479 us, SiLU 509 -> 482.)
__device__ __forceinline__ float gate_up(int act, float z, float u) {
  if (act == 0) return z <= 0.f ? 0.f : z * u;
  const float g = __fdividef(z, 1.f + __expf(-z));
  return (act == ACT_SILU ? g == 0.f : z <= 0.f) ? 0.f : g * u;
}

template <int CTAS, int MODE, bool KN>
__global__ void __launch_bounds__(MODE == TG_I8 ? TG_THREADS_I8 : TG_THREADS, 1)
    gmm_tc_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mW3,
                  const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mXb, const TgArgs p) {
  static_assert(MODE != TG_I8 || CTAS == 1, "the converters arrive on their own block's barriers");
  constexpr bool GATED = MODE == TG_GATED, I8 = MODE == TG_I8, F16 = MODE == TG_I8 || MODE == TG_F16;
  constexpr int EW = I8 ? 4 : 8;  // epilogue warps
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  constexpr uint32_t AB = 128u * 128u;  // one A region: 128 rows x 128 bytes
  const uint32_t NTl = (uint32_t)p.NT / CTAS;
  const uint32_t bb = (NTl + 7) / 8 * 1024u;                 // B region
  // an operand stage; int8: 128 codes of x widened (two 64-wide tiles; the weights' are in TMEM), a raw stage both's
  const uint32_t st_bytes = I8 ? 2 * bb : (GATED ? 2 : 1) * AB + bb, raw_bytes = AB + bb;
  const uint32_t raw0 = (uint32_t)p.S * st_bytes;
  const uint32_t epi0 = raw0 + (I8 ? (uint32_t)p.SR * raw_bytes : 0u);  // the epilogue's scratch, then the barriers
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + epi0 + EW * TG_EPI_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = full + p.S;
  uint64_t* rfull = empty + p.S;
  uint64_t* rempty = rfull + p.SR;
  uint64_t* accf = rempty + p.SR;  // [2]
  uint64_t* acce = accf + 2;       // [2]
  uint64_t* partf = acce + 2;      // K cut: every block's partial tile is in its shared memory,
  uint64_t* partd = partf + 1;     // and every block has read its share of them
  uint32_t* tslot = reinterpret_cast<uint32_t*>(partd + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int* s_off = reinterpret_cast<int*>(tslot + 2);  // [E + 1]
  int* s_pre = s_off + p.g.E + 1;                  // [E + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  const int ks = CTAS == 1 ? p.ks : 1;
  const int kr = ks > 1 ? (int)cluster_rank() : 0;  // this block's share of K: chunks [cb, ce), whole pairs of them
  const int KP = (p.KC + 1) / 2, cb = 2 * (int)((long long)KP * kr / ks);
  const int ce = min(p.KC, 2 * (int)((long long)KP * (kr + 1) / ks));

  if (tid == 0) {
    for (int s = 0; s < p.S; ++s) {
      mbar_init(&full[s], I8 ? TG_CONV_WARPS / TG_CONV_GROUPS : 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < p.SR; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], TG_CONV_WARPS / TG_CONV_GROUPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], EW * CTAS);
    }
    mbar_init(partf, EW * ks);
    mbar_init(partd, EW * ks);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&mW);
    tma_prefetch_map(&mX);
    if (GATED) tma_prefetch_map(&mW3);
  }
  if (warp == 2) tg_alloc<CTAS>(tslot, (uint32_t)p.cols);
  // what needs nothing of the kernel before this one comes before the wait for it
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2 || ks > 1) cluster_sync_all();  // the other blocks' barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tslot;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();  // the offsets, x and the index come from earlier kernels
  if (warp == 3) {  // group bounds and the prefix sum of their tiles
    // bounds that go back or past the end are cut: a group starts where the ones before it ended at the latest
    int carry = 0, last = p.g.offsets ? min(max(p.g.offsets[0], 0), p.g.R) : 0;
    for (int e0 = 0; e0 < p.g.E; e0 += 32) {
      const int e = e0 + lane;
      int hi = 0;  // the end of group e, then the largest end up to it
      if (e < p.g.E) hi = p.g.offsets ? min(max(p.g.offsets[e + 1], 0), p.g.R) : p.g.R;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, hi, o);
        if (lane >= o) hi = max(hi, v);
      }
      hi = max(hi, last);
      int before = __shfl_up_sync(0xffffffffu, hi, 1);
      if (lane == 0) before = last;
      const int v = (hi - before + p.NT - 1) / p.NT * p.MT;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < p.g.E) {
        s_off[e] = before;
        s_pre[e] = carry + x - v;
        if (e == p.g.E - 1) {
          s_off[e + 1] = hi;
          s_pre[e + 1] = carry + x;
        }
      }
      carry += __shfl_sync(0xffffffffu, x, 31);
      last = __shfl_sync(0xffffffffu, hi, 31);
    }
  }
  __syncthreads();
  const int total = s_pre[p.g.E];
  const int first = blockIdx.x / (CTAS * ks), step = gridDim.x / (CTAS * ks);
  const uint32_t smb = smem_u32(sm);
  const int n0r = 128 * (int)rank;  // this block's rows inside a weight tile

  if (warp == 0 || warp == 3) {
    // ---------------------------------------------------------------- TMA producers: warp 0 w, warp 3 x
    const bool xside = warp == 3;
    uint64_t* fb = I8 ? rfull : full;
    uint64_t* eb = I8 ? rempty : empty;
    const int S = I8 ? p.SR : p.S, KW = I8 ? 128 : 64;
    const int kb = I8 ? cb / 2 : cb, ke = I8 ? (ce + 1) / 2 : ce;
    const uint32_t base = I8 ? smb + raw0 : smb, stage = I8 ? raw_bytes : st_bytes;
    uint32_t it = 0, s = 0, par = 1;  // par: parity of the wait for stage s (a fresh barrier passes parity 1)
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Tile q = tile_at<CTAS>(p, s_off, s_pre, t);
      const int nl = q.n / CTAS, nb = q.mt * 128 * CTAS + n0r;
      const int xr = q.r0 + (int)rank * nl;  // this block's rows of x
      const bool big = nl > p.bxr;           // one copy of the whole region, or one small box
      const uint32_t xbytes = p.g.index ? (uint32_t)nl * 128u : (big ? NTl : (uint32_t)p.bxr) * 128u;
      const uint32_t tx = ((GATED ? 2 : 1) * AB + xbytes) * CTAS;
      int gy[2][4];
      if (xside && p.g.index) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = xr + (lane + 32 * h) * 4 + j;
            int src = p.g.XR;  // out of range: zeros
            if (r < q.r1) {
              const int i = p.g.index[r];
              if (i >= 0) src = min(i / p.g.index_div, p.g.XR);
            }
            gy[h][j] = src;
          }
      }
      if (ks > 1 && t != first) {  // the stages held the last tile's partial sums
        if (!__all_sync(0xffffffffu, tg_wait<true>(partd, (uint32_t)((t - first) / step - 1) & 1, abort_flag, p.err))) break;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      for (int c = kb; c < ke; ++c, ++it) {
        if (!__all_sync(0xffffffffu, tg_wait<false>(&eb[s], par, abort_flag, p.err))) {
          ok = false;
          break;
        }
        const uint32_t st = base + s * stage;
        // a pair's stages complete on the first block's barrier
        const uint32_t bar = CTAS == 2 ? cluster_map(smem_u32(&fb[s]), 0) : smem_u32(&fb[s]);
        if (!xside) {
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&fb[s], tx);
            if constexpr (KN) {
              tma_w3d<CTAS>(st, &mW, nb, c * KW, q.e, bar);
              tma_w3d<CTAS>(st + AB / 2, &mW, nb + 64, c * KW, q.e, bar);
            } else {
              tma_w3d<CTAS>(st, &mW, c * KW, nb, q.e, bar);
            }
            if (GATED) tma_w3d<CTAS>(st + AB, &mW3, c * KW, nb, q.e, bar);
          }
        } else {
          const uint32_t bst = st + (GATED ? 2 : 1) * AB;
          if (p.g.index) {
            if (lane < nl / 4) tma_gather4<CTAS>(bst + lane * 512u, &mX, c * KW, gy[0], bar);
            if (lane + 32 < nl / 4) tma_gather4<CTAS>(bst + (lane + 32) * 512u, &mX, c * KW, gy[1], bar);
          } else if (lane == 0) {
            tma_x2d<CTAS>(bst, big ? &mXb : &mX, c * KW, xr, bar);
          }
        }
        if (++s == (uint32_t)S) {
          s = 0;
          par ^= 1;
        }
      }
    }
    // after a failed wait copies may still be in flight: let them land before the block ends
    if (!ok && lane == 0 && rank == 0)
      for (int i = 0; i < S && (uint32_t)i < it; ++i) {
        const uint32_t use = (it - 1 - i) / S;
        mbar_wait_drain(&fb[i], use & 1, TG_TIMEOUT_NS);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (first block of a pair)
    // The warp stays converged; one lane issues a stage's MMAs and their commit together.  Up to 64 columns the issue
    // is what an MMA costs, so the loop holds nothing but 32-bit adds.
    if (rank == 0) {
      const uint32_t st0 = (smb >> 4) & 0x3fffu;  // (in a cluster an address holds the block's rank above its offset)
      uint32_t s = 0, par = 0, tl = 0, st = st0;   // st: the stage's address in 16-byte units
      const uint32_t st16 = st_bytes >> 4, eb = smem_u32(empty);
      const uint32_t hi = (uint32_t)(smem_desc(0, 0, 1024, SMEM_LAYOUT_SW128) >> 32);
      const uint32_t alo0 = (KN ? AB / 2 : 16) >> 4 << 16, blo0 = 1u << 16;  // the leading byte offset
      bool ok = true;
      for (int t = first; t < total && ok; t += step, ++tl) {
        const Tile q = tile_at<CTAS>(p, s_off, s_pre, t);
        const uint32_t idesc = (F16 ? 1u << 4 : (1u << 4) | (1u << 7) | (1u << 10)) | ((KN ? 1u : 0u) << 15) |
                               ((uint32_t)(q.n >> 3) << 17) | ((uint32_t)(128 * CTAS >> 4) << 24);
        const uint32_t b = p.nacc == 2 ? tl & 1 : 0, use = p.nacc == 2 ? tl >> 1 : tl;
        if (use > 0 && !__all_sync(0xffffffffu, tg_wait<CTAS == 2>(&acce[b], (use - 1) & 1, abort_flag, p.err))) break;
        tc_fence_after();
        const uint32_t d = tmem + b * (uint32_t)((GATED ? 2 : 1) * p.NT);
        uint32_t acc = 0;
        for (int c = I8 ? cb / 2 : cb; c < (I8 ? (ce + 1) / 2 : ce); ++c) {
          if (!__all_sync(0xffffffffu, tg_wait<false>(full + s, par, abort_flag, p.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t al = alo0 + st, bl = blo0 + st + ((I8 ? 0 : GATED ? 2 : 1) * AB >> 4);
          if (elect_one()) {
            if constexpr (I8) {
              const uint32_t at = tmem + (uint32_t)p.wcol + 64u * s;  // the stage's weights
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tg_mma_t(d, at + 8 * k, bl + (k >> 2) * (bb >> 4) + 2 * (k & 3), hi, idesc, k == 0 ? acc : 1u);
            }
#pragma unroll
            for (int k = 0; k < (I8 ? 0 : 4); ++k) {
              const uint32_t ak = al + (KN ? (k * 2048) >> 4 : 2 * k);
              tg_mma<CTAS>(d, ak, hi, bl + 2 * k, hi, idesc, k == 0 ? acc : 1u);
              if (GATED) tg_mma<CTAS>(d + p.NT, ak + (AB >> 4), hi, bl + 2 * k, hi, idesc, k == 0 ? acc : 1u);
            }
            tg_commit<CTAS>(eb + 8 * s);
          }
          acc = 1;
          st += st16;
          if (++s == (uint32_t)p.S) {
            s = 0;
            par ^= 1;
            st = st0;
          }
        }
        if (ok && elect_one()) tg_commit<CTAS>(smem_u32(&accf[b]));
      }
    }
    __syncwarp();
  } else if (I8 && warp >= TG_CONV_WARP0) {
    // ---------------------------------------------------------------- int8 -> fp16 operand tiles
    // Two groups of eight warps take every other raw stage of 128 codes each, a warp 64 of them.
    const int cg = (warp - TG_CONV_WARP0) >> 3, half = (warp - TG_CONV_WARP0) >> 2 & 1, cw = warp & 3;
    const int row8 = lane & 7, cj = lane >> 3;
    // Stages and their phases are counted up, never divided for: a division costs as much as the widening.
    const int n = (ce + 1) / 2 - cb / 2;  // raw stages of a tile
    uint32_t s = 0, epar = 1;             // operand stage of the next one; parity of the wait for it (fresh: passes)
    uint32_t rs = 0, rpar = 0;            // its raw stage, parity of its wait
    int skip = cg;                        // raw stages to go on to the group's next one
    bool ok = true;
    auto forward = [&](int by) {
      s += by;
      while (s >= (uint32_t)p.S) {
        s -= p.S;
        epar ^= 1;
      }
      rs += by;
      while (rs >= (uint32_t)p.SR) {
        rs -= p.SR;
        rpar ^= 1;
      }
    };
    for (int t = first; t < total && ok; t += step) {
      const Tile q = tile_at<CTAS>(p, s_off, s_pre, t);
      const int groups = q.n / 8;  // 8-row groups of x
      int c = 0;
      for (;;) {
        if (c + skip >= n) {  // the next one is in a later tile
          forward(n - c);
          skip -= n - c;
          break;
        }
        forward(skip);
        c += skip;
        skip = TG_CONV_GROUPS;
        // A parity wait must not run two phases ahead.  The group's last wait for `empty`, two raw stages ago, showed
        // that stage it - 2 - S was multiplied, so with S >= 2 the phase before this one (it - 2 S) is over; this wait
        // shows that it - S and all before are, so with SR >= S the raw stage's phase before this one is over, too.
        ok = tg_wait<false>(&empty[s], epar, abort_flag, p.err);
        if (ok) ok = tg_wait<false>(&rfull[rs], rpar, abort_flag, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t rw = smb + raw0 + rs * raw_bytes;
        {  // weights: a lane's row, 64 codes, into its TMEM lane
          tc_fence_after();
          const uint32_t src = rw + (uint32_t)(32 * cw + lane) * 128u;
          uint4 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = lds16a(src + ((uint32_t)((half * 4 + j) ^ row8) << 4));
          const uint32_t at = tmem + (uint32_t)p.wcol + 64u * s + 32u * half + ((uint32_t)(32 * cw) << 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              widen4(v[2 * h + j].x, o + 8 * j);
              widen4(v[2 * h + j].y, o + 8 * j + 2);
              widen4(v[2 * h + j].z, o + 8 * j + 4);
              widen4(v[2 * h + j].w, o + 8 * j + 6);
            }
            tmem_st16(at + 16 * h, o);
          }
        }
        const uint32_t src = rw + AB + (uint32_t)row8 * 128u + ((uint32_t)((half * 4 + cj) ^ row8) << 4);
        const uint32_t dst = smb + s * st_bytes + half * bb + (uint32_t)row8 * 128u;
        const uint32_t d0 = dst + ((uint32_t)((2 * cj) ^ row8) << 4), d1 = dst + ((uint32_t)((2 * cj + 1) ^ row8) << 4);
        for (int g0 = cw; g0 < groups; g0 += 16) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (g0 + 4 * i < groups) v[i] = lds16a(src + (uint32_t)(g0 + 4 * i) * 1024u);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (g0 + 4 * i < groups) {
              const uint32_t off = (uint32_t)(g0 + 4 * i) * 1024u;
              uint32_t o[8];
              widen4(v[i].x, o);
              widen4(v[i].y, o + 2);
              widen4(v[i].z, o + 4);
              widen4(v[i].w, o + 6);
              sts16(d0 + off, o[0], o[1], o[2], o[3]);
              sts16(d1 + off, o[4], o[5], o[6], o[7]);
            }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[s]);
          mbar_arrive(&rempty[rs]);
        }
      }
    }
  } else if (warp >= TG_EPI_WARP0 && warp < TG_EPI_WARP0 + EW) {
    // ---------------------------------------------------------------- epilogue: lane = one row of w
    // Warp ew empties TMEM lanes 32 (ew % 4) .., and of the 32-column pieces every EW / 4-th.
    const int ew = warp - TG_EPI_WARP0;
    uint32_t tl = 0;
    for (int t = first; t < total; t += step, ++tl) {
      const Tile q = tile_at<CTAS>(p, s_off, s_pre, t);
      const uint32_t b = p.nacc == 2 ? tl & 1 : 0, use = p.nacc == 2 ? tl >> 1 : tl;
      const int n = q.mt * 128 * CTAS + n0r + 32 * (ew & 3) + lane;
      const bool nok = n < p.g.N;
      if (!__all_sync(0xffffffffu, tg_wait<false>(&accf[b], use & 1, abort_flag, p.err))) break;
      tc_fence_after();
      const uint32_t ta = tmem + b * (uint32_t)((GATED ? 2 : 1) * p.NT) + ((uint32_t)(32 * (ew & 3)) << 16);
      const float sw = F16 && nok ? p.g.sw[(size_t)q.e * p.g.N + n] : 0.f;
      const int rows = q.r1 - q.r0;
      if (CTAS == 1 && ks > 1) {
        // K is cut over the cluster: every block leaves its partial tile, [row of x][128 rows of w], in the stages
        // (their copies and MMAs are done, and the producers wait for `partd`); then each sums its share of the
        // rows over the blocks in their order, so the result does not depend on timing.  Gate and up: two tiles.
        const uint32_t up = (uint32_t)(p.NT * TG_PART) * 4u;
        for (int c0 = 32 * (ew >> 2); c0 < rows; c0 += 32 * (EW / 4)) {
#pragma unroll
          for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            uint32_t v[32];
            tmem_ld32(ta + h * p.NT + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c0 + j < rows) sts4(smb + h * up + (uint32_t)((c0 + j) * TG_PART + 32 * (ew & 3) + lane) * 4u, v[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[b]);
        if (lane < ks) arrive_remote(cluster_map(smem_u32(partf), (uint32_t)lane));
        if (!__all_sync(0xffffffffu, tg_wait<true>(partf, tl & 1, abort_flag, p.err))) break;
        const int t0 = (int)((long long)rows * kr / ks), t1 = (int)((long long)rows * (kr + 1) / ks);
        const int nc = q.mt * 128 + 4 * lane;
        float s4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s4[i] = F16 && nc + i < p.g.N ? p.g.sw[(size_t)q.e * p.g.N + nc + i] : 1.f;
        for (int r = t0 + ew; r < t1; r += EW) {
          const uint32_t at = smb + (uint32_t)(r * TG_PART + 4 * lane) * 4u;
          auto sum_of = [&](uint32_t where, float (&f)[4]) {
            float4 v[8];  // every block's part in flight together, added in their order
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < ks) v[k] = ld_cluster_f4(cluster_map(where, (uint32_t)k));
            f[0] = f[1] = f[2] = f[3] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < ks) {
                f[0] += v[k].x;
                f[1] += v[k].y;
                f[2] += v[k].z;
                f[3] += v[k].w;
              }
          };
          float f[4];
          sum_of(at, f);
          if (GATED) {
            float u[4];
            sum_of(at + up, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = gate_up(p.g.act, f[i], u[i]);
          }
          const int gr = q.r0 + r;
          if (F16) {
            int src = gr;
            if (p.g.index) {
              const int i = p.g.index[gr];
              src = i >= 0 && i / p.g.index_div < p.g.XR ? i / p.g.index_div : -1;
            }
            const float sx = src >= 0 ? p.g.sx[src] : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = f[i] * sx * s4[i];
          }
          const uint64_t o = (uint64_t)(uint32_t)gr * (uint64_t)p.g.ldy + nc;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (nc + i < p.g.N) {
              if (p.g.y_f32)
                reinterpret_cast<float*>(p.g.y)[o + i] = f[i];
              else
                reinterpret_cast<__nv_bfloat16*>(p.g.y)[o + i] = __float2bfloat16_rn(f[i]);
            }
        }
        __syncwarp();
        if (lane < ks) arrive_remote(cluster_map(smem_u32(partd), (uint32_t)lane));
        if (t + step < total && !__all_sync(0xffffffffu, tg_wait<true>(partd, tl & 1, abort_flag, p.err))) break;
        continue;
      }
      for (int c0 = 32 * (ew >> 2); c0 < rows; c0 += 32 * (EW / 4)) {
        uint32_t v[32];
        tmem_ld32(ta + c0, v);
        const int left = min(rows - c0, 32);  // rows of this piece, r0 + c0 on
        const uint64_t y0 = (uint64_t)(uint32_t)(q.r0 + c0) * (uint64_t)p.g.ldy;
        float sx = 0.f;  // lane j: the scale of row j
        if (F16 && lane < left) {
          int src = q.r0 + c0 + lane;
          if (p.g.index) {
            const int i = p.g.index[src];
            src = i >= 0 && i / p.g.index_div < p.g.XR ? i / p.g.index_div : -1;
          }
          sx = src >= 0 ? p.g.sx[src] : 0.f;
        }
        if constexpr (GATED) {
          uint32_t u[32];
          tmem_ld32(ta + p.NT + c0, u);
          tmem_ld_wait();
          if (p.g.act == 0) {  // hoisted: as a branch of each value ReLU pays for the others
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(gate_up(0, __uint_as_float(v[j]), __uint_as_float(u[j])));
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = __float_as_uint(gate_up(p.g.act, __uint_as_float(v[j]), __uint_as_float(u[j])));
          }
        } else {
          tmem_ld_wait();
        }
        if (c0 + 32 * (EW / 4) >= rows) {  // this warp has read its last columns
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CTAS == 2)
              arrive_remote(cluster_map(smem_u32(&acce[b]), 0));
            else
              mbar_arrive(&acce[b]);
          }
        }
        if (p.vec) {
          // through this warp's shared scratch, so that a store carries 16 bytes of a row a lane
          const uint32_t buf = smb + epi0 + (uint32_t)ew * TG_EPI_BYTES;
          const int nc = q.mt * 128 * CTAS + n0r + 32 * (ew & 3);  // the warp's first column of y
          if (p.g.y_f32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16 rows x 32 columns
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float f = __uint_as_float(v[16 * h + j]);
                if (F16) f = f * __shfl_sync(0xffffffffu, sx, 16 * h + j) * sw;
                sts4(buf + (uint32_t)(j * TG_EPI_PITCH + lane) * 4u, __float_as_uint(f));
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = 4 * i + (lane >> 3), c = 4 * (lane & 7);
                const uint4 d = lds16a(buf + (uint32_t)(j * TG_EPI_PITCH + c) * 4u);
                if (16 * h + j < left && nc + c < p.g.NY)
                  *reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.g.y) + y0 +
                                            (uint64_t)(16 * h + j) * (uint64_t)p.g.ldy + nc + c) = d;
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // rows 2 j and 2 j + 1 in one word
              float f0 = __uint_as_float(v[2 * j]), f1 = __uint_as_float(v[2 * j + 1]);
              if (F16) {
                f0 = f0 * __shfl_sync(0xffffffffu, sx, 2 * j) * sw;
                f1 = f1 * __shfl_sync(0xffffffffu, sx, 2 * j + 1) * sw;
              }
              sts4(buf + (uint32_t)(j * TG_EPI_PITCH + lane) * 4u, pack_bf16x2_rn(f0, f1));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int j = 8 * i + (lane >> 2), c = 8 * (lane & 3);
              const uint32_t at = buf + (uint32_t)(j * TG_EPI_PITCH + c) * 4u;
              const uint4 d = lds16a(at), e = lds16a(at + 16);
              __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.g.y) + y0 + (uint64_t)(2 * j) * (uint64_t)p.g.ldy + nc + c;
              if (nc + c < p.g.NY) {
                if (2 * j < left)
                  *reinterpret_cast<uint4*>(y) =
                      make_uint4(__byte_perm(d.x, d.y, 0x5410), __byte_perm(d.z, d.w, 0x5410),
                                 __byte_perm(e.x, e.y, 0x5410), __byte_perm(e.z, e.w, 0x5410));
                if (2 * j + 1 < left)
                  *reinterpret_cast<uint4*>(y + p.g.ldy) =
                      make_uint4(__byte_perm(d.x, d.y, 0x7632), __byte_perm(d.z, d.w, 0x7632),
                                 __byte_perm(e.x, e.y, 0x7632), __byte_perm(e.z, e.w, 0x7632));
              }
            }
            __syncwarp();
          }
        } else {
          const uint32_t size = p.g.y_f32 ? 4 : 2;
          uint8_t* to = reinterpret_cast<uint8_t*>(p.g.y) + (y0 + n) * size;
          const uint64_t pitch = (uint64_t)p.g.ldy * size;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float f = __uint_as_float(v[j]);
            if (F16) f = f * __shfl_sync(0xffffffffu, sx, j) * sw;
            if (nok && j < left) {
              if (p.g.y_f32)
                *reinterpret_cast<float*>(to) = f;
              else
                *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16_rn(f);
            }
            to += pitch;
          }
        }
      }
      if (32 * (ew >> 2) >= rows) {  // no columns for this warp
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CTAS == 2)
            arrive_remote(cluster_map(smem_u32(&acce[b]), 0));
          else
            mbar_arrive(&acce[b]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2 || ks > 1) cluster_sync_all();  // no block leaves while another may still signal its barriers
  tc_fence_after();
  if (warp == 2) tg_dealloc<CTAS>(tmem, (uint32_t)p.cols);
}

// ------------------------------------------------------------------ host side

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, bool i8) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base),
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_w(CUtensorMap* m, const void* w, const GmmArgs& a) {
  const cuuint64_t eb = a.i8 ? 1 : 2, N = (cuuint64_t)a.N, K = (cuuint64_t)a.K;
  const cuuint64_t in = a.kn ? N : K, out = a.kn ? K : N;
  const cuuint64_t dims[3] = {in, out, (cuuint64_t)a.E};
  const cuuint64_t strides[2] = {in * eb, N * K * eb};
  const cuuint32_t box[3] = {a.i8 ? 128u : 64u, a.kn ? 64u : 128u, 1u};
  return encode(m, w, 3, dims, strides, box, a.i8 != 0);
}

template <int CTAS, int MODE, bool KN>
cudaError_t tg_go(const CUtensorMap& mW, const CUtensorMap& mW3, const CUtensorMap& mX, const CUtensorMap& mXb,
                  TgArgs p, size_t smem, int sms, cudaStream_t s) {
  auto kernel = gmm_tc_kernel<CTAS, MODE, KN>;
  constexpr int threads = MODE == TG_I8 ? TG_THREADS_I8 : TG_THREADS;
  struct Setup {
    std::once_flag once;
    cudaError_t attr = cudaSuccess;
    int clusters[9] = {};  // clusters that fit at once, by their blocks (a pair, or the cut of K)
  };
  static Setup setups[TG_DEVICES];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= TG_DEVICES) return cudaErrorInvalidDevice;
  int (&clusters)[9] = setups[dev].clusters;
  cudaError_t& attr = setups[dev].attr;
  std::call_once(setups[dev].once, [&] {
    attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TG_SMEM);
    clusters[1] = sms;
    for (int c = 2; attr == cudaSuccess && c <= (CTAS == 2 ? 2 : 8); ++c) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(sms / c * c));
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = TG_SMEM;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)c;
      at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) clusters[c] = std::min(sms / c, n);
    }
    (void)cudaGetLastError();
  });
  if (attr != cudaSuccess) return attr;
  const GmmArgs& a = p.g;
  const long long most = (long long)p.MT * ((long long)a.R / p.NT + std::min(a.E, a.R));  // tiles at most
  int c = CTAS;
  if (CTAS == 1) {
    // Fewer tiles than half the SMs (as far as sizes tell: groups of equal length): a cluster cuts K, as often as the
    // tiles' clusters fit at once.  A cut costs a tile's exchange, about two microseconds, so a share keeps 4 pairs of
    // chunks at least.
    const int busy = std::min(a.E, a.R);
    const long long tiles = (long long)p.MT * busy * (((a.R + busy - 1) / busy + p.NT - 1) / p.NT);
    for (int k = 2; k <= std::min(8, (p.KC + 1) / 8); ++k)
      if (clusters[k] >= tiles) c = k;
  }
  p.ks = CTAS == 1 ? c : 1;
  if (clusters[c] < 1) return cudaErrorInvalidConfiguration;
  const int n = (int)std::min<long long>(clusters[c], std::max(1ll, most));
  return ops_launch(kernel, dim3((unsigned)(n * c)), threads, smem, s, c, mW, mW3, mX, mXb, p);
}

// shared memory beside the stages: the epilogue warps' scratch, barriers, the groups' tables
constexpr size_t tg_fixed(int epilogue_warps, int E) {
  return epilogue_warps * TG_EPI_BYTES + 1024 + 8 * (2 * 16 + 2 * 16 + 6) + 8 + sizeof(int) * 2 * ((size_t)E + 1) + 64;
}

}  // namespace

cudaError_t launch_gmm_tc(const GmmArgs& a, int ctas, int nt, cudaStream_t s) {
  TgArgs p;
  p.g = a;
  p.NT = nt;
  p.MT = (a.N + 128 * ctas - 1) / (128 * ctas);
  p.KC = (a.K + 63) / 64;
  const bool gated = a.w3 != nullptr;
  cudaError_t e = ops_error_word(&p.err);
  if (e != cudaSuccess) return e;
  const size_t yb = a.y_f32 ? 4 : 2;
  p.g.NY = std::max(a.N, a.NY);
  p.vec = ((uintptr_t)a.y & 15) == 0 && a.ldy * yb % 16 == 0 && p.g.NY * yb % 16 == 0;
  const size_t fixed = tg_fixed(a.i8 ? 4 : 8, a.E);
  const int room = (int)(TG_SMEM - fixed);
  const int ntl = p.NT / ctas, bb = (ntl + 7) / 8 * 1024;
  // int8: three operand stages (two are 10 to 15 % slower) and as many raw ones at least (see the converters' waits);
  // 128 rows a tile leave room for them with the tables of as many experts as there may be
  constexpr int least = 3;
  static_assert(tg_fixed(4, SFFN_MAX_EXPERTS) + least * (2 * 16384 + 16384 + 16384) <= TG_SMEM, "int8 stages");
  const int st = a.i8 ? 2 * bb : (gated ? 2 : 1) * 16384 + bb, raw = a.i8 ? 16384 + bb : 0;
  p.S = a.i8 ? least : std::min(16, room / st);
  p.SR = a.i8 ? std::min(12, (room - p.S * st) / raw) : 0;
  const int wide = (gated ? 2 : 1) * p.NT, wcols = a.i8 ? 64 * p.S : 0;  // TMEM columns: an accumulator, the weights
  p.nacc = 2 * wide + wcols <= 512 ? 2 : 1;
  p.wcol = p.nacc * wide;
  int cols = 32;
  while (cols < p.wcol + wcols) cols <<= 1;
  p.cols = cols;
  p.bxr = std::min(ntl, 32);
  CUtensorMap mW, mW3, mX, mXb;
  if (!encode_w(&mW, a.w, a) || !encode_w(&mW3, gated ? a.w3 : a.w, a)) return cudaErrorInvalidValue;
  {
    const cuuint64_t eb = a.i8 ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)a.XR}, strides[1] = {(cuuint64_t)a.ldx * eb};
    const cuuint32_t box[2] = {a.i8 ? 128u : 64u, a.index ? 1u : (cuuint32_t)p.bxr};
    const cuuint32_t boxb[2] = {a.i8 ? 128u : 64u, a.index ? 1u : (cuuint32_t)ntl};
    if (!encode(&mX, a.x, 2, dims, strides, box, a.i8 != 0) || !encode(&mXb, a.x, 2, dims, strides, boxb, a.i8 != 0))
      return cudaErrorInvalidValue;
  }
  const size_t smem = fixed + (size_t)p.S * st + (size_t)p.SR * raw;
  const int sms = ops_num_sms();
  if (a.i8) return tg_go<1, TG_I8, false>(mW, mW3, mX, mXb, p, smem, sms, s);
  if (a.f16) return tg_go<2, TG_F16, false>(mW, mW3, mX, mXb, p, smem, sms, s);
  if (gated)
    return ctas == 2 ? tg_go<2, TG_GATED, false>(mW, mW3, mX, mXb, p, smem, sms, s)
                     : tg_go<1, TG_GATED, false>(mW, mW3, mX, mXb, p, smem, sms, s);
  if (a.kn)
    return ctas == 2 ? tg_go<2, TG_BF16, true>(mW, mW3, mX, mXb, p, smem, sms, s)
                     : tg_go<1, TG_BF16, true>(mW, mW3, mX, mXb, p, smem, sms, s);
  return ctas == 2 ? tg_go<2, TG_BF16, false>(mW, mW3, mX, mXb, p, smem, sms, s)
                   : tg_go<1, TG_BF16, false>(mW, mW3, mX, mXb, p, smem, sms, s);
}

// fp16 copies of x's and w's codes for the products whose groups are long.
__global__ void __launch_bounds__(256) widen_kernel(const uint8_t* __restrict__ x, long long ldx, int K16,
                                                    long long nx, const uint4* __restrict__ w, long long nw,
                                                    uint4* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < nx + nw; i += (long long)gridDim.x * 256) {
    uint4 v;
    if (i < nx) {
      const long long r = i / K16;
      v = *reinterpret_cast<const uint4*>(x + r * ldx + (i - r * K16) * 16);
    } else {
      v = __ldcs(w + (i - nx));
    }
    uint32_t o[8];
    widen4(v.x, o);
    widen4(v.y, o + 2);
    widen4(v.z, o + 4);
    widen4(v.w, o + 6);
    out[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    out[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// fp16 copies of the codes, made once, against widening in flight: copies let 256 x 256 pair tiles run at full tensor
// rate, so a round of tiles over the SMs, 0.28 us per 64 codes either way, does four times the work on two SMs; they
// cost a launch and an exposed epilogue, 5 us, and three bytes of traffic a code.  (us, in flight / copies, K = 4096:
// 1024 rows, N = 14336 116 / 103; 2048 rows, N = 512 22 / 31, 1024 25 / 34, 2048 42 / 37, 14336 221 / 161; 8192 rows, N =
// 16 25 / 47, 512 45 / 50, 1024 81 / 69; 16 experts of 1000 x 2560: 1024 rows each 106 / 111, 1536 145 / 145.)
// Below TG_WIDE_ROWS an expert they never pay (768 rows, N = 14336: 97 / 103), and no workspace is asked for.
constexpr int TG_WIDE_ROWS = 832;

bool wide(int R, int E, int i8) { return i8 && R / E >= TG_WIDE_ROWS; }

bool copies_pay(const GmmArgs& a) {
  const long long rows = a.R / a.E, sms = ops_num_sms();
  const long long small = (long long)a.E * ((a.N + 127) / 128) * ((rows + 127) / 128);
  const long long pairs = (long long)a.E * ((a.N + 255) / 256) * ((rows + 255) / 256);
  const long long rounds = (small + sms - 1) / sms - (2 * pairs + sms - 1) / sms;
  const long long codes = ((long long)a.XR + (long long)a.E * a.N) * a.K;
  return rounds * ((a.K + 63) / 64) * 280 > 5000 + codes / 2000;  // ns
}

size_t gmm_workspace(int R, int XR, int N, int K, int E, int i8) {
  return wide(R, E, i8) ? 2 * ((size_t)XR * K + (size_t)E * N * K) : 0;
}

cudaError_t launch_gmm(const GmmArgs& a, cudaStream_t s) {
  const int busy = std::min(a.E, a.R);
  if (wide(a.R, a.E, a.i8) && a.workspace && copies_pay(a)) {
    const long long nx = (long long)a.XR * (a.K / 16), nw = (long long)a.E * a.N * (a.K / 16);
    const int grid = (int)std::min<long long>((nx + nw + 255) / 256, 8ll * ops_num_sms());
    const cudaError_t e = ops_launch(widen_kernel, dim3((unsigned)grid), 256, 0, s, 1, (const uint8_t*)a.x, a.ldx,
                                     a.K / 16, nx, (const uint4*)a.w, nw, (uint4*)a.workspace);
    if (e != cudaSuccess) return e;
    GmmArgs b = a;
    b.x = a.workspace;
    b.w = static_cast<uint16_t*>(a.workspace) + 16 * nx;
    b.ldx = a.K;
    b.i8 = 0;
    b.f16 = 1;
    return launch_gmm_tc(b, 2, 256, s);
  }
  if (a.i8) return a.R <= std::max(a.E, 4) ? launch_gmm_rows(a, s) : launch_gmm_tc(a, 1, 128, s);
  // A pair's 256 x 256 tiles from 96 rows a group on, where they fill the SMs (us, 128 x 128 / pair tiles; 64 experts, N =
  // 1024, K = 2560: 64 rows each 63 / 65, 96 72 / 68, 256 102 / 83; one, N = K = 4096: 256 rows 17 / 24, 512 19 / 24)
  // and N fills more than one of the pair's blocks (16384 rows, 16 experts, N = 100, K = 2560: 21 / 25).
  const long long pairs = (long long)((a.N + 255) / 256) * busy * (((a.R + busy - 1) / busy + 255) / 256);
  const bool fill = 2 * pairs >= ops_num_sms();
  // Gate and up together: 256 rows a tile take all of TMEM, so their epilogue is not hidden, and still win from 128
  // rows a group on (4096 tokens, 8 of 64 experts, D = 2560, H = 1024: 561 against 643 us; 512 tokens 225 / 211).
  if (a.w3) return a.R >= 128 * busy && fill && a.N > 128 ? launch_gmm_tc(a, 2, 256, s) : launch_gmm_tc(a, 1, 128, s);
  return a.R >= 96 * busy && fill && a.N > 128 ? launch_gmm_tc(a, 2, 256, s) : launch_gmm_tc(a, 1, 128, s);
}

}  // namespace sffn

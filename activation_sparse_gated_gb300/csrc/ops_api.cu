// ops_api.cu -- the handle-free entry points of include/sffn.h: the router,
// per-token int8 codes, the int8 product, the products grouped by expert, the
// gated experts' forward, 4-bit weights and their products, and the gated block
// with its backward pass.  Argument checks come before any CUDA call.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "ops.h"
#include "sffn.h"

using namespace sffn;

namespace {

__device__ int g_ops_error = 0;  // DEV_ERR_TIMEOUT, once a wait of an operator's kernel on this device ran out

int fail(int code, const char* fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return code;
}

int cuda_fail(const char* what, cudaError_t e) {
  return fail(e == cudaErrorMemoryAllocation ? SFFN_ERR_NOMEM : SFFN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool misaligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

bool overlap(const void* a, unsigned long long na, const void* b, unsigned long long nb) {
  const unsigned long long pa = (uintptr_t)a, pb = (uintptr_t)b;
  return a && b && pa < pb + nb && pb < pa + na;
}

}  // namespace

cudaError_t sffn::ops_error_word(int** p) {
  static int* at[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!at[dev]) {
    void* q = nullptr;
    if ((e = cudaGetSymbolAddress(&q, g_ops_error)) != cudaSuccess) return e;
    at[dev] = static_cast<int*>(q);
  }
  *p = at[dev];
  return cudaSuccess;
}

int sffn::ops_num_sms() {
  static std::atomic<int> at[64];  // by device: threads may ask at once, and devices differ
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  int n = at[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    at[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

extern "C" {

size_t sffn_route_workspace(int T, int E, int k) {
  if (T < 1 || E < 1 || E > SFFN_MAX_EXPERTS || k < 1 || k > SFFN_MAX_CHOICES) return 0;
  return route_workspace(T, E, k);
}

int sffn_route(const void* logits, long long ld, float* weights, int* ids, int* offsets, int* rows, int T, int E,
               int k, int dtype, int flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != SFFN_F32 && dtype != SFFN_BF16) return fail(SFFN_ERR_DTYPE, "sffn_route: logits are f32 or bf16");
  if (flags & ~(SFFN_ROUTE_SIGMOID | SFFN_ROUTE_NORMALIZE))
    return fail(SFFN_ERR_ARG, "sffn_route: flags 0x%x has unknown bits", flags);
  if (E < 1 || E > SFFN_MAX_EXPERTS) return fail(SFFN_ERR_ARG, "sffn_route: E=%d outside 1..%d", E, SFFN_MAX_EXPERTS);
  if (k < 1 || k > SFFN_MAX_CHOICES || k > E)
    return fail(SFFN_ERR_ARG, "sffn_route: k=%d outside 1..min(%d, E)", k, SFFN_MAX_CHOICES);
  if (T < 0 || (long long)T * k > SFFN_MAX_ROWS)
    return fail(SFFN_ERR_ARG, "sffn_route: T=%d, k=%d: more than %d choices", T, k, SFFN_MAX_ROWS);
  if (ld < E) return fail(SFFN_ERR_ARG, "sffn_route: the logits' row pitch %lld is below E=%d", ld, E);
  if (!offsets || (T > 0 && (!logits || !weights || !ids || !rows)))
    return fail(SFFN_ERR_ARG, "sffn_route: null pointer");
  if (misaligned(logits, dtype == SFFN_F32 ? 4 : 2) || misaligned(weights, 4) || misaligned(ids, 4) ||
      misaligned(offsets, 4) || misaligned(rows, 4))
    return fail(SFFN_ERR_ALIGN, "sffn_route: a pointer is not aligned to its element");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(offsets, 0, sizeof(int) * (E + 1), s);
    return e == cudaSuccess ? SFFN_OK : cuda_fail("cudaMemsetAsync", e);
  }
  const unsigned long long nz = ((unsigned long long)(T - 1) * ld + E) * (dtype == SFFN_F32 ? 4 : 2), nc = 4ull * T * k;
  if (overlap(logits, nz, weights, nc) || overlap(logits, nz, ids, nc) || overlap(logits, nz, rows, nc) ||
      overlap(logits, nz, offsets, 4ull * (E + 1)))
    return fail(SFFN_ERR_ARG, "sffn_route: an output overlaps the logits");
  const size_t need = route_workspace(T, E, k);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(SFFN_ERR_ARG, "sffn_route: workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0,
                need);
  if (need > 0 && misaligned(workspace, 16)) return fail(SFFN_ERR_ALIGN, "sffn_route: workspace is not 16-byte aligned");
  RouteArgs a;
  a.logits = logits;
  a.ld = ld;
  a.weights = weights;
  a.ids = ids;
  a.offsets = offsets;
  a.rows = rows;
  a.hist = static_cast<int*>(workspace);
  a.T = T;
  a.E = E;
  a.k = k;
  a.bf16 = dtype == SFFN_BF16;
  a.sigmoid = (flags & SFFN_ROUTE_SIGMOID) != 0;
  a.normalize = (flags & SFFN_ROUTE_NORMALIZE) != 0;
  a.vec = !misaligned(logits, 16) && ld * (a.bf16 ? 2 : 4) % 16 == 0;
  const cudaError_t e = launch_route(a, s);
  return e == cudaSuccess ? SFFN_OK : cuda_fail("sffn_route", e);
}

int sffn_quantize_tokens(const void* x, long long ldx, int8_t* q, float* scales, int T, int K, void* stream) {
  if (T < 0 || K < 1) return fail(SFFN_ERR_ARG, "sffn_quantize_tokens: T=%d, K=%d", T, K);
  if (ldx < K) return fail(SFFN_ERR_ARG, "sffn_quantize_tokens: the row pitch %lld is below K=%d", ldx, K);
  if (T == 0) return SFFN_OK;
  if (!x || !q || !scales) return fail(SFFN_ERR_ARG, "sffn_quantize_tokens: null pointer");
  if (misaligned(x, 2) || misaligned(scales, 4))
    return fail(SFFN_ERR_ALIGN, "sffn_quantize_tokens: a pointer is not aligned to its element");
  const unsigned long long nx = ((unsigned long long)(T - 1) * ldx + K) * 2;
  if (overlap(x, nx, q, (unsigned long long)T * K) || overlap(x, nx, scales, 4ull * T))
    return fail(SFFN_ERR_ARG, "sffn_quantize_tokens: an output overlaps x");
  const cudaError_t e = launch_quantize_tokens(x, ldx, q, scales, T, K, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail("sffn_quantize_tokens", e);
}

int sffn_grouped_matmul(const void* x, long long ldx, const float* sx, const void* w, const float* sw,
                        const int* offsets, const int* index, int index_div, void* y, long long ldy, int R, int XR,
                        int N, int K, int E, int dtype, int y_dtype, int flags, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const char* fn = "sffn_grouped_matmul";
  if (dtype != SFFN_BF16 && dtype != SFFN_I8) return fail(SFFN_ERR_DTYPE, "%s: operands are bf16 or int8 codes", fn);
  if (y_dtype != SFFN_BF16 && y_dtype != SFFN_F32) return fail(SFFN_ERR_DTYPE, "%s: y is bf16 or f32", fn);
  if (flags & ~SFFN_W_KN) return fail(SFFN_ERR_ARG, "%s: flags 0x%x has unknown bits", fn, flags);
  const bool i8 = dtype == SFFN_I8, kn = (flags & SFFN_W_KN) != 0;
  if (i8 && kn) return fail(SFFN_ERR_DTYPE, "%s: int8 weights are [E, N, K]", fn);
  if (R < 0 || R > SFFN_MAX_ROWS || XR < 0 || N < 1 || N > SFFN_MAX_ROWS || K < 1 || E < 1 || E > SFFN_MAX_EXPERTS)
    return fail(SFFN_ERR_ARG, "%s: R=%d, XR=%d, N=%d, K=%d, E=%d (1..%d experts)", fn, R, XR, N, K, E, SFFN_MAX_EXPERTS);
  const int per = i8 ? 16 : 8;
  if (K % per != 0) return fail(SFFN_ERR_ARG, "%s: K=%d must be a multiple of %d", fn, K, per);
  if (K > SFFN_MAX_SUM) return fail(SFFN_ERR_ARG, "%s: K=%d above %d", fn, K, SFFN_MAX_SUM);
  if (kn && N % 8 != 0) return fail(SFFN_ERR_ARG, "%s: N=%d must be a multiple of 8 for [E, K, N] weights", fn, N);
  if (ldx < K || ldx % per != 0)
    return fail(SFFN_ERR_ARG, "%s: x's row pitch %lld must be a multiple of %d and at least K=%d", fn, ldx, per, K);
  if (ldy < N) return fail(SFFN_ERR_ARG, "%s: y's row pitch %lld is below N=%d", fn, ldy, N);
  if (index && index_div < 1) return fail(SFFN_ERR_ARG, "%s: index_div=%d must be at least 1", fn, index_div);
  if (R == 0) return SFFN_OK;
  if (XR < (index ? 1 : R)) return fail(SFFN_ERR_ARG, "%s: x has %d rows, %d needed", fn, XR, index ? 1 : R);
  if (!x || !w || !y || (E > 1 && !offsets)) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (i8 && (!sx || !sw)) return fail(SFFN_ERR_ARG, "%s: int8 operands need sx and sw", fn);
  if (misaligned(x, 16) || misaligned(w, 16)) return fail(SFFN_ERR_ALIGN, "%s: x and w must be 16-byte aligned", fn);
  if (misaligned(y, y_dtype == SFFN_F32 ? 4 : 2) || misaligned(offsets, 4) || misaligned(index, 4) ||
      (i8 && (misaligned(sx, 4) || misaligned(sw, 4))))
    return fail(SFFN_ERR_ALIGN, "%s: a pointer is not aligned to its element", fn);
  const size_t need = gmm_workspace(R, XR, N, K, E, i8);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(SFFN_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace ? workspace_bytes : (size_t)0, need);
  if (need > 0 && misaligned(workspace, 16)) return fail(SFFN_ERR_ALIGN, "%s: workspace is not 16-byte aligned", fn);
  const unsigned long long eb = i8 ? 1 : 2, yb = y_dtype == SFFN_F32 ? 4 : 2;
  const unsigned long long ny = ((unsigned long long)(R - 1) * ldy + N) * yb;
  if (overlap(x, ((unsigned long long)(XR - 1) * ldx + K) * eb, y, ny) ||
      overlap(w, (unsigned long long)E * N * K * eb, y, ny) || (need > 0 && overlap(workspace, need, y, ny)) ||
      overlap(offsets, 4ull * (E + 1), y, ny) || overlap(index, 4ull * R, y, ny) ||
      (i8 && (overlap(sx, 4ull * XR, y, ny) || overlap(sw, 4ull * E * N, y, ny))))
    return fail(SFFN_ERR_ARG, "%s: y overlaps an operand or the workspace", fn);
  GmmArgs a;
  a.workspace = need > 0 ? workspace : nullptr;
  a.x = x;
  a.w = w;
  a.sx = i8 ? sx : nullptr;
  a.sw = i8 ? sw : nullptr;
  a.offsets = offsets;
  a.index = index;
  a.index_div = index ? index_div : 1;
  a.y = y;
  a.ldx = ldx;
  a.ldy = ldy;
  a.R = R;
  a.XR = XR;
  a.N = N;
  a.K = K;
  a.E = E;
  a.i8 = i8;
  a.y_f32 = y_dtype == SFFN_F32;
  a.kn = kn;
  const cudaError_t e = launch_gmm(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

size_t sffn_grouped_workspace(int R, int XR, int N, int K, int E, int dtype) {
  if (R < 1 || XR < 1 || N < 1 || K < 1 || E < 1) return 0;
  return gmm_workspace(R, XR, N, K, E, dtype == SFFN_I8);
}

int sffn_matmul_int8(const int8_t* xq, long long ldx, const float* sx, const int8_t* wq, const float* sw, void* y,
                     long long ldy, int T, int N, int K, int y_dtype, void* workspace, size_t workspace_bytes,
                     void* stream) {
  return sffn_grouped_matmul(xq, ldx, sx, wq, sw, nullptr, nullptr, 1, y, ldy, T, T, N, K, 1, SFFN_I8, y_dtype, 0,
                             workspace, workspace_bytes, stream);
}

size_t sffn_experts_workspace(int T, int k, int D, int H) {
  if (T < 1 || k < 1 || k > SFFN_MAX_CHOICES || D < 1 || H < 1) return 0;
  return experts_workspace(T, k, D, H);
}

int sffn_experts_forward(const void* x, long long ldx, const float* weights, const int* ids, const int* offsets,
                         const int* rows, const void* W1, const void* W3, const void* W2t, void* y, int T, int E, int k,
                         int D, int H, int act, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "sffn_experts_forward";
  if (act != SFFN_ACT_RELU && act != SFFN_ACT_RSP && act != SFFN_ACT_SILU)
    return fail(SFFN_ERR_ARG, "%s: act %d unknown", fn, act);
  if (T < 0 || H < 1 || E < 1 || E > SFFN_MAX_EXPERTS || k < 1 || k > SFFN_MAX_CHOICES || k > E)
    return fail(SFFN_ERR_ARG, "%s: T=%d, E=%d, k=%d, H=%d", fn, T, E, k, H);
  if (D < 8 || D % 8 != 0 || D > SFFN_MAX_SUM || H > SFFN_MAX_SUM)
    return fail(SFFN_ERR_ARG, "%s: D=%d must be a multiple of 8, D and H at most %d", fn, D, SFFN_MAX_SUM);
  if ((long long)T * k > SFFN_MAX_ROWS)
    return fail(SFFN_ERR_ARG, "%s: T=%d, k=%d: more than %d choices", fn, T, k, SFFN_MAX_ROWS);
  if (ldx < D || ldx % 8 != 0)
    return fail(SFFN_ERR_ARG, "%s: x's row pitch %lld must be a multiple of 8 and at least D=%d", fn, ldx, D);
  if (T == 0) return SFFN_OK;
  if (!x || !weights || !ids || !offsets || !rows || !W1 || !W3 || !W2t || !y)
    return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(x, 16) || misaligned(W1, 16) || misaligned(W3, 16) || misaligned(W2t, 16) || misaligned(y, 16))
    return fail(SFFN_ERR_ALIGN, "%s: x, W1, W3, W2t and y must be 16-byte aligned", fn);
  if (misaligned(weights, 4) || misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(rows, 4))
    return fail(SFFN_ERR_ALIGN, "%s: a pointer is not aligned to its element", fn);
  const size_t need = experts_workspace(T, k, D, H);
  if (!workspace || workspace_bytes < need)
    return fail(SFFN_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace ? workspace_bytes : (size_t)0, need);
  if (misaligned(workspace, 16)) return fail(SFFN_ERR_ALIGN, "%s: workspace is not 16-byte aligned", fn);
  const unsigned long long ny = 2ull * T * D, nw = 2ull * E * H * D, nc = 4ull * T * k;
  if (overlap(x, 2ull * ((unsigned long long)(T - 1) * ldx + D), y, ny) || overlap(W1, nw, y, ny) ||
      overlap(W3, nw, y, ny) || overlap(W2t, nw, y, ny) || overlap(workspace, need, y, ny) ||
      overlap(weights, nc, y, ny) || overlap(ids, nc, y, ny) || overlap(rows, nc, y, ny) ||
      overlap(offsets, 4ull * (E + 1), y, ny))
    return fail(SFFN_ERR_ARG, "%s: y overlaps an operand or the workspace", fn);
  ExpertsArgs a;
  a.x = x;
  a.ldx = ldx;
  a.weights = weights;
  a.ids = ids;
  a.offsets = offsets;
  a.rows = rows;
  a.W1 = W1;
  a.W3 = W3;
  a.W2t = W2t;
  a.y = y;
  a.workspace = workspace;
  a.T = T;
  a.E = E;
  a.k = k;
  a.D = D;
  a.H = H;
  a.act = act;
  const cudaError_t e = launch_experts(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

// The checks that the 4-bit entry points share; G: scales a row.
static int check_int4(const char* fn, long long N, int K, int group, int* G) {
  if (N < 1 || N > SFFN_MAX_ROWS) return fail(SFFN_ERR_ARG, "%s: %lld rows of weights, 1..%d are taken", fn, N, SFFN_MAX_ROWS);
  if (K < 16 || K % 16 != 0 || K > SFFN_MAX_SUM)
    return fail(SFFN_ERR_ARG, "%s: %d columns of weights: a multiple of 16, at most %d, is taken", fn, K, SFFN_MAX_SUM);
  if (group < 0 || group % 64 != 0)
    return fail(SFFN_ERR_ARG, "%s: group=%d must be a multiple of 64, or 0 for one scale a row", fn, group);
  *G = group > 0 && group < K ? (K - 1) / group + 1 : 1;
  return SFFN_OK;
}

int sffn_quantize_int4(const void* w, long long ldw, uint8_t* codes, float* scales, int N, int K, int group, void* stream) {
  const char* fn = "sffn_quantize_int4";
  if (N < 0) return fail(SFFN_ERR_ARG, "%s: N=%d", fn, N);
  int G = 0;
  const int rc = check_int4(fn, N < 1 ? 1 : N, K, group, &G);
  if (rc != SFFN_OK) return rc;
  if (ldw < K || ldw % 8 != 0)
    return fail(SFFN_ERR_ARG, "%s: w's row pitch %lld must be a multiple of 8 and at least K=%d", fn, ldw, K);
  if (N == 0) return SFFN_OK;
  if (!w || !codes || !scales) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(w, 16) || misaligned(codes, 16)) return fail(SFFN_ERR_ALIGN, "%s: w and codes must be 16-byte aligned", fn);
  if (misaligned(scales, 4)) return fail(SFFN_ERR_ALIGN, "%s: scales are not aligned to their element", fn);
  const unsigned long long nw = ((unsigned long long)(N - 1) * ldw + K) * 2, nq = (unsigned long long)N * K / 2, ns = 4ull * N * G;
  if (overlap(w, nw, codes, nq) || overlap(w, nw, scales, ns) || overlap(codes, nq, scales, ns))
    return fail(SFFN_ERR_ARG, "%s: an output overlaps w or the other one", fn);
  const cudaError_t e = launch_quantize_int4(w, ldw, codes, scales, N, K, group, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

int sffn_dequantize_int4(const uint8_t* codes, const float* scales, void* y, long long ldy, int N, int K, int group,
                         int y_dtype, void* stream) {
  const char* fn = "sffn_dequantize_int4";
  if (y_dtype != SFFN_BF16 && y_dtype != SFFN_F32) return fail(SFFN_ERR_DTYPE, "%s: y is bf16 or f32", fn);
  if (N < 0) return fail(SFFN_ERR_ARG, "%s: N=%d", fn, N);
  int G = 0;
  const int rc = check_int4(fn, N < 1 ? 1 : N, K, group, &G);
  if (rc != SFFN_OK) return rc;
  if (ldy < K || ldy % 8 != 0)
    return fail(SFFN_ERR_ARG, "%s: y's row pitch %lld must be a multiple of 8 and at least K=%d", fn, ldy, K);
  if (N == 0) return SFFN_OK;
  if (!y || !codes || !scales) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(y, 16) || misaligned(codes, 16)) return fail(SFFN_ERR_ALIGN, "%s: codes and y must be 16-byte aligned", fn);
  if (misaligned(scales, 4)) return fail(SFFN_ERR_ALIGN, "%s: scales are not aligned to their element", fn);
  const unsigned long long ny = ((unsigned long long)(N - 1) * ldy + K) * (y_dtype == SFFN_F32 ? 4 : 2);
  if (overlap(y, ny, codes, (unsigned long long)N * K / 2) || overlap(y, ny, scales, 4ull * N * G))
    return fail(SFFN_ERR_ARG, "%s: y overlaps codes or scales", fn);
  const cudaError_t e = launch_dequantize_int4(codes, scales, y, ldy, N, K, group, y_dtype == SFFN_F32,
                                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

size_t sffn_int4_workspace(int T, int N, int K, int y_dtype, int gated) {
  if (T < 1 || N < 1 || K < 1) return 0;
  return int4_workspace(T, N, K, y_dtype == SFFN_F32 || gated, gated != 0);
}

// Both products by 4-bit weights; w3 and s3 null: the plain one.
static int run_int4(const char* fn, const void* x, long long ldx, const uint8_t* w, const float* sw, const uint8_t* w3,
                    const float* s3, bool gated, void* y, long long ldy, int T, int N, int K, int group, int y_dtype,
                    int act, void* workspace, size_t workspace_bytes, void* stream) {
  int G = 0;
  const int rc = check_int4(fn, N, K, group, &G);
  if (rc != SFFN_OK) return rc;
  if (T < 0 || T > SFFN_MAX_ROWS) return fail(SFFN_ERR_ARG, "%s: T=%d outside 0..%d", fn, T, SFFN_MAX_ROWS);
  if (ldx < K || ldx % 8 != 0)
    return fail(SFFN_ERR_ARG, "%s: x's row pitch %lld must be a multiple of 8 and at least %d", fn, ldx, K);
  if (ldy < N) return fail(SFFN_ERR_ARG, "%s: the result's row pitch %lld is below %d", fn, ldy, N);
  if (T == 0) return SFFN_OK;
  if (!x || !w || !sw || !y || (gated && (!w3 || !s3))) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(w3, 16))
    return fail(SFFN_ERR_ALIGN, "%s: x and the codes must be 16-byte aligned", fn);
  if (misaligned(y, y_dtype == SFFN_F32 ? 4 : 2) || misaligned(sw, 4) || misaligned(s3, 4))
    return fail(SFFN_ERR_ALIGN, "%s: a pointer is not aligned to its element", fn);
  const size_t need = int4_workspace(T, N, K, y_dtype == SFFN_F32 || gated, gated);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(SFFN_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace ? workspace_bytes : (size_t)0, need);
  if (need > 0 && misaligned(workspace, 16)) return fail(SFFN_ERR_ALIGN, "%s: workspace is not 16-byte aligned", fn);
  const unsigned long long ny = ((unsigned long long)(T - 1) * ldy + N) * (y_dtype == SFFN_F32 ? 4 : 2);
  const unsigned long long nx = ((unsigned long long)(T - 1) * ldx + K) * 2, nw = (unsigned long long)N * K / 2, ns = 4ull * N * G;
  if (overlap(x, nx, y, ny) || overlap(w, nw, y, ny) || overlap(sw, ns, y, ny) || (gated && (overlap(w3, nw, y, ny) || overlap(s3, ns, y, ny))) ||
      (need > 0 && overlap(workspace, need, y, ny)))
    return fail(SFFN_ERR_ARG, "%s: the result overlaps an operand or the workspace", fn);
  if (need > 0 && (overlap(workspace, need, x, nx) || overlap(workspace, need, w, nw) || overlap(workspace, need, sw, ns) ||
                   (gated && (overlap(workspace, need, w3, nw) || overlap(workspace, need, s3, ns)))))
    return fail(SFFN_ERR_ARG, "%s: the workspace overlaps an operand", fn);
  Int4Args a;
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.w3 = gated ? w3 : nullptr;
  a.sw = sw;
  a.s3 = gated ? s3 : nullptr;
  a.y = y;
  a.ldy = ldy;
  a.T = T;
  a.N = N;
  a.K = K;
  a.group = group;
  a.y_f32 = y_dtype == SFFN_F32;
  a.act = act;
  a.workspace = workspace;
  const cudaError_t e = launch_matmul_int4(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

int sffn_matmul_int4(const void* x, long long ldx, const uint8_t* wq, const float* sw, void* y, long long ldy, int T, int N,
                     int K, int group, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (y_dtype != SFFN_BF16 && y_dtype != SFFN_F32) return fail(SFFN_ERR_DTYPE, "sffn_matmul_int4: y is bf16 or f32");
  return run_int4("sffn_matmul_int4", x, ldx, wq, sw, nullptr, nullptr, false, y, ldy, T, N, K, group, y_dtype, 0, workspace,
                  workspace_bytes, stream);
}

int sffn_gated_up_int4(const void* x, long long ldx, const uint8_t* w1, const float* s1, const uint8_t* w3, const float* s3,
                       void* h, long long ldh, int T, int D, int H, int group, int act, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (act != SFFN_ACT_RELU && act != SFFN_ACT_RSP && act != SFFN_ACT_SILU)
    return fail(SFFN_ERR_ARG, "sffn_gated_up_int4: act %d unknown", act);
  return run_int4("sffn_gated_up_int4", x, ldx, w1, s1, w3, s3, true, h, ldh, T, H, D, group, SFFN_BF16, act, workspace,
                  workspace_bytes, stream);
}

// The checks that the gated block's two passes share.
static int check_gated(const char* fn, const void* x, long long ldx, const void* W1, const void* W3, int T, int D, int H,
                       int act) {
  if (act != SFFN_ACT_RELU && act != SFFN_ACT_RSP && act != SFFN_ACT_SILU)
    return fail(SFFN_ERR_ARG, "%s: act %d unknown", fn, act);
  if (D < 8 || D % 8 != 0 || D > SFFN_MAX_SUM || H < 1 || H > SFFN_MAX_SUM)
    return fail(SFFN_ERR_ARG, "%s: D=%d must be a multiple of 8, D and H=%d at most %d", fn, D, H, SFFN_MAX_SUM);
  if (T < 0 || T > SFFN_MAX_ROWS) return fail(SFFN_ERR_ARG, "%s: T=%d outside 0..%d", fn, T, SFFN_MAX_ROWS);
  if (ldx < D || ldx % 8 != 0)
    return fail(SFFN_ERR_ARG, "%s: x's row pitch %lld must be a multiple of 8 and at least D=%d", fn, ldx, D);
  if (T > 0 && (!x || !W1 || !W3)) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(x, 16) || misaligned(W1, 16) || misaligned(W3, 16))
    return fail(SFFN_ERR_ALIGN, "%s: x, W1 and W3 must be 16-byte aligned", fn);
  return SFFN_OK;
}

int sffn_gated_up(const void* x, long long ldx, const void* W1, const void* W3, void* h, long long ldh, float* z, float* u,
                  long long ldz, int T, int D, int H, int act, void* stream) {
  const char* fn = "sffn_gated_up";
  const int rc = check_gated(fn, x, ldx, W1, W3, T, D, H, act);
  if (rc != SFFN_OK) return rc;
  if (ldh < H) return fail(SFFN_ERR_ARG, "%s: h's row pitch %lld is below H=%d", fn, ldh, H);
  if (!z != !u) return fail(SFFN_ERR_ARG, "%s: z and u go together", fn);
  if (z && (ldz < H || ldz > SFFN_MAX_ROWS))
    return fail(SFFN_ERR_ARG, "%s: z's and u's row pitch %lld is outside H=%d..%d", fn, ldz, H, SFFN_MAX_ROWS);
  if (T == 0) return SFFN_OK;
  if (!h) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(h, 2) || misaligned(z, 4) || misaligned(u, 4))
    return fail(SFFN_ERR_ALIGN, "%s: a pointer is not aligned to its element", fn);
  const unsigned long long nx = ((unsigned long long)(T - 1) * ldx + D) * 2, nw = 2ull * H * D;
  const unsigned long long nh = ((unsigned long long)(T - 1) * ldh + H) * 2, nz = z ? ((unsigned long long)(T - 1) * ldz + H) * 4 : 0;
  const void* out[3] = {h, z, u};
  const unsigned long long size[3] = {nh, nz, nz};
  for (int i = 0; i < 3; ++i)
    if (overlap(out[i], size[i], x, nx) || overlap(out[i], size[i], W1, nw) || overlap(out[i], size[i], W3, nw) ||
        overlap(out[i], size[i], out[(i + 1) % 3], size[(i + 1) % 3]))
      return fail(SFFN_ERR_ARG, "%s: an output overlaps an operand or another output", fn);
  GatedArgs a;
  a.x = x;
  a.ldx = ldx;
  a.W1 = W1;
  a.W3 = W3;
  a.h = h;
  a.ldh = ldh;
  a.z = z;
  a.u = u;
  a.ldz = z ? ldz : 0;
  a.T = T;
  a.D = D;
  a.H = H;
  a.act = act;
  const cudaError_t e = launch_gated_up(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

size_t sffn_gated_up_backward_workspace(int T, int H) { return T < 1 || H < 1 ? 0 : gated_grad_workspace(T, H); }

int sffn_gated_up_backward(const void* dh, long long lddh, const float* z, const float* u, long long ldz, const void* x,
                           long long ldx, const void* W1, const void* W3, void* dx, void* dW1, void* dW3, int T, int D,
                           int H, int act, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "sffn_gated_up_backward";
  const int rc = check_gated(fn, x, ldx, W1, W3, T, D, H, act);
  if (rc != SFFN_OK) return rc;
  if (lddh < H || ldz < H) return fail(SFFN_ERR_ARG, "%s: a row pitch (dh %lld, z and u %lld) is below H=%d", fn, lddh, ldz, H);
  if (misaligned(dx, 16) || misaligned(dW1, 16) || misaligned(dW3, 16))
    return fail(SFFN_ERR_ALIGN, "%s: dx, dW1 and dW3 must be 16-byte aligned", fn);
  const unsigned long long nw = 2ull * H * D;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (overlap(dW1, nw, dW3, nw)) return fail(SFFN_ERR_ARG, "%s: dW1 and dW3 overlap", fn);
  if (T == 0) {  // a sum over no tokens
    for (void* p : {dW1, dW3})
      if (p) {
        const cudaError_t e = cudaMemsetAsync(p, 0, nw, s);
        if (e != cudaSuccess) return cuda_fail("cudaMemsetAsync", e);
      }
    return SFFN_OK;
  }
  if (!dh || !z || !u) return fail(SFFN_ERR_ARG, "%s: null pointer", fn);
  if (misaligned(dh, 2) || misaligned(z, 4) || misaligned(u, 4))
    return fail(SFFN_ERR_ALIGN, "%s: a pointer is not aligned to its element", fn);
  const size_t need = gated_grad_workspace(T, H);
  if (!workspace || workspace_bytes < need)
    return fail(SFFN_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace ? workspace_bytes : (size_t)0, need);
  if (misaligned(workspace, 16)) return fail(SFFN_ERR_ALIGN, "%s: workspace is not 16-byte aligned", fn);
  const unsigned long long nx = ((unsigned long long)(T - 1) * ldx + D) * 2, ndh = ((unsigned long long)(T - 1) * lddh + H) * 2;
  const unsigned long long nz = ((unsigned long long)(T - 1) * ldz + H) * 4, ndx = 2ull * T * D;
  const void* in[7] = {dh, z, u, x, W1, W3, workspace};
  const unsigned long long in_size[7] = {ndh, nz, nz, nx, nw, nw, need};
  const void* out[3] = {dx, dW1, dW3};
  const unsigned long long size[3] = {ndx, nw, nw};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 7; ++j)
      if (overlap(out[i], size[i], in[j], in_size[j]))
        return fail(SFFN_ERR_ARG, "%s: a gradient overlaps an operand or the workspace", fn);
    if (overlap(out[i], size[i], out[(i + 1) % 3], size[(i + 1) % 3]))
      return fail(SFFN_ERR_ARG, "%s: a gradient overlaps another", fn);
  }
  for (int j = 0; j < 6; ++j)
    if (overlap(workspace, need, in[j], in_size[j])) return fail(SFFN_ERR_ARG, "%s: the workspace overlaps an operand", fn);
  if (!dx && !dW1 && !dW3) return SFFN_OK;
  GatedGradArgs a;
  a.dh = dh;
  a.lddh = lddh;
  a.z = z;
  a.u = u;
  a.ldz = ldz;
  a.x = x;
  a.ldx = ldx;
  a.W1 = W1;
  a.W3 = W3;
  a.dx = dx;
  a.dW1 = dW1;
  a.dW3 = dW3;
  a.T = T;
  a.D = D;
  a.H = H;
  a.act = act;
  a.workspace = workspace;
  const cudaError_t e = launch_gated_grad(a, s);
  return e == cudaSuccess ? SFFN_OK : cuda_fail(fn, e);
}

int sffn_check(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail("cudaStreamSynchronize", e);
  int* word = nullptr;
  if ((e = ops_error_word(&word)) != cudaSuccess) return cuda_fail("sffn_check", e);
  int v = 0;
  if ((e = cudaMemcpy(&v, word, sizeof v, cudaMemcpyDeviceToHost)) != cudaSuccess) return cuda_fail("cudaMemcpy", e);
  if (v == 0) return SFFN_OK;
  if ((e = cudaMemset(word, 0, sizeof v)) != cudaSuccess) return cuda_fail("cudaMemset", e);
  return fail(SFFN_ERR_TIMEOUT, "an operator's device-side wait ran out of time (error word 0x%x); its outputs are "
              "invalid", v);
}

}  // extern "C"

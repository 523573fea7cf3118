// ops_api.cu -- the handle-free entry points of include/sffn.h: the router,
// per-token int8 codes, the int8 product, the products grouped by expert and
// the gated experts' forward.  Argument checks come before any CUDA call.
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

// ops.h -- launchers of the mixture-of-experts and 8-bit operators (handle-free
// entry points of include/sffn.h; not installed).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sffn {

// The per-device error word of the handle-free operators (0 or DEV_ERR_TIMEOUT).
cudaError_t ops_error_word(int** p);
int ops_num_sms();

// ---- route.cu
struct RouteArgs {
  const void* logits;
  long long ld;
  float* weights;
  int *ids, *offsets, *rows, *hist;
  int T, E, k, bf16, sigmoid, normalize;
  int vec;  // rows of logits are 16-byte aligned
};
size_t route_workspace(int T, int E, int k);
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);

// ---- quant_tokens.cu
cudaError_t launch_quantize_tokens(const void* x, long long ld, int8_t* q, float* sc, int T, int K, cudaStream_t s);

// ---- the products.  Operands: x rows of `ldx` elements, w [E, N, K] (kn: [E, K, N]); row r of the
// result belongs to the expert e with offsets[e] <= r < offsets[e + 1] (offsets null: one expert, all rows).
struct GmmArgs {
  const void* x = nullptr;
  const void* w = nullptr;
  const void* w3 = nullptr;       // gated form: h = A(x W1^T) .* (x W3^T)
  const float* sx = nullptr;      // int8: scale of source row s(r)
  const float* sw = nullptr;      // int8: [E, N]
  const int* offsets = nullptr;   // [E + 1]
  const int* index = nullptr;     // source row of row r is index[r] / index_div
  int index_div = 1;
  void* y = nullptr;
  long long ldx = 0, ldy = 0;
  int R = 0, XR = 0, N = 0, K = 0, E = 1;  // XR: rows of x
  int i8 = 0, y_f32 = 0, kn = 0, act = 0;
  int NY = 0;                     // columns of y that may be written (past N: zeros), if more than N
  int f16 = 0;                    // x and w are fp16 copies of int8 codes (with their scales)
  float *z = nullptr, *u = nullptr;  // gated: the two products themselves, fp32, row pitch ldz
  long long ldz = 0;
  int split = 0;                  // w's rows hold two parts of round_up(K, 64) columns each, both multiplied by x
  int K1 = 0;                     // kn: rows 0 .. K1 of K are w's, rows K / 2 .. K / 2 + K1 w3's (K / 2 = round_up(K1, 64))
  int xt = 0;                     // kn: x is [K, rows]; group e's rows are its columns from e * xper on, w is every group's
  int per = 0, xper = 0;          // xt: rows of a group
  void* y2 = nullptr;             // xt: the second group's result (its first row)
  long long ldw = 0;              // kn: row pitch of w, if not N
  void* workspace = nullptr;      // gmm_workspace() bytes
};
constexpr int GATE_ROWS = 16;  // rows of z whose norms are side by side; a tile of x starts at a multiple of it
cudaError_t launch_gmm_rows(const GmmArgs& a, cudaStream_t s);
cudaError_t launch_gmm_tc(const GmmArgs& a, int ctas, int nt, cudaStream_t s);  // ctas 1 or 2, nt 32 .. 256 (gated: 128)
cudaError_t launch_gate_norms(const GmmArgs& a, int per, cudaStream_t s);  // gated.cu; per: rows of x a tile
cudaError_t launch_gmm(const GmmArgs& a, cudaStream_t s);
size_t gmm_workspace(int R, int XR, int N, int K, int E, int i8);

// ---- experts.cu
struct ExpertsArgs {
  const void* x;
  long long ldx;
  const float* weights;  // [T, k]
  const int* ids;        // [T, k]
  const int* offsets;    // [E + 1]
  const int* rows;       // [T * k]
  const void *W1, *W3, *W2t;
  void* y;
  void* workspace;
  int T, E, k, D, H, act;
};
size_t experts_workspace(int T, int k, int D, int H);
cudaError_t launch_experts(const ExpertsArgs& a, cudaStream_t s);

// ---- int4.cu
struct Int4Args {
  const void* x;
  long long ldx;
  const uint8_t *w, *w3;  // w3: the gated block, else null
  const float *sw, *s3;
  void* y;
  long long ldy;
  int T, N, K, group, y_f32, act;
  void* workspace;  // int4_workspace() bytes
};
cudaError_t launch_quantize_int4(const void* w, long long ldw, uint8_t* q, float* sc, int N, int K, int group,
                                 cudaStream_t s);
cudaError_t launch_dequantize_int4(const uint8_t* q, const float* sc, void* y, long long ldy, int N, int K, int group,
                                   int y_f32, cudaStream_t s);
size_t int4_workspace(int T, int N, int K, int split, int gated);  // split: y is fp32, or gated
cudaError_t launch_matmul_int4(const Int4Args& a, cudaStream_t s);

// ---- gated.cu
struct GatedArgs {
  const void* x;
  long long ldx;
  const void *W1, *W3;
  void* h;
  long long ldh;
  float *z, *u;  // may be null (both)
  long long ldz;
  int T, D, H, act;
};
cudaError_t launch_gated_up(const GatedArgs& a, cudaStream_t s);
struct GatedGradArgs {
  const void* dh;
  long long lddh;
  const float *z, *u;
  long long ldz;
  const void* x;
  long long ldx;
  const void *W1, *W3;
  void *dx, *dW1, *dW3;  // each may be null
  int T, D, H, act;
  void* workspace;  // gated_grad_workspace() bytes
};
size_t gated_grad_workspace(int T, int H);
cudaError_t launch_gated_grad(const GatedGradArgs& a, cudaStream_t s);

// A launch whose blocks may start while the kernel before it in the stream
// ends (each kernel waits for that one's results itself).
template <typename... KArgs, typename... Args>
inline cudaError_t ops_launch(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                              int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sffn

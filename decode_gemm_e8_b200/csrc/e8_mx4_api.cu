// C ABI of the microscaled 4-bit form and of the mixture-of-experts layer
// (declared in include/e8.h): argument checks, workspace carving, launches.
#include <cstdint>

#include "e8.h"
#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace {

using e8::aligned16;

bool valid_shape(int64_t rows, int64_t K) {
  return rows >= 0 && rows <= INT32_MAX && K >= 1 && K <= INT32_MAX;
}
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? E8_OK : E8_ECUDA; }

// The last check before the first launch: argument errors come before any CUDA call.
int check_device(const e8_codebook* cb) {
  (void)cudaGetLastError();  // a failed earlier launch must not be reported here
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return E8_ECUDA;
  return dev == cb->device ? E8_OK : E8_EDEVICE;
}

uintptr_t elem_bytes(int dtype) { return dtype == E8_DT_F32 ? 4 : 2; }
bool valid_dtype(int dtype) { return dtype >= E8_DT_BF16 && dtype <= E8_DT_F32; }

}  // namespace

extern "C" {

int64_t e8_mx4_code_bytes(int64_t rows, int64_t K) {
  return valid_shape(rows, K) ? rows * e8::mx4::code_stride(K) : -1;
}

int64_t e8_mx4_scale_bytes(int64_t rows, int64_t K) {
  return valid_shape(rows, K) ? e8::mx4::scale_bytes(rows, K) : -1;
}

int e8_mx4_encode(const e8_codebook* cb, const void* X, int dtype, int64_t batch, int64_t rows,
                  int64_t K, int64_t ldx, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!cb || !valid_dtype(dtype) || batch < 0 || batch > INT32_MAX || !valid_shape(rows, K) ||
      ldx < K || ldx > INT32_MAX)
    return E8_EINVAL;
  if (batch == 0 || rows == 0) return E8_OK;
  if (!X || !codes || !scales || !aligned(X, elem_bytes(dtype)) || !aligned16(codes) ||
      !aligned16(scales))
    return E8_EINVAL;
  const int rc = check_device(cb);
  if (rc != E8_OK) return rc;
  return cuda_status(
      e8::launch_mx4_encode(X, dtype, batch, rows, K, ldx, codes, scales,
                            cb->sm_count, (cudaStream_t)stream));
}

int e8_mx4_decode_to_bf16(const e8_codebook* cb, const uint8_t* codes, const uint8_t* scales,
                          int64_t batch, int64_t rows, int64_t K, uint16_t* out, void* stream) {
  if (!cb || batch < 0 || batch > INT32_MAX || !valid_shape(rows, K)) return E8_EINVAL;
  if (batch == 0 || rows == 0) return E8_OK;
  if (!codes || !scales || !out || !aligned16(codes) || !aligned16(scales) || !aligned16(out))
    return E8_EINVAL;
  const int rc = check_device(cb);
  if (rc != E8_OK) return rc;
  return cuda_status(
      e8::launch_mx4_decode(codes, scales, batch, rows, K, out, (cudaStream_t)stream));
}

// The partial sums of a split product stay in the SMs of its cluster.
size_t e8_mx4_gemm_codes_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

// [codes of X][scales of X], each on 256 bytes
size_t e8_mx4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!valid_shape(M, K) || !valid_shape(N, K) || M == 0 || N == 0) return 0;
  return round256((size_t)e8_mx4_code_bytes(M, K)) + round256((size_t)e8_mx4_scale_bytes(M, K));
}

int e8_mx4_gemm_codes(const e8_codebook* cb, const uint8_t* a_codes, const uint8_t* a_scales,
                      int64_t M, const uint8_t* w_codes, const uint8_t* w_scales, int64_t N,
                      int64_t K, uint16_t* Y, void*, size_t, void* stream) {
  if (!cb || !valid_shape(M, K) || !valid_shape(N, K)) return E8_EINVAL;
  if (M == 0 || N == 0) return E8_OK;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !Y || !aligned16(a_codes) ||
      !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(Y))
    return E8_EINVAL;
  const int rc = check_device(cb);
  if (rc != E8_OK) return rc;
  return cuda_status(e8::launch_mx4_gemm(a_codes, a_scales, M, w_codes, w_scales, N, K, Y,
                                         cb->status, cb->sm_count, 0, (cudaStream_t)stream));
}

int e8_mx4_gemm(const e8_codebook* cb, const void* X, int dtype, int64_t M, int64_t ldx,
                const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int64_t K,
                uint16_t* Y, void* workspace, size_t ws_bytes, void* stream) {
  if (!cb || !valid_dtype(dtype) || !valid_shape(M, K) || !valid_shape(N, K) || ldx < K ||
      ldx > INT32_MAX)
    return E8_EINVAL;
  if (M == 0 || N == 0) return E8_OK;
  if (!X || !w_codes || !w_scales || !Y || !aligned(X, elem_bytes(dtype)) ||
      !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(Y))
    return E8_EINVAL;
  const size_t need = e8_mx4_gemm_workspace_bytes(M, N, K);
  if (!workspace || !aligned16(workspace) || ws_bytes < need) return E8_EWORKSPACE;
  const int rc = check_device(cb);
  if (rc != E8_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (M <= e8::kMx4Small)
    return cuda_status(e8::launch_mx4_gemm_small(X, dtype, M, ldx, w_codes, w_scales, N, K, Y,
                                                 cb->status, cb->sm_count, st));
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + round256((size_t)e8_mx4_code_bytes(M, K));
  if (e8::launch_mx4_encode(X, dtype, 1, M, K, ldx, codes, scales, cb->sm_count, st) != cudaSuccess)
    return E8_ECUDA;
  return cuda_status(e8::launch_mx4_gemm(codes, scales, M, w_codes, w_scales, N, K, Y, cb->status,
                                         cb->sm_count, 1, st));
}

static bool moe_shape(int64_t T, int64_t H, int64_t E, int topk, int64_t I) {
  return T >= 0 && T <= E8_MOE_MAX_TOKENS && E >= 1 && E <= E8_MOE_MAX_EXPERTS && topk >= 1 &&
         topk <= E && topk <= E8_MOE_MAX_TOPK && H >= 128 && H % 128 == 0 && I >= 128 &&
         I % 128 == 0 && H <= 32768 && I <= 65536;
}

size_t e8_mx4_moe_workspace_bytes(int64_t T, int64_t H, int64_t E, int topk, int64_t I) {
  if (!moe_shape(T, H, E, topk, I) || T == 0) return 0;
  return e8::moe_workspace(T, H, E, topk, I);
}

int e8_mx4_moe(const e8_codebook* cb, const uint16_t* X, int64_t T, int64_t H,
               const uint16_t* router, int64_t E, int topk, int renormalize,
               const uint8_t* w13_codes, const uint8_t* w13_scales, int64_t I,
               const uint8_t* w2_codes, const uint8_t* w2_scales, uint16_t* Y, int32_t* experts,
               float* probs, void* workspace, size_t ws_bytes, void* stream) {
  if (!cb || !moe_shape(T, H, E, topk, I)) return E8_EINVAL;
  if (T == 0) return E8_OK;
  if (!X || !router || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !Y ||
      !aligned16(X) || !aligned16(router) || !aligned(w13_codes, 32) || !aligned(w13_scales, 32) ||
      !aligned(w2_codes, 32) || !aligned(w2_scales, 32) || !aligned16(Y) ||
      !aligned16(experts) || !aligned16(probs))
    return E8_EINVAL;
  const size_t need = e8_mx4_moe_workspace_bytes(T, H, E, topk, I);
  if (!workspace || !aligned16(workspace) || ws_bytes < need) return E8_EWORKSPACE;
  const int rc = check_device(cb);
  if (rc != E8_OK) return rc;
  e8::MoeArgs a;
  a.X = X;
  a.router = router;
  a.w13_codes = w13_codes;
  a.w13_scales = w13_scales;
  a.w2_codes = w2_codes;
  a.w2_scales = w2_scales;
  a.Y = Y;
  a.experts = experts;
  a.probs = probs;
  a.workspace = workspace;
  a.T = (int)T;
  a.H = (int)H;
  a.E = (int)E;
  a.topk = topk;
  a.renorm = renormalize != 0;
  a.I = (int)I;
  a.status = cb->status;
  return cuda_status(e8::launch_moe(a, cb->sm_count, (cudaStream_t)stream));
}

}  // extern "C"

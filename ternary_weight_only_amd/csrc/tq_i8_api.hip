// tq_i8_api.hip -- the extern "C" entry points of the norms that make 8-bit rows
// and of the products that read them (declared in include/tq.h): host-side
// argument validation, then the launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/tq.h"
#include "../../include/tq_probe.h"
#include "tq_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxK = int64_t(1) << 21;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 40;  // every byte count stays below 2^62
constexpr int64_t kMaxExperts = 65536;
constexpr double kMinEps = 0x1p-252;  // where rstd is written: a row of zeros has 2^126 there, which fp32 holds
constexpr int64_t kMaxGather = int64_t(1) << 32;  // bytes of x, read by 32-bit offsets where rows are given by index

bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

bool type_ok(int t) { return t == TQ_BF16 || t == TQ_F32; }
uintptr_t size_of(int t) { return t == TQ_F32 ? 4 : 2; }

int check_norm_shape(int64_t M, int64_t K) {
  if (M < 0 || M > kMaxRows || K < 1 || K > kMaxK || !product_ok(M, K)) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int check_product(int64_t T, int64_t N, int64_t K, int G, int64_t experts) {
  if (G != 64 && G != 128) return TQ_ERR_GROUP;
  if (T < 0 || T > kMaxRows || N < 1 || N > kMaxRows || K < 1 || K > kMaxK || K % G != 0) return TQ_ERR_SHAPE;
  if (experts < 1 || experts > kMaxExperts) return TQ_ERR_SHAPE;
  if (!product_ok(T, N) || !product_ok(T, K) || !product_ok(N, K) || !product_ok(experts, N * K)) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int check_workspace(const void *workspace, int64_t have, int64_t need) {
  if (need == 0) return TQ_OK;
  if (have < need) return TQ_ERR_WORKSPACE;
  if (!workspace) return TQ_ERR_NULL;
  return aligned(workspace, 16) ? TQ_OK : TQ_ERR_ALIGN;
}

int finish_launch() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? TQ_OK : TQ_ERR_LAUNCH;
}

// The arguments that both forms of the norm have; `out` is q or h.
int check_norm(const void *x, int x_type, const void *residual, int residual_type, const void *weight,
               int weight_type, int64_t M, int64_t K, double eps, double least, const void *out, const void *y,
               const int32_t *d_status) {
  const int rc = check_norm_shape(M, K);
  if (rc) return rc;
  if (!type_ok(x_type) || (residual && !type_ok(residual_type)) || (weight && !type_ok(weight_type)))
    return TQ_ERR_TYPE;
  if (!(eps > 0.0) || !isfinite(eps) || eps < least) return TQ_ERR_VALUE;
  if (M == 0) return TQ_OK;
  if (!x || !out || !residual != !y) return TQ_ERR_NULL;
  if (!aligned(x, size_of(x_type)) || !aligned(d_status, 4) ||
      (residual && (!aligned(residual, size_of(residual_type)) || !aligned(y, size_of(residual_type)))) ||
      (weight && !aligned(weight, size_of(weight_type))))
    return TQ_ERR_ALIGN;
  return TQ_OK;
}

// Both forms of the product; offsets null: one matrix.
int product(const int8_t *x, const float *x_scales, int64_t sources, const int32_t *rows, const uint8_t *packed,
            const uint16_t *scales, const int32_t *offsets, bool grouped, int64_t experts, const void *bias,
            int bias_type, int act, const void *residual, int64_t T, int64_t N, int64_t K, int G, void *out,
            int out_type, void *workspace, int64_t workspace_bytes, int32_t *d_status, void *stream) {
  int rc = check_product(T, N, K, G, experts);
  if (rc) return rc;
  if (sources < 0 || sources > kMaxRows || !product_ok(sources, K) || (!rows && sources < T)) return TQ_ERR_SHAPE;
  if (rows && sources * K > kMaxGather) return TQ_ERR_SHAPE;
  if (act != TQ_ACT_SILU && act != TQ_ACT_GELU && act != TQ_ACT_NONE && act != TQ_ACT_RELU2) return TQ_ERR_ACT;
  if (!type_ok(out_type) || (bias && !type_ok(bias_type))) return TQ_ERR_TYPE;
  if (T == 0) return TQ_OK;
  if (sources < 1) return TQ_ERR_SHAPE;  // nothing that a row index could name
  if (!x || !x_scales || !packed || !scales || !out || (grouped && !offsets)) return TQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(x_scales, 4) || !aligned(scales, 2) || !aligned(offsets, 4) ||
      !aligned(rows, 4) || (bias && !aligned(bias, size_of(bias_type))) || !aligned(out, size_of(out_type)) ||
      !aligned(residual, size_of(out_type)) || !aligned(d_status, 4))
    return TQ_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, tq::gemm_i8_workspace(T, N, K, G, experts, grouped));
  if (rc) return rc;
  (void)hipGetLastError();
  tq::launch_gemm_i8(x, x_scales, packed, scales, offsets, experts, rows, sources, bias, bias_type == TQ_F32, act,
                     residual, T, N, K, G, out, out_type == TQ_F32, workspace, d_status, (hipStream_t)stream);
  return finish_launch();
}

}  // namespace

extern "C" {

int tq_rms_norm_i8(const void *x, int x_type, const void *residual, int residual_type, const void *weight,
                   int weight_type, int64_t M, int64_t K, double eps, int8_t *q, float *scales, void *y,
                   int32_t *d_status, void *stream) {
  const int rc = check_norm(x, x_type, residual, residual_type, weight, weight_type, M, K, eps, 0.0, q, y, d_status);
  if (rc || M == 0) return rc;
  if (!scales) return TQ_ERR_NULL;
  if (!aligned(scales, 4)) return TQ_ERR_ALIGN;
  (void)hipGetLastError();
  tq::launch_rms_norm(x, x_type == TQ_F32, residual, residual_type == TQ_F32, weight, weight_type == TQ_F32, M, K,
                      eps, q, scales, nullptr, y, nullptr, d_status, (hipStream_t)stream);
  return finish_launch();
}

int tq_rms_norm_forward(const void *x, int x_type, const void *residual, int residual_type, const void *weight,
                        int weight_type, int64_t M, int64_t K, double eps, uint16_t *h, void *y, float *rstd,
                        int32_t *d_status, void *stream) {
  const int rc = check_norm(x, x_type, residual, residual_type, weight, weight_type, M, K, eps, rstd ? kMinEps : 0.0, h,
                            y, d_status);
  if (rc || M == 0) return rc;
  if (!aligned(h, 2) || !aligned(rstd, 4)) return TQ_ERR_ALIGN;
  (void)hipGetLastError();
  tq::launch_rms_norm(x, x_type == TQ_F32, residual, residual_type == TQ_F32, weight, weight_type == TQ_F32, M, K,
                      eps, nullptr, nullptr, h, y, rstd, d_status, (hipStream_t)stream);
  return finish_launch();
}

int64_t tq_rms_norm_backward_workspace(int64_t M, int64_t K) {
  return check_norm_shape(M, K) || M == 0 ? 0 : tq::rms_norm_backward_workspace(M, K);
}

int tq_rms_norm_backward(const uint16_t *dh, const void *y, int y_type, const float *rstd, const void *weight,
                         int weight_type, const void *dy, int64_t M, int64_t K, void *dx, void *dweight,
                         void *workspace, int64_t workspace_bytes, void *stream) {
  int rc = check_norm_shape(M, K);
  if (rc) return rc;
  if (!type_ok(y_type) || (weight && !type_ok(weight_type))) return TQ_ERR_TYPE;
  if (dweight && !weight) return TQ_ERR_NULL;
  if (M > 0 && (!dh || !y || !rstd || !dx)) return TQ_ERR_NULL;
  const uintptr_t size = size_of(y_type);
  if (!aligned(dh, 2) || !aligned(y, size) || !aligned(rstd, 4) || !aligned(dy, size) || !aligned(dx, size) ||
      (weight && (!aligned(weight, size_of(weight_type)) || !aligned(dweight, size_of(weight_type)))))
    return TQ_ERR_ALIGN;
  if (M > 0) {
    rc = check_workspace(workspace, workspace_bytes, tq::rms_norm_backward_workspace(M, K));
    if (rc) return rc;
  }
  (void)hipGetLastError();
  tq::launch_rms_norm_backward(dh, y, y_type == TQ_F32, rstd, weight, weight_type == TQ_F32, dy, M, K, dx, dweight,
                               workspace, (hipStream_t)stream);
  return finish_launch();
}

int64_t tq_gemm_i8_workspace(int64_t M, int64_t N, int64_t K, int G) {
  return check_product(M, N, K, G, 1) || M == 0 ? 0 : tq::gemm_i8_workspace(M, N, K, G, 1, false);
}

int tq_gemm_i8(const int8_t *x, const float *x_scales, const uint8_t *packed, const uint16_t *scales,
               const void *bias, int bias_type, int act, const void *residual, int64_t M, int64_t N, int64_t K,
               int G, void *out, int out_type, void *workspace, int64_t workspace_bytes, int32_t *d_status,
               void *stream) {
  return product(x, x_scales, M, nullptr, packed, scales, nullptr, false, 1, bias, bias_type, act, residual, M, N,
                 K, G, out, out_type, workspace, workspace_bytes, d_status, stream);
}

int64_t tq_expert_gemm_i8_workspace(int64_t T, int64_t N, int64_t K, int G, int64_t experts) {
  return check_product(T, N, K, G, experts) || T == 0 ? 0 : tq::gemm_i8_workspace(T, N, K, G, experts, true);
}

int tq_expert_gemm_i8(const int8_t *x, const float *x_scales, int64_t sources, const int32_t *rows,
                      const uint8_t *packed, const uint16_t *scales, const int32_t *offsets, int64_t experts,
                      const void *bias, int bias_type, int act, const void *residual, int64_t T, int64_t N,
                      int64_t K, int G, void *out, int out_type, void *workspace, int64_t workspace_bytes,
                      int32_t *d_status, void *stream) {
  return product(x, x_scales, sources, rows, packed, scales, offsets, true, experts, bias, bias_type, act, residual,
                 T, N, K, G, out, out_type, workspace, workspace_bytes, d_status, stream);
}

int tq_probe_i8_plan(int64_t M, int64_t N, int64_t K, int G, int64_t experts, int64_t *plan) {
  const int rc = check_product(M, N, K, G, experts ? experts : 1);
  if (rc) return rc;
  if (M < 1) return TQ_ERR_SHAPE;
  if (!plan) return TQ_ERR_NULL;
  tq::i8_plan(M, N, K, G, experts, plan);
  return TQ_OK;
}

}  // extern "C"

// tq_ffn_api.hip -- the extern "C" entry points of the gated feed-forward and
// adapter calls (declared in include/tq.h): host-side argument validation,
// then the launches on the caller's stream, as tq_api.hip does for the rest.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tq.h"
#include "../../include/tq_probe.h"
#include "tq_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxK = int64_t(1) << 21;  // a 256-row slab of x stays below 2^31 bytes
constexpr int64_t kMaxRows = int64_t(1) << 30;  // tiles times threads fit a launch
constexpr int64_t kMaxElems = int64_t(1) << 40;          // every byte count stays below 2^62

bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

int check_mnk(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || M > kMaxRows || N < 1 || N > kMaxRows || K < 1 || K > kMaxK) return TQ_ERR_SHAPE;
  if (!product_ok(M, N) || !product_ok(M, K) || !product_ok(N, K)) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int check_packed_shape(int64_t M, int64_t N, int64_t K, int G) {
  if (G != 64 && G != 128) return TQ_ERR_GROUP;
  const int rc = check_mnk(M, N, K);
  if (rc) return rc;
  return K % G == 0 ? TQ_OK : TQ_ERR_SHAPE;
}

int check_train_shape(int64_t M, int64_t N, int64_t K) {
  const int rc = check_mnk(M, N, K);
  if (rc) return rc;
  return K % 64 == 0 && N <= kMaxK ? TQ_OK : TQ_ERR_SHAPE;  // N is a reduction length too
}

int check_rank(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t R) {
  if (adapters < 0 || adapters > kMaxRows || R < 8 || R > 256 || R % 8 != 0) return TQ_ERR_SHAPE;
  if (!product_ok(adapters, N * R) || !product_ok(adapters, K * R) || !product_ok(M, R))
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

int check_workspace(const void *workspace, int64_t have, int64_t need) {
  if (need == 0) return TQ_OK;
  if (have < need) return TQ_ERR_WORKSPACE;
  if (!workspace) return TQ_ERR_NULL;
  return aligned(workspace, 16) ? TQ_OK : TQ_ERR_ALIGN;
}

bool act_ok(int act) { return act == TQ_ACT_SILU || act == TQ_ACT_GELU; }

int finish_launch() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? TQ_OK : TQ_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int64_t tq_glu_workspace(int64_t M, int64_t N, int64_t K, int G) {
  return check_packed_shape(M, N, K, G) || M == 0 ? 0 : tq::glu_workspace(M, N, K, G);
}

int tq_glu(const uint16_t *x, const uint8_t *gate_packed, const uint16_t *gate_scales,
           const uint8_t *up_packed, const uint16_t *up_scales, int64_t M, int64_t N, int64_t K,
           int G, int act, uint16_t *h, void *workspace, int64_t workspace_bytes,
           int32_t *d_status, void *stream) {
  int rc = check_packed_shape(M, N, K, G);
  if (rc) return rc;
  if (!act_ok(act)) return TQ_ERR_ACT;
  if (M == 0) return TQ_OK;
  if (!x || !gate_packed || !gate_scales || !up_packed || !up_scales || !h) return TQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(gate_scales, 2) || !aligned(up_scales, 2) || !aligned(h, 2) ||
      !aligned(d_status, 4))
    return TQ_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, tq::glu_workspace(M, N, K, G));
  if (rc) return rc;
  (void)hipGetLastError();
  tq::launch_glu(x, gate_packed, gate_scales, up_packed, up_scales, M, N, K, G, act, h, workspace,
                 d_status, (hipStream_t)stream);
  return finish_launch();
}

int64_t tq_lora_workspace(int64_t M, int64_t N, int64_t K, int G, int64_t R) {
  if (check_packed_shape(M, N, K, G) || check_rank(M, N, K, 0, R) || M == 0) return 0;
  return tq::lora_workspace(M, N, K, G, (int)R);
}

int tq_lora_matmul(const uint16_t *x, const uint8_t *packed, const uint16_t *scales,
                   const int32_t *ids, const uint16_t *A, const uint16_t *B,
                   const float *scaling, int64_t M, int64_t N, int64_t K, int G,
                   int64_t adapters, int64_t R, float *y, void *workspace,
                   int64_t workspace_bytes, int32_t *d_status, void *stream) {
  int rc = check_packed_shape(M, N, K, G);
  if (!rc) rc = check_rank(M, N, K, adapters, R);
  if (rc) return rc;
  if (M == 0) return TQ_OK;
  if (!x || !packed || !scales || !ids || !y) return TQ_ERR_NULL;
  if (adapters > 0 && (!A || !B || !scaling)) return TQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(scales, 2) || !aligned(ids, 4) || !aligned(A, 16) ||
      !aligned(B, 16) || !aligned(scaling, 4) || !aligned(y, 4) || !aligned(d_status, 4))
    return TQ_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, tq::lora_workspace(M, N, K, G, (int)R));
  if (rc) return rc;
  (void)hipGetLastError();
  tq::launch_lora(x, packed, scales, M, N, K, G, ids, A, B, scaling, (int)adapters, (int)R, y,
                  workspace, d_status, (hipStream_t)stream);
  return finish_launch();
}

int tq_probe_projection_plan(int64_t M, int64_t N, int64_t K, int G, int matrices, int64_t R,
                             int64_t *plan) {
  int rc = check_packed_shape(M, N, K, G);
  if (!rc && matrices == 1) rc = check_rank(M, N, K, 0, R);
  if (rc) return rc;
  if (M < 1 || matrices < 1 || matrices > 2) return TQ_ERR_SHAPE;
  if (!plan) return TQ_ERR_NULL;
  tq::projection_plan(M, N, K, G, matrices, (int)R, plan);
  return TQ_OK;
}

int tq_glu_forward(const uint16_t *x, const uint16_t *wg, const uint16_t *wu, int64_t M,
                   int64_t N, int64_t K, int act, uint16_t *h, uint16_t *g, uint16_t *u,
                   void *stream) {
  const int rc = check_train_shape(M, N, K);
  if (rc) return rc;
  if (!act_ok(act)) return TQ_ERR_ACT;
  if (M == 0) return TQ_OK;
  if (!x || !wg || !wu || !h || !g != !u) return TQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(wg, 16) || !aligned(wu, 16) || !aligned(h, 16) ||
      !aligned(g, 16) || !aligned(u, 16))
    return TQ_ERR_ALIGN;
  (void)hipGetLastError();
  tq::launch_glu_forward(x, wg, wu, M, N, K, act, h, g, u, (hipStream_t)stream);
  return finish_launch();
}

int64_t tq_glu_backward_workspace(int64_t M, int64_t N, int64_t K) {
  return check_train_shape(M, N, K) || M == 0 ? 0 : tq::glu_backward_workspace(M, N, K);
}

int tq_glu_backward(const uint16_t *dh, const uint16_t *x, const uint16_t *wg,
                    const uint16_t *wu, const uint16_t *g, const uint16_t *u, int64_t M,
                    int64_t N, int64_t K, int act, uint16_t *dx, uint16_t *dwg, uint16_t *dwu,
                    void *workspace, int64_t workspace_bytes, void *stream) {
  int rc = check_train_shape(M, N, K);
  if (rc) return rc;
  if (!act_ok(act)) return TQ_ERR_ACT;
  if (!wg || !wu || !dwg || !dwu) return TQ_ERR_NULL;
  if (M > 0 && (!dh || !x || !g || !u || !dx)) return TQ_ERR_NULL;
  if (!aligned(dh, 16) || !aligned(x, 16) || !aligned(wg, 16) || !aligned(wu, 16) ||
      !aligned(g, 16) || !aligned(u, 16) || !aligned(dx, 16) || !aligned(dwg, 16) ||
      !aligned(dwu, 16))
    return TQ_ERR_ALIGN;
  if (M > 0) {
    rc = check_workspace(workspace, workspace_bytes, tq::glu_backward_workspace(M, N, K));
    if (rc) return rc;
  }
  (void)hipGetLastError();
  tq::launch_glu_backward(dh, x, wg, wu, g, u, M, N, K, act, dx, dwg, dwu, workspace,
                          (hipStream_t)stream);
  return finish_launch();
}

int tq_probe_train_plan(int64_t M, int64_t N, int64_t K, int64_t *plan) {
  const int rc = check_train_shape(M, N, K);
  if (rc) return rc;
  if (M < 1) return TQ_ERR_SHAPE;
  if (!plan) return TQ_ERR_NULL;
  tq::train_plan(M, N, K, plan);
  return TQ_OK;
}

}  // extern "C"

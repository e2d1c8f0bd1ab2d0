// tq_glu_train.hip -- the gated feed-forward block on bf16 weights, forward
// and backward (quantization-aware training: the weights are the bf16 w_hat
// of tq_fake_quantize, whose gradient is straight-through).
//
//   forward    g = x Wg^T, u = x Wu^T, h = act(g) u
//   backward   dg = dh u act'(g), du = dh act(g)
//              dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_ffn.h"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int T = 64, KS = 32, PITCH = KS + 8;

// An operand element (row, k) at p[row * rs + k * ks].
struct Operand {
  const uint16_t *p;
  int64_t rs, ks;
};

constexpr int kEpiStore = 0, kEpiGlu = 1;

// kEpiStore: c0 = sum over both pairs of a_i b_i^T (pair 1 absent: b1.p null)
// kEpiGlu:   g = a0 b0^T, u = a0 b1^T -> c0 = h, c1 = g, c2 = u
template <int EPI, int ACT>
__global__ __launch_bounds__(256) void dense_kernel(Operand a0, Operand b0, Operand a1, Operand b1,
                                                    int64_t rows, int64_t cols, int64_t depth,
                                                    uint16_t *__restrict__ c0,
                                                    uint16_t *__restrict__ c1,
                                                    uint16_t *__restrict__ c2) {
  __shared__ __align__(16) uint16_t as[T * PITCH], bs[T * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.y * T, q0 = (int64_t)blockIdx.x * T;
  constexpr int NA = EPI == kEpiGlu ? 2 : 1;
  f32x4 acc[NA][4];
  for (int i = 0; i < NA; ++i)
    for (int a = 0; a < 4; ++a) acc[i][a] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int pair = 0; pair < 2; ++pair) {
    const Operand A = EPI == kEpiGlu || pair == 0 ? a0 : a1, B = pair == 0 ? b0 : b1;
    if (!B.p) break;
    for (int64_t k0 = 0; k0 < depth; k0 += KS) {
      for (int e = tid; e < T * KS; e += 256) {
        const int r = e / KS, k = e % KS;
        const bool kin = k0 + k < depth;
        as[r * PITCH + k] = kin && r0 + r < rows ? A.p[(r0 + r) * A.rs + (k0 + k) * A.ks] : 0;
        bs[r * PITCH + k] = kin && q0 + r < cols ? B.p[(q0 + r) * B.rs + (k0 + k) * B.ks] : 0;
      }
      __syncthreads();
      const bf16x8 bv = *(const bf16x8 *)(bs + (16 * wv + (lane & 15)) * PITCH + 8 * (lane >> 4));
      f32x4 *ac = acc[EPI == kEpiGlu ? pair : 0];
      for (int a = 0; a < 4; ++a)
        ac[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            *(const bf16x8 *)(as + (16 * a + (lane & 15)) * PITCH + 8 * (lane >> 4)), bv, ac[a], 0,
            0, 0);
      __syncthreads();
    }
  }
  const int64_t q = q0 + 16 * wv + (lane & 15);
  for (int a = 0; a < 4; ++a)
    for (int i = 0; i < 4; ++i) {
      const int64_t r = r0 + 16 * a + 4 * (lane >> 4) + i;
      if (r >= rows || q >= cols) continue;
      if constexpr (EPI == kEpiGlu) {
        const float g = acc[0][a][i], u = acc[NA - 1][a][i];
        c0[r * cols + q] = f32_to_bf16(act_value<ACT>(g) * u);
        if (c1) {
          c1[r * cols + q] = f32_to_bf16(g);
          c2[r * cols + q] = f32_to_bf16(u);
        }
      } else {
        c0[r * cols + q] = f32_to_bf16(acc[0][a][i]);
      }
    }
}

// dg and du, rounded once to bf16 (the type the matrix cores take).
template <int ACT>
__global__ __launch_bounds__(256) void gate_grad_kernel(const uint16_t *__restrict__ dh,
                                                        const uint16_t *__restrict__ g,
                                                        const uint16_t *__restrict__ u, int64_t n,
                                                        uint16_t *__restrict__ dg,
                                                        uint16_t *__restrict__ du) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float value, slope;
    const float d = bf16_to_f32(dh[i]);
    act_and_slope<ACT>(bf16_to_f32(g[i]), value, slope);
    dg[i] = f32_to_bf16(d * bf16_to_f32(u[i]) * slope);
    du[i] = f32_to_bf16(d * value);
  }
}

}  // namespace

void launch_glu_forward(const uint16_t *x, const uint16_t *wg, const uint16_t *wu, int64_t M,
                        int64_t N, int64_t K, int act, uint16_t *h, uint16_t *g, uint16_t *u,
                        hipStream_t stream) {
  const dim3 grid((unsigned)((N + T - 1) / T), (unsigned)((M + T - 1) / T));
  auto kernel = act == kActSilu ? dense_kernel<kEpiGlu, kActSilu> : dense_kernel<kEpiGlu, kActGelu>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, Operand{x, K, 1}, Operand{wg, K, 1},
                     Operand{x, K, 1}, Operand{wu, K, 1}, M, N, K, h, g, u);
}

int64_t glu_backward_workspace(int64_t M, int64_t N, int64_t K) { return 4 * M * N; }

void launch_glu_backward(const uint16_t *dh, const uint16_t *x, const uint16_t *wg,
                         const uint16_t *wu, const uint16_t *g, const uint16_t *u, int64_t M,
                         int64_t N, int64_t K, int act, uint16_t *dx, uint16_t *dwg, uint16_t *dwu,
                         void *workspace, hipStream_t stream) {
  uint16_t *dg = (uint16_t *)workspace, *du = dg + M * N;
  if (M > 0) {
    const int64_t blocks = (M * N + 255) / 256;
    hipLaunchKernelGGL(act == kActSilu ? gate_grad_kernel<kActSilu> : gate_grad_kernel<kActGelu>,
                       dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, dh, g,
                       u, M * N, dg, du);
    hipLaunchKernelGGL((dense_kernel<kEpiStore, kActSilu>),
                       dim3((unsigned)((K + T - 1) / T), (unsigned)((M + T - 1) / T)), dim3(256), 0,
                       stream, Operand{dg, N, 1}, Operand{wg, 1, K}, Operand{du, N, 1},
                       Operand{wu, 1, K}, M, K, N, dx, nullptr, nullptr);
  }
  const dim3 grid((unsigned)((K + T - 1) / T), (unsigned)((N + T - 1) / T));
  hipLaunchKernelGGL((dense_kernel<kEpiStore, kActSilu>), grid, dim3(256), 0, stream,
                     Operand{dg, 1, N}, Operand{x, 1, K}, Operand{}, Operand{}, N, K, M, dwg,
                     nullptr, nullptr);
  hipLaunchKernelGGL((dense_kernel<kEpiStore, kActSilu>), grid, dim3(256), 0, stream,
                     Operand{du, 1, N}, Operand{x, 1, K}, Operand{}, Operand{}, N, K, M, dwu,
                     nullptr, nullptr);
}

}  // namespace tq

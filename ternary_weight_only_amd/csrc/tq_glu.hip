// tq_glu.hip -- the packed-ternary projection behind tq_glu and
// tq_lora_matmul: one or two weight matrices against the same activations,
// with the epilogue that makes the operator.
//
//   P_i[m,n] = sum_g s_i[n,g] * sum_{j<G} x[m, gG+j] * c_i[n, gG+j]
//   glu:   h = bf16(act(P_0) * P_1)
//   lora:  y = P_0 + scaling_a * sum_r t[m,r] * B_a[n,r],  t[m,r] = sum_k x[m,k] A_a[r,k],
//          a = ids[m]; an id of -1 adds nothing.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_ffn.h"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int BM = 64, BN = 64, KS = 64, PITCH = KS + 8;

// 64 x 64 tile of the output, four waves, each 64 rows of x by 16 of W.
template <int G, int NB, int ACT>
__global__ __launch_bounds__(256) void proj_kernel(
    const uint16_t *__restrict__ x, const uint8_t *__restrict__ p0,
    const uint16_t *__restrict__ s0, const uint8_t *__restrict__ p1,
    const uint16_t *__restrict__ s1, int64_t M, int N, int K, const int32_t *__restrict__ ids,
    const float *__restrict__ t, const uint16_t *__restrict__ b,
    const float *__restrict__ scaling, int adapters, int R, void *__restrict__ out,
    int32_t *__restrict__ d_status) {
  constexpr int B = bytes_per_group(G);
  __shared__ __align__(16) uint16_t xs[BM * PITCH];
  __shared__ __align__(16) uint16_t cs[NB][BN * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t m0 = (int64_t)blockIdx.y * BM;
  const int n0 = blockIdx.x * BN, nG = K / G;
  f32x4 acc[NB][4], part[NB][4];
  for (int i = 0; i < NB; ++i)
    for (int a = 0; a < 4; ++a) acc[i][a] = part[i][a] = f32x4{0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  for (int k0 = 0; k0 < K; k0 += KS) {
    for (int c = tid; c < BM * KS / 8; c += 256) {
      const int r = c / 8, kc = c % 8;
      u32x4 v{0, 0, 0, 0};
      if (m0 + r < M) v = *(const u32x4 *)(x + (m0 + r) * K + k0 + 8 * kc);
      *(u32x4 *)(xs + r * PITCH + 8 * kc) = v;
    }
    {
      const int r = tid / 4, j0 = k0 % G + 16 * (tid % 4);
      for (int i = 0; i < NB; ++i) {
        const uint8_t *row = (i ? p1 : p0) + ((int64_t)(n0 + r) * nG + k0 / G) * B;
        for (int j = 0; j < 16; ++j) {
          uint16_t code = 0;
          if (n0 + r < N) {
            uint32_t v = row[(j0 + j) / 5];
            bad |= v >= 243;
            for (int d = 0; d < (j0 + j) % 5; ++d) v /= 3;
            v %= 3;
            code = v == 0 ? 0xBF80 : v == 2 ? 0x3F80 : 0;
          }
          cs[i][r * PITCH + 16 * (tid % 4) + j] = code;
        }
      }
    }
    __syncthreads();
    for (int ks = 0; ks < KS / 32; ++ks)
      for (int i = 0; i < NB; ++i) {
        const int col = 32 * ks + 8 * (lane >> 4);
        const bf16x8 bv = *(const bf16x8 *)(cs[i] + (16 * wv + (lane & 15)) * PITCH + col);
        for (int a = 0; a < 4; ++a)
          part[i][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              *(const bf16x8 *)(xs + (16 * a + (lane & 15)) * PITCH + col), bv, part[i][a], 0, 0, 0);
      }
    __syncthreads();
    if ((k0 + KS) % G == 0) {
      const int n = n0 + 16 * wv + (lane & 15);
      for (int i = 0; i < NB; ++i) {
        const float s =
            n < N ? __half2float(__ushort_as_half((i ? s1 : s0)[(int64_t)n * nG + k0 / G])) : 0.f;
        for (int a = 0; a < 4; ++a) {
          acc[i][a] += s * part[i][a];
          part[i][a] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
    }
  }
  const int n = n0 + 16 * wv + (lane & 15);
  for (int a = 0; a < 4; ++a)
    for (int r = 0; r < 4; ++r) {
      const int64_t m = m0 + 16 * a + 4 * (lane >> 4) + r;
      if (m >= M || n >= N) continue;
      if constexpr (NB == 2) {
        ((uint16_t *)out)[m * N + n] = f32_to_bf16(act_value<ACT>(acc[0][a][r]) * acc[1][a][r]);
      } else {
        float y = acc[0][a][r];
        const int id = ids[m];
        if (id >= 0 && id < adapters) {
          float sum = 0.f;
          for (int q = 0; q < R; ++q)
            sum += t[m * R + q] * bf16_to_f32(b[((int64_t)id * N + n) * R + q]);
          y += scaling[id] * sum;
        }
        ((float *)out)[m * N + n] = y;
      }
    }
  if (bad && d_status) atomicOr(d_status, kDevInvalidByte);
}

// t[m,r]: one wave a row of x and a rank; ids outside [-1, adapters) are
// flagged and count as -1.
__global__ __launch_bounds__(256) void shrink_kernel(const uint16_t *__restrict__ x, int64_t M,
                                                     int K, const int32_t *__restrict__ ids,
                                                     const uint16_t *__restrict__ A, int adapters,
                                                     int R, float *__restrict__ t,
                                                     int32_t *__restrict__ d_status) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t m = w / R;
  const int r = (int)(w % R);
  if (m >= M) return;
  const int id = ids[m];
  if (id < 0 || id >= adapters) {
    if (id != -1 && d_status && lane == 0) atomicOr(d_status, kDevBadAdapter);
    return;
  }
  const uint16_t *xr = x + m * K, *ar = A + ((int64_t)id * R + r) * K;
  float sum = 0.f;
  for (int k = lane; k < K; k += 64) sum += bf16_to_f32(xr[k]) * bf16_to_f32(ar[k]);
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) t[m * R + r] = sum;
}

}  // namespace

void launch_glu(const uint16_t *x, const uint8_t *pg, const uint16_t *sg, const uint8_t *pu,
                const uint16_t *su, int64_t M, int64_t N, int64_t K, int G, int act, uint16_t *h,
                void *workspace, int32_t *d_status, hipStream_t stream) {
  const dim3 grid((unsigned)((N + BN - 1) / BN), (unsigned)((M + BM - 1) / BM));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, x, pg, sg, pu, su, M, (int)N, (int)K,
                       nullptr, nullptr, nullptr, nullptr, 0, 0, h, d_status);
  };
  if (G == 64)
    act == kActSilu ? go(proj_kernel<64, 2, kActSilu>) : go(proj_kernel<64, 2, kActGelu>);
  else
    act == kActSilu ? go(proj_kernel<128, 2, kActSilu>) : go(proj_kernel<128, 2, kActGelu>);
}

void launch_lora(const uint16_t *x, const uint8_t *packed, const uint16_t *scales, int64_t M,
                 int64_t N, int64_t K, int G, const int32_t *ids, const uint16_t *a,
                 const uint16_t *b, const float *scaling, int adapters, int R, float *y,
                 void *workspace, int32_t *d_status, hipStream_t stream) {
  float *t = (float *)workspace;
  hipLaunchKernelGGL(shrink_kernel, dim3((unsigned)((M * R + 3) / 4)), dim3(256), 0, stream, x, M,
                     (int)K, ids, a, adapters, R, t, d_status);
  const dim3 grid((unsigned)((N + BN - 1) / BN), (unsigned)((M + BM - 1) / BM));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, x, packed, scales, nullptr, nullptr, M,
                       (int)N, (int)K, ids, t, b, scaling, adapters, R, y, d_status);
  };
  G == 64 ? go(proj_kernel<64, 1, kActSilu>) : go(proj_kernel<128, 1, kActSilu>);
}

int64_t glu_workspace(int64_t M, int64_t N, int64_t K, int G) { return 0; }

int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int G, int R) { return M * R * 4; }

}  // namespace tq

// tq_glu_train.hip -- the gated feed-forward block on bf16 weights, forward
// and backward (quantization-aware training: the weights are the bf16 w_hat
// of tq_fake_quantize, whose gradient is straight-through).
//
//   forward    g = x Wg^T, u = x Wu^T, h = act(g) u
//   backward   dg = dh u act'(g), du = dh act(g)
//              dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
//
// All four are the tile product of tq_mm.h with the operands as they lie in
// memory:
//   forward  P = gate and up rows side by side (a wave holds both of its
//            columns, so act(g) u is formed in registers), Q = x
//   dx       P = columns of Wg, then of Wu; Q = rows of [dg | du]; k = n
//   dW       P = columns of x, Q = columns of [dg | du]; k = m
// [dg | du] is made once by an elementwise pass, each half padded with zeros
// to a multiple of 64 columns.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tq_ffn.h"
#include "tq_internal.h"
#include "tq_mm.h"

namespace tq {
namespace {

constexpr int kFwd = 0, kDx = 1, kDw = 2;

struct TrainArgs {
  const uint16_t *p0, *p1;  // weights (kFwd, kDx) or x (kDw: p0)
  const uint16_t *q;        // x (kFwd), [dg | du] (kDx, kDw)
  uint16_t *o0, *o1, *o2;   // kFwd: h, g, u; kDx: dx; kDw: dwg, dwu
  float *partial;           // splits > 1: fp32 [split][rows of q][K]
  int64_t M;
  int N, K, Np;             // Np: columns of half of [dg | du]
  int tp, tq;               // tiles along p and q
  int stages, splits;       // stages of 32 k in all (even), and the blocks they are shared by
};

template <int MODE, int ACT, int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ)
__attribute__((amdgpu_waves_per_eu(2, 2))) void train_kernel(const TrainArgs A) {
  constexpr int NT = 64 * WP * WQ, TP = BP / WP / 16, TQ = BQ / WQ / 16;
  constexpr int PK = MODE == kFwd ? kRows : kCols, QK = MODE == kDw ? kCols : kRows;
  typedef Stream<PK, BP, NT> PS;
  typedef Stream<QK, BQ, NT> QS;
  constexpr uint32_t kQOff = kRing * PS::kSlot;
  __shared__ __align__(16) unsigned char smem_raw[kRing * (PS::kSlot + QS::kSlot)];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wv / WQ, wq = wv % WQ;

  int ip, iq;
  const int tiles = A.tp * A.tq, split = (int)blockIdx.x / tiles;
  tile_of_block((int)blockIdx.x - split * tiles, tiles, A.tp, A.tq, ip, iq);
  // this block's stages [s0, s1), an even number of them
  const int pairs = A.stages / 2;
  const int s0 = 2 * (int)((int64_t)pairs * split / A.splits);
  const int s1 = 2 * (int)((int64_t)pairs * (split + 1) / A.splits);

  PS ps;
  QS qs;
  constexpr int HP = BP / WP / 2;  // kFwd: gate (and up) columns of a wave
  const int n0 = ip * (BP / 2);    // kFwd: first column of the tile
  const int64_t q0 = (int64_t)iq * BQ;
  if constexpr (MODE == kFwd) {
    // slot row r: wave column r / 2HP, gate if (r % 2HP) < HP, else up
    ps.init_rows(tid, (uint32_t)A.K, [&](int r) -> int64_t {
      const int n = (r / (2 * HP)) * HP + r % HP;
      return n0 + n < A.N ? n : -1;
    });
  } else {
    ps.init_cols(tid, (uint32_t)A.K, A.K - ip * BP);
  }
  if constexpr (MODE == kDw)
    qs.init_cols(tid, (uint32_t)(2 * A.Np), 2 * A.Np - (int)q0);
  else
    qs.init_rows(tid, (uint32_t)(MODE == kFwd ? A.K : 2 * A.Np),
                 [&](int r) -> int64_t { return q0 + r < A.M ? r : -1; });

  const uint16_t *qbase = A.q + (MODE == kDw ? q0 : q0 * (MODE == kFwd ? A.K : 2 * A.Np));
  // The requests of one stage: L loads a thread, loads 0..1 of P then of Q.
  constexpr int L = PS::kLoads + QS::kLoads;
  struct Request {
    const uint16_t *p, *p_up, *q;  // kFwd: p holds gate rows, p_up up rows
    lds_bytes *pslot, *qslot;
    int prem, qrem;
  };
  int rslot = 0;  // slot of the next request; stage s0 is in slot 0
  auto request_of = [&](int s) {
    Request r;
    r.pslot = smem + (uint32_t)rslot * PS::kSlot;
    r.qslot = smem + kQOff + (uint32_t)rslot * QS::kSlot;
    rslot = next_slot(rslot);
    const bool in = s < s1;
    if constexpr (MODE == kFwd) {
      const int64_t k = (int64_t)s * kKS;
      r.p = A.p0 + (int64_t)n0 * A.K + k;
      r.p_up = A.p1 + (int64_t)n0 * A.K + k;
      r.q = qbase + k;
      r.prem = r.qrem = in ? 1 : 0;
    } else if constexpr (MODE == kDx) {
      const int half = A.Np / kKS, sn = s < half ? s : s - half;
      r.p = (s < half ? A.p0 : A.p1) + (int64_t)sn * kKS * A.K + ip * BP;
      r.q = qbase + (int64_t)s * kKS;
      r.prem = in ? A.N - sn * kKS : 0;
      r.qrem = in ? 1 : 0;
    } else {
      const int64_t m = (int64_t)s * kKS;
      r.p = A.p0 + m * A.K + ip * BP;
      r.q = qbase + m * (2 * A.Np);
      r.prem = r.qrem = !in ? 0 : A.M - m < kKS ? (int)(A.M - m) : kKS;
    }
    return r;
  };
  auto request = [&](const Request &r, int i) {
    if (i >= PS::kLoads) {
      qs.load(i - PS::kLoads, r.q, r.qslot, (uint32_t)wv, r.qrem);
    } else if constexpr (MODE == kFwd) {
      // the 64 lanes cover 16 slot rows, all gate or all up
      const bool gate = (i * NT + 64 * wv) / 4 % (2 * HP) < HP;
      ps.load(i, gate ? r.p : r.p_up, r.pslot, (uint32_t)wv, r.prem);
    } else {
      ps.load(i, r.p, r.pslot, (uint32_t)wv, r.prem);
    }
  };

  Frags<PK, BP, TP> pf;
  Frags<QK, BQ, TQ> qf;
  pf.init(lane, wp * (BP / WP));
  qf.init(lane, wq * (BQ / WQ));

  f32x4 acc[TP][TQ];
#pragma unroll
  for (int a = 0; a < TP; ++a)
#pragma unroll
    for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  static_assert(TP >= TQ && TP >= L, "rows of MFMAs to put the reads and requests between");
  bf16x8 pa[TP], qa[TQ], qb[TQ];
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) {
    const Request r = request_of(s0 + s);
#pragma unroll
    for (int i = 0; i < L; ++i) request(r, i);
  }
  static_assert(kRing == 5, "the waits count the loads of four stages in flight");
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(3 * L) : "memory");
#pragma unroll
  for (int b = 0; b < TQ; ++b) qa[b] = qf.read(smem, kQOff, b);
#pragma unroll
  for (int a = 0; a < TP; ++a) pa[a] = pf.read(smem, 0, a);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * L) : "memory");

  // Stage s: its fragments are pa and qc; those of s + 1 are read into pa (as
  // its blocks are used up) and qn.
  int fslot = 1;  // slot of stage s + 1
  auto stage = [&](int s, bf16x8(&qc)[TQ], bf16x8(&qn)[TQ]) {
    const uint32_t pn = (uint32_t)fslot * PS::kSlot;
    const uint32_t qn0 = kQOff + (uint32_t)fslot * QS::kSlot;
    fslot = next_slot(fslot);
    __builtin_amdgcn_sched_barrier(0);
    const Request r = request_of(s + kRing - 1);
#pragma unroll
    for (int a = 0; a < TP; ++a) {
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = mfma32<false>(pa[a], qc[b], acc[a][b]);
      if (a < TQ) qn[a] = qf.read(smem, qn0, a);
      pa[a] = pf.read(smem, pn, a);
      if (a < L) request(r, a);
    }
    order_stage<PK, QK, TP, TQ>();
    __builtin_amdgcn_sched_barrier(0);
    // stage s + 2 has landed when only the loads of s + 3 and s + 4 are out
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * L) : "memory");
  };
  for (int s = s0; s < s1; s += 2) {
    stage(s, qa, qb);
    stage(s + 1, qb, qa);
  }
  // no load may still be writing this block's LDS when it exits
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- epilogue: lane holds rows p = 16 a + 4 (lane / 16) + r, column
  // q = 16 b + lane % 16 ----
  const int lp = 4 * (lane >> 4);
  const int64_t lq = q0 + wq * (BQ / WQ) + (lane & 15);
  if constexpr (MODE == kFwd) {
#pragma unroll
    for (int b = 0; b < TQ; ++b) {
      const int64_t m = lq + 16 * b;
      if (m >= A.M) continue;
#pragma unroll
      for (int a = 0; a < TP / 2; ++a) {
        const int n = n0 + wp * HP + 16 * a + lp;
        const f32x4 g = acc[a][b], u = acc[a + TP / 2][b];
        f32x4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = act_value<ACT>(g[r]) * u[r];
        const int64_t o = m * A.N + n;
        if ((A.N & 3) == 0 && n < A.N) {  // four columns, 8-byte aligned
          store4(A.o0 + o, h);
          if (A.o1) {
            store4(A.o1 + o, g);
            store4(A.o2 + o, u);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (n + r >= A.N) continue;
            A.o0[o + r] = f32_to_bf16(h[r]);
            if (A.o1) {
              A.o1[o + r] = f32_to_bf16(g[r]);
              A.o2[o + r] = f32_to_bf16(u[r]);
            }
          }
        }
      }
    }
  } else {
    const int64_t rows = MODE == kDx ? A.M : 2 * (int64_t)A.Np;
#pragma unroll
    for (int b = 0; b < TQ; ++b) {
      const int64_t q = lq + 16 * b;
      if (q >= rows) continue;
      if (A.splits > 1) {
        float *o = A.partial + ((int64_t)split * rows + q) * A.K;
#pragma unroll
        for (int a = 0; a < TP; ++a) {
          const int p = ip * BP + wp * (BP / WP) + 16 * a + lp;
          if (p < A.K) *(f32x4 *)(o + p) = acc[a][b];
        }
        continue;
      }
      uint16_t *o;
      if constexpr (MODE == kDx) {
        o = A.o0 + q * A.K;
      } else {
        const bool up = q >= A.Np;
        const int64_t n = up ? q - A.Np : q;
        if (n >= A.N) continue;
        o = (up ? A.o1 : A.o0) + n * A.K;
      }
#pragma unroll
      for (int a = 0; a < TP; ++a) {
        const int p = ip * BP + wp * (BP / WP) + 16 * a + lp;
        if (p < A.K) store4(o + p, acc[a][b]);
      }
    }
  }
}

// Sum the splits' partial sums in order and round: rows of [rows, K], four
// columns a thread.  The rows of dW go to dwg and dwu.
__global__ __launch_bounds__(256) void reduce_kernel(const float *__restrict__ partial, int64_t rows,
                                                     int K, int splits, int Np, int N,
                                                     uint16_t *__restrict__ o0,
                                                     uint16_t *__restrict__ o1) {
  const int64_t n4 = rows * (K / 4);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    f32x4 v = *(const f32x4 *)(partial + 4 * i);
    for (int s = 1; s < splits; ++s) v += *(const f32x4 *)(partial + ((int64_t)s * n4 + i) * 4);
    if (!o1) {
      store4(o0 + 4 * i, v);
    } else {
      const int64_t q = i / (K / 4), p = 4 * (i - q * (K / 4));
      const bool up = q >= Np;
      const int64_t n = up ? q - Np : q;
      if (n < N) store4((up ? o1 : o0) + n * K + p, v);
    }
  }
}

// [dg | du], each rounded once to bf16 (the type the matrix cores take); the
// columns past N of each half are zeros.  Eight columns a thread; VEC: N % 8
// == 0, so the inputs' eight are one aligned load.
template <int ACT, bool VEC>
__global__ __launch_bounds__(256) void gate_grad_kernel(const uint16_t *__restrict__ dh,
                                                        const uint16_t *__restrict__ g,
                                                        const uint16_t *__restrict__ u, int64_t M,
                                                        int N, int Np, uint16_t *__restrict__ out) {
  const int64_t per = Np / 8, total = M * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per, o = m * N;
    const int n = 8 * (int)(i - m * per);
    uint16_t d[8], gv[8], uv[8], dg[8], du[8];
    if (VEC && n < N) {
      *(u32x4 *)d = *(const u32x4 *)(dh + o + n);
      *(u32x4 *)gv = *(const u32x4 *)(g + o + n);
      *(u32x4 *)uv = *(const u32x4 *)(u + o + n);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = n + j < N;
        d[j] = in ? dh[o + n + j] : 0;
        gv[j] = in ? g[o + n + j] : 0;
        uv[j] = in ? u[o + n + j] : 0;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float value, slope;
      const float f = bf16_to_f32(d[j]);
      act_and_slope<ACT>(bf16_to_f32(gv[j]), value, slope);
      dg[j] = f32_to_bf16(f * bf16_to_f32(uv[j]) * slope);
      du[j] = f32_to_bf16(f * value);
    }
    *(u32x4 *)(out + m * (2 * Np) + n) = *(u32x4 *)dg;
    *(u32x4 *)(out + m * (2 * Np) + Np + n) = *(u32x4 *)du;
  }
}

// Tile size and k split of one product of p x q outputs.
struct Plan {
  bool big;
  int tp, tq, splits;
};

Plan plan_of(int64_t p, int64_t q, int stages, bool may_split) {
  auto up = [](int64_t a, int64_t b) { return (int)((a + b - 1) / b); };
  Plan r;
  r.tp = up(p, 256), r.tq = up(q, 256), r.splits = 1;
  r.big = (int64_t)r.tp * r.tq >= 192;
  if (r.big) return r;
  r.tp = up(p, 128), r.tq = up(q, 128);
  const int tiles = r.tp * r.tq, most = stages / 16;
  if (may_split && tiles > 0 && tiles <= 256 && most > 1) r.splits = std::min(512 / tiles, most);
  return r;
}

int pad64(int64_t n) { return (int)((n + 63) / 64 * 64); }
int even_stages(int64_t k) { return 2 * (int)((k + 2 * kKS - 1) / (2 * kKS)); }

template <int MODE, int ACT>
void launch_product(const TrainArgs &a, bool big, hipStream_t stream) {
  const dim3 grid((unsigned)(a.tp * a.tq * a.splits));
  if (big)
    hipLaunchKernelGGL((train_kernel<MODE, ACT, 256, 256, 2, 4>), grid, dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((train_kernel<MODE, ACT, 128, 128, 2, 2>), grid, dim3(256), 0, stream, a);
}

struct BackwardPlan {
  Plan dx, dw;
  int Np, sx, sw;          // stages
  int64_t gates, partial;  // workspace bytes: [dg | du], then the larger partial array
};

BackwardPlan plan_backward(int64_t M, int64_t N, int64_t K) {
  BackwardPlan b;
  b.Np = pad64(N);
  b.sx = 2 * b.Np / kKS;
  b.sw = even_stages(M);
  b.dx = plan_of(K, M, b.sx, true);
  b.dw = plan_of(K, 2 * (int64_t)b.Np, b.sw, true);
  b.gates = M * 4 * b.Np;
  const int64_t px = b.dx.splits > 1 ? b.dx.splits * M * K * 4 : 0;
  const int64_t pw = b.dw.splits > 1 ? b.dw.splits * 2 * (int64_t)b.Np * K * 4 : 0;
  b.partial = px > pw ? px : pw;
  return b;
}

}  // namespace

void launch_glu_forward(const uint16_t *x, const uint16_t *wg, const uint16_t *wu, int64_t M,
                        int64_t N, int64_t K, int act, uint16_t *h, uint16_t *g, uint16_t *u,
                        hipStream_t stream) {
  const Plan p = plan_of(2 * N, M, (int)(K / kKS), false);
  TrainArgs a{};
  a.p0 = wg, a.p1 = wu, a.q = x, a.o0 = h, a.o1 = g, a.o2 = u;
  a.M = M, a.N = (int)N, a.K = (int)K;
  a.tp = p.tp, a.tq = p.tq, a.stages = (int)(K / kKS), a.splits = 1;
  if (act == kActSilu)
    launch_product<kFwd, kActSilu>(a, p.big, stream);
  else
    launch_product<kFwd, kActGelu>(a, p.big, stream);
}

int64_t glu_backward_workspace(int64_t M, int64_t N, int64_t K) {
  const BackwardPlan b = plan_backward(M, N, K);
  return b.gates + b.partial;
}

void launch_glu_backward(const uint16_t *dh, const uint16_t *x, const uint16_t *wg,
                         const uint16_t *wu, const uint16_t *g, const uint16_t *u, int64_t M,
                         int64_t N, int64_t K, int act, uint16_t *dx, uint16_t *dwg, uint16_t *dwu,
                         void *workspace, hipStream_t stream) {
  const BackwardPlan b = plan_backward(M, N, K);
  uint16_t *gates = (uint16_t *)workspace;
  TrainArgs a{};
  a.q = gates;
  a.partial = (float *)((char *)workspace + b.gates);
  a.M = M, a.N = (int)N, a.K = (int)K, a.Np = b.Np;
  auto blocks = [](int64_t threads) {
    const int64_t n = (threads + 255) / 256;
    return dim3((unsigned)(n < 8192 ? n : 8192));
  };
  if (M > 0) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, blocks(M * (b.Np / 8)), dim3(256), 0, stream, dh, g, u, M, (int)N,
                         b.Np, gates);
    };
    if (N % 8 == 0)
      act == kActSilu ? go(gate_grad_kernel<kActSilu, true>) : go(gate_grad_kernel<kActGelu, true>);
    else
      act == kActSilu ? go(gate_grad_kernel<kActSilu, false>) : go(gate_grad_kernel<kActGelu, false>);
    a.p0 = wg, a.p1 = wu, a.o0 = dx;
    a.tp = b.dx.tp, a.tq = b.dx.tq, a.stages = b.sx, a.splits = b.dx.splits;
    launch_product<kDx, kActSilu>(a, b.dx.big, stream);
    if (a.splits > 1)
      hipLaunchKernelGGL(reduce_kernel, blocks(M * (K / 4)), dim3(256), 0, stream, a.partial, M,
                         (int)K, a.splits, 0, 0, dx, nullptr);
  }
  a.p0 = x, a.p1 = nullptr, a.o0 = dwg, a.o1 = dwu;
  a.tp = b.dw.tp, a.tq = b.dw.tq, a.stages = b.sw, a.splits = b.dw.splits;
  launch_product<kDw, kActSilu>(a, b.dw.big, stream);
  if (a.splits > 1)
    hipLaunchKernelGGL(reduce_kernel, blocks(2 * (int64_t)b.Np * (K / 4)), dim3(256), 0, stream,
                       a.partial, 2 * (int64_t)b.Np, (int)K, a.splits, b.Np, (int)N, dwg, dwu);
}

}  // namespace tq

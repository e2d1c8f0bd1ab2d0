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
  int blocks;               // blocks of the launch that work on this product
};

// One tile of one split of K.
struct Item {
  int ip, iq, split, s0, s1;  // stages [s0, s1), an even number
};

__device__ __forceinline__ Item item_of(const TrainArgs &A, int w) {
  Item r;
  const int tiles = A.tp * A.tq, pairs = A.stages / 2;
  const int split = w / tiles;
  int ip, iq;
  tile_of_block(w - split * tiles, tiles, A.tp, A.tq, ip, iq);
  // the same for the wave: kept in scalar registers, as load addresses need
  r.split = __builtin_amdgcn_readfirstlane(split);
  r.ip = __builtin_amdgcn_readfirstlane(ip);
  r.iq = __builtin_amdgcn_readfirstlane(iq);
  r.s0 = __builtin_amdgcn_readfirstlane(2 * (pairs * split / A.splits));
  r.s1 = __builtin_amdgcn_readfirstlane(2 * (pairs * (split + 1) / A.splits));
  return r;
}

// Persistent blocks: block b of `grid` computes items b, b + grid, ...  The
// requests run on across items, so an item's first stages load while the one before is
// multiplied and stored, and the stores of one drain under the next.  (A block
// an item cost 12 to 16 us an item beside its stages, most of it stores.)
template <int MODE, int ACT, int BP, int BQ, int WP, int WQ>
__device__ __forceinline__ void product(const TrainArgs &A, int block, int grid, lds_bytes *smem) {
  constexpr int NT = 64 * WP * WQ, TP = BP / WP / 16, TQ = BQ / WQ / 16;
  constexpr int PK = MODE == kFwd ? kRows : kCols, QK = MODE == kDw ? kCols : kRows;
  typedef Stream<PK, BP, NT> PS;
  typedef Stream<QK, BQ, NT> QS;
  constexpr uint32_t kQOff = kRing * PS::kSlot;
  constexpr int L = PS::kLoads + QS::kLoads;  // loads a thread and stage: P's, then Q's
  static_assert(2 * TQ % TP == 0 && TP >= L, "rows of MFMAs to put the reads and requests between");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wv / WQ, wq = wv % WQ;
  constexpr int HP = BP / WP / 2;  // kFwd: gate (and up) columns of a wave
  const int total = A.tp * A.tq * A.splits;

  // ---- requests ----
  PS ps;
  QS qs;
  Item rq;                              // item of the next request
  int rw = block, rs = 0;               // its index; stage
  const uint16_t *rp0, *rp1, *rqb;      // its operands at k = 0: P (kDx: of the first and the
                                        // second half of k; kFwd: gate and up), Q
  auto open = [&]() {
    rq = item_of(A, rw);
    rs = rq.s0;
    const int64_t q0 = (int64_t)rq.iq * BQ;
    if constexpr (MODE == kFwd) {
      const int n0 = rq.ip * (BP / 2);
      // slot row r: wave column r / 2HP, gate if (r % 2HP) < HP, else up
      ps.init_rows(tid, (uint32_t)A.K, [&](int r) -> int64_t {
        const int n = (r / (2 * HP)) * HP + r % HP;
        return n0 + n < A.N ? n : -1;
      });
      rp0 = A.p0 + (int64_t)n0 * A.K;
      rp1 = A.p1 + (int64_t)n0 * A.K;
    } else {
      ps.init_cols(tid, (uint32_t)A.K, A.K - rq.ip * BP);
      rp0 = A.p0 + rq.ip * BP;
      rp1 = A.p1 + rq.ip * BP;
    }
    if constexpr (MODE == kDw) {
      qs.init_cols(tid, (uint32_t)(2 * A.Np), 2 * A.Np - (int)q0);
      rqb = A.q + q0;
    } else {
      const int64_t ld = MODE == kFwd ? A.K : 2 * A.Np;
      qs.init_rows(tid, (uint32_t)ld, [&](int r) -> int64_t { return q0 + r < A.M ? r : -1; });
      rqb = A.q + q0 * ld;
    }
  };
  struct Request {
    const uint16_t *p, *p_up, *q;  // kFwd: p holds gate rows, p_up up rows
    lds_bytes *pslot, *qslot;
    int prem, qrem;
  };
  int rslot = 0;  // slot of the next request; the first item's first stage is in slot 0
  auto request_of = [&]() {
    Request r;
    r.pslot = smem + (uint32_t)rslot * PS::kSlot;
    r.qslot = smem + kQOff + (uint32_t)rslot * QS::kSlot;
    rslot = next_slot(rslot);
    const bool in = rw < total;  // past the last item: zeros that nothing uses
    if constexpr (MODE == kFwd) {
      const int64_t k = (int64_t)rs * kKS;
      r.p = rp0 + k;
      r.p_up = rp1 + k;
      r.q = rqb + k;
      r.prem = r.qrem = in ? 1 : 0;
    } else if constexpr (MODE == kDx) {
      const int half = A.Np / kKS, sn = rs < half ? rs : rs - half;
      r.p = (rs < half ? rp0 : rp1) + (int64_t)sn * kKS * A.K;
      r.q = rqb + (int64_t)rs * kKS;
      r.prem = in ? A.N - sn * kKS : 0;
      r.qrem = in ? 1 : 0;
    } else {
      const int64_t m = (int64_t)rs * kKS;
      r.p = rp0 + m * A.K;
      r.q = rqb + m * (2 * A.Np);
      r.prem = r.qrem = !in ? 0 : A.M - m < kKS ? (int)(A.M - m) : kKS;
    }
    ++rs;
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
  auto advance = [&]() {  // to the next item after an item's last request
    if (rs == rq.s1 && rw < total) {
      rw += grid;
      if (rw < total) open();
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
  bf16x8 pa[TP], qa[TQ], qb[TQ];
  open();
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) {
    const Request r = request_of();
#pragma unroll
    for (int i = 0; i < L; ++i) request(r, i);
    advance();
  }
  static_assert(kRing == 5, "the waits count the loads of four stages in flight");
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(3 * L) : "memory");
#pragma unroll
  for (int b = 0; b < TQ; ++b) qa[b] = qf.read(smem, kQOff, b);
#pragma unroll
  for (int a = 0; a < TP; ++a) pa[a] = pf.read(smem, 0, a);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * L) : "memory");

  // A stage: its fragments are pa and qc; those of the next are read into pa
  // (as its blocks are used up) and qn.  `stores`: how many stores at least
  // were issued between the requests of the two stages before the last two and
  // those of the last two.
  int fslot = 1;  // slot of the next stage
  auto stage = [&](bf16x8(&qc)[TQ], bf16x8(&qn)[TQ], int stores) {
    const uint32_t pn = (uint32_t)fslot * PS::kSlot;
    const uint32_t qn0 = kQOff + (uint32_t)fslot * QS::kSlot;
    fslot = next_slot(fslot);
    __builtin_amdgcn_sched_barrier(0);
    const Request r = request_of();
#pragma unroll
    for (int a = 0; a < TP; ++a) {
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = mfma32<false>(pa[a], qc[b], acc[a][b]);
      constexpr int R = 2 * TQ / TP;  // Q's fragments in the first half of the rows
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (R * a + i < TQ) qn[R * a + i] = qf.read(smem, qn0, R * a + i);
      pa[a] = pf.read(smem, pn, a);
      if (a < L) request(r, a);
    }
    order_stage<PK, QK, TP, TQ>();
    __builtin_amdgcn_sched_barrier(0);
    // Stage s + 2 has landed when only the loads of s + 3 and s + 4 are out,
    // and the stores issued after its own.
    if (stores >= 16)
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * L + 16) : "memory");
    else if (stores >= 8)
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * L + 8) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2 * L) : "memory");
    advance();
  };

  const int h = lane >> 4, l = lane & 15;
  const int p8 = pack8_row(lane);
  // All of a wave's columns and rows are inside and aligned: returns the
  // number of stores issued, which every such wave issues alike; else 0.
  auto store = [&](const Item &t) -> int {
    const int64_t q0 = (int64_t)t.iq * BQ + wq * (BQ / WQ);
    const bool rows_in = q0 + BQ / WQ <= (MODE == kDw ? 2 * (int64_t)A.Np : A.M);
    if constexpr (MODE == kFwd) {
      static_assert(TP / 2 % 2 == 0, "pairs of tiles");
      const int n0 = t.ip * (BP / 2) + wp * HP;
      const bool full = rows_in && n0 + HP <= A.N && (A.N & 7) == 0;
#pragma unroll
      for (int b = 0; b < TQ; ++b) {
        const int64_t m = q0 + 16 * b + l;
        f32x4 hv[TP / 2];
#pragma unroll
        for (int a = 0; a < TP / 2; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) hv[a][r] = act_value<ACT>(acc[a][b][r]) * acc[a + TP / 2][b][r];
        if (full) {
#pragma unroll
          for (int a = 0; a < TP / 2; a += 2) {
            const int64_t o = m * A.N + n0 + 16 * a + p8;
            *(u32x4 *)(A.o0 + o) = pack8(hv[a], hv[a + 1]);
            if (A.o1) {
              *(u32x4 *)(A.o1 + o) = pack8(acc[a][b], acc[a + 1][b]);
              *(u32x4 *)(A.o2 + o) = pack8(acc[a + TP / 2][b], acc[a + 1 + TP / 2][b]);
            }
          }
        } else if (m < A.M) {
#pragma unroll
          for (int a = 0; a < TP / 2; ++a)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int n = n0 + 16 * a + 4 * h + r;
              if (n >= A.N) continue;
              const int64_t o = m * A.N + n;
              A.o0[o] = f32_to_bf16(hv[a][r]);
              if (A.o1) {
                A.o1[o] = f32_to_bf16(acc[a][b][r]);
                A.o2[o] = f32_to_bf16(acc[a + TP / 2][b][r]);
              }
            }
        }
      }
      return full ? TQ * (TP / 4) : 0;  // h alone; more with g and u
    } else {
      const int64_t rows = MODE == kDw ? 2 * (int64_t)A.Np : A.M;
      const int p0 = t.ip * BP + wp * (BP / WP);
      const bool full = rows_in && p0 + BP / WP <= A.K && (MODE == kDx || A.N == A.Np);
#pragma unroll
      for (int b = 0; b < TQ; ++b) {
        const int64_t q = q0 + 16 * b + l;
        if (!full && q >= rows) continue;
        if (A.splits > 1) {
          float *o = A.partial + ((int64_t)t.split * rows + q) * A.K + p0;
#pragma unroll
          for (int a = 0; a < TP; ++a)
            if (full || p0 + 16 * a < A.K) *(f32x4 *)(o + 16 * a + 4 * h) = acc[a][b];
          continue;
        }
        uint16_t *o;
        if constexpr (MODE == kDx) {
          o = A.o0 + q * A.K + p0;
        } else {
          const bool up = q >= A.Np;
          const int64_t n = up ? q - A.Np : q;
          if (!full && n >= A.N) continue;
          o = (up ? A.o1 : A.o0) + n * A.K + p0;
        }
#pragma unroll
        for (int a = 0; a < TP; a += 2)
          if (full || p0 + 16 * a < A.K)  // K % 64 == 0: both tiles or neither
            *(u32x4 *)(o + 16 * a + p8) = pack8(acc[a][b], acc[a + 1][b]);
      }
      return full ? TQ * (TP / 2) : 0;
    }
  };

  int stores = 0;
  for (int w = block; w < total; w += grid) {
    const Item t = item_of(A, w);
    for (int s = t.s0; s < t.s1; s += 2) {
      stage(qa, qb, stores);
      stage(qb, qa, stores);
      stores = 0;
    }
    stores = store(t);
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // no load may still be writing this block's LDS when it exits
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

constexpr int lds_of(int BP, int BQ) { return kRing * kKS * 2 * (BP + BQ); }

// 4096 rows by 2 x [3584,1024]: 63 us, 0.95 PFLOP/s; 1.75 tiles a CU and 88 MB
// of results (17 us at copy rate) beside 41 us of multiplying at a library's rate.
template <int ACT, int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ)
__attribute__((amdgpu_waves_per_eu(2, 2))) void forward_kernel(const TrainArgs A) {
  __shared__ __align__(16) unsigned char smem[lds_of(BP, BQ)];
  product<kFwd, ACT, BP, BQ, WP, WQ>(A, (int)blockIdx.x, A.blocks, (lds_bytes *)smem);
}

// dW, dx, or both side by side, each on its share of the chip: alone, either
// may leave CUs idle in its last round or have to split K, whose sums cross
// memory twice.  4096 rows, [3584,1024]: 110 us side by side, 1.09 PFLOP/s; 2048
// rows, [14336,4096]: 374 us each, 1.29 PFLOP/s (a
// library's product of such a size 1.44).
template <int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ)
__attribute__((amdgpu_waves_per_eu(2, 2))) void backward_kernel(const TrainArgs W, const TrainArgs X) {
  __shared__ __align__(16) unsigned char smem[lds_of(BP, BQ)];
  if ((int)blockIdx.x < W.blocks)
    product<kDw, kActSilu, BP, BQ, WP, WQ>(W, (int)blockIdx.x, W.blocks, (lds_bytes *)smem);
  else
    product<kDx, kActSilu, BP, BQ, WP, WQ>(X, (int)blockIdx.x - W.blocks, X.blocks, (lds_bytes *)smem);
}

// Sum a product's splits in order and round, four columns a thread; dW's rows
// go to dwg and dwu.
template <int MODE>
__device__ __forceinline__ void reduce_product(const TrainArgs &A, int64_t first, int64_t stride) {
  const int64_t rows = MODE == kDx ? A.M : 2 * (int64_t)A.Np, n4 = rows * (A.K / 4);
  for (int64_t i = first; i < n4; i += stride) {
    f32x4 v = *(const f32x4 *)(A.partial + 4 * i);
    for (int s = 1; s < A.splits; ++s) v += *(const f32x4 *)(A.partial + ((int64_t)s * n4 + i) * 4);
    if constexpr (MODE == kDx) {
      store4(A.o0 + 4 * i, v);
    } else {
      const int64_t q = i / (A.K / 4), p = 4 * (i - q * (A.K / 4));
      const bool up = q >= A.Np;
      const int64_t n = up ? q - A.Np : q;
      if (n < A.N) store4((up ? A.o1 : A.o0) + n * A.K + p, v);
    }
  }
}

// The products whose K is split, W's on the first `w_blocks` blocks.
__global__ __launch_bounds__(256) void reduce_kernel(const TrainArgs W, const TrainArgs X, int w_blocks) {
  const int b = (int)blockIdx.x;
  if (b < w_blocks)
    reduce_product<kDw>(W, (int64_t)b * 256 + threadIdx.x, (int64_t)w_blocks * 256);
  else
    reduce_product<kDx>(X, (int64_t)(b - w_blocks) * 256 + threadIdx.x,
                        (int64_t)((int)gridDim.x - w_blocks) * 256);
}

// [dg | du], each rounded once to bf16, the type the matrix cores take: it is
// all that a gradient loses beside its own rounding (error 0.0023 in root mean
// square, where that rounding alone makes 0.0017).  With a second bf16 piece of
// each multiplied too the error was 0.0017, and the matrix cores' work twice as
// much: 4096 rows of [3584,1024] 269 us instead of 148, 2048 rows of
// [14336,4096] 1631 instead of 842.
// The columns past N of each half are zeros.  Eight columns a thread; VEC: N % 8
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

// Microseconds by measured rates.  A stage of a 256 x 256 tile takes a CU 0.78
// us, one of two 128 x 128 tiles side by side 0.60 us (half the work), one of
// such a tile alone 0.40 us; an item costs 4 us more than its stages; split
// sums cross memory twice at about 4 TB/s, in a launch of 4 us; two products
// side by side find less of their operands in the L2s and take 8% longer.
struct Rates {
  int size, slots;  // tile, and how many the chip works on at once
  double stage, alone;
};
constexpr Rates kRates[2] = {{256, 256, 0.78, 0.78}, {128, 512, 0.60, 0.40}};
constexpr double kItem = 4.0, kLaunch = 4.0, kPartialBytesPerUs = 4e6, kJoint = 1.08;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One product of p x q outputs: its tiles, split `splits` ways on `slots`.
struct Tiling {
  int tp, tq, splits, blocks;
};
Tiling tiling_of(const Rates &r, int64_t p, int64_t q, int splits, int64_t slots) {
  const int64_t tp = ceil_div(p, r.size), tq = ceil_div(q, r.size);
  return Tiling{(int)tp, (int)tq, splits, (int)std::min(slots, tp * tq * splits)};
}
double product_us(const Rates &r, int64_t p, int64_t q, int stages, int splits, int64_t slots) {
  const int64_t items = ceil_div(p, r.size) * ceil_div(q, r.size) * splits;
  const double stage = 2 * items <= slots ? r.alone : r.stage;
  return (double)ceil_div(items, slots) * ((double)stages / splits * stage + kItem);
}
double partial_us(int64_t p, int64_t q, int splits) {
  return splits > 1 ? 8.0 * (double)p * (double)q * splits / kPartialBytesPerUs : 0.0;
}

int pad64(int64_t n) { return (int)((n + 63) / 64 * 64); }
// At least one pair: of no rows it adds zeros.
int even_stages(int64_t k) { return k ? 2 * (int)((k + 2 * kKS - 1) / (2 * kKS)) : 2; }

void set_tiling(TrainArgs &a, const Tiling &t, int stages) {
  a.tp = t.tp, a.tq = t.tq, a.splits = t.splits, a.blocks = t.blocks, a.stages = stages;
}

struct BackwardPlan {
  bool big, joint;
  Tiling w, x;
  int Np, sw, sx;                      // stages
  int64_t gates, partial_w, partial_x;  // workspace bytes: [dg | du], then the partial sums
};

// dW and dx one after the other on the whole chip, or side by side on shares
// of it (in eights, one an XCD): tile size, shares and splits that take least.
BackwardPlan plan_backward(int64_t M, int64_t N, int64_t K) {
  BackwardPlan b{};
  b.Np = pad64(N);
  b.sx = 2 * b.Np / kKS;
  b.sw = even_stages(M);
  b.gates = M * 4 * b.Np;
  const int64_t qw = 2 * (int64_t)b.Np;
  double least = 1e30;
  auto look = [&](int i, bool joint, int64_t cw, int64_t cx) {
    const Rates &r = kRates[i];
    for (int sw = 1; sw <= 16 && (sw == 1 || b.sw / sw >= 8); sw *= 2) {
      const double w = product_us(r, K, qw, b.sw, sw, cw), pw = partial_us(K, qw, sw);
      for (int sx = 1; sx <= 16 && (sx == 1 || b.sx / sx >= 8); sx *= 2) {
        const double x = M ? product_us(r, K, M, b.sx, sx, cx) : 0.0;
        const double us = (joint ? kJoint * std::max(w, x) : w + x + kLaunch) + pw + partial_us(K, M, sx) +
                          (sw > 1 || sx > 1 ? kLaunch : 0.0);
        if (us < least) {
          least = us;
          b.big = i == 0, b.joint = joint;
          b.w = tiling_of(r, K, qw, sw, cw);
          b.x = tiling_of(r, K, M, sx, cx);
        }
      }
    }
  };
  for (int i = 0; i < 2; ++i) {
    const Rates &r = kRates[i];
    look(i, false, r.slots, r.slots);
    const double work_w = (double)ceil_div(qw, r.size) * b.sw, work_x = (double)ceil_div(M, r.size) * b.sx;
    const int eights = r.slots / 8, share = (int)(eights * work_w / (work_w + work_x) + 0.5);
    for (int e = std::max(share - 1, 1); M && e <= std::min(share + 1, eights - 1); ++e)
      look(i, true, 8 * e, r.slots - 8 * e);
  }
  b.partial_w = b.w.splits > 1 ? b.w.splits * qw * K * 4 : 0;
  b.partial_x = b.x.splits > 1 ? b.x.splits * M * K * 4 : 0;
  return b;
}

// 256 x 256 tiles unless the smaller ones fill the chip better.
bool forward_big(int64_t M, int64_t N, int stages) {
  return product_us(kRates[0], 2 * N, M, stages, 1, kRates[0].slots) <=
         product_us(kRates[1], 2 * N, M, stages, 1, kRates[1].slots);
}

}  // namespace

void train_plan(int64_t M, int64_t N, int64_t K, int64_t *plan) {
  const BackwardPlan b = plan_backward(M, N, K);
  plan[0] = kRates[forward_big(M, N, (int)(K / kKS)) ? 0 : 1].size;
  plan[1] = kRates[b.big ? 0 : 1].size, plan[2] = b.joint;
  plan[3] = b.w.splits, plan[4] = b.x.splits;
}

void launch_glu_forward(const uint16_t *x, const uint16_t *wg, const uint16_t *wu, int64_t M,
                        int64_t N, int64_t K, int act, uint16_t *h, uint16_t *g, uint16_t *u,
                        hipStream_t stream) {
  const int stages = (int)(K / kKS);
  const bool big = forward_big(M, N, stages);
  const Rates &r = kRates[big ? 0 : 1];
  TrainArgs a{};
  a.p0 = wg, a.p1 = wu, a.q = x, a.o0 = h, a.o1 = g, a.o2 = u;
  a.M = M, a.N = (int)N, a.K = (int)K;
  set_tiling(a, tiling_of(r, 2 * N, M, 1, r.slots), stages);
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)a.blocks), dim3(threads), 0, stream, a);
  };
  if (act == kActSilu)
    big ? go(forward_kernel<kActSilu, 256, 256, 4, 2>, 512) : go(forward_kernel<kActSilu, 128, 128, 2, 2>, 256);
  else
    big ? go(forward_kernel<kActGelu, 256, 256, 4, 2>, 512) : go(forward_kernel<kActGelu, 128, 128, 2, 2>, 256);
}

int64_t glu_backward_workspace(int64_t M, int64_t N, int64_t K) {
  const BackwardPlan b = plan_backward(M, N, K);
  return b.gates + b.partial_w + b.partial_x;
}

void launch_glu_backward(const uint16_t *dh, const uint16_t *x, const uint16_t *wg,
                         const uint16_t *wu, const uint16_t *g, const uint16_t *u, int64_t M,
                         int64_t N, int64_t K, int act, uint16_t *dx, uint16_t *dwg, uint16_t *dwu,
                         void *workspace, hipStream_t stream) {
  const BackwardPlan b = plan_backward(M, N, K);
  uint16_t *gates = (uint16_t *)workspace;
  TrainArgs w{}, v{};  // dW, dx
  w.p0 = x, w.q = gates, w.o0 = dwg, w.o1 = dwu;
  v.p0 = wg, v.p1 = wu, v.q = gates, v.o0 = dx;
  w.M = v.M = M, w.N = v.N = (int)N, w.K = v.K = (int)K, w.Np = v.Np = b.Np;
  w.partial = (float *)((char *)workspace + b.gates);
  v.partial = (float *)((char *)workspace + b.gates + b.partial_w);
  set_tiling(w, b.w, b.sw);
  set_tiling(v, b.x, b.sx);
  auto blocks = [](int64_t threads) { return (unsigned)std::min<int64_t>(8192, ceil_div(threads, 256)); };
  if (M > 0) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(blocks(M * (b.Np / 8))), dim3(256), 0, stream, dh, g, u, M, (int)N,
                         b.Np, gates);
    };
    if (N % 8 == 0)
      act == kActSilu ? go(gate_grad_kernel<kActSilu, true>) : go(gate_grad_kernel<kActGelu, true>);
    else
      act == kActSilu ? go(gate_grad_kernel<kActSilu, false>) : go(gate_grad_kernel<kActGelu, false>);
  }
  auto products = [&](TrainArgs pw, TrainArgs px) {
    const dim3 grid((unsigned)(pw.blocks + px.blocks));
    if (grid.x == 0) return;
    if (b.big)
      hipLaunchKernelGGL((backward_kernel<256, 256, 4, 2>), grid, dim3(512), 0, stream, pw, px);
    else
      hipLaunchKernelGGL((backward_kernel<128, 128, 2, 2>), grid, dim3(256), 0, stream, pw, px);
  };
  if (b.joint) {
    products(w, v);
  } else {
    TrainArgs none{};
    products(w, none);
    products(none, v);
  }
  const unsigned rw = w.splits > 1 ? blocks(2 * (int64_t)b.Np * (K / 4)) : 0;
  const unsigned rx = v.splits > 1 ? blocks(M * (K / 4)) : 0;
  if (rw + rx > 0)
    hipLaunchKernelGGL(reduce_kernel, dim3(rw + rx), dim3(256), 0, stream, w, v, (int)rw);
}

}  // namespace tq

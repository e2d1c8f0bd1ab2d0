// tq_glu.hip -- the packed-ternary projections behind tq_glu and
// tq_lora_matmul: one or two weight matrices against the same activations,
// with the epilogue that makes the operator.
//
//   P_i[m,n] = sum_g s_i[n,g] * sum_{j<G} x[m, gG+j] * c_i[n, gG+j]
//   glu:   h = bf16(act(P_0) * P_1)
//   lora:  y = P_0 + sum_r t[m,r] * B_a[n,r],  t[m,r] = scaling_a * sum_k x[m,k] A_a[r,k],
//          a = ids[m]; an id of -1 adds nothing.
//
// A sum over k may take its terms in any order, and base-3 bytes hold five
// codes, which no matrix operand's eight divides into.  So the codes of a
// group go to the matrix cores in the order in which whole bytes yield them
// (five of each byte, and the few of the last byte or two shared out), and x
// is put into the same order once, by whoever reads it (tq_ternary.h).
//
// Two kernels multiply:
//   dec_kernel    few rows: every packed byte is decoded in registers by the
//                 lane that feeds it to the matrix cores; the waves of a block
//                 share the groups of the same 16 or 32 weight rows.
//   wide_kernel   many rows: 256 x 256 tiles (tq_mm.h); each block decodes its
//                 weight rows into LDS, where 256 rows of x use them.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tq_ffn.h"
#include "tq_internal.h"
#include "tq_mm.h"
#include "tq_ternary.h"

namespace tq {
namespace {

// What both kernels read and write.
struct ProjArgs {
  const uint16_t *x;              // bf16 [M,K] (staged), or x in fragment order, or f16 rows
  const uint8_t *packed[2];
  const uint16_t *scales[2];
  const int32_t *shift;           // wide: x of row m is stored times 2^shift[m]
  const int32_t *ids;             // lora
  const float *t;                 // lora: [M,R] fp32, scaled
  const uint16_t *b;              // lora: [adapters,N,R]
  int adapters, R;
  void *out;                      // bf16 [M,N] (glu) or fp32 [M,N] (lora)
  float *partial;                 // splits > 1: fp32 [split][NB][M][N]
  int64_t M;
  int N, K;
  int splits, chunks;             // dec: blocks along K, and chunks of rows
  int tp, tq;                     // wide: tiles
  int32_t *status;
};

// ---------------------------------------------------------------------------
// adapters
// ---------------------------------------------------------------------------

// The distinct adapters among the ids that a wave's lanes hold, as a mask of
// the first lane of each.
__device__ __forceinline__ uint64_t adapter_leaders(int id, int lane) {
  bool first = id >= 0;
  for (int j = 0; j < 63; ++j) {
    const int other = __builtin_amdgcn_readlane(id, j);
    if (j < lane && other == id) first = false;
  }
  return __ballot(first);
}

// A row's t in three bf16 pieces (24 bits together): eight ranks of it.
struct Pieces {
  bf16x8 p[3];
};
__device__ __forceinline__ Pieces split_t(const float *t, bool in) {
  Pieces r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = in ? t[i] : 0.f;
    const __bf16 a = (__bf16)v;
    const float ra = v - (float)a;
    const __bf16 b = (__bf16)ra;
    r.p[0][i] = a;
    r.p[1][i] = b;
    r.p[2][i] = (__bf16)(ra - (float)b);
  }
  return r;
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

constexpr int kDecWaves = 8, kDecThreads = 64 * kDecWaves;
constexpr int kStagedRows = 4;            // rows of x a block puts in order itself
constexpr uint32_t kStagedBytes = 48 << 10;  // and the LDS for them

// One lane's bytes of one group of one weight row.
struct Raw {
  uint32_t w0, w1, tail, scale;
};

template <int G>
__device__ __forceinline__ Raw load_raw(const uint8_t *row, const uint16_t *srow, int g, int q) {
  Raw r;
  const uint8_t *p = row + (int64_t)g * bytes_per_group(G);
  if constexpr (G == 128) {
    uint64_t w;
    uint16_t tail;
    __builtin_memcpy(&w, p + 6 * q, 8);  // six bytes of it; q = 3 ends at the group's end
    __builtin_memcpy(&tail, p + 24, 2);
    r.w0 = (uint32_t)w;
    r.w1 = (uint32_t)(w >> 32);
    r.tail = tail;
  } else {
    __builtin_memcpy(&r.w0, p + 3 * q, 4);  // three bytes of it; q = 3 ends at the group's end
    r.w1 = 0;
    r.tail = p[12];
  }
  r.scale = srow[g];
  return r;
}

// A block: RT tiles of 16 rows of W (of each matrix), one chunk of 16 MT rows
// of x, the groups of one split; wave w takes groups w, w + 8, ...
// STAGED: x is bf16 [M,K], M <= 4, and each block puts its slice in order in
// LDS; else x comes in fragment order from frag_role, a fragment 1 KB.
// The matrix cores take x as the row operand and W as the column operand, so
// a lane's partial sums belong to the weight row whose bytes it decoded.
template <int G, int NB, int MT, int RT, bool STAGED, int ACT>
__global__ __launch_bounds__(kDecThreads) void dec_kernel(const ProjArgs A) {
  constexpr int S32 = G / 32;
  constexpr uint32_t kRedBytes = kDecWaves * MT * 1024;
  constexpr uint32_t kBuf = STAGED ? kStagedBytes : kRedBytes;
  static_assert(kBuf >= kRedBytes, "the sums of the waves reuse x's LDS");
  __shared__ __align__(16) unsigned char smem_raw[kLutBytes + kBuf];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  lds_bytes *buf = smem + kLutBytes;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nG = A.K / G;

  int b = (int)blockIdx.x;
  const int chunk = b % A.chunks;
  b /= A.chunks;
  const int split = b % A.splits, n0 = b / A.splits * (16 * RT);
  const int g0 = (int)((int64_t)nG * split / A.splits);
  const int g1 = (int)((int64_t)nG * (split + 1) / A.splits);
  const int64_t m0 = (int64_t)chunk * (16 * MT);

  // rows past N read row N - 1; their sums are not stored
  const uint8_t *row[RT][NB];
  const uint16_t *srow[RT][NB];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t n = min(n0 + 16 * rt + l, A.N - 1);
      row[rt][i] = A.packed[i] + n * nG * bytes_per_group(G);
      srow[rt][i] = A.scales[i] + n * nG;
    }

  // the first bytes are requested before the table is built and x put in
  // order, which take as long as the bytes do
  constexpr int U = RT * NB >= 4 ? 2 : 4;  // groups in flight
  Raw raw[U][RT][NB];
  auto fetch = [&](int u, int g) {
    const int gc = min(g, nG - 1);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < NB; ++i) raw[u][rt][i] = load_raw<G>(row[rt][i], srow[rt][i], gc, q);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(u, g0 + wv + kDecWaves * u);

  build_lut<kLutBf16>(smem, tid, kDecThreads);
  if constexpr (STAGED) {
    // unit (g, quarter, m): a quarter's codes of a group of one row
    const int M = (int)A.M, units = (g1 - g0) * 4 * M;
    for (int e = tid; e < units; e += kDecThreads) {
      const int m = e % M, gq = e / M, g = gq >> 2, uq = gq & 3;
      u32x4 f[S32];
      order_quarter<G>(A.x + (int64_t)m * A.K + (int64_t)(g0 + g) * G, uq, f);
#pragma unroll
      for (int s = 0; s < S32; ++s)
        *(lds_u32x4 *)(buf + 16u * (uint32_t)(((g * S32 + s) * 4 + uq) * M + m)) = f[s];
    }
  }
  __syncthreads();

  f32x4 acc[RT][NB][MT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[rt][i][mt] = f32x4{0.f, 0.f, 0.f, 0.f};

  const uint32_t lut = lut_lane(lane);
  uint32_t flags = 0;
  for (int g = g0 + wv; g < g1; g += kDecWaves * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gu = g + kDecWaves * u;
      if (gu >= g1) break;
      bf16x8 xf[S32][MT];
#pragma unroll
      for (int s = 0; s < S32; ++s)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (STAGED) {
            // rows past M read row M - 1
            const int M = (int)A.M;
            xf[s][mt] = *(lds_bf16x8_c *)(buf + 16u * (uint32_t)((((gu - g0) * S32 + s) * 4 + q) * M +
                                                                 min(l, M - 1)));
          } else {
            xf[s][mt] = *(const bf16x8 *)(A.x + ((((int64_t)chunk * nG + gu) * S32 + s) * MT + mt) * 512 +
                                          lane * 8);
          }
        }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const Raw r = raw[u][rt][i];
          uint32_t d[4 * S32];
          decode_quarter<G>(smem, lut, r.w0, r.w1, r.tail, q, d, flags);
          f32x4 part[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < S32; ++s) {
            const bf16x8 w = __builtin_bit_cast(bf16x8, u32x4{d[4 * s], d[4 * s + 1], d[4 * s + 2], d[4 * s + 3]});
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) part[mt] = mfma32<false>(xf[s][mt], w, part[mt]);
          }
          // codes entered as 2c
          const float sh = 0.5f * __half2float(__ushort_as_half((unsigned short)r.scale));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[rt][i][mt][j] = fmaf(sh, part[mt][j], acc[rt][i][mt][j]);
        }
      fetch(u, gu + kDecWaves * U);
    }
  }
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);

  if constexpr (NB == 1) {
    // adapters, once per output (split 0); the waves take the distinct ones
    // in turn and add to their partial sums.  A product of one adapter is
    // made for all rows of the chunk and kept for its own, so nothing in an
    // adapter reaches another's rows.
    if (split == 0 && A.adapters > 0) {
      int id = -1;
      if (lane < 16 * MT && m0 + lane < A.M) id = A.ids[m0 + lane];
      if (id >= A.adapters) id = -1;
      uint64_t todo = adapter_leaders(id, lane);
      for (int turn = 0; todo; ++turn) {
        const int first = __builtin_ctzll(todo);
        todo &= todo - 1;
        if (turn % kDecWaves != wv) continue;
        const int a = __builtin_amdgcn_readlane(id, first);
        f32x4 add[RT][MT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) add[rt][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int r0 = 0; r0 < A.R; r0 += 32) {
          const bool in = r0 + 8 * q < A.R;
          bf16x8 bv[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const int64_t n = min(n0 + 16 * rt + l, A.N - 1);
            u32x4 v{0u, 0u, 0u, 0u};
            if (in) v = *(const u32x4 *)(A.b + ((int64_t)a * A.N + n) * A.R + r0 + 8 * q);
            bv[rt] = __builtin_bit_cast(bf16x8, v);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int own = __shfl(id, 16 * mt + l);
            const Pieces p = split_t(A.t + (m0 + 16 * mt + l) * A.R + r0 + 8 * q, in && own == a);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int i = 0; i < 3; ++i) add[rt][mt] = mfma32<false>(p.p[i], bv[rt], add[rt][mt]);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool mine = __shfl(id, 16 * mt + 4 * q + j) == a;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[rt][0][mt][j] += mine ? add[rt][mt][j] : 0.f;
          }
      }
    }
  }

  // sums of the waves, in wave order
  constexpr int E = (MT * 256 + kDecThreads - 1) / kDecThreads;  // outputs a thread and matrix
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float v[NB][E];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        *(__attribute__((address_space(3))) f32x4 *)(buf + 16u * (uint32_t)((wv * MT + mt) * 64 + lane)) =
            acc[rt][i][mt];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int o = e * kDecThreads + tid;
        v[i][e] = 0.f;
        if (o < MT * 256)
#pragma unroll
          for (int w = 0; w < kDecWaves; ++w)
            v[i][e] += *(__attribute__((address_space(3))) float *)(buf + 4u * (uint32_t)(w * MT * 256 + o));
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int o = e * kDecThreads + tid;  // [mt][lane][j]
      const int j = o & 3, ol = (o >> 2) & 63;
      const int64_t m = m0 + 16 * (o >> 8) + 4 * (ol >> 4) + j;
      const int n = n0 + 16 * rt + (ol & 15);
      if (o >= MT * 256 || m >= A.M || n >= A.N) continue;
      if (A.splits > 1) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
          A.partial[(((int64_t)split * NB + i) * A.M + m) * A.N + n] = v[i][e];
      } else if constexpr (NB == 2) {
        ((uint16_t *)A.out)[m * A.N + n] = f32_to_bf16(act_value<ACT>(v[0][e]) * v[1][e]);
      } else {
        ((float *)A.out)[m * A.N + n] = v[0][e];
      }
    }
  }
}

// The splits' partial sums, in order, and the operator's last step.
template <int NB, int ACT>
__global__ __launch_bounds__(256) void combine_kernel(const float *__restrict__ partial, int splits,
                                                      int64_t mn, void *__restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < mn; i += (int64_t)gridDim.x * 256) {
    float v[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) v[k] = 0.f;
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int k = 0; k < NB; ++k) v[k] += partial[((int64_t)s * NB + k) * mn + i];
    if constexpr (NB == 2)
      ((uint16_t *)out)[i] = f32_to_bf16(act_value<ACT>(v[0]) * v[1]);
    else
      ((float *)out)[i] = v[0];
  }
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kWideP = 256, kWideQ = 256, kWideThreads = 512;
constexpr int kWideRing = 4;  // slots of x, and of codes

// 256 rows of W (NB = 1) or 128 of each of two (NB = 2) by 256 rows of x, in
// stages of 32 k; codes times their scale and x as f16 (both exact, see
// f16_role), so that one fp32 sum runs over all of K.
// While the MFMAs of stage s run, a wave
//   - reads the fragments of s + 1,
//   - decodes the codes of s + 3: two threads a weight row, three bytes and
//     one of the group's left-over codes each,
//   - requests x of s + 3 and the bytes of s + 5.
// LDS: 64 KB x, 64 KB codes, 32 KB table.
template <int G, int NB, int ACT>
__global__ __launch_bounds__(kWideThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void wide_kernel(const ProjArgs A) {
  constexpr int S32 = G / 32, WP = 2, WQ = 4, TP = 8, TQ = 4, B = bytes_per_group(G);
  typedef Stream<kRows, kWideQ, kWideThreads> QS;
  constexpr uint32_t kPSlot = kWideP * kKS * 2;
  constexpr uint32_t kQOff = kWideRing * kPSlot, kLutOff = kQOff + kWideRing * QS::kSlot;
  __shared__ __align__(16) unsigned char smem_raw[kLutOff + kLutBytes];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wv / WQ, wq = wv % WQ;
  const int nG = A.K / G, S = A.K / kKS;

  int ip, iq;
  tile_of_block((int)blockIdx.x, A.tp * A.tq, A.tp, A.tq, ip, iq);
  constexpr int HP = kWideP / WP / NB;  // rows of one matrix in a wave
  const int n0 = ip * (kWideP / NB);
  const int64_t q0 = (int64_t)iq * kWideQ;

  // this thread's weight row: slot row tid / 2; rows past N read row N - 1
  const int sr = tid >> 1, hf = tid & 1;
  const uint8_t *prow;
  const uint16_t *srow;
  {
    const int which = NB == 1 ? 0 : sr % (NB * HP) / HP;
    const int64_t n = min(n0 + sr / (NB * HP) * HP + sr % HP, A.N - 1);
    prow = A.packed[which] + n * nG * B;
    srow = A.scales[which] + n * nG;
  }
  uint32_t raw[2], tail = 0, tail_next, flags = 0;
  uint32_t scale = 0, scale_next;
  u32x2 left{0u, 0u};  // high bytes of the group's left-over codes
  // bytes of stage s, J = s % S32 (past the end: of the last group)
  auto load_raw = [&](int s, auto jc) {
    constexpr int J = decltype(jc)::value;
    const int g = min(s / S32, nG - 1);
    __builtin_memcpy(&raw[J & 1], prow + (int64_t)g * B + 6 * J + 3 * hf, 4);
  };
  auto load_group = [&](int s) {
    const int g = min(s / S32, nG - 1);
    const uint8_t *p = prow + (int64_t)g * B;
    if constexpr (G == 128) {
      uint16_t v;
      __builtin_memcpy(&v, p + 24, 2);
      tail_next = v;
    } else {
      tail_next = p[12];
    }
    scale_next = srow[g];
  };
  const uint32_t lut = kLutOff + lut_lane(lane);
  const uint32_t put0 = rows_at((uint32_t)sr, 2u * hf), put1 = rows_at((uint32_t)sr, 2u * hf + 1u);
  // codes of the stage whose bytes are loaded (J = its index % S32) -> slot
  auto decode = [&](auto jc, uint32_t slot) {
    constexpr int J = decltype(jc)::value;
    if constexpr (J == 0) {
      tail = tail_next;
      scale = scale_next * 0x10001u;
      left = leftover_pool<G>(smem, lut, tail, flags);
    }
    u32x4 c0, c1;
    decode_eighth(smem, lut, raw[J & 1], left, (uint32_t)(2 * J + hf), scale, c0, c1, flags);
    *(lds_u32x4 *)(smem + slot + put0) = c0;
    *(lds_u32x4 *)(smem + slot + put1) = c1;
  };

  QS qs;
  qs.init_rows(tid, (uint32_t)A.K, [&](int r) -> int64_t { return q0 + r < A.M ? r : -1; });
  const uint16_t *qbase = A.x + q0 * A.K;
  auto request = [&](int s, int i) {
    qs.load_tracked(i, qbase + (int64_t)s * kKS, smem + kQOff + (uint32_t)(s % kWideRing) * QS::kSlot,
                    (uint32_t)wv, s < S ? 1 : 0);
  };

  // ---- prologue: bytes of stages 0 .. 4, x of 0 .. 2, codes of 0 .. 2 ----
  load_group(0);
  load_raw(0, Int<0>{});
  load_raw(1, Int<1>{});
#pragma unroll
  for (int s = 0; s < kWideRing - 1; ++s)
#pragma unroll
    for (int i = 0; i < QS::kLoads; ++i) request(s, i);
  build_lut<kLutF16>(smem + kLutOff, tid, kWideThreads);
  __syncthreads();
  decode(Int<0>{}, 0);
  load_raw(2, Int<2 % S32>{});
  if constexpr (S32 == 2) load_group(2);
  decode(Int<1>{}, kPSlot);
  load_raw(3, Int<3 % S32>{});
  decode(Int<2 % S32>{}, 2 * kPSlot);
  load_raw(4, Int<0>{});
  load_group(4);

  Frags<kRows, kWideP, TP> pf;
  Frags<kRows, kWideQ, TQ> qf;
  pf.init(lane, wp * (kWideP / WP));
  qf.init(lane, wq * (kWideQ / WQ));
  f32x4 acc[TP][TQ];
#pragma unroll
  for (int a = 0; a < TP; ++a)
#pragma unroll
    for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  bf16x8 pa[TP], qa[TQ], qb[TQ];
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int b = 0; b < TQ; ++b) qa[b] = qf.read(smem, kQOff, b);
#pragma unroll
  for (int a = 0; a < TP; ++a) pa[a] = pf.read(smem, 0, a);

  auto stage = [&](int s, auto jc, bf16x8(&qc)[TQ], bf16x8(&qn)[TQ]) {
    constexpr int J = decltype(jc)::value;
    const uint32_t pn = (uint32_t)((s + 1) % kWideRing) * kPSlot;
    const uint32_t qn0 = kQOff + (uint32_t)((s + 1) % kWideRing) * QS::kSlot;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int a = 0; a < TP; ++a) {
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = mfma32<true>(pa[a], qc[b], acc[a][b]);
      if (a < TQ) qn[a] = qf.read(smem, qn0, a);
      pa[a] = pf.read(smem, pn, a);
      if (a < QS::kLoads) request(s + kWideRing - 1, a);
      if (a == 3) {
        decode(Int<(J + 3) % S32>{}, (uint32_t)((s + 3) % kWideRing) * kPSlot);
        load_raw(s + 5, Int<(J + 5) % S32>{});
        if constexpr ((J + 5) % S32 == 0) load_group(s + 5);
        // the codes are written before the fragments of rows 4 .. 7 are read:
        // when the last of those is used, in stage s + 1, the writes are done,
        // a barrier before stage s + 2 reads them
        asm volatile("" ::: "memory");
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // every stage issues at least three loads after x of stage s + 2
    asm volatile("s_waitcnt vmcnt(3)\n\ts_barrier" ::: "memory");
  };
  for (int s = 0; s < S; s += S32) {
    stage(s, Int<0>{}, qa, qb);
    stage(s + 1, Int<1>{}, qb, qa);
    if constexpr (S32 == 4) {
      stage(s + 2, Int<2>{}, qa, qb);
      stage(s + 3, Int<3>{}, qb, qa);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);

  // ---- epilogue: lane holds rows n = 16 a + 4 (lane / 16) + r, column
  // m = 16 b + lane % 16 ----
  const int l = lane & 15, q = lane >> 4;
  const int64_t mq = q0 + wq * (kWideQ / WQ) + l;
#pragma unroll
  for (int b = 0; b < TQ; ++b) {
    const int64_t m = mq + 16 * b;
    const int sh = m < A.M ? -A.shift[m] : 0;
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[a][b][r] = ldexpf(acc[a][b][r], sh);
  }
  if constexpr (NB == 2) {
    uint16_t *h = (uint16_t *)A.out;
#pragma unroll
    for (int b = 0; b < TQ; ++b) {
      const int64_t m = mq + 16 * b;
      if (m >= A.M) continue;
#pragma unroll
      for (int a = 0; a < TP / 2; ++a) {
        const int n = n0 + wp * HP + 16 * a + 4 * q;
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = act_value<ACT>(acc[a][b][r]) * acc[a + TP / 2][b][r];
        uint16_t *o = h + m * A.N + n;
        if ((A.N & 3) == 0 && (reinterpret_cast<uintptr_t>(h) & 7) == 0 && n < A.N) {
          store4(o, v);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < A.N) o[r] = f32_to_bf16(v[r]);
        }
      }
    }
  } else {
    const int nw = n0 + wp * HP;  // first row of this wave
    if (A.adapters > 0) {
      // the wave's 64 columns, one a lane
      const int64_t mw = q0 + wq * (kWideQ / WQ);
      int id = mw + lane < A.M ? A.ids[mw + lane] : -1;
      if (id >= A.adapters) id = -1;
      uint64_t todo = adapter_leaders(id, lane);
      while (todo) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= todo - 1;
        bool mine[TQ];
#pragma unroll
        for (int b = 0; b < TQ; ++b) mine[b] = __shfl(id, 16 * b + l) == a;
        for (int r0 = 0; r0 < A.R; r0 += 32) {
          const bool in = r0 + 8 * q < A.R;
          Pieces tp[TQ];
#pragma unroll
          for (int b = 0; b < TQ; ++b)
            tp[b] = split_t(A.t + (mw + 16 * b + l) * A.R + r0 + 8 * q, in && mine[b]);
#pragma unroll
          for (int t = 0; t < TP; ++t) {
            const int64_t n = min(nw + 16 * t + l, A.N - 1);
            u32x4 v{0u, 0u, 0u, 0u};
            if (in) v = *(const u32x4 *)(A.b + ((int64_t)a * A.N + n) * A.R + r0 + 8 * q);
            const bf16x8 bv = __builtin_bit_cast(bf16x8, v);
#pragma unroll
            for (int b = 0; b < TQ; ++b) {
              f32x4 add{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < 3; ++i) add = mfma32<false>(bv, tp[b].p[i], add);
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[t][b][r] += mine[b] ? add[r] : 0.f;
            }
          }
        }
      }
    }
    float *y = (float *)A.out;
#pragma unroll
    for (int b = 0; b < TQ; ++b) {
      const int64_t m = mq + 16 * b;
      if (m >= A.M) continue;
#pragma unroll
      for (int a = 0; a < TP; ++a) {
        const int n = nw + 16 * a + 4 * q;
        float *o = y + m * A.N + n;
        if ((A.N & 3) == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0 && n < A.N) {
          *(f32x4 *)o = acc[a][b];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < A.N) o[r] = acc[a][b][r];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// before the product: x in order, and t
// ---------------------------------------------------------------------------

constexpr int kPreThreads = 512, kPreWaves = 8;
constexpr int kShrinkTile = 256;  // rows among which equal adapters are gathered

struct PreArgs {
  const uint16_t *x, *a;
  const int32_t *ids;
  const float *scaling;
  uint16_t *xo;     // fragments or f16 rows
  int32_t *shift;   // f16 rows
  float *t;
  int64_t M;
  int K, adapters, R, mt;
  int shrink_blocks, units, rtiles;  // shrink: blocks, units a tile of rows, tiles of 16 ranks
  int32_t *status;
};

// t of one unit: up to 16 rows of one adapter, 16 ranks.  The rows of a tile
// that name the same adapter are numbered in order and cut into units of 16,
// so rows in any order share the adapter's A.  Waves split K; sums of the
// waves in order.
__device__ void shrink_role(const PreArgs &A, int64_t blk, unsigned char *smem_raw) {
  int *ids = (int *)smem_raw;                       // [256]
  int *rows = ids + kShrinkTile;                    // [16]
  int *info = rows + 16;                            // adapter, leader's rank
  int *counts = info + 4;                           // [8] leaders of each wave
  float *red = (float *)(counts + 12);              // [8][64][4]
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, l = lane & 15, q = lane >> 4;
  const int rt = (int)(blk % A.rtiles), unit = (int)(blk / A.rtiles % A.units);
  const int64_t m0 = blk / A.rtiles / A.units * kShrinkTile;
  const int nrows = (int)min((int64_t)kShrinkTile, A.M - m0);
  int id = -1;
  if (tid < nrows) {
    id = A.ids[m0 + tid];
    if (id < -1 || id >= A.adapters) {
      if (unit == 0 && rt == 0 && A.status) atomicOr(A.status, kDevBadAdapter);
      id = -1;
    }
  }
  if (tid < kShrinkTile) ids[tid] = id;
  if (tid < 16) rows[tid] = -1;
  if (tid == 0) info[0] = -1;
  __syncthreads();
  int rank = 0;  // among the rows of this adapter
  if (id >= 0)
    for (int j = 0; j < tid; ++j) rank += ids[j] == id;
  const bool leads = id >= 0 && rank % 16 == 0;
  const uint64_t mask = __ballot(leads);
  if (lane == 0) counts[wv] = __popcll(mask);
  __syncthreads();
  int before = __popcll(mask & ((1ull << lane) - 1));
  for (int w = 0; w < wv; ++w) before += counts[w];
  if (leads && before == unit) {
    info[0] = id;
    info[1] = rank;
  }
  __syncthreads();
  const int a = info[0];
  if (a < 0) return;  // fewer units than this
  if (id == a && rank / 16 == info[1] / 16) rows[rank % 16] = tid;
  __syncthreads();

  // columns: the unit's rows (the first one in place of absent ones); rows:
  // ranks 16 rt + l
  const int own = rows[l], mr = own < 0 ? rows[0] : own;
  const uint16_t *xr = A.x + (m0 + mr) * A.K + 8 * q;
  const int r = min(16 * rt + l, A.R - 1);
  const uint16_t *ar = A.a + ((int64_t)a * A.R + r) * A.K + 8 * q;
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  const int steps = A.K / 32;
#pragma unroll 4
  for (int s = wv; s < steps; s += kPreWaves)
    acc = mfma32<false>(*(const bf16x8 *)(ar + 32 * s), *(const bf16x8 *)(xr + 32 * s), acc);
  *(f32x4 *)(red + 4 * tid) = acc;
  __syncthreads();
  if (tid < 256) {
    float sum = 0.f;
    for (int w = 0; w < kPreWaves; ++w) sum += red[w * 256 + tid];
    const int ol = tid >> 2, rr = 16 * rt + 4 * (ol >> 4) + (tid & 3), row = rows[ol & 15];
    if (row >= 0 && rr < A.R) A.t[(m0 + row) * A.R + rr] = A.scaling[a] * sum;
  }
}

// x in the fragment order of dec_kernel: [chunk][group][step][16-row tile]
// [lane][8]; rows past M are zeros.
template <int G>
__device__ void frag_role(const PreArgs &A, int64_t first, int64_t stride) {
  constexpr int S32 = G / 32;
  const int nG = A.K / G, rows = 16 * A.mt;
  const int64_t chunks = (A.M + rows - 1) / rows, units = chunks * nG * 4 * rows;
  for (int64_t e = first; e < units; e += stride) {
    // a wave's lanes take neighbouring quarters of one row
    const int uq = (int)(e & 3);
    const int64_t rest = e >> 2;
    const int g = (int)(rest % nG);
    const int64_t row = rest / nG, chunk = row / rows;
    const int rr = (int)(row - chunk * rows);
    u32x4 f[S32];
#pragma unroll
    for (int s = 0; s < S32; ++s) f[s] = u32x4{0u, 0u, 0u, 0u};
    if (row < A.M) order_quarter<G>(A.x + row * A.K + (int64_t)g * G, uq, f);
#pragma unroll
    for (int s = 0; s < S32; ++s)
      *(u32x4 *)(A.xo + (((chunk * nG + g) * S32 + s) * A.mt + (rr >> 4)) * 512 + (uq * 16 + (rr & 15)) * 8) =
          f[s];
  }
}

// Row m of x as f16 times a power of two that brings its largest finite value
// to [2^14, 2^15): a bf16 value's eight bits fit f16's eleven, so every
// element down to 2^-32 of the row's largest is exact, and a smaller one is
// off by at most 2^-40 of it.  In the order of wide_kernel's codes.
template <int G>
__device__ void f16_role(const PreArgs &A, int64_t m) {
  const int lane = threadIdx.x & 63;
  const uint16_t *xr = A.x + m * A.K;
  uint32_t top = 0;
  for (int k = 8 * lane; k < A.K; k += 512) {
    uint16_t v[8];
    *(u32x4 *)v = *(const u32x4 *)(xr + k);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = v[j] & 0x7FFFu;
      top = b < 0x7F80u && b > top ? b : top;
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  int exponent;  // top is in [2^(exponent - 1), 2^exponent)
  (void)frexpf(bf16_to_f32(top), &exponent);
  const int shift = top ? 15 - exponent : 0;
  if (lane == 0) A.shift[m] = shift;
  uint16_t *o = A.xo + m * A.K;
  for (int e = lane; e < A.K / 16; e += 64) {
    const int g = e / (G / 16), part = e % (G / 16);
    const uint16_t *p = xr + g * G;
    _Float16 f[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      f[j] = (_Float16)ldexpf(bf16_to_f32(p[eighth_source<G>(part, j)]), shift);
    *(u32x4 *)(o + 16 * e) = *(u32x4 *)f;
    *(u32x4 *)(o + 16 * e + 8) = *(u32x4 *)(f + 8);
  }
}

constexpr int64_t kMaxPreBlocks = 1 << 16;  // of a role; each strides over its work
constexpr int kPreNone = 0, kPreFrag = 1, kPreF16 = 2;

template <int G, int MODE>
__global__ __launch_bounds__(kPreThreads) void pre_kernel(const PreArgs A) {
  __shared__ __align__(16) unsigned char smem[4 * (kShrinkTile + 32) + 16 * kPreThreads];
  if ((int)blockIdx.x < A.shrink_blocks) {
    const int64_t work = (A.M + kShrinkTile - 1) / kShrinkTile * A.units * A.rtiles;
    for (int64_t w = blockIdx.x; w < work; w += A.shrink_blocks) {
      shrink_role(A, w, smem);
      __syncthreads();
    }
    return;
  }
  const int64_t blk = (int64_t)blockIdx.x - A.shrink_blocks;
  const int64_t blocks = (int64_t)gridDim.x - A.shrink_blocks;
  if constexpr (MODE == kPreFrag) {
    frag_role<G>(A, blk * kPreThreads + threadIdx.x, blocks * kPreThreads);
  } else if constexpr (MODE == kPreF16) {
    for (int64_t m = blk * kPreWaves + (threadIdx.x >> 6); m < A.M; m += blocks * kPreWaves)
      f16_role<G>(A, m);
  }
}

// ---------------------------------------------------------------------------
// which kernel, and the workspace
// ---------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

struct Plan {
  bool wide, staged;
  int mt, rt, splits, chunks;
  int64_t x, shift, t, partial;  // workspace bytes, each a multiple of 16, in this order
  int64_t total() const { return x + shift + t + partial; }
};

Plan plan_of(int64_t M, int64_t N, int64_t K, int G, int NB, int R) {
  Plan p{};
  p.t = R ? round16(M * R * 4) : 0;
  // wide: from about half the chip's CUs on, a tile each
  p.wide = ceil_div(NB * N, kWideP) * ceil_div(M, kWideQ) >= 128 && M > 128;
  if (p.wide) {
    p.x = round16(M * K * 2);
    p.shift = round16(M * 4);
    return p;
  }
  p.staged = M <= kStagedRows;
  p.mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  p.chunks = (int)ceil_div(M, 16 * p.mt);
  const int64_t tiles = ceil_div(N, 16), nG = K / G;
  p.rt = !p.staged && tiles * p.chunks >= 1024 ? 2 : 1;
  const int64_t blocks = ceil_div(tiles, p.rt) * p.chunks;
  // staged: a block's slice of x fits its LDS.  Otherwise K is split only
  // while blocks are few and every wave keeps two groups.
  int64_t s = p.staged ? ceil_div(nG, std::max<int64_t>(1, kStagedBytes / (M * G * 2))) : 1;
  while (blocks * s < 192 && nG / (2 * s) >= 2 * kDecWaves) s *= 2;
  p.splits = (int)std::min(s, nG);
  if (!p.staged) p.x = (int64_t)p.chunks * 16 * p.mt * K * 2;
  if (p.splits > 1) p.partial = round16((int64_t)p.splits * NB * M * N * 4);
  return p;
}

template <int G, int NB, int ACT>
void launch_dec(const Plan &p, const ProjArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)(ceil_div(ceil_div(a.N, 16), p.rt) * p.splits * p.chunks));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kDecThreads), 0, stream, a);
  };
  if (p.staged)
    go(dec_kernel<G, NB, 1, 1, true, ACT>);
  else if (p.mt == 1)
    p.rt == 1 ? go(dec_kernel<G, NB, 1, 1, false, ACT>) : go(dec_kernel<G, NB, 1, 2, false, ACT>);
  else if (p.mt == 2)
    p.rt == 1 ? go(dec_kernel<G, NB, 2, 1, false, ACT>) : go(dec_kernel<G, NB, 2, 2, false, ACT>);
  else
    p.rt == 1 ? go(dec_kernel<G, NB, 4, 1, false, ACT>) : go(dec_kernel<G, NB, 4, 2, false, ACT>);
}

// All launches of a call; `a` and `pre` hold the caller's arguments.
template <int G, int NB, int ACT>
void launch_proj(const Plan &p, ProjArgs a, PreArgs pre, void *workspace, hipStream_t stream) {
  char *ws = (char *)workspace;
  pre.x = a.x;
  pre.xo = (uint16_t *)ws;
  pre.shift = (int32_t *)(ws + p.x);
  pre.t = (float *)(ws + p.x + p.shift);
  a.partial = (float *)(ws + p.x + p.shift + p.t);
  a.t = pre.t;
  a.shift = pre.shift;
  pre.M = a.M, pre.K = a.K, pre.mt = p.mt, pre.status = a.status;
  pre.ids = a.ids, pre.adapters = a.adapters, pre.R = a.R;
  if (NB == 1) {
    const int64_t tiles = ceil_div(a.M, kShrinkTile);
    const int64_t rows = std::min<int64_t>(a.M, kShrinkTile);
    // units of a tile: one for each 16 rows and one more for each adapter
    pre.units = (int)std::max<int64_t>(1, std::min(rows, ceil_div(rows, 16) + std::min<int64_t>(rows, a.adapters)));
    pre.rtiles = (int)ceil_div(a.R, 16);
    if (a.adapters == 0) pre.units = pre.rtiles = 1;  // the ids are still checked
    pre.shrink_blocks = (int)std::min(kMaxPreBlocks, tiles * pre.units * pre.rtiles);
  }
  if (p.wide) {
    const dim3 grid((unsigned)(pre.shrink_blocks + std::min(kMaxPreBlocks, ceil_div(a.M, kPreWaves))));
    hipLaunchKernelGGL((pre_kernel<G, kPreF16>), grid, dim3(kPreThreads), 0, stream, pre);
    a.x = pre.xo;
  } else if (!p.staged) {
    const int64_t units = (int64_t)p.chunks * 16 * p.mt * (a.K / G) * 4;
    const dim3 grid((unsigned)(pre.shrink_blocks + std::min<int64_t>(4096, ceil_div(units, kPreThreads))));
    hipLaunchKernelGGL((pre_kernel<G, kPreFrag>), grid, dim3(kPreThreads), 0, stream, pre);
    a.x = pre.xo;
  } else if (pre.shrink_blocks) {
    hipLaunchKernelGGL((pre_kernel<G, kPreNone>), dim3((unsigned)pre.shrink_blocks),
                       dim3(kPreThreads), 0, stream, pre);
  }
  if (p.wide) {
    a.tp = (int)ceil_div(NB * (int64_t)a.N, kWideP);
    a.tq = (int)ceil_div(a.M, kWideQ);
    hipLaunchKernelGGL((wide_kernel<G, NB, ACT>), dim3((unsigned)(a.tp * a.tq)), dim3(kWideThreads), 0,
                       stream, a);
    return;
  }
  a.splits = p.splits;
  a.chunks = p.chunks;
  launch_dec<G, NB, ACT>(p, a, stream);
  if (p.splits > 1) {
    const int64_t mn = a.M * a.N;
    hipLaunchKernelGGL((combine_kernel<NB, ACT>), dim3((unsigned)std::min<int64_t>(4096, ceil_div(mn, 256))),
                       dim3(256), 0, stream, a.partial, p.splits, mn, a.out);
  }
}

}  // namespace

int64_t glu_workspace(int64_t M, int64_t N, int64_t K, int G) { return plan_of(M, N, K, G, 2, 0).total(); }

void launch_glu(const uint16_t *x, const uint8_t *pg, const uint16_t *sg, const uint8_t *pu,
                const uint16_t *su, int64_t M, int64_t N, int64_t K, int G, int act, uint16_t *h,
                void *workspace, int32_t *d_status, hipStream_t stream) {
  const Plan p = plan_of(M, N, K, G, 2, 0);
  ProjArgs a{};
  a.x = x, a.packed[0] = pg, a.packed[1] = pu, a.scales[0] = sg, a.scales[1] = su;
  a.out = h, a.M = M, a.N = (int)N, a.K = (int)K, a.status = d_status;
  if (G == 64)
    act == kActSilu ? launch_proj<64, 2, kActSilu>(p, a, PreArgs{}, workspace, stream)
                    : launch_proj<64, 2, kActGelu>(p, a, PreArgs{}, workspace, stream);
  else
    act == kActSilu ? launch_proj<128, 2, kActSilu>(p, a, PreArgs{}, workspace, stream)
                    : launch_proj<128, 2, kActGelu>(p, a, PreArgs{}, workspace, stream);
}

int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int G, int R) {
  return plan_of(M, N, K, G, 1, R).total();
}

void launch_lora(const uint16_t *x, const uint8_t *packed, const uint16_t *scales, int64_t M,
                 int64_t N, int64_t K, int G, const int32_t *ids, const uint16_t *a,
                 const uint16_t *b, const float *scaling, int adapters, int R, float *y,
                 void *workspace, int32_t *d_status, hipStream_t stream) {
  const Plan p = plan_of(M, N, K, G, 1, R);
  ProjArgs pa{};
  pa.x = x, pa.packed[0] = packed, pa.scales[0] = scales, pa.ids = ids, pa.b = b;
  pa.adapters = adapters, pa.R = R, pa.out = y, pa.M = M, pa.N = (int)N, pa.K = (int)K;
  pa.status = d_status;
  PreArgs pre{};
  pre.a = a, pre.scaling = scaling;
  G == 64 ? launch_proj<64, 1, kActSilu>(p, pa, pre, workspace, stream)
          : launch_proj<128, 1, kActSilu>(p, pa, pre, workspace, stream);
}

}  // namespace tq

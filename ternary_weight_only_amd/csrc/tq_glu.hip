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
// Three kernels multiply:
//   few_kernel    up to 32 rows: bound by the weights' bytes.  Every byte is
//                 decoded in registers by the lane that feeds it to the matrix
//                 cores; the waves of a block share the groups of a tile of 16
//                 weight rows, x stays in LDS.
//   mid_kernel    some more rows: the same decode, a tile of weight rows a
//                 wave, 64 rows of x streamed through LDS for all eight.
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

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What the kernels read and write.
struct ProjArgs {
  const uint16_t *x;              // bf16 [M,K], or as f16_role leaves it
  const uint8_t *packed[2];
  const uint16_t *scales[2];
  const uint16_t *x0;             // bf16 [M,K]
  const u32x2 *rows;              // mid, wide: x of row m is stored times 2^rows[m].x, and the
                                  // magnitudes that it lost by that are rows[m].y (fp32) in all
  const int32_t *ids;             // lora
  const float *t;                 // lora: [tsplits][M,R] fp32, scaled
  int tsplits;
  const uint16_t *b;              // lora: [adapters,N,R]
  int adapters, R;
  void *out;                      // bf16 [M,N] (glu) or fp32 [M,N] (lora)
  float *partial;                 // splits > 1: fp32 [split][NB][M][N]
  int64_t M;
  int N, K;
  int splits;                     // blocks along K
  int wk, wt;                     // few: waves of a tile (along K), tiles of a set
  int chunks;                     // mid: chunks of rows
  int tp, tq;                     // wide: tiles
  int32_t *status;
};

// ---------------------------------------------------------------------------
// what x loses as f16
// ---------------------------------------------------------------------------

// A row whose elements spread over more than 2^32 loses some of its smallest
// (tq_ternary.h): in a sum, at most the magnitudes lost times the largest
// scale.  A sum at least 2^22 times that has it within an fp32 sum's own
// roundings; one below -- where the row's largest elements meet codes 0, or
// cancel -- gets the lost part added, a wave a sum.  Rows that lose something
// are known when x is converted, so others cost a load and a ballot.  (One
// element of 2^40 in every row of normal ones: a third of the sums get theirs.)
constexpr float kLostCounts = 4194304.f;

// The same value, known only here: what follows from it is not computed ahead
// of a loop around, where it would hold registers that the loop needs.
__device__ __forceinline__ int uniform_here(int v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+s"(v));
#endif
  return v;
}
// The lane, from no register that a loop before had to keep.
__device__ __forceinline__ int lane_here() {
#if defined(__HIP_DEVICE_COMPILE__)
  int lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  asm volatile("" : "+v"(lane));
  return lane;
#else
  return 0;
#endif
}

// Largest magnitude among the scales of `rows` weight rows from n0 on.
__device__ __forceinline__ float scale_top(const ProjArgs &A, int i, int n0, int rows, int nG) {
  const int lane = lane_here();
  nG = uniform_here(nG);
  const uint16_t *s = A.scales[i] + (int64_t)n0 * nG;
  const int64_t count = (int64_t)max(0, min(rows, A.N - n0)) * nG;
  uint32_t top = 0;
  for (int64_t e = lane; e < count; e += 64) top = max(top, (uint32_t)s[e] & 0x7FFFu);
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  return (float)__builtin_bit_cast(_Float16, (uint16_t)top);
}

// The lost part (WHOLE: all) of the sum of x's row m (times 2^shift) and row n
// of matrix i over groups g0 .. g1 - 1; by a whole wave, the same in every
// lane.  A byte a lane at a time, decoded by division: few registers beside
// those of the kernel around it, and no table need be there.
template <int G, bool WHOLE>
__device__ __forceinline__ float lost_part(const ProjArgs &A, int i, int64_t m, int64_t n, int g0, int g1,
                                           int shift) {
  constexpr int B = bytes_per_group(G);
  const int nG = uniform_here(A.K / G);
  const uint8_t *p = A.packed[i] + (n * nG + g0) * B;
  const uint16_t *s = A.scales[i] + n * nG + g0;
  const uint16_t *x = A.x0 + (m * nG + g0) * G;
  float sum = 0.f;
#pragma unroll 1
  for (int e = lane_here(); e < (g1 - g0) * B; e += 64) {
    const int g = e / B, k = 5 * (e - g * B);
    uint32_t byte = p[e];
    float part = 0.f;
#pragma unroll
    for (int d = 0; d < 5; ++d) {  // the last byte's codes past G are 0
      const uint32_t b = x[g * G + min(k + d, G - 1)];
      part = fmaf((float)(int)(byte % 3u) - 1.f, WHOLE ? bf16_to_f32(b) : lost_of(b, shift), part);
      byte /= 3u;
    }
    sum = fmaf(part, (float)__builtin_bit_cast(_Float16, s[g]), sum);
  }
  return wave_sum(sum);
}

// The lost part added to what a split of groups g0 .. g1 - 1 stored for row m
// of x and column n, by the lane that stored it (`mine`; in order for it).
// Where that is the gated product, it is made anew, and any lane may write it.
template <int G, int NB, int ACT>
__device__ __forceinline__ void mend_result(const ProjArgs &A, int64_t m, int64_t n, int split, int g0, int g1,
                                            bool mine) {
  const int64_t o = m * A.N + n;
  if (NB == 2 && A.splits == 1) {
    const float g = lost_part<G, true>(A, 0, m, n, g0, g1, 0), u = lost_part<G, true>(A, 1, m, n, g0, g1, 0);
    if (mine) ((uint16_t *)A.out)[o] = f32_to_bf16(act_value<ACT>(g) * u);
    return;
  }
  const int shift = (int)A.rows[m].x;
#pragma unroll 1
  for (int i = 0; i < NB; ++i) {
    const float add = lost_part<G, false>(A, i, m, n, g0, g1, shift);
    float *y = (A.splits > 1 ? A.partial + ((int64_t)split * NB + i) * A.M * A.N : (float *)A.out) + o;
    if (mine) *y += add;
  }
}

// ---------------------------------------------------------------------------
// adapters
// ---------------------------------------------------------------------------

// The distinct adapters among the ids that a wave's lanes hold, as a mask of the first lane of each: the lanes of the first
// one left are struck out in turn.
__device__ __forceinline__ uint64_t adapter_leaders(int id) {
  uint64_t left = __ballot(id >= 0), leaders = 0;
  while (left) {
    const int j = __builtin_ctzll(left);
    leaders |= 1ull << j;
    left &= ~__ballot(id == __builtin_amdgcn_readlane(id, j));
  }
  return leaders;
}

// Eight ranks of row m's t in three bf16 pieces (24 bits together); zeros
// unless `in`.
struct Pieces {
  bf16x8 p[3];
};
__device__ __forceinline__ Pieces split_t(const ProjArgs &A, int64_t m, int r, bool in) {
  f32x4 lo{0.f, 0.f, 0.f, 0.f}, hi = lo;
  if (in) {
    const f32x4 *t = (const f32x4 *)(A.t + m * A.R + r);
    lo = t[0];
    hi = t[1];
    for (int s = 1; s < A.tsplits; ++s) {
      const f32x4 *u = (const f32x4 *)(A.t + (s * A.M + m) * A.R + r);
      lo += u[0];
      hi += u[1];
    }
  }
  Pieces out;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = i < 4 ? lo[i] : hi[i - 4];
    const __bf16 a = (__bf16)v;
    const float ra = v - (float)a;
    const __bf16 b = (__bf16)ra;
    out.p[0][i] = a;
    out.p[1][i] = b;
    out.p[2][i] = (__bf16)(ra - (float)b);
  }
  return out;
}

// Add the adapters' part to T tiles of 16 weight rows (n0 + 16 t + ..) by C
// of 16 rows of x (m0 + i, named by lane i's id, -1 for none): acc[t][c] has
// the weight rows as the matrix cores' rows if WROWS, else as their columns.
// The distinct adapters are taken in turn, those with turn % share == mine
// here, the next one's B requested while one is multiplied.  A row's t is its
// own adapter's; a product with an adapter is made for all the rows and kept
// for those that name it, so nothing in an adapter reaches another's rows.
template <bool WROWS, int T, int C>
__device__ __forceinline__ void add_adapters(const ProjArgs &A, int64_t m0, int n0, int id, int share,
                                             int mine, f32x4 (&acc)[T][C]) {
  const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const uint64_t leaders = adapter_leaders(id);
  int64_t n[T];
#pragma unroll
  for (int t = 0; t < T; ++t) n[t] = min(n0 + 16 * t + l, A.N - 1);
  for (int r0 = 0; r0 < A.R; r0 += 32) {
    const int r = r0 + 8 * q;
    Pieces x[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      x[c] = split_t(A, m0 + 16 * c + l, r, __shfl(id, 16 * c + l) >= 0 && r < A.R);
    uint64_t todo = leaders;
    int turn = 0;
    auto next = [&]() {  // the next adapter of ours, or -1
      while (todo) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= todo - 1;
        if (turn++ % share == mine) return a;
      }
      return -1;
    };
    u32x4 b[T];
    auto fetch = [&](int a) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        b[t] = u32x4{0u, 0u, 0u, 0u};
        if (r < A.R) b[t] = *(const u32x4 *)(A.b + ((int64_t)a * A.N + n[t]) * A.R + r);
      }
    };
    int a = next();
    if (a >= 0) fetch(a);
    while (a >= 0) {
      bf16x8 w[T];
#pragma unroll
      for (int t = 0; t < T; ++t) w[t] = __builtin_bit_cast(bf16x8, b[t]);
      const int an = next();
      if (an >= 0) fetch(an);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!__ballot(__shfl(id, 16 * c + l) == a)) continue;
        bool own[4];  // WROWS: of this lane's column; else of its four rows
        if constexpr (WROWS) {
          own[0] = __shfl(id, 16 * c + l) == a;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) own[j] = __shfl(id, 16 * c + 4 * q + j) == a;
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          f32x4 add{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 3; ++i)
            add = WROWS ? mfma32<false>(w[t], x[c].p[i], add) : mfma32<false>(x[c].p[i], w[t], add);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][c][j] += own[WROWS ? 0 : j] ? add[j] : 0.f;
        }
      }
      a = an;
    }
  }
}

// As add_adapters with the weight rows as columns (this lane's is n), a result
// at a time in fp32, from its own row's t and adapter: the same time whatever
// the ids are.  The splits share the results.
template <int C>
__device__ __forceinline__ void add_own_adapters(const ProjArgs &A, int64_t m0, int64_t n, int id, int share,
                                                 int mine, f32x4 (&acc)[C]) {
  const int q = (threadIdx.x & 63) >> 4;
  int turn = 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 16 * c + 4 * q + j, a = __shfl(id, i);
      const bool ours = turn == mine;
      turn = turn + 1 == share ? 0 : turn + 1;
      if (!ours || a < 0) continue;
      const uint16_t *b = A.b + ((int64_t)a * A.N + n) * A.R;
      const float *t = A.t + (m0 + i) * A.R;
      float sum = 0.f;
#pragma unroll 2
      for (int r = 0; r < A.R; r += 8) {
        const u32x4 w = *(const u32x4 *)(b + r);
        f32x4 lo = *(const f32x4 *)(t + r), hi = *(const f32x4 *)(t + r + 4);
        for (int s = 1; s < A.tsplits; ++s) {
          lo += *(const f32x4 *)(t + s * A.M * A.R + r);
          hi += *(const f32x4 *)(t + s * A.M * A.R + r + 4);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sum = fmaf(k < 4 ? lo[k] : hi[k - 4], bf16_to_f32((uint16_t)(w[k / 2] >> (k & 1 ? 16 : 0))), sum);
      }
      acc[c][j] += sum;
    }
}

// What the product's kernels need of row m; zeros past the last.
__device__ __forceinline__ u32x2 row_scale(const ProjArgs &A, int64_t m) {
  return m < A.M ? A.rows[m] : u32x2{0u, 0u};
}

// The id of row m as add_adapters takes it.
__device__ __forceinline__ int adapter_of(const ProjArgs &A, int64_t m, bool in) {
  const int id = in && m < A.M ? A.ids[m] : -1;
  return id < A.adapters ? id : -1;
}

// ---------------------------------------------------------------------------
// t
// ---------------------------------------------------------------------------

constexpr int kPreThreads = 1024, kPreWaves = 16;
constexpr int kRowLds = 16384;    // elements of a row of x in LDS
constexpr int kShrinkTile = 256;  // rows among which equal adapters are gathered
constexpr int kShrinkRanks = 4;   // tiles of 16 ranks that share a read of x
constexpr int kPreTiles = 2;      // tiles of 16 rows of a unit of pre_kernel, one in few_kernel

struct PreArgs {
  const uint16_t *x, *a;
  const int32_t *ids;
  const float *scaling;
  uint16_t *xo;     // x as f16_role leaves it
  u32x2 *rows;      // as in ProjArgs
  float *t;
  int64_t M;
  int K, adapters, R, rpb;
  // shrink: blocks, units a tile of rows, tiles of 16 RT ranks, splits of K
  int shrink_blocks, units, rtiles, tsplits;
  int32_t *status;
};

// t of one unit: up to 16 CT rows of one adapter, 16 RT ranks.  The rows of a
// tile that name the same adapter are numbered in order and cut into units, so
// rows in any order share the adapter's A.  One split of K, which the waves
// share; their sums are added in order.  A wave's steps of 32 k go through a
// ring of its own in LDS, where 4 lanes bring a row's 64 bytes: loads straight
// into the matrix cores' operands have 16 lanes on 16 rows, 16 bytes each (64
// ranks of 1900 rows of 14336: 63 us that way, 52 this way, by itself).
constexpr int kShrinkRing = 3;
template <int RT, int CT>
constexpr int shrink_waves() {  // as many as have room, two blocks a CU if CT is 2
  constexpr int n = ((CT == 2 ? 72 : 144) << 10) / (kShrinkRing * (RT + CT) * 1024);
  return n < kPreWaves ? n : kPreWaves;
}
template <int RT, int CT>
constexpr int shrink_lds() {
  return 4 * (kShrinkTile + 16 * CT + 32) + shrink_waves<RT, CT>() * kShrinkRing * (RT + CT) * 1024;
}
template <int RT, int CT>
__device__ __forceinline__ void shrink_role(const PreArgs &A, int64_t blk, unsigned char *smem_raw) {
  constexpr int kUnit = 16 * CT, L = RT + CT, W = shrink_waves<RT, CT>();
  constexpr uint32_t kSlot = L * 1024, kRingOff = 4 * (kShrinkTile + kUnit + 32);
  static_assert(kRingOff % 16 == 0, "");
  int *ids = (int *)smem_raw;                       // [256]
  int *rows = ids + kShrinkTile;                    // [kUnit]
  int *info = rows + kUnit;                         // adapter, leader's rank
  int *counts = info + 4;                           // [16] leaders of each wave
  float *red = (float *)(smem_raw + kRingOff);      // [W][RT][CT][64][4], after the rings
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the same for the block: kept in scalar registers
  const int split = __builtin_amdgcn_readfirstlane((int)(blk % A.tsplits));
  blk /= A.tsplits;
  const int rt = __builtin_amdgcn_readfirstlane((int)(blk % A.rtiles));
  blk /= A.rtiles;
  const int64_t tiles = ceil_div(A.M, kShrinkTile);
  const int unit = (int)(blk / tiles);  // slowest: the last ones may be absent
  const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane((int)(blk % tiles)) * kShrinkTile;
  const int nrows = (int)min((int64_t)kShrinkTile, A.M - m0);
  int id = -1;
  if (tid < nrows) {
    id = A.ids[m0 + tid];
    if (id < -1 || id >= A.adapters) {
      if (unit == 0 && rt == 0 && split == 0 && A.status) atomicOr(A.status, kDevBadAdapter);
      id = -1;
    }
  }
  if (tid < kShrinkTile) ids[tid] = id;
  if (tid < kUnit) rows[tid] = -1;
  if (tid == 0) info[0] = -1;
  __syncthreads();
  int rank = 0;  // among the rows of this adapter
  if (id >= 0) {
#pragma unroll 4
    for (int j = 0; j <= tid / 4; ++j) {
      const u32x4 other = ((const u32x4 *)ids)[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) rank += (int)other[i] == id && 4 * j + i < tid;
    }
  }
  const bool leads = id >= 0 && rank % kUnit == 0;
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
  const int a = __builtin_amdgcn_readfirstlane(info[0]);
  if (a < 0) return;  // fewer units than this
  if (id == a && rank / kUnit == info[1] / kUnit) rows[rank % kUnit] = tid;
  __syncthreads();

  if (wv < W) {
    // slot rows: the unit's rows, then ranks 16 RT rt on; zeros for absent ones
    lds_bytes *ring = (lds_bytes *)smem_raw + kRingOff + (uint32_t)wv * (kShrinkRing * kSlot);
    const uint32_t ld = 2u * (uint32_t)A.K, sl = lane >> 2;
    const uint32_t at = 16u * ((lane & 3u) ^ rows_swz(sl));  // rows 16 apart alike
    const uint16_t *xb = A.x + m0 * A.K, *ab = A.a + (int64_t)a * A.R * A.K;
    uint32_t off[L];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int own = rows[16 * c + sl];
      off[c] = own < 0 ? kNoRow : (uint32_t)own * ld + at;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = 16 * (RT * rt + i) + (int)sl;
      off[CT + i] = r < A.R ? (uint32_t)r * ld + at : kNoRow;
    }
    const int steps = A.K / 32;
    const int s0 = steps * split / A.tsplits, s1 = steps * (split + 1) / A.tsplits;
    // in pairs: 128 consecutive bytes of a row
    const int share = (s1 - s0 + 2 * W - 1) / (2 * W) * 2;
    const int first = min(s0 + wv * share, s1), n = min(first + share, s1) - first;
    auto request = [&](int s, int slot) {  // steps past the end: the last one again, unused
      const int k = __builtin_amdgcn_readfirstlane(32 * max(0, first + min(s, n - 1)));
#pragma unroll
      for (int i = 0; i < L; ++i)
        dma16((i < CT ? xb : ab) + k, ring + (uint32_t)slot * kSlot + 1024u * (uint32_t)i, off[i]);
    };
    f32x4 acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kShrinkRing - 1; ++s) request(s, s);
    const uint32_t get = rows_at((uint32_t)l, (uint32_t)q);
    int slot = 0, put = kShrinkRing - 1;
    for (int s = 0; s < n; ++s) {
      // the slot before has been read; then step s is here when only the
      // newest kShrinkRing - 1 are not
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      request(s + kShrinkRing - 1, put);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kShrinkRing - 1) * L) : "memory");
      bf16x8 v[L];
#pragma unroll
      for (int i = 0; i < L; ++i)
        v[i] = *(lds_bf16x8_c *)(ring + (uint32_t)slot * kSlot + 1024u * (uint32_t)i + get);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = mfma32<false>(v[CT + i], v[c], acc[i][c]);
      put = slot;
      slot = slot == kShrinkRing - 1 ? 0 : slot + 1;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();  // no ring is in use
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c) *(f32x4 *)(red + (((wv * RT + i) * CT + c) * 64 + lane) * 4) = acc[i][c];
  } else {
    __syncthreads();
  }
  __syncthreads();
  for (int o = tid; o < RT * CT * 256; o += kPreThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red[w * (RT * CT * 256) + o];
    const int i = o / (CT * 256), c = o / 256 % CT, ol = o >> 2 & 63;
    const int rr = 16 * (RT * rt + i) + 4 * (ol >> 4) + (o & 3), row = rows[16 * c + (ol & 15)];
    if (row >= 0 && rr < A.R) A.t[((int64_t)split * A.M + m0 + row) * A.R + rr] = A.scaling[a] * sum;
  }
}

// The share of one of A.shrink_blocks blocks of kPreThreads.
template <int RT, int CT>
__device__ __forceinline__ void shrink_all(const PreArgs &A, int block, unsigned char *smem) {
  const int64_t work = ceil_div(A.M, kShrinkTile) * A.units * A.rtiles * A.tsplits;
  for (int64_t w = block; w < work; w += A.shrink_blocks) {
    shrink_role<RT, CT>(A, w, smem);
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// up to 32 rows
// ---------------------------------------------------------------------------

constexpr int kFewRows = 32;           // two 16-row tiles of x
constexpr int kFewWaves = 16;          // most waves of a block
constexpr int kOwnT = -1;
// Most bytes of A that a block reads to make its own t.  One row, 8 ranks: K =
// 1024 (16 KB) 8.1 us this way, 10.6 the other; 3584 (56 KB) 9.9 and 11.4.  64
// KB: one row, 32 ranks of 1024, 11.1 and 10.7; two rows of 16, 11.4 and 10.3.
constexpr int64_t kOwnTBytes = 60 << 10;
constexpr int kFewSetUp = 8;           // least: they share the table and x
constexpr uint32_t kFewX = 64 << 10;   // LDS for a block's slice of x

// Consecutive bytes of a row and their group's scale, or two groups' scales.
template <int BYTES>
struct Raw {
  Bytes<BYTES> w;
  uint32_t scale;
};

// A block: one split of K, and tiles of 16 weight rows (of each matrix) one
// set after another, wt tiles a set; wk waves share a tile.  A unit is 128
// codes, a group or (G = 64) two; a wave works on four units of the 16 rows at
// a time, lane (l, q) on unit q of row l, so that its bytes are two wide loads
// and the four lanes of a row read 104 neighbouring ones.  (With each group
// dealt to four lanes instead, three small loads each, the address units took
// four times as long as the bytes; with 13-byte groups singly, twice.)  Where
// a row has an odd number of 64-groups, its last unit is the last two groups,
// the first of them with scale 0.  Scales are multiplied into the codes, since
// a lane's sums run over all groups.
// x [M,K] (M <= 16 MT) of the split, as f16 times a power of two for each row,
// is put in order once, in LDS; it is the row operand of the matrix cores and W
// the column operand.
// A wave requests its next four units when it has decoded the last, across the
// ends of tiles, and the first before the table is built.  (Two or three ahead
// cost 2 to 4 us more at M = 7, 2 x [14336,4096]: x's loads wait behind them.)
// LDS: 64 KB table, 64 KB x, up to 32 KB for the sums of the waves.
// 2 x [14336,4096], G = 64, takes 19.4 us at 7 rows (28 MB: 1.4 TB/s; 5.4 us at
// copy rate): about 8 before the first sum (a launch's own 4 to 5, the table, x
// put in order), then the decode, 0.25 us a CU for 16 rows by 512 codes of both
// matrices, in which VALU issue is 0.7 busy (0.33 of the whole).  2 x [3584,1024]
// at one row: 7.8 us.
// lora: the projection alone; the first blocks make t meanwhile (RT as in
// shrink_role, 0 for none), and expand_kernel adds the adapters.  Of few rows
// and ranks (RT = kOwnT) every block makes the t of its split, in fp32 beside
// setting up, and adds the adapters to its results: one launch less.
template <int G, int NB, int MT, int ACT, int RT>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(const ProjArgs A, const PreArgs P) {
  constexpr int T = 16, B = bytes_per_group(G), GU = 128 / G;  // matrix steps and groups of a unit
  typedef Lut<32> L;
  constexpr uint32_t kXOff = L::kBytes, kRedOff = kXOff + kFewX;
  __shared__ __align__(16) unsigned char smem_raw[L::kBytes + kFewX + kFewWaves * 2048];
  const int work_blocks = (int)gridDim.x - P.shrink_blocks;
  int block = (int)blockIdx.x;
  constexpr uint32_t kTOff = kRedOff + kFewWaves * 1024;  // kOwnT: t [M][R], behind the sums
  static_assert(RT != kOwnT || (NB == 1 && MT == 1), "the sums leave room");
  if constexpr (RT > 0) {
    if (block < P.shrink_blocks) {
      shrink_all<RT, 1>(P, block, smem_raw);
      return;
    }
    block -= P.shrink_blocks;
  }
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6;
  const int nG = A.K / G, M = (int)A.M;
  const int split = block % A.splits, b0 = block / A.splits;
  const int blocks = work_blocks / A.splits;
  const int nU = (nG + GU - 1) / GU, nQ = (nU + 3) / 4;  // units, and fours of them
  // (at most 4096 fours and as many splits: the products fit)
  const int u0 = 4 * (nQ * split / A.splits), u1 = min(nU, 4 * (nQ * (split + 1) / A.splits));
  const int wk = A.wk, wt = A.wt;        // waves of a tile, tiles of a set
  const int kw = wv % wk, tw = wv / wk;  // this wave's place (tw >= wt: it helps set up)
  const int tiles = (A.N + 15) / 16, sets = (tiles + wt - 1) / wt;
  const int steps = b0 < sets ? (sets - b0 + blocks - 1) / blocks : 0;
  const int quads = (u1 - u0 + 3) / 4, batches = (quads + wk - 1) / wk;  // of a tile

  // the set of step j is b0 + j * blocks
  auto tile_row = [&](int j) { return ((b0 + j * blocks) * wt + tw) * 16; };
  const bool active = tw < wt;
  int fj = 0, fk = 0;  // step and batch of the next request
  Raw<26> f[NB];
  auto fetch = [&]() {
    if (!active) return;
    const int n0 = tile_row(fj), quad = kw + wk * fk;
    // rows past N read row N - 1 and units past the last read it, with scales
    // 0; neither is stored or counts
    const int64_t n = min(n0 + l, A.N - 1);
    const int u = u0 + 4 * quad + q, g = GU * min(u, u1 - 1);
    const int64_t at = n * nG + min(g, nG - GU);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      f[i].w = load_bytes<26>(A.packed[i] + at * B);
      uint32_t sc;
      if constexpr (G == 128) {
        sc = A.scales[i][at];
      } else {
        __builtin_memcpy(&sc, A.scales[i] + at, 4);
        if (g + 1 == nG) sc &= 0xFFFF0000u;  // the first of the two belongs to the unit before
      }
      f[i].scale = u < u1 ? sc : 0u;
    }
    if (++fk == batches) {
      fk = 0;
      ++fj;
    }
  };

  // the first bytes are requested before the table is built and x put in order
  fetch();
  L::build(smem, tid, threads);
  // spans of the rows, [wave][row], where the sums will be
  auto span_at = [&](int w, int m) {
    return (__attribute__((address_space(3))) uint32_t *)(smem + kRedOff + 4u * (uint32_t)(w * kFewRows + m));
  };
  // rows are shared by the waves, `parts` waves a row
  const int parts = max(1, waves / M);
  const uint16_t *xs = A.x + (int64_t)u0 * 128;
  const int len = min(A.K - u0 * 128, (u1 - u0) * 128);
  {
    const int part = wv % parts;
    for (int m = wv / parts; m < M; m += waves / parts) {
      SpanOf of;
#pragma unroll 4
      for (int k = 8 * (64 * part + lane); k < len; k += 512 * parts)
        of.take(*(const u32x4 *)(xs + (int64_t)m * A.K + k));
      const uint32_t span = span_wave(of.word());
      if (lane == 0) *span_at(part, m) = span;
    }
    if constexpr (RT == kOwnT) {
      if (block == 0 && tid < M && A.status) {
        const int id = A.ids[tid];
        if (id < -1 || id >= A.adapters) atomicOr(A.status, kDevBadAdapter);
      }
      for (int o = wv; o < M * A.R; o += waves) {  // a wave a rank
        const int m = o / A.R, r = o - m * A.R, id = A.ids[m];
        float sum = 0.f;
        if (id >= 0 && id < A.adapters) {
          const uint16_t *ar = P.a + ((int64_t)id * A.R + r) * A.K + (int64_t)u0 * 128;
          const uint16_t *xr = xs + (int64_t)m * A.K;
#pragma unroll 8
          for (int k = 8 * lane; k < len; k += 512) {
            const u32x4 av = *(const u32x4 *)(ar + k), xv = *(const u32x4 *)(xr + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum = fmaf(bf16_to_f32((uint16_t)av[i]), bf16_to_f32((uint16_t)xv[i]), sum);
              sum = fmaf(bf16_to_f32((uint16_t)(av[i] >> 16)), bf16_to_f32((uint16_t)(xv[i] >> 16)), sum);
            }
          }
#pragma unroll
          for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
          sum *= P.scaling[id];
        }
        if (lane == 0) *(__attribute__((address_space(3))) float *)(smem + kTOff + 4u * (uint32_t)o) = sum;
      }
    }
  }
  __syncthreads();
  auto span_of = [&](int m) {
    uint32_t span = 0;
    for (int w = 0; w < parts; ++w) span = span_join(span, *span_at(w, m));
    return span;
  };
  // of row `lane`: its power of two, and what it loses; and the rows that lose
  // something, the same in every wave
  const uint32_t span_own = span_of(min(lane, M - 1));
  const int shift_own = f16_shift(span_top(span_own));
  float lost = 0.f;
  const uint32_t lossy = (uint32_t)__ballot(lane < M && span_loses(span_own));
#pragma unroll 1
  for (uint32_t todo = lossy; todo; todo &= todo - 1) {
    const int m = __builtin_ctz(todo), shift = __builtin_amdgcn_readlane(shift_own, m);
    float sum = 0.f;
    for (int k = 8 * lane; k < len; k += 512) sum += lost_of(*(const u32x4 *)(xs + (int64_t)m * A.K + k), shift);
    sum = wave_sum(sum);
    lost = lane == m ? sum : lost;
  }
  {
    // a piece: the five steps of 40 codes, or those that are left, of a group
    // of a row
    constexpr int U = (G + 39) / 40, kLast = G - 40 * (U - 1);
    const int pieces = quads * 4 * GU * U;
    for (int o = tid; o < pieces * M; o += threads) {
      const int m = o / pieces, e = o - m * pieces, shift = f16_shift(span_top(span_of(m)));
      const int slot = e / U, piece = e - slot * U;  // slot: a group's place
      // in a row's odd last unit the last group comes second
      int g = GU * u0 + slot;
      if (GU == 2 && (nG & 1)) g = g == nG ? nG - 1 : g == nG - 1 ? nG : g;
      const bool in = g < min(nG, GU * u1), last = piece == U - 1;
      const int count = last ? kLast : 40;
      const uint16_t *p = A.x + (int64_t)m * A.K + (int64_t)(in ? g : 0) * G + 40 * piece;
      uint16_t v[40];
#pragma unroll
      for (int s = 0; s < 5; ++s) *(u32x4 *)(v + 8 * s) = *(const u32x4 *)(p + (8 * s < count ? 8 * s : 0));
#pragma unroll
      for (int s = 0; s < 5; ++s) {
        if (8 * s >= count) break;
        _Float16 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // the codes past a group's tens are in their own order
          const int c = 8 * s + i;
          const uint16_t tens = v[group_source<40>(c)];
          f[i] = f16_of(!in ? 0 : last && c >= kLast / 10 * 10 ? v[c] : tens, shift);
        }
        // [quad][step][unit of the quad][row]
        const int unit = slot / GU, step = (slot % GU) * (T / GU) + 5 * piece + s;
        *(lds_u32x4 *)(smem + kXOff + 16u * (uint32_t)((((unit >> 2) * T + step) * 4 + (unit & 3)) * M + m)) =
            *(u32x4 *)f;
      }
    }
  }
  __syncthreads();

  const L lut(0, lane);
  uint32_t xlane[MT];  // rows past M: row M - 1
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) xlane[mt] = kXOff + 16u * (uint32_t)(q * M + min(16 * mt + l, M - 1));
  uint32_t flags = 0;
  f32x4 acc[NB][MT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[i][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
  int j = 0, k = 0;  // step and batch being worked on
  const int total = steps * batches;
  for (int t = 0; t < total; ++t) {
    const int n0 = tile_row(j), quad = kw + wk * k;
    if (active && n0 < A.N && quad < quads) {
      const uint32_t xq = 64u * (uint32_t)(quad * T * M);
      // five steps at a time: eight bytes of each matrix, of the group at byte
      // OFF whose steps start at S
      auto part = [&](auto p0, auto p1, auto tail, auto which) {
        constexpr int P0 = decltype(p0)::value, P1 = decltype(p1)::value, H = decltype(which)::value;
        constexpr int S = H * (T / GU), OFF = H * B;
        constexpr int S0 = 5 * P0 / 4, S1 = decltype(tail)::value ? G / 8 : 5 * P1 / 4;
        bf16x8 xf[S1 - S0][MT];
#pragma unroll
        for (int s = S0; s < S1; ++s)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            xf[s - S0][mt] = *(lds_bf16x8_c *)(smem + xlane[mt] + xq + 64u * (uint32_t)((S + s) * M));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          uint32_t d[G / 2];
          const uint32_t sc = f[i].scale;
          const f16x2 two = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(sc, sc, H ? 0x03020302u : 0x01000100u));
          decode_group<G, P0, P1, decltype(tail)::value, OFF>(smem, lut, f[i].w, two, d, flags);
#pragma unroll
          for (int s = S0; s < S1; ++s)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              acc[i][mt] = mfma32<true>(
                  xf[s - S0][mt],
                  __builtin_bit_cast(bf16x8, u32x4{d[4 * s], d[4 * s + 1], d[4 * s + 2], d[4 * s + 3]}),
                  acc[i][mt]);
          __builtin_amdgcn_sched_barrier(0);  // one part's registers at a time
        }
      };
      if constexpr (G == 128) {
        part(Int<0>{}, Int<4>{}, Int<0>{}, Int<0>{});
        part(Int<4>{}, Int<8>{}, Int<0>{}, Int<0>{});
        part(Int<8>{}, Int<12>{}, Int<1>{}, Int<0>{});
      } else {
        part(Int<0>{}, Int<4>{}, Int<0>{}, Int<0>{});
        part(Int<4>{}, Int<6>{}, Int<1>{}, Int<0>{});
        part(Int<0>{}, Int<4>{}, Int<0>{}, Int<1>{});
        part(Int<4>{}, Int<6>{}, Int<1>{}, Int<1>{});
      }
    }
    fetch();
    if (++k < batches) continue;
    k = 0;
    // the tile's last batch: the waves' sums, in wave order; a matrix and 16
    // rows of x at a time where LDS holds no more
    constexpr int kOnce = NB * MT > 2 ? 1 : MT;  // 16-row tiles a pass (with all matrices)
    static_assert(kFewWaves * NB * kOnce * 1024 <= kFewWaves * 2048, "the sums' LDS");
#pragma unroll
    for (int c0 = 0; c0 < MT; c0 += kOnce) {
      __syncthreads();  // the sums before have been read
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int ct = 0; ct < kOnce; ++ct) {
          const int mt = c0 + ct;
          f32x4 v;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = ldexpf(acc[i][mt][c], -__shfl(shift_own, 16 * mt + 4 * q + c));
          *(__attribute__((address_space(3))) f32x4 *)(smem + kRedOff + 16u * (uint32_t)(((i * kOnce + ct) * waves + wv) * 64 + lane)) = v;
          acc[i][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      __syncthreads();
      for (int o = tid; o < wt * kOnce * 256; o += threads) {  // [tile][16-row tile][row][column]
        const int ct = (o >> 8) % kOnce, ts = (o >> 8) / kOnce;
        const int mr = (o >> 4) & 15, m = 16 * (c0 + ct) + mr;
        const int n0 = ((b0 + j * blocks) * wt + ts) * 16, n = n0 + (o & 15);
        const bool in = m < M && n < A.N;
        if (!lossy && !in) continue;
        // row mr of column c is element mr % 4 of lane 16 (mr / 4) + c
        const uint32_t at = kRedOff + 16u * (uint32_t)(ts * wk * 64 + (mr >> 2) * 16 + (o & 15)) + 4u * (mr & 3);
        float v[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          v[i] = 0.f;
          for (int w = 0; w < wk; ++w)
            v[i] += *(__attribute__((address_space(3))) float *)(smem + at + 1024u * (uint32_t)((i * kOnce + ct) * waves + w));
        }
        if (lossy) {  // a wave's 64 results are of one tile
          const float mine = __shfl(lost, m);
          bool low = false;
#pragma unroll
          for (int i = 0; i < NB; ++i)
            low = low || fabsf(v[i]) < kLostCounts * mine * scale_top(A, i, n0, 16, nG);
          for (uint64_t todo = __ballot(in && low); todo; todo &= todo - 1) {
            const int r = __builtin_ctzll(todo);
            const int mm = __builtin_amdgcn_readlane(m, r), nn = __builtin_amdgcn_readlane(n, r);
            const int sh = __builtin_amdgcn_readlane(shift_own, mm);
            const int sp = uniform_here(split), g0 = GU * 4 * (nQ * sp / A.splits);
            const int g1 = min(nG, GU * 4 * (nQ * (sp + 1) / A.splits));
#pragma unroll 1
            for (int i = 0; i < NB; ++i) {
              const float add = lost_part<G, false>(A, i, mm, nn, g0, g1, sh);
#pragma unroll
              for (int k = 0; k < NB; ++k) v[k] += lane == r && k == i ? add : 0.f;
            }
          }
          if (!in) continue;
        }
        if constexpr (RT == kOwnT) {
          const int id = A.ids[m];
          if (id >= 0 && id < A.adapters) {
            const uint16_t *br = A.b + ((int64_t)id * A.N + n) * A.R;
            float add = 0.f;
            for (int r = 0; r < A.R; r += 8) {
              const u32x4 bv = *(const u32x4 *)(br + r);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float t = *(__attribute__((address_space(3))) float *)(smem + kTOff + 4u * (uint32_t)(m * A.R + r + i));
                add = fmaf(t, bf16_to_f32((uint16_t)(bv[i / 2] >> (i & 1 ? 16 : 0))), add);
              }
            }
            v[0] += add;
          }
        }
        const int64_t at_out = (int64_t)m * A.N + n;
        if (A.splits > 1) {
#pragma unroll
          for (int i = 0; i < NB; ++i) A.partial[((int64_t)split * NB + i) * M * A.N + at_out] = v[i];
        } else if constexpr (NB == 2) {
          ((uint16_t *)A.out)[at_out] = f32_to_bf16(act_value<ACT>(v[0]) * v[1]);
        } else {
          ((float *)A.out)[at_out] = v[0];
        }
      }
    }
    ++j;
  }
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);
}

// ---------------------------------------------------------------------------
// some rows
// ---------------------------------------------------------------------------

constexpr int kMidWaves = 8, kMidThreads = 64 * kMidWaves;
constexpr int kMidRows = 64;  // of x a block

// A block: 128 weight rows (of each matrix), a tile of 16 a wave; one chunk of
// 64 rows of x; one split of K, in whole quads of groups.  Lane (l, q) decodes
// group q of a quad of row l; x comes in the same order and as f16 (f16_role), four
// matrix steps at a time, through a ring of LDS slots that all waves read.
// A quad's decode, its x from LDS and its MFMAs take, by count, 2000, 4000 and
// 2000 cycles of a CU with two blocks and overlap in part: 3.8 us for 256 k of one
// matrix, 5 of two.  333 rows by 2 x [3584,1024]: 17 us, 0.3 PFLOP/s.
template <int G, int NB, int ACT>
__global__ __launch_bounds__(kMidThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void mid_kernel(const ProjArgs A) {
  constexpr int MT = kMidRows / 16, T = G / 8, B = bytes_per_group(G), SQ = T / 4;  // SQ: stages of a quad
  typedef Lut<8> L;
  constexpr uint32_t kSlot = 4 * MT * 1024, kLoad = 16 * kMidThreads;
  constexpr int kD = kSlot / kLoad;      // loads of x a thread and stage
  constexpr int kSlots = 65536 / kSlot;  // 80 KB in all: two blocks a CU
  __shared__ __align__(16) unsigned char smem_raw[L::kBytes + kSlots * kSlot];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  lds_bytes *ring = smem + L::kBytes;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nG = A.K / G, nQ = (nG + 3) / 4;
  int b = (int)blockIdx.x;
  const int chunk = b % A.chunks;
  b /= A.chunks;
  const int split = b % A.splits, n0 = (b / A.splits) * 128 + 16 * wv;
  const int q0 = (int)((int64_t)nQ * split / A.splits);
  const int q1 = (int)((int64_t)nQ * (split + 1) / A.splits);
  const int64_t m0 = (int64_t)chunk * (16 * MT);

  // rows past N read row N - 1; their sums are not stored
  const int64_t n = min(n0 + l, A.N - 1);
  Raw<B> ra[NB], rb[NB];
  auto fetch = [&](Raw<B>(&r)[NB], int quad) {  // always: the waits below count on its loads
    // groups past the last read it, with scale 0
    const int g = 4 * quad + q;
    const int64_t at = n * nG + min(g, nG - 1);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      r[i].w = load_bytes<B>(A.packed[i] + at * B);
      const uint32_t sc = A.scales[i][at];
      r[i].scale = g < nG ? sc : 0u;
    }
  };
  const uint16_t *xbase = A.x + (int64_t)chunk * nQ * SQ * (kSlot / 2);
  int put = 0;  // slot of the next request
  auto request = [&](int s) {  // stage s of the whole of K
#pragma unroll
    for (int i = 0; i < kD; ++i)
      dma16_tracked(xbase + (int64_t)s * (kSlot / 2),
                    ring + (uint32_t)put * kSlot + (uint32_t)(i * kLoad) + 1024u * (uint32_t)wv,
                    s < q1 * SQ ? (uint32_t)(i * kLoad + 16 * tid) : kNoRow);
    put = put == kSlots - 1 ? 0 : put + 1;
  };

  fetch(ra, q0);
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) request(q0 * SQ + s);
  L::build(smem, tid, kMidThreads);
  f32x4 acc[NB][MT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[i][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto shift_rows = [&](int sign, u32x2 of_row, int q) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int sh = sign * __shfl((int)of_row.x, 16 * mt + 4 * q + c);
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i][mt][c] = ldexpf(acc[i][mt][c], sh);
      }
  };
  if constexpr (NB == 1) {
    // the adapters' part while the first bytes are on their way, times
    // 2^shift as the sums that follow; the splits share the adapters.  (What is
    // below 2^-140 of the row's largest element loses bits by that; after the
    // product instead, 1 to 6% slower, it would not.)
    if (A.adapters > 0 && n0 < A.N) {
      const int id = adapter_of(A, m0 + lane, lane < 16 * MT);
      // Adapters one after another, or results one after another: 4000 rows of
      // 592 columns, 8 and 16 ranks, with 32 adapters 71 and 55 us, with 4 45 and
      // 49; with 64 ranks 99 and 124, 55 and 107.
      if (2 * __popcll(adapter_leaders(id)) > A.R)
        add_own_adapters(A, m0, n, id, A.splits, split, acc[0]);
      else
        add_adapters<false>(A, m0, n0, id, A.splits, split, acc);
      shift_rows(1, row_scale(A, m0 + lane), q);
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const L lut(0, lane);
  uint32_t flags = 0;
  int get = 0;
  auto quad_of = [&](int quad, Raw<B>(&r)[NB], Raw<B>(&next)[NB]) {
    uint32_t d[NB][G / 2];
    auto stage = [&](auto sc) {
      constexpr int S = decltype(sc)::value;
      request(quad * SQ + S + kSlots - 1);
      if constexpr (S == 0) fetch(next, quad + 1);
      lds_bytes *x = ring + (uint32_t)get * kSlot + 16u * (uint32_t)lane;
      get = get == kSlots - 1 ? 0 : get + 1;
      // the byte pairs whose first dword is among this stage's sixteen
      constexpr int P = G / 10, P0 = (16 * S + 4) / 5, P1 = (16 * S + 20) / 5 < P ? (16 * S + 20) / 5 : P;
#pragma unroll
      for (int i = 0; i < NB; ++i)
        decode_group<G, P0, P1, S == SQ - 1, 0>(
            smem, lut, r[i].w, __builtin_bit_cast(f16x2, r[i].scale * 0x10001u), d[i], flags);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const bf16x8 xf = *(lds_bf16x8_c *)(x + 1024u * (uint32_t)(s * MT + mt));
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const uint32_t *w = d[i] + 16 * S + 4 * s;
            acc[i][mt] =
                mfma32<true>(xf, __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]}), acc[i][mt]);
          }
        }
      // x of the next stage was requested kSlots - 2 stages ago, before at
      // least the x requests of the stages since and, if the quad's first
      // stage is one of them, three loads a matrix
      constexpr int kSince = kSlots - 2;
      constexpr bool kFetched = S < kSince;
      constexpr int kOut = kSince * kD + (kFetched ? 3 * NB : 0);
      // every read of this stage's slot is done before the barrier: the next
      // stage's request may fill it at once (one past the end needs no memory)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kOut) : "memory");
    };
    stage(Int<0>{});
    stage(Int<1>{});
    if constexpr (SQ == 4) {
      stage(Int<2>{});
      stage(Int<3>{});
    }
  };
  for (int quad = q0; quad < q1; quad += 2) {
    quad_of(quad, ra, rb);
    if (quad + 1 < q1) quad_of(quad + 1, rb, ra);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may still write this block's LDS
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);

  {
    static_assert(kMidRows == 64, "a row of x a lane");
    // from here on: kept through the loop they would cost it registers
    const int lane = lane_here(), l = lane & 15, q = lane >> 4;
    const u32x2 of_row = row_scale(A, m0 + lane);
    shift_rows(-1, of_row, q);
    const float lost = __uint_as_float(of_row.y);
    uint32_t low = 0;  // sums that may lack something: bit 4 mt + c, of either matrix
    if (__ballot(lost > 0.f)) {
      float most[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) most[i] = kLostCounts * scale_top(A, i, n0, 16, nG);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float mine = __shfl(lost, 16 * mt + 4 * q + c);
#pragma unroll
          for (int i = 0; i < NB; ++i)
            if (m0 + 16 * mt + 4 * q + c < A.M && n0 + l < A.N && fabsf(acc[i][mt][c]) < most[i] * mine)
              low |= 1u << (4 * mt + c);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t m = m0 + 16 * mt + 4 * q + c;
        if (m >= A.M || n0 + l >= A.N) continue;
        const int64_t o = m * A.N + n0 + l;
        if (A.splits > 1) {
#pragma unroll
          for (int i = 0; i < NB; ++i) A.partial[((int64_t)split * NB + i) * A.M * A.N + o] = acc[i][mt][c];
        } else if constexpr (NB == 2) {
          ((uint16_t *)A.out)[o] = f32_to_bf16(act_value<ACT>(acc[0][mt][c]) * acc[1][mt][c]);
        } else {
          ((float *)A.out)[o] = acc[0][mt][c];
        }
      }
    while (const uint64_t todo = __ballot(low != 0)) {
      const int r = __builtin_ctzll(todo);
      const int e = __builtin_ctz((uint32_t)__builtin_amdgcn_readlane((int)low, r));
      low &= lane == r ? ~(1u << e) : ~0u;
      mend_result<G, NB, ACT>(A, m0 + 16 * (e / 4) + 4 * (r / 16) + e % 4, n0 + r % 16, split, 4 * q0,
                              min(nG, 4 * q1), lane == r);
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

// After few_kernel: y = the splits' partial sums in order (y itself where
// there is one split) + the adapters' part.  A block: 16 columns, all rows, a
// result a thread: its row's t comes from LDS and its row of B, whose
// neighbours lie beside it, from memory; fp32 throughout.  (On the matrix cores,
// each adapter for all rows, 32 adapters of 16 ranks by 4096 columns took 10.3 us
// and this 5.8.)
template <int MT>
__global__ __launch_bounds__(256 * MT) void expand_kernel(const ProjArgs A) {
  constexpr int kHeld = 4;                   // eights of ranks held in registers
  __shared__ __align__(16) float t[16 * MT * 260];  // [row][R + 4]: rows in different banks
  const int tid = threadIdx.x, m = tid >> 4, n = (int)blockIdx.x * 16 + (tid & 15), ld = A.R + 4;
  const bool mine = m < A.M && n < A.N;
  const int id = mine ? A.ids[m] : -1;
  const bool has = id >= 0 && id < A.adapters;
  const uint16_t *b = A.b + (has ? ((int64_t)id * A.N + n) * A.R : 0);
  u32x4 held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (has && 8 * i < A.R) held[i] = *(const u32x4 *)(b + 8 * i);
  const int MR = (int)A.M * A.R;
  for (int o = tid; A.adapters > 0 && o < MR; o += 256 * MT) {
    float v = A.t[o];
    for (int s = 1; s < A.tsplits; ++s) v += A.t[(int64_t)s * MR + o];
    t[o / A.R * ld + o % A.R] = v;
  }
  float v = 0.f;
  if (mine) {
    const float *p = (A.splits > 1 ? A.partial : (const float *)A.out) + (int64_t)m * A.N + n;
    const int64_t mn = A.M * A.N;
#pragma unroll 8
    for (int s = 0; s < A.splits; ++s) v += p[s * mn];
  }
  __syncthreads();
  if (!mine) return;
  if (has) {
    float add = 0.f;
    auto eight = [&](u32x4 w, int r) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        add = fmaf(t[m * ld + r + i], bf16_to_f32((uint16_t)(w[i / 2] >> (i & 1 ? 16 : 0))), add);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (8 * i < A.R) eight(held[i], 8 * i);
    for (int r = 8 * kHeld; r < A.R; r += 8) eight(*(const u32x4 *)(b + r), r);
    v += add;
  }
  ((float *)A.out)[(int64_t)m * A.N + n] = v;
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kWideP = 256, kWideQ = 256, kWideThreads = 512;
constexpr int kWideX = 5, kWideC = 4;  // slots of x, and of codes

// 256 rows of W (NB = 1) or 128 of each of two (NB = 2) by 256 rows of x, in
// stages of 32 k; codes times their scale and x as f16 (both exact, see
// f16_role), so that one fp32 sum runs over all of K.
// While the MFMAs of stage s run, a wave
//   - reads the fragments of s + 1,
//   - decodes the codes of s + 3: two threads a weight row, three bytes and
//     one of the group's left-over codes each,
//   - requests x of s + 4 and the bytes of s + 7.
// LDS: 80 KB x, 64 KB codes, 16 KB table.  K is split between blocks when the
// tiles are few.
// A stage takes 0.85 us (1.26 PFLOP/s on all CUs; a library's bf16 product
// reaches 1.45): LDS is busy 0.4 of it, the MFMAs 0.55 to 0.6.  2 x
// [14336,4096] by 2048 rows: 442 us a call, 11 of them before it, 1.12 PFLOP/s,
// 3.5 tiles a CU.
template <int G, int NB, int ACT>
__global__ __launch_bounds__(kWideThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void wide_kernel(const ProjArgs A) {
  constexpr int S32 = G / 32, WP = 2, WQ = 4, TP = 8, TQ = 4, B = bytes_per_group(G);
  typedef Lut<8> L;
  constexpr uint32_t kPSlot = kWideP * kKS * 2, kQSlot = kWideQ * kKS * 2;
  constexpr int kXLoads = kQSlot / 16 / kWideThreads;  // a thread's requests of x in a stage
  constexpr uint32_t kQOff = kWideC * kPSlot, kLutOff = kQOff + kWideX * kQSlot;
  __shared__ __align__(16) unsigned char smem_raw[kLutOff + L::kBytes];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wv / WQ, wq = wv % WQ;
  const int nG = A.K / G, tiles = A.tp * A.tq, split = (int)blockIdx.x / tiles;
  // this block's groups, and its stages counted from the first
  const int g0 = (int)((int64_t)nG * split / A.splits);
  const int g1 = (int)((int64_t)nG * (split + 1) / A.splits);
  const int S = (g1 - g0) * S32;

  int ip, iq;
  tile_of_block((int)blockIdx.x - split * tiles, tiles, A.tp, A.tq, ip, iq);
  constexpr int HP = kWideP / WP / NB;  // rows of one matrix in a wave
  const int n0 = ip * (kWideP / NB);
  const int64_t q0 = (int64_t)iq * kWideQ;

  // this thread's weight row: slot row tid / 2; rows past N read row N - 1.  A
  // wave's 32 slot rows are of one matrix: the tile starts at a scalar address.
  static_assert(HP % 32 == 0, "");
  const int sr = tid >> 1, hf = tid & 1;
  const int which = NB == 1 ? 0 : wv * 32 % (NB * HP) / HP;
  const uint32_t first = (uint32_t)min(sr / (NB * HP) * HP + sr % HP, A.N - 1 - n0) * (uint32_t)nG;
  const uint32_t poff = first * B + 3u * hf, toff = first * B, soff = first * 2u;
  const Scalar bytes(A.packed[which] + ((int64_t)n0 * nG + g0) * B);
  const Scalar values(A.scales[which] + (int64_t)n0 * nG + g0);
  // bytes and group values are requested four stages before they are decoded
  constexpr int kGroups = 4 / S32;  // groups of four stages
  uint32_t raw[4], tail_next[kGroups], scale_next[kGroups], scale = 0, flags = 0;
  u32x2 left{0u, 0u};  // high bytes of the group's left-over codes
  // bytes of stage s, J = s % 4 (past the end: of the last group)
  auto load_raw = [&](int s, auto jc) {
    constexpr int J = decltype(jc)::value;
    const int g = min(s / S32, nG - 1 - g0);
    raw[J] = bytes.load4(poff, g * B + 6 * (J % S32));
    if constexpr (J % S32 == 0) {
      tail_next[J / S32] = G == 128 ? bytes.load2(toff, g * B + 24) : bytes.load1(toff, g * B + 12);
      scale_next[J / S32] = values.load2(soff, g * 2);
    }
  };
  const L lut(kLutOff, tid & 63);
  const uint32_t put0 = rows_at((uint32_t)sr, 2u * hf), put1 = rows_at((uint32_t)sr, 2u * hf + 1u);
  // codes of the stage whose bytes are raw[J], J = its index % 4, -> slot: the
  // table's entries first, some work of others' between, then the rest
  auto look_up = [&](auto jc) {
    constexpr int J = decltype(jc)::value;
    if constexpr (J % S32 == 0) {
      scale = scale_next[J / S32] * 0x10001u;
      left = leftover_pool<G>(smem, lut, tail_next[J / S32], flags);
    }
    return look_up_eighth(smem, lut, raw[J]);
  };
  auto decode = [&](auto jc, const Eighth &t, uint32_t slot) {
    constexpr int J = decltype(jc)::value;
    u32x4 c0, c1;
    decode_eighth(t, left, (uint32_t)(2 * (J % S32) + hf), scale, c0, c1, flags);
    *(lds_u32x4 *)(smem + slot + put0) = c0;
    *(lds_u32x4 *)(smem + slot + put1) = c1;
  };

  // a stage of x is the image of its slot; past the end the last one again
  const uint16_t *qbase = A.x + q0 * A.K + (int64_t)g0 * S32 * (kWideQ * kKS);
  const uint32_t xoff = 16u * (uint32_t)tid;
  int xput = 0;  // slot of the next request
  auto request = [&](int s, int i) {
    dma16_tracked(qbase + (int64_t)min(s, S - 1) * (kWideQ * kKS) + i * (8 * kWideThreads),
                  smem + kQOff + (uint32_t)xput * kQSlot + 16u * (uint32_t)(i * kWideThreads + 64 * wv), xoff);
    if (i == kXLoads - 1) xput = xput == kWideX - 1 ? 0 : xput + 1;
  };

  // ---- prologue: bytes of stages 0 .. 6, x of 0 .. 3, codes of 0 .. 2 ----
  load_raw(0, Int<0>{});
  load_raw(1, Int<1>{});
  load_raw(2, Int<2>{});
  load_raw(3, Int<3>{});
#pragma unroll
  for (int s = 0; s < kWideX - 1; ++s)
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) request(s, i);
  L::build(smem + kLutOff, tid, kWideThreads);
  __syncthreads();
  decode(Int<0>{}, look_up(Int<0>{}), 0);
  load_raw(4, Int<0>{});
  decode(Int<1>{}, look_up(Int<1>{}), kPSlot);
  load_raw(5, Int<1>{});
  decode(Int<2>{}, look_up(Int<2>{}), 2 * kPSlot);
  load_raw(6, Int<2>{});

  Frags<kRows, kWideP, TP> pf;
  Frags<kRows, kWideQ, TQ> qf;
  pf.init(tid & 63, wp * (kWideP / WP));
  qf.init(tid & 63, wq * (kWideQ / WQ));
  f32x4 acc[TP][TQ];
#pragma unroll
  for (int a = 0; a < TP; ++a)
#pragma unroll
    for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  bf16x8 pa[TP], qa[TQ], qb[TQ];
  // a wait that the compiler sees: inside the loop it then counts only the
  // loop's own loads, instead of waiting, on every pass, for the newest ones in
  // case they were these
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int b = 0; b < TQ; ++b) qa[b] = qf.read(smem, kQOff, b);
#pragma unroll
  for (int a = 0; a < TP; ++a) pa[a] = pf.read(smem, 0, a);

  int xget = 1;  // slot of x of stage s + 1
  auto stage = [&](int s, auto jc, bf16x8(&qc)[TQ], bf16x8(&qn)[TQ]) {
    constexpr int J = decltype(jc)::value;  // s % 4
    const uint32_t pn = (uint32_t)((J + 1) % kWideC) * kPSlot;
    const uint32_t qn0 = kQOff + (uint32_t)xget * kQSlot;
    xget = xget == kWideX - 1 ? 0 : xget + 1;
    Eighth next;
#pragma unroll
    for (int a = 0; a < TP; ++a) {
      // rows stay apart: reads spread between the MFMAs, the table's entries
      // three rows before their use
      __builtin_amdgcn_sched_barrier(0);
      if (a == 0) next = look_up(Int<(J + 3) % 4>{});
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = mfma32<true>(pa[a], qc[b], acc[a][b]);
      // the codes are written before the fragments of rows 4 .. 7 are read:
      // when the last of those is used, in stage s + 1, the writes are done, a
      // barrier before stage s + 2 reads them
      if (a == 3) decode(Int<(J + 3) % 4>{}, next, (uint32_t)((J + 3) % kWideC) * kPSlot);
      if (a >= 3 && a < 3 + TQ) qn[a - 3] = qf.read(smem, qn0, a - 3);
      pa[a] = pf.read(smem, pn, a);
      if (a >= 1 && a <= kXLoads) request(s + kWideX - 1, a - 1);
      if (a == 5) load_raw(s + 7, Int<(J + 7) % 4>{});
    }
    __builtin_amdgcn_sched_barrier(0);
    // x of stage s + 2 was requested in stage s - 2: at least the bytes of
    // that stage and three loads of each of s - 1 and s follow it
    asm volatile("s_waitcnt vmcnt(7)\n\ts_barrier" ::: "memory");
  };
  int s = 0;
  for (; s + 4 <= S; s += 4) {
    stage(s, Int<0>{}, qa, qb);
    stage(s + 1, Int<1>{}, qb, qa);
    stage(s + 2, Int<2>{}, qa, qb);
    stage(s + 3, Int<3>{}, qb, qa);
  }
  if (S32 == 2 && s < S) {
    stage(s, Int<0>{}, qa, qb);
    stage(s + 1, Int<1>{}, qb, qa);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);

  // ---- epilogue: lane holds rows n = 16 a + 4 (lane / 16) + r, column
  // m = 16 b + lane % 16 ----
  const int lane = lane_here(), l = lane & 15, q = lane >> 4;
  const int64_t mq = q0 + wq * (kWideQ / WQ) + l;
  const int64_t mw = q0 + wq * (kWideQ / WQ);  // the wave's 64 rows of x, one a lane
  static_assert(kWideQ / WQ == 64 && 16 * TQ == 64, "");
  // what x's row of column b needs: read by each lane, or one a lane and handed
  // over (each way leaves the loop above without spills where it is used)
  struct Rows {
    u32x2 own;
    __device__ __forceinline__ u32x2 of(const ProjArgs &A, int64_t mw, int l, int b) const {
      if constexpr (NB == 2) return row_scale(A, mw + 16 * b + l);
      return u32x2{(uint32_t)__shfl((int)own.x, 16 * b + l), (uint32_t)__shfl((int)own.y, 16 * b + l)};
    }
  };
  const Rows for_shift{NB == 2 ? u32x2{} : row_scale(A, mw + lane)};
#pragma unroll
  for (int b = 0; b < TQ; ++b) {
    const int sh = -(int)for_shift.of(A, mw, l, b).x;
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[a][b][r] = ldexpf(acc[a][b][r], sh);
  }
  const bool vec = (A.N & 3) == 0 && (reinterpret_cast<uintptr_t>(A.out) & 15) == 0;
  const int nw = n0 + wp * HP;  // first row of this wave
  const bool rows8 = nw + HP <= A.N && (A.N & 7) == 0 && (reinterpret_cast<uintptr_t>(A.out) & 15) == 0;
  auto store_f32 = [&](float *y, int64_t m, int n, f32x4 v, bool aligned) {
    float *o = y + m * A.N + n;
    if (aligned && n < A.N) {
      *(f32x4 *)o = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < A.N) o[r] = v[r];
    }
  };
  if constexpr (NB == 1) {
    if (A.adapters > 0) {
      // the wave's 64 columns, one a lane; the splits share the adapters
      add_adapters<true>(A, mw, nw, adapter_of(A, mw + lane, true), A.splits, split, acc);
    }
  }
  const Rows for_lost{row_scale(A, mw + lane_here())};
  uint32_t low[TQ] = {};  // sums that may lack something: bit 4 a + r, of either matrix
  if (__ballot(__uint_as_float(for_lost.own.y) > 0.f)) {
    float most[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) most[i] = kLostCounts * scale_top(A, i, nw, HP, nG);
#pragma unroll
    for (int b = 0; b < TQ; ++b) {
      const float lost = __uint_as_float(for_lost.of(A, mw, l, b).y);
#pragma unroll
      for (int a = 0; a < TP; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int of = a % (TP / NB);
          if (mq + 16 * b < A.M && nw + 16 * of + 4 * q + r < A.N &&
              fabsf(acc[a][b][r]) < most[a / (TP / NB)] * lost)
            low[b] |= 1u << (4 * of + r);
        }
    }
  }
#pragma unroll
  for (int b = 0; b < TQ; ++b) {
    const int64_t m = mq + 16 * b;
    if (A.splits > 1) {
      if (m >= A.M) continue;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int a = 0; a < TP / NB; ++a)
          store_f32(A.partial + ((int64_t)split * NB + i) * A.M * A.N, m, nw + 16 * a + 4 * q,
                    acc[a + i * (TP / NB)][b], (A.N & 3) == 0);
    } else if constexpr (NB == 2) {
#pragma unroll
      for (int a = 0; a < TP / 2; a += 2) {
        f32x4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[i][r] = act_value<ACT>(acc[a + i][b][r]) * acc[a + i + TP / 2][b][r];
        uint16_t *o = (uint16_t *)A.out + m * A.N + nw + 16 * a;
        if (rows8) {  // the same for the wave: lanes exchange values
          const u32x4 d = pack8(v[0], v[1]);
          if (m < A.M) *(u32x4 *)(o + pack8_row(lane)) = d;
        } else if (m < A.M) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (nw + 16 * (a + i) + 4 * q + r < A.N) o[16 * i + 4 * q + r] = f32_to_bf16(v[i][r]);
        }
      }
    } else if (m < A.M) {
#pragma unroll
      for (int a = 0; a < TP; ++a) store_f32((float *)A.out, m, nw + 16 * a + 4 * q, acc[a][b], vec);
    }
  }
  if (!__ballot((low[0] | low[1] | low[2] | low[3]) != 0)) return;
  // a gated result may have been stored by a neighbour (pack8): it has to be there first
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll 1
  for (int b = 0; b < TQ; ++b) {
    while (const uint64_t todo = __ballot(low[0] != 0)) {
      const int j = __builtin_ctzll(todo);
      const int e = __builtin_ctz((uint32_t)__builtin_amdgcn_readlane((int)low[0], j));
      low[0] &= lane == j ? ~(1u << e) : ~0u;
      mend_result<G, NB, ACT>(A, mw + 16 * b + j % 16, nw + 16 * (e / 4) + 4 * (j / 16) + e % 4, split, g0, g1,
                              lane == j);
    }
#pragma unroll
    for (int k = 0; k + 1 < TQ; ++k) low[k] = low[k + 1];
  }
}

// ---------------------------------------------------------------------------
// before the product, in a launch of its own
// ---------------------------------------------------------------------------

constexpr int kPreHead = 2 * 4 * kPreWaves;  // LDS bytes before the rows

// The first kRowLds / rpb elements of a row, 16 a thread; zeros past its end.
__device__ __forceinline__ void load_row(const PreArgs &A, int64_t first, u32x4 (&v)[2]) {
  const int threads = kPreThreads / A.rpb, tid = threadIdx.x % threads;
  const int64_t m = first + threadIdx.x / threads;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = 8 * (tid + i * threads);
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (m < A.M && k < A.K) v[i] = *(const u32x4 *)(A.x + m * A.K + k);
  }
}

// Row m of x as f16 times a power of two, and what it loses by that, for mid_kernel in its fragments
// [chunk][quad][step][16-row tile][lane][8] (rows past M and groups past the
// last are zeros), for wide_kernel as images of its LDS slots [256 rows][stage
// of 32 k][slot], in the order of its codes.
// Rows pass through LDS, from which their elements are picked; a block takes
// `rpb` rows at a time (1, 2 or 4, so that they fit), threads / rpb each.  `v`
// is load_row of these rows and, on return, of those `step` on, which are on
// their way while these are converted.
template <int G, bool FRAG>
__device__ __forceinline__ void f16_role(const PreArgs &A, int64_t first, int64_t step, int64_t rows_in_all,
                                         u32x4 (&v)[2], unsigned char *smem_raw) {
  uint32_t *spans = (uint32_t *)smem_raw;            // [16] of the waves' parts of rows
  float *losses = (float *)(spans + kPreWaves);      // [16]
  const int threads = kPreThreads / A.rpb, room = kRowLds / A.rpb;
  const int tid = threadIdx.x % threads, part = threadIdx.x / threads;
  uint16_t *row = (uint16_t *)(smem_raw + kPreHead) + part * room;
  const int64_t m = first + part;
  const uint16_t *xr = A.x + m * A.K;
  const bool in = m < A.M;
  __syncthreads();  // the rows before have been read
  SpanOf mine;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    mine.take(v[i]);
    *(u32x4 *)(row + 8 * (tid + i * threads)) = v[i];
  }
  if (in)
    for (int k = room + 8 * tid; k < A.K; k += 8 * threads) mine.take(*(const u32x4 *)(xr + k));
  if (first + step < rows_in_all) load_row(A, first + step, v);
  const uint32_t of_wave = span_wave(mine.word());
  if ((threadIdx.x & 63) == 0) spans[threadIdx.x >> 6] = of_wave;
  __syncthreads();
  // joined by four waves (rpb is 4, 2 or 1): of this row, and of all the block's
  uint32_t four[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const u32x4 s = ((const u32x4 *)spans)[w];
    four[w] = span_join(span_join(s[0], s[1]), span_join(s[2], s[3]));
  }
  const uint32_t lower = span_join(four[0], four[1]), upper = span_join(four[2], four[3]);
  const uint32_t all = span_join(lower, upper);
  const uint32_t span = A.rpb == 1 ? all : A.rpb == 2 ? (part ? upper : lower)
                        : part < 2 ? (part ? four[1] : four[0]) : (part == 2 ? four[2] : four[3]);
  const int shift = f16_shift(span_top(span));
  float lost = 0.f;
  if (span_loses(all)) {  // then a row of the block may; the same for all threads
    if (in && span_loses(span))
      for (int k = 8 * tid; k < A.K; k += 8 * threads) lost += lost_of(*(const u32x4 *)(xr + k), shift);
    lost = wave_sum(lost);
    if ((threadIdx.x & 63) == 0) losses[threadIdx.x >> 6] = lost;
    __syncthreads();
    lost = 0.f;
    for (int w = 0; w < threads / 64; ++w) lost += losses[part * (threads / 64) + w];
  }
  if (in && tid == 0) A.rows[m] = u32x2{(uint32_t)shift, __float_as_uint(lost)};
  constexpr int T = G / 8;
  const int nG = A.K / G, nQ = (nG + 3) / 4, rows = kMidRows;
  const int64_t chunk = FRAG ? m / rows : 0;
  const int r = FRAG ? (int)(m - chunk * rows) : 0;
  for (int k0 = 0; k0 < A.K; k0 += room) {  // pieces of whole quads of groups; one if rpb > 1
    const int len = min(A.K - k0, room);
    if (k0 > 0) {
      __syncthreads();
      if (in)
        for (int k = 8 * tid; k < len; k += 8 * threads) *(u32x4 *)(row + k) = *(const u32x4 *)(xr + k0 + k);
      __syncthreads();
    }
    if constexpr (FRAG) {
      const int g0 = k0 / G, quads = (len / G + 3) / 4;
      for (int e = tid; m < rows_in_all && e < quads * 4 * T; e += threads) {
        const int g = e / T, t = e % T;
        const bool has = in && g0 + g < nG;
        _Float16 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = f16_of(has ? row[g * G + group_source<G>(8 * t + i)] : 0, shift);
        *(u32x4 *)(A.xo + (((chunk * nQ + ((g0 + g) >> 2)) * T + t) * (kMidRows / 16) + (r >> 4)) * 512 +
                   ((g & 3) * 16 + (r & 15)) * 8) = *(u32x4 *)f;
      }
    } else {
      const uint32_t r = (uint32_t)(m & (kWideQ - 1));
      const int64_t s0 = m / kWideQ * (A.K / kKS) + k0 / kKS;
      for (int e = tid; in && e < len / 16; e += threads) {
        const int g = e / (G / 16), part16 = e % (G / 16);
        _Float16 f[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = f16_of(row[g * G + eighth_source<G>(part16, j)], shift);
        unsigned char *o = (unsigned char *)A.xo + (s0 + (e >> 1)) * (kWideQ * kKS * 2);
        const uint32_t c = 2u * (e & 1);
        *(u32x4 *)(o + rows_at(r, c)) = *(u32x4 *)f;
        *(u32x4 *)(o + rows_at(r, c + 1)) = *(u32x4 *)(f + 8);
      }
    }
  }
}

constexpr int64_t kMaxPreBlocks = 1 << 16;  // of a role; each strides over its work
constexpr int kPreFrag = 1, kPreRows = 2;

// The last A.shrink_blocks blocks make t (16 RT ranks at a time, none if 0),
// the others convert rows; two blocks are on a CU.  Converting streams x once
// in and once out and takes its bytes' time (1900 rows of 14336: 22 us, 109
// MB); making t waits for loads, and runs in the gaps (together 55 us with 64
// ranks, 39 with 16; in launches of their own 67 and 47).
template <int G, int MODE, int RT>
__global__ __launch_bounds__(kPreThreads) __attribute__((amdgpu_waves_per_eu(8, 8)))
void pre_kernel(const PreArgs A) {
  constexpr int kShrinkLds = RT ? shrink_lds<RT, kPreTiles>() : 0, kRowBytes = kPreHead + 2 * kRowLds;
  __shared__ __align__(16) unsigned char smem[kShrinkLds > kRowBytes ? kShrinkLds : kRowBytes];
  const int row_blocks = (int)gridDim.x - A.shrink_blocks;
  if constexpr (RT > 0) {
    if ((int)blockIdx.x >= row_blocks) {
      shrink_all<RT, kPreTiles>(A, (int)blockIdx.x - row_blocks, smem);
      return;
    }
  }
  const int64_t blk = blockIdx.x, step = (int64_t)row_blocks * A.rpb;
  const int64_t rows = MODE == kPreFrag ? ceil_div(A.M, kMidRows) * kMidRows : A.M;
  u32x4 v[2];
  load_row(A, blk * A.rpb, v);
  for (int64_t m = blk * A.rpb; m < rows; m += step) f16_role<G, MODE == kPreFrag>(A, m, step, rows, v, smem);
}

// ---------------------------------------------------------------------------
// which kernel, and the workspace
// ---------------------------------------------------------------------------

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

constexpr int kFew = 0, kMid = 1, kWide = 2;

int shrink_tiles(int R) { return R > 16 ? kShrinkRanks : 1; }

struct Plan {
  int kind, wk, wt, splits, tsplits;
  bool own_t;
  int64_t blocks, chunks;
  int64_t x, rows, t, partial;  // workspace bytes, each a multiple of 16, in this order
  int64_t total() const { return x + rows + t + partial; }
};

// The number of splits of K that costs least, in us: blocks of `steps` steps,
// `places` at a time, after `start`; a step takes `full` with every place taken,
// down to `alone` with few.  Splits keep `least` steps, and their sums are
// written, read and joined in a launch more.  The rates are measured ones:
// wide_kernel takes 0.85 us for 32 k after 16 (28 where adapters follow); mid_kernel, for 256 k after 4, 2
// alone and, with two blocks on every CU, 3.9 with one matrix and 5 with two.
// (300 rows by 4096 x 14336, one matrix: mid, 3 splits, 96 us; 4 splits, in two
// waves of blocks, 114; wide 120.  4000 rows by 1024 x 3584: mid 88, wide 153.
// 700 rows by 4096 x 14336: wide 146, mid 180.)
struct Split {
  int splits;
  double cost;
};
Split split_of(int64_t blocks, int64_t steps, int64_t least, int64_t places, double start, double alone,
               double full, double sums) {
  Split best{1, 1e30};
  for (int s = 1; s == 1 || (s <= 16 && steps / s >= least); ++s) {
    const int64_t waves = blocks * s / places, rest = blocks * s - waves * places;
    const double last = rest ? alone + (full - alone) * rest / places : 0;
    const double join = s > 1 ? 5 + s * sums * 8 / 5.2e6 : 0;
    const double cost = start + (double)ceil_div(steps, s) * (waves * full + last) + join;
    if (cost < best.cost) best = Split{s, cost};
  }
  return best;
}

// few_kernel's waves of a tile and tiles of a set: those that take least by
// measured rates, in us.  A block works on its sets one after another; of a set,
// each wave takes 1.5 for every four units, all of them together 0.25, and
// gathering the sums 1.  With fewer waves a tile a set is larger and a block has
// fewer: as few sets as its 16 waves allow, of equal size.  (M = 1, two matrices,
// waves by tiles: [14336,4096] 8 x 1 21.4 us, 8 x 2 18.9, 4 x 4 18.1, 2 x 8 25.1,
// 1 x 16 40.4; [11008,8192] 16 x 1 30.9, 8 x 2 33.9, 4 x 4 32.2, 4 x 3 25.7;
// [512,4096] 8 x 1 9.8, 4 x 1 10.1, 2 x 1 12.5, 1 x 1 18.8, 8 x 2 12.8.)
void set_waves(Plan &p, int64_t tiles, int64_t quads, int64_t blocks) {
  double least = 1e30;
  for (int64_t wk = std::min<int64_t>(quads, kFewWaves);; wk = ceil_div(wk, 2)) {
    const int64_t sets = ceil_div(tiles, blocks * (kFewWaves / wk));  // of a block
    const int64_t wt = ceil_div(tiles, blocks * sets);
    const double cost = sets * (std::max(1.5 * ceil_div(quads, wk), 0.25 * wt * quads) + 1);
    if (cost < least) least = cost, p.wk = (int)wk, p.wt = (int)wt;
    if (wk == 1) break;
  }
}

Plan plan_of(int64_t M, int64_t N, int64_t K, int G, int NB, int R) {
  Plan p{};
  const int64_t nG = K / G;
  p.splits = 1;
  if (R) {
    // where the units are few K is split, while a wave keeps several steps
    const bool few = M <= kFewRows && K >= 128;
    const int64_t units = ceil_div(M, few ? 16 : 16 * kPreTiles) * ceil_div(R, 16 * shrink_tiles(R));
    p.tsplits = 1;
    while (p.tsplits < (few ? 2 : 4) && units * p.tsplits < 128 && K / p.tsplits > 4096) p.tsplits *= 2;
    p.t = round16(p.tsplits * M * R * 4);
  }
  const int64_t wide_tiles = ceil_div(NB * N, kWideP) * ceil_div(M, kWideQ);
  // few against mid_kernel at 32 rows: 28.7 us and 36.4 ([4096,14336], 16 ranks),
  // 31 and 40 (2 x [14336,4096]), 12.2 and 20.7 (2 x [3584,1024]); at 16 rows of
  // the first 19.5 and 33.5
  if (M <= kFewRows && K >= 128) {
    p.kind = kFew;
    // a block's slice of x, in whole fours of units, fits its LDS
    const int64_t fours = ceil_div(K, 512);
    p.splits = (int)ceil_div(fours, kFewX / (M * 512 * 2));
    p.own_t = R && M <= 16 && M * R * ceil_div(fours, p.splits) * 512 * 2 <= kOwnTBytes;
    // (the workspace has room for t either way: callers need not know which)
    const int64_t quads = ceil_div(fours, p.splits), tiles = ceil_div(N, 16);
    // a block a CU, beside those that make t
    const int64_t cus = 256 - (R && !p.own_t ? std::min<int64_t>(64, M * p.tsplits) : 0);
    const int64_t most = std::max<int64_t>(1, cus / p.splits);  // blocks of a split
    set_waves(p, tiles, quads, most);
    p.blocks = std::min(ceil_div(tiles, p.wt), most) * p.splits;
  } else {
    // the cheaper of the two by the model of split_of
    const int64_t quads = ceil_div(nG, 4), chunks = ceil_div(M, kMidRows);
    const double sums = (double)NB * M * N;
    const Split wide = split_of(wide_tiles, K / 32, 16, 256, NB == 1 ? 28 : 16, 0.85, 0.85, sums);
    const Split mid =
        split_of(ceil_div(N, 128) * chunks, quads, 2, 512, 4, G / 32, (NB == 1 ? 3.9 : 5.0) * G / 64, sums);
    // mid_kernel's results go out in runs of 32 bytes
    p.kind = wide.cost < mid.cost + 1.4e-6 * M * N ? kWide : kMid;
    p.rows = round16(M * 8);
    if (p.kind == kWide) {
      p.splits = wide.splits;
      p.blocks = wide_tiles * p.splits;
      p.x = ceil_div(M, kWideQ) * kWideQ * K * 2;  // rows past M are never read back
    } else {
      p.splits = mid.splits;
      p.chunks = chunks;
      p.blocks = ceil_div(N, 128) * chunks * p.splits;
      p.x = p.chunks * kMidRows * quads * 4 * G * 2;
    }
  }
  if (p.splits > 1) p.partial = round16((int64_t)p.splits * NB * M * N * 4);
  return p;
}

template <int G, int NB, int MT, int ACT>
void launch_few(const Plan &p, const ProjArgs &a, const PreArgs &pre, hipStream_t stream) {
  if constexpr (NB == 2) {
    hipLaunchKernelGGL((few_kernel<G, NB, MT, ACT, 0>), dim3((unsigned)p.blocks),
                       dim3(64 * std::max(kFewSetUp, p.wk * p.wt)), 0, stream, a, pre);
  } else {
    if constexpr (MT == 1) {
      if (p.own_t) {
        hipLaunchKernelGGL((few_kernel<G, NB, MT, ACT, kOwnT>), dim3((unsigned)p.blocks),
                           dim3(64 * std::max(kFewSetUp, p.wk * p.wt)), 0, stream, a, pre);
        return;
      }
    }
    const dim3 grid((unsigned)(p.blocks + pre.shrink_blocks));
    auto kernel = shrink_tiles(a.R) == 1 ? few_kernel<G, NB, MT, ACT, 1> : few_kernel<G, NB, MT, ACT, kShrinkRanks>;
    hipLaunchKernelGGL(kernel, grid, dim3(kPreThreads), 0, stream, a, pre);
    hipLaunchKernelGGL(expand_kernel<MT>, dim3((unsigned)ceil_div(a.N, 16)), dim3(256 * MT), 0, stream, a);
  }
}

template <int G, int NB, int ACT>
void launch_product(const Plan &p, const ProjArgs &a, const PreArgs &pre, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  if (p.kind == kFew)
    a.M <= 16 ? launch_few<G, NB, 1, ACT>(p, a, pre, stream) : launch_few<G, NB, 2, ACT>(p, a, pre, stream);
  else if (p.kind == kWide)
    hipLaunchKernelGGL((wide_kernel<G, NB, ACT>), grid, dim3(kWideThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((mid_kernel<G, NB, ACT>), grid, dim3(kMidThreads), 0, stream, a);
}

// All launches of a call; `a` and `pre` hold the caller's arguments.
template <int G, int NB, int ACT>
void launch_proj(const Plan &p, ProjArgs a, PreArgs pre, void *workspace, hipStream_t stream) {
  char *ws = (char *)workspace;
  pre.x = a.x;
  pre.xo = (uint16_t *)ws;
  pre.rows = (u32x2 *)(ws + p.x);
  pre.t = (float *)(ws + p.x + p.rows);
  a.partial = (float *)(ws + p.x + p.rows + p.t);
  a.t = pre.t;
  a.x0 = a.x;
  a.rows = pre.rows;
  a.tsplits = pre.tsplits = p.tsplits;
  a.splits = p.splits;
  a.wk = p.wk;
  a.wt = p.wt;
  a.chunks = (int)p.chunks;
  a.tp = (int)ceil_div(NB * (int64_t)a.N, kWideP);
  a.tq = (int)ceil_div(a.M, kWideQ);
  pre.M = a.M, pre.K = a.K, pre.status = a.status;
  pre.ids = a.ids, pre.adapters = a.adapters, pre.R = a.R;
  if (NB == 1 && !p.own_t) {
    const int64_t tiles = ceil_div(a.M, kShrinkTile);
    const int64_t rows = std::min<int64_t>(a.M, kShrinkTile);
    // units of a tile: one for each 16 (32) rows and one more for each adapter
    const int64_t unit = p.kind == kFew ? 16 : 16 * kPreTiles;
    pre.units = (int)std::min(rows, ceil_div(rows, unit) + std::min<int64_t>(rows, a.adapters));
    pre.rtiles = (int)ceil_div(a.R, 16 * shrink_tiles(a.R));
    if (a.adapters == 0) pre.units = pre.rtiles = pre.tsplits = 1;  // the ids are still checked
    pre.shrink_blocks = (int)std::min(kMaxPreBlocks, tiles * pre.units * pre.rtiles * pre.tsplits);
  }
  pre.rpb = a.K <= kRowLds / 4 ? 4 : a.K <= kRowLds / 2 ? 2 : 1;
  if (p.kind != kFew) {
    // two blocks a CU, each with a row on its way while it converts another; one
    // beside those that make t
    auto prepare = [&](auto kernel, int64_t rows) {
      const int64_t convert = std::min<int64_t>(pre.shrink_blocks > 8 ? 256 : 512, ceil_div(rows, pre.rpb));
      hipLaunchKernelGGL(kernel, dim3((unsigned)(convert + pre.shrink_blocks)), dim3(kPreThreads), 0, stream, pre);
    };
    const int64_t rows = p.kind == kWide ? a.M : p.chunks * kMidRows;
    if constexpr (NB == 2)
      p.kind == kWide ? prepare(pre_kernel<G, kPreRows, 0>, rows) : prepare(pre_kernel<G, kPreFrag, 0>, rows);
    else if (shrink_tiles(a.R) > 1)
      p.kind == kWide ? prepare(pre_kernel<G, kPreRows, kShrinkRanks>, rows)
                      : prepare(pre_kernel<G, kPreFrag, kShrinkRanks>, rows);
    else
      p.kind == kWide ? prepare(pre_kernel<G, kPreRows, 1>, rows) : prepare(pre_kernel<G, kPreFrag, 1>, rows);
    a.x = pre.xo;
  }
  launch_product<G, NB, ACT>(p, a, pre, stream);
  if (p.splits > 1 && !(p.kind == kFew && NB == 1 && !p.own_t)) {
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

void projection_plan(int64_t M, int64_t N, int64_t K, int G, int matrices, int R, int64_t *plan) {
  const Plan p = plan_of(M, N, K, G, matrices, matrices == 1 ? R : 0);
  plan[0] = p.kind, plan[1] = p.splits, plan[2] = p.tsplits, plan[3] = p.own_t;
  plan[4] = p.wk, plan[5] = p.wt;
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

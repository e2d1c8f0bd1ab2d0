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
//   few_kernel    up to 16 rows: bound by the weights' bytes.  Every byte is
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

// What both kernels read and write.
struct ProjArgs {
  const uint16_t *x;              // bf16 [M,K] (staged), or x in fragment order, or f16 rows
  const uint8_t *packed[2];
  const uint16_t *scales[2];
  const int32_t *shift;           // wide: x of row m is stored times 2^shift[m]
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
  int wk;                         // few: waves along K (a power of two)
  int chunks;                     // mid: chunks of rows
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

// Eight ranks of row m's t in three bf16 pieces (24 bits together); zeros
// unless `in`.
struct Pieces {
  bf16x8 p[3];
};
__device__ __forceinline__ Pieces split_t(const ProjArgs &A, int64_t m, int r, bool in) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (in)
    for (int k = 0; k < A.tsplits; ++k) {
      const f32x4 *t = (const f32x4 *)(A.t + ((int64_t)k * A.M + m) * A.R + r);
      const f32x4 lo = t[0], hi = t[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += lo[i];
        v[4 + i] += hi[i];
      }
    }
  Pieces out;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __bf16 a = (__bf16)v[i];
    const float ra = v[i] - (float)a;
    const __bf16 b = (__bf16)ra;
    out.p[0][i] = a;
    out.p[1][i] = b;
    out.p[2][i] = (__bf16)(ra - (float)b);
  }
  return out;
}

// Add the adapters' part to one tile of 16 weight rows (columns n0 + lane %
// 16) by 16 MT rows of x (row m0 + i named by lane i's id, -1 for none).  The
// distinct adapters are taken in turn, those with turn % share == mine here.
// A product of one adapter is made for all the rows and kept for its own, so
// nothing in an adapter reaches another's rows.
template <int MT>
__device__ void add_adapters(const ProjArgs &A, int64_t m0, int n0, int id, int share, int mine,
                             f32x4 (&acc)[MT]) {
  const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int64_t n = min(n0 + l, A.N - 1);
  uint64_t todo = adapter_leaders(id, lane);
  for (int turn = 0; todo; ++turn) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= todo - 1;
    if (turn % share != mine) continue;
    f32x4 add[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) add[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < A.R; r0 += 32) {
      const int r = r0 + 8 * q;
      u32x4 v{0u, 0u, 0u, 0u};
      if (r < A.R) v = *(const u32x4 *)(A.b + ((int64_t)a * A.N + n) * A.R + r);
      const bf16x8 bv = __builtin_bit_cast(bf16x8, v);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bool own = __shfl(id, 16 * mt + l) == a;
        if (!__ballot(own)) continue;
        const Pieces p = split_t(A, m0 + 16 * mt + l, r, own && r < A.R);
#pragma unroll
        for (int i = 0; i < 3; ++i) add[mt] = mfma32<false>(p.p[i], bv, add[mt]);
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[mt][j] += __shfl(id, 16 * mt + 4 * q + j) == a ? add[mt][j] : 0.f;
  }
}

// The id of row m as add_adapters takes it.
__device__ __forceinline__ int adapter_of(const ProjArgs &A, int64_t m, bool in) {
  const int id = in && m < A.M ? A.ids[m] : -1;
  return id < A.adapters ? id : -1;
}

// ---------------------------------------------------------------------------
// up to 16 rows
// ---------------------------------------------------------------------------

// One lane's bytes of one group of one weight row.
struct Raw {
  uint32_t w0, w1, tail, scale;
};

// `tile` is the group's bytes in the tile's first row and `stile` its scale
// there (both the same for the wave); row, srow the lane's row within the tile
// in bytes and in scales.
template <int G>
__device__ __forceinline__ Raw load_raw(const uint8_t *tile, const uint16_t *stile, uint32_t row,
                                        uint32_t srow, uint32_t q) {
  Raw r;
  if constexpr (G == 128) {
    uint64_t w;
    uint16_t tail;
    __builtin_memcpy(&w, tile + (row + 6u * q), 8);  // six of them; q = 3 ends at the group's end
    __builtin_memcpy(&tail, tile + (row + 24u), 2);
    r.w0 = (uint32_t)w;
    r.w1 = (uint32_t)(w >> 32);
    r.tail = tail;
  } else {
    __builtin_memcpy(&r.w0, tile + (row + 3u * q), 4);  // three; q = 3 ends at the group's end
    r.w1 = 0;
    r.tail = tile[row + 12u];
  }
  r.scale = stile[srow];
  return r;
}

constexpr int kFewRows = 16;
constexpr int kFewWaves = 16, kFewThreads = 64 * kFewWaves;
constexpr uint32_t kFewX = 64 << 10;  // LDS for a block's slice of x
// Groups a wave requests together: what 128 registers a lane leave room for.
constexpr int few_u(int G, int NB) { return G == 128 && NB == 2 ? 2 : 4; }

// A block: one split of K, and tiles of 16 weight rows (of each matrix) one
// set after another, kFewWaves / wk tiles a set; wk waves share the groups of
// a tile.  x [M,K] (M <= 16) of the split is put in order once, in LDS.
// The matrix cores take x as the row operand and W as the column operand, so
// a lane's partial sums belong to the weight row whose bytes it decoded.
// A wave requests few_u groups of bytes while it works on as many others,
// across the ends of tiles.  One block a CU: 64 KB table, 64 KB x, 16 KB a matrix for
// the sums of the waves.
template <int G, int NB, int ACT>
__global__ __launch_bounds__(kFewThreads) void few_kernel(const ProjArgs A) {
  constexpr int S32 = G / 32, B = bytes_per_group(G), kFewU = few_u(G, NB);
  typedef Lut<kLutBf16, 32> L;
  constexpr uint32_t kXOff = L::kBytes, kRedOff = kXOff + kFewX;
  __shared__ __align__(16) unsigned char smem_raw[kRedOff + kFewWaves * NB * 1024];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nG = A.K / G, M = (int)A.M;
  const int split = (int)blockIdx.x % A.splits, b0 = (int)blockIdx.x / A.splits;
  const int blocks = (int)gridDim.x / A.splits;
  const int g0 = (int)((int64_t)nG * split / A.splits);
  const int g1 = (int)((int64_t)nG * (split + 1) / A.splits);
  const int wk = A.wk, wt = kFewWaves / wk;       // waves of a tile, tiles of a set
  const int kw = wv % wk, tw = wv / wk;           // this wave's place
  const int tiles = (A.N + 15) / 16, sets = (tiles + wt - 1) / wt;
  const int steps = b0 < sets ? (sets - b0 + blocks - 1) / blocks : 0;
  const int batches = (g1 - g0 + wk * kFewU - 1) / (wk * kFewU);  // of a tile

  // the set of step j is b0 + j * blocks
  auto tile_row = [&](int j) { return ((b0 + j * blocks) * wt + tw) * 16; };
  struct Batch {
    Raw r[kFewU][NB];
  };
  int fj = 0, fk = 0;  // step and batch of the next request
  auto fetch = [&](Batch &f) {
    const int n0 = tile_row(fj);
    if (fj < steps && n0 < A.N) {
      // rows past N read row N - 1; their sums are not stored
      const uint32_t ln = (uint32_t)min(l, A.N - 1 - n0);
      const uint32_t row = ln * (uint32_t)nG * B, srow = ln * (uint32_t)nG;
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
        const int g = g0 + kw + wk * (fk * kFewU + u);
        if (g >= g1) break;
        const int64_t at = (int64_t)n0 * nG + g;
#pragma unroll
        for (int i = 0; i < NB; ++i)
          f.r[u][i] = load_raw<G>(A.packed[i] + at * B, A.scales[i] + at, row, srow, (uint32_t)q);
      }
    }
    if (++fk == batches) {
      fk = 0;
      ++fj;
    }
  };

  // the first bytes are requested before the table is built and x put in order
  Batch ba, bb;
  fetch(ba);
  L::build(smem, tid, kFewThreads);
  {
    // unit: a quarter's codes of a group of one row
    const int quarters = 4 * (g1 - g0), units = quarters * M;
    for (int e = tid; e < units; e += kFewThreads) {
      const int m = e / quarters, gq = e - m * quarters, g = gq >> 2, uq = gq & 3;
      u32x4 f[S32];
      order_quarter<G>(A.x + (int64_t)m * A.K + (int64_t)(g0 + g) * G, uq, f);
#pragma unroll
      for (int s = 0; s < S32; ++s)
        *(lds_u32x4 *)(smem + kXOff + 16u * (uint32_t)(((g * S32 + s) * 4 + uq) * M + m)) = f[s];
    }
  }
  __syncthreads();

  const L lut(0, lane);
  const uint32_t xlane = kXOff + 16u * (uint32_t)(q * M + min(l, M - 1));  // rows past M: row M - 1
  int id = -1;
  if constexpr (NB == 1) id = adapter_of(A, lane, lane < 16);
  uint32_t flags = 0;
  f32x4 acc[NB][1];
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  int j = 0, k = 0;  // step and batch being worked on
  auto work = [&](Batch &f, Batch &next) {
    fetch(next);
    const int n0 = tile_row(j);
    if (n0 < A.N) {
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
        const int g = g0 + kw + wk * (k * kFewU + u);
        if (g >= g1) break;
        bf16x8 xf[S32];
#pragma unroll
        for (int s = 0; s < S32; ++s)
          xf[s] = *(lds_bf16x8_c *)(smem + xlane + 64u * (uint32_t)(((g - g0) * S32 + s) * M));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const Raw r = f.r[u][i];
          uint32_t d[G / 8];
          decode_quarter<G>(smem, lut, r.w0, r.w1, r.tail, q, d, flags);
          f32x4 part{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < S32; ++s)
            part = mfma32<false>(
                xf[s], __builtin_bit_cast(bf16x8, u32x4{d[4 * s], d[4 * s + 1], d[4 * s + 2], d[4 * s + 3]}),
                part);
          // codes entered as 2c
          const float sh = 0.5f * __half2float(__ushort_as_half((unsigned short)r.scale));
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][0][c] = fmaf(sh, part[c], acc[i][0][c]);
        }
      }
    }
    if (++k < batches) return;
    k = 0;
    // the tile's last batch: adapters (split 0), then the waves' sums in order
    if constexpr (NB == 1)
      if (split == 0 && A.adapters > 0 && n0 < A.N) add_adapters<1>(A, 0, n0, id, wk, kw, acc[0]);
    __syncthreads();  // the sums of the set before have been read
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      *(__attribute__((address_space(3))) f32x4 *)(smem + kRedOff + 16u * (uint32_t)((i * kFewWaves + wv) * 64 + lane)) =
          acc[i][0];
      acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __syncthreads();
    for (int o = tid; o < wt * 256; o += kFewThreads) {  // [tile][row][column]
      const int m = (o >> 4) & 15, n = ((b0 + j * blocks) * wt + (o >> 8)) * 16 + (o & 15);
      if (m >= M || n >= A.N) continue;
      // row m of column c is element m % 4 of lane 16 (m / 4) + c
      const uint32_t at = kRedOff + 16u * (uint32_t)((o >> 8) * wk * 64 + (m >> 2) * 16 + (o & 15)) + 4u * (m & 3);
      float v[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        v[i] = 0.f;
        for (int w = 0; w < wk; ++w)
          v[i] += *(__attribute__((address_space(3))) float *)(smem + at + 1024u * (uint32_t)(i * kFewWaves + w));
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
    ++j;
  };
  const int total = steps * batches;
  for (int t = 0; t < total; t += 2) {
    work(ba, bb);
    if (t + 1 < total) work(bb, ba);
  }
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);
}

// ---------------------------------------------------------------------------
// some rows
// ---------------------------------------------------------------------------

constexpr int kMidWaves = 8, kMidThreads = 64 * kMidWaves;

// A block: 128 weight rows (of each matrix), a tile of 16 a wave; one chunk of
// 16 MT rows of x; one split of K.  x comes in fragment order (frag_role), a
// group at a time, through a ring of LDS slots that all waves read.
template <int G, int NB, int MT, int ACT>
__global__ __launch_bounds__(kMidThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void mid_kernel(const ProjArgs A) {
  constexpr int S32 = G / 32, B = bytes_per_group(G);
  typedef Lut<kLutBf16, 16> L;
  constexpr uint32_t kStage = S32 * MT * 1024, kLoad = 16 * kMidThreads;
  constexpr uint32_t kSlot = kStage > kLoad ? kStage : kLoad;
  constexpr int kD = kSlot / kLoad;                             // loads a thread and stage
  constexpr int kSlots = 49152 / kSlot > 6 ? 6 : 49152 / kSlot;  // 80 KB in all: two blocks a CU
  __shared__ __align__(16) unsigned char smem_raw[L::kBytes + kSlots * kSlot];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  lds_bytes *ring = smem + L::kBytes;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nG = A.K / G;
  int b = (int)blockIdx.x;
  const int chunk = b % A.chunks;
  b /= A.chunks;
  const int split = b % A.splits, n0 = (b / A.splits) * 128 + 16 * wv;
  const int g0 = (int)((int64_t)nG * split / A.splits);
  const int g1 = (int)((int64_t)nG * (split + 1) / A.splits);
  const int64_t m0 = (int64_t)chunk * (16 * MT);

  // rows past N read row N - 1; their sums are not stored
  const int nt = min(n0, A.N - 1);
  const uint32_t ln = (uint32_t)min(l, A.N - 1 - nt);
  const uint32_t row = ln * (uint32_t)nG * B, srow = ln * (uint32_t)nG;
  Raw ra[NB], rb[NB];
  auto fetch = [&](Raw(&r)[NB], int g) {  // always: the waits below count its loads
    const int64_t at = (int64_t)nt * nG + min(g, nG - 1);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      r[i] = load_raw<G>(A.packed[i] + at * B, A.scales[i] + at, row, srow, (uint32_t)q);
  };
  uint32_t off[kD];
#pragma unroll
  for (int i = 0; i < kD; ++i) {
    off[i] = (uint32_t)(i * kLoad + 16 * tid);
    if (off[i] >= kStage) off[i] = kNoRow;
  }
  const uint16_t *xbase = A.x + (int64_t)chunk * nG * (kStage / 2);
  int put = 0;  // slot of the next request
  auto request = [&](int g) {
#pragma unroll
    for (int i = 0; i < kD; ++i)
      dma16_tracked(xbase + (int64_t)g * (kStage / 2),
                    ring + (uint32_t)put * kSlot + (uint32_t)(i * kLoad) + 1024u * (uint32_t)wv,
                    g < g1 ? off[i] : kNoRow);
    put = put == kSlots - 1 ? 0 : put + 1;
  };

  fetch(ra, g0);
  fetch(rb, g0 + 1);
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) request(g0 + s);
  L::build(smem, tid, kMidThreads);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  f32x4 acc[NB][MT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[i][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
  const L lut(0, lane);
  uint32_t flags = 0;
  int get = 0;
  auto stage = [&](int g, Raw(&r)[NB]) {
    request(g + kSlots - 1);
    lds_bytes *x = ring + (uint32_t)get * kSlot + 16u * (uint32_t)lane;
    get = get == kSlots - 1 ? 0 : get + 1;
    uint32_t d[NB][G / 8];
    float sh[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      decode_quarter<G>(smem, lut, r[i].w0, r[i].w1, r[i].tail, q, d[i], flags);
      // codes entered as 2c
      sh[i] = 0.5f * __half2float(__ushort_as_half((unsigned short)r[i].scale));
    }
    fetch(r, g + 2);
    f32x4 part[NB][MT];
#pragma unroll
    for (int s = 0; s < S32; ++s)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bf16x8 xf = *(lds_bf16x8_c *)(x + 1024u * (uint32_t)(s * MT + mt));
#pragma unroll
        for (int i = 0; i < NB; ++i)
          part[i][mt] = mfma32<false>(
              xf,
              __builtin_bit_cast(bf16x8, u32x4{d[i][4 * s], d[i][4 * s + 1], d[i][4 * s + 2], d[i][4 * s + 3]}),
              s == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : part[i][mt]);
      }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][mt][c] = fmaf(sh[i], part[i][mt][c], acc[i][mt][c]);
    // x of group g + 1 has landed when what was requested after it is all
    // that is out: the rest of its stage at the least, and kSlots - 2 stages
    // of kD loads of x and 3 NB of bytes and scales
    constexpr int kOut = (kSlots - 2) * (kD + 3 * NB);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kOut > 63 ? 63 : kOut) : "memory");
  };
  for (int g = g0; g < g1; g += 2) {
    stage(g, ra);
    if (g + 1 < g1) stage(g + 1, rb);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may still write this block's LDS
  if ((flags & kBadFlag) && A.status) atomicOr(A.status, kDevInvalidByte);

  if constexpr (NB == 1) {
    // the splits share the adapters
    const int64_t m = m0 + lane;
    if (A.adapters > 0 && n0 < A.N)
      add_adapters<MT>(A, m0, n0, adapter_of(A, m, lane < 16 * MT), A.splits, split, acc[0]);
  }
  const int n = n0 + l;
  if (n >= A.N) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t m = m0 + 16 * mt + 4 * q + c;
      if (m >= A.M) continue;
      const int64_t o = m * A.N + n;
      if (A.splits > 1) {
#pragma unroll
        for (int i = 0; i < NB; ++i) A.partial[((int64_t)split * NB + i) * A.M * A.N + o] = acc[i][mt][c];
      } else if constexpr (NB == 2) {
        ((uint16_t *)A.out)[o] = f32_to_bf16(act_value<ACT>(acc[0][mt][c]) * acc[1][mt][c]);
      } else {
        ((float *)A.out)[o] = acc[0][mt][c];
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
template <int G, int NB, int ACT>
__global__ __launch_bounds__(kWideThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void wide_kernel(const ProjArgs A) {
  constexpr int S32 = G / 32, WP = 2, WQ = 4, TP = 8, TQ = 4, B = bytes_per_group(G);
  typedef Stream<kRows, kWideQ, kWideThreads> QS;
  typedef Lut<kLutF16, 8> L;
  constexpr uint32_t kPSlot = kWideP * kKS * 2;
  constexpr uint32_t kQOff = kWideC * kPSlot, kLutOff = kQOff + kWideX * QS::kSlot;
  __shared__ __align__(16) unsigned char smem_raw[kLutOff + L::kBytes];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63;
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
  // bytes and group values are requested four stages before they are decoded
  constexpr int kGroups = 4 / S32;  // groups of four stages
  uint32_t raw[4], tail_next[kGroups], scale_next[kGroups], scale = 0, flags = 0;
  u32x2 left{0u, 0u};  // high bytes of the group's left-over codes
  // bytes of stage s, J = s % 4 (past the end: of the last group)
  auto load_raw = [&](int s, auto jc) {
    constexpr int J = decltype(jc)::value;
    const int g = min(g0 + s / S32, nG - 1);
    const uint8_t *p = prow + (int64_t)g * B;
    __builtin_memcpy(&raw[J], p + 6 * (J % S32) + 3 * hf, 4);
    if constexpr (J % S32 == 0) {
      if constexpr (G == 128) {
        uint16_t v;
        __builtin_memcpy(&v, p + 24, 2);
        tail_next[J / S32] = v;
      } else {
        tail_next[J / S32] = p[12];
      }
      scale_next[J / S32] = srow[g];
    }
  };
  const L lut(kLutOff, lane);
  const uint32_t put0 = rows_at((uint32_t)sr, 2u * hf), put1 = rows_at((uint32_t)sr, 2u * hf + 1u);
  // codes of the stage whose bytes are raw[J], J = its index % 4, -> slot
  auto decode = [&](auto jc, uint32_t slot) {
    constexpr int J = decltype(jc)::value;
    if constexpr (J % S32 == 0) {
      scale = scale_next[J / S32] * 0x10001u;
      left = leftover_pool<G>(smem, lut, tail_next[J / S32], flags);
    }
    u32x4 c0, c1;
    decode_eighth(smem, lut, raw[J], left, (uint32_t)(2 * (J % S32) + hf), scale, c0, c1, flags);
    *(lds_u32x4 *)(smem + slot + put0) = c0;
    *(lds_u32x4 *)(smem + slot + put1) = c1;
  };

  QS qs;
  qs.init_rows(tid, (uint32_t)A.K, [&](int r) -> int64_t { return q0 + r < A.M ? r : -1; });
  const uint16_t *qbase = A.x + q0 * A.K + (int64_t)g0 * G;
  int xput = 0;  // slot of the next request
  auto request = [&](int s, int i) {
    qs.load_tracked(i, qbase + (int64_t)s * kKS, smem + kQOff + (uint32_t)xput * QS::kSlot, (uint32_t)wv,
                    s < S ? 1 : 0);
    if (i == QS::kLoads - 1) xput = xput == kWideX - 1 ? 0 : xput + 1;
  };

  // ---- prologue: bytes of stages 0 .. 6, x of 0 .. 3, codes of 0 .. 2 ----
  load_raw(0, Int<0>{});
  load_raw(1, Int<1>{});
  load_raw(2, Int<2>{});
  load_raw(3, Int<3>{});
#pragma unroll
  for (int s = 0; s < kWideX - 1; ++s)
#pragma unroll
    for (int i = 0; i < QS::kLoads; ++i) request(s, i);
  L::build(smem + kLutOff, tid, kWideThreads);
  __syncthreads();
  decode(Int<0>{}, 0);
  load_raw(4, Int<0>{});
  decode(Int<1>{}, kPSlot);
  load_raw(5, Int<1>{});
  decode(Int<2>{}, 2 * kPSlot);
  load_raw(6, Int<2>{});

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

  int xget = 1;  // slot of x of stage s + 1
  auto stage = [&](int s, auto jc, bf16x8(&qc)[TQ], bf16x8(&qn)[TQ]) {
    constexpr int J = decltype(jc)::value;  // s % 4
    const uint32_t pn = (uint32_t)((J + 1) % kWideC) * kPSlot;
    const uint32_t qn0 = kQOff + (uint32_t)xget * QS::kSlot;
    xget = xget == kWideX - 1 ? 0 : xget + 1;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int a = 0; a < TP; ++a) {
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = mfma32<true>(pa[a], qc[b], acc[a][b]);
      if (a < TQ) qn[a] = qf.read(smem, qn0, a);
      pa[a] = pf.read(smem, pn, a);
      if (a < QS::kLoads) request(s + kWideX - 1, a);
      if (a == 3) {
        decode(Int<(J + 3) % 4>{}, (uint32_t)((J + 3) % kWideC) * kPSlot);
        load_raw(s + 7, Int<(J + 7) % 4>{});
        // the codes are written before the fragments of rows 4 .. 7 are read:
        // when the last of those is used, in stage s + 1, the writes are done,
        // a barrier before stage s + 2 reads them
        asm volatile("" ::: "memory");
      }
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
  const bool vec = (A.N & 3) == 0 && (reinterpret_cast<uintptr_t>(A.out) & 15) == 0;
  const int nw = n0 + wp * HP;  // first row of this wave
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
      const int64_t mw = q0 + wq * (kWideQ / WQ);
      const int id = adapter_of(A, mw + lane, true);
      uint64_t todo = adapter_leaders(id, lane);
      for (int turn = 0; todo; ++turn) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= todo - 1;
        if (turn % A.splits != split) continue;
        for (int r0 = 0; r0 < A.R; r0 += 32) {
          const int r = r0 + 8 * q;
#pragma unroll
          for (int b = 0; b < TQ; ++b) {
            const bool own = __shfl(id, 16 * b + l) == a;
            if (!__ballot(own)) continue;
            const Pieces t = split_t(A, mw + 16 * b + l, r, own && r < A.R);
#pragma unroll
            for (int p = 0; p < TP; ++p) {
              const int64_t n = min(nw + 16 * p + l, A.N - 1);
              u32x4 v{0u, 0u, 0u, 0u};
              if (r < A.R) v = *(const u32x4 *)(A.b + ((int64_t)a * A.N + n) * A.R + r);
              const bf16x8 bv = __builtin_bit_cast(bf16x8, v);
              f32x4 add{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < 3; ++i) add = mfma32<false>(bv, t.p[i], add);
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[p][b][c] += own ? add[c] : 0.f;
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < TQ; ++b) {
    const int64_t m = mq + 16 * b;
    if (m >= A.M) continue;
    if (A.splits > 1) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int a = 0; a < TP / NB; ++a)
          store_f32(A.partial + ((int64_t)split * NB + i) * A.M * A.N, m, nw + 16 * a + 4 * q,
                    acc[a + i * (TP / NB)][b], (A.N & 3) == 0);
    } else if constexpr (NB == 2) {
#pragma unroll
      for (int a = 0; a < TP / 2; ++a) {
        const int n = nw + 16 * a + 4 * q;
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = act_value<ACT>(acc[a][b][r]) * acc[a + TP / 2][b][r];
        uint16_t *o = (uint16_t *)A.out + m * A.N + n;
        if (vec && n < A.N) {
          store4(o, v);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < A.N) o[r] = f32_to_bf16(v[r]);
        }
      }
    } else {
#pragma unroll
      for (int a = 0; a < TP; ++a) store_f32((float *)A.out, m, nw + 16 * a + 4 * q, acc[a][b], vec);
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
  // shrink: blocks, units a tile of rows, tiles of 16 ranks, splits of K
  int shrink_blocks, units, rtiles, tsplits;
  int32_t *status;
};

// t of one unit: up to 16 rows of one adapter, 16 ranks.  The rows of a tile
// that name the same adapter are numbered in order and cut into units of 16,
// so rows in any order share the adapter's A.  One split of K; its waves
// share the split, and their sums are added in order.
__device__ void shrink_role(const PreArgs &A, int64_t blk, unsigned char *smem_raw) {
  int *ids = (int *)smem_raw;                       // [256]
  int *rows = ids + kShrinkTile;                    // [16]
  int *info = rows + 16;                            // adapter, leader's rank
  int *counts = info + 4;                           // [8] leaders of each wave
  float *red = (float *)(counts + 12);              // [8][64][4]
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, l = lane & 15, q = lane >> 4;
  const int split = (int)(blk % A.tsplits);
  blk /= A.tsplits;
  const int rt = (int)(blk % A.rtiles), unit = (int)(blk / A.rtiles % A.units);
  const int64_t m0 = blk / A.rtiles / A.units * kShrinkTile;
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
  const int s0 = (int)((int64_t)steps * split / A.tsplits), s1 = (int)((int64_t)steps * (split + 1) / A.tsplits);
  for (int s = s0 + wv; s < s1; s += kPreWaves * 8) {
    // eight steps requested together; those past the end read the last one
    // and add nothing
    bf16x8 av[8], xv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int si = min(s + kPreWaves * i, steps - 1);
      av[i] = *(const bf16x8 *)(ar + 32 * si);
      xv[i] = *(const bf16x8 *)(xr + 32 * si);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s + kPreWaves * i < s1) acc = mfma32<false>(av[i], xv[i], acc);
  }
  *(f32x4 *)(red + 4 * tid) = acc;
  __syncthreads();
  if (tid < 256) {
    float sum = 0.f;
    for (int w = 0; w < kPreWaves; ++w) sum += red[w * 256 + tid];
    const int ol = tid >> 2, rr = 16 * rt + 4 * (ol >> 4) + (tid & 3), row = rows[ol & 15];
    if (row >= 0 && rr < A.R) A.t[((int64_t)split * A.M + m0 + row) * A.R + rr] = A.scaling[a] * sum;
  }
}

// x in the fragment order of mid_kernel: [chunk][group][step][16-row tile]
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
__device__ void f16_role(const PreArgs &A, int64_t m, unsigned char *smem_raw) {
  uint32_t *tops = (uint32_t *)smem_raw;  // [8]
  const int tid = threadIdx.x, lane = tid & 63;
  const uint16_t *xr = A.x + m * A.K;
  uint32_t top = 0;
  for (int k = 8 * tid; k < A.K; k += 8 * kPreThreads) {
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
  __syncthreads();  // the row before has been read
  if (lane == 0) tops[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPreWaves; ++w) top = max(top, tops[w]);
  int exponent;  // top is in [2^(exponent - 1), 2^exponent)
  (void)frexpf(bf16_to_f32(top), &exponent);
  const int shift = top ? 15 - exponent : 0;
  if (tid == 0) A.shift[m] = shift;
  uint16_t *o = A.xo + m * A.K;
  for (int e = tid; e < A.K / 16; e += kPreThreads) {
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
    const int64_t work = (A.M + kShrinkTile - 1) / kShrinkTile * A.units * A.rtiles * A.tsplits;
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
    for (int64_t m = blk; m < A.M; m += blocks) f16_role<G>(A, m, smem);
  }
}

// ---------------------------------------------------------------------------
// which kernel, and the workspace
// ---------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

constexpr int kFew = 0, kMid = 1, kWide = 2;

struct Plan {
  int kind, wk, mt, splits, tsplits;
  int64_t blocks, chunks;
  int64_t x, shift, t, partial;  // workspace bytes, each a multiple of 16, in this order
  int64_t total() const { return x + shift + t + partial; }
};

Plan plan_of(int64_t M, int64_t N, int64_t K, int G, int NB, int R) {
  Plan p{};
  const int64_t nG = K / G;
  p.splits = 1;
  const int64_t wide_tiles = ceil_div(NB * N, kWideP) * ceil_div(M, kWideQ);
  if (M <= kFewRows) {
    p.kind = kFew;
    // a block's slice of x fits its LDS
    p.splits = (int)ceil_div(nG, kFewX / (M * G * 2));
    // waves along K: few_u groups a wave, more waves while the sets of tiles
    // are fewer than the CUs
    const int64_t ng = ceil_div(nG, p.splits), tiles = ceil_div(N, 16);
    p.wk = 1;
    while (p.wk < kFewWaves && (ng > few_u(G, NB) * p.wk || tiles * p.wk / kFewWaves * p.splits < 192)) p.wk *= 2;
    p.blocks = std::min(ceil_div(tiles, kFewWaves / p.wk), std::max<int64_t>(1, 256 / p.splits)) * p.splits;
  } else if (M > 128 && wide_tiles >= 64) {
    p.kind = kWide;
    // a tile a CU; K is split while every block keeps 64 stages
    while (wide_tiles * p.splits < 160 && nG / (2 * p.splits) * (G / 32) >= 64) p.splits *= 2;
    p.blocks = wide_tiles * p.splits;
    p.x = round16(M * K * 2);
    p.shift = round16(M * 4);
  } else {
    p.kind = kMid;
    p.mt = M <= 32 ? 2 : 4;
    p.chunks = ceil_div(M, 16 * p.mt);
    const int64_t blocks = ceil_div(N, 128) * p.chunks;
    // two blocks a CU; K is split while every block keeps four groups
    while (blocks * p.splits < 384 && nG / (2 * p.splits) >= 4) p.splits *= 2;
    p.blocks = blocks * p.splits;
    p.x = p.chunks * 16 * p.mt * K * 2;
  }
  if (p.splits > 1) p.partial = round16((int64_t)p.splits * NB * M * N * 4);
  if (R) {
    // t: about eight steps a wave of a block
    p.tsplits = (int)std::min<int64_t>(8, ceil_div(K / 32, 8 * kPreWaves));
    if (M > 64) p.tsplits = std::min(p.tsplits, 2);
    p.t = round16(p.tsplits * M * R * 4);
  }
  return p;
}

template <int G, int NB, int ACT>
void launch_product(const Plan &p, const ProjArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  if (p.kind == kFew)
    hipLaunchKernelGGL((few_kernel<G, NB, ACT>), grid, dim3(kFewThreads), 0, stream, a);
  else if (p.kind == kWide)
    hipLaunchKernelGGL((wide_kernel<G, NB, ACT>), grid, dim3(kWideThreads), 0, stream, a);
  else if (p.mt == 2)
    hipLaunchKernelGGL((mid_kernel<G, NB, 2, ACT>), grid, dim3(kMidThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((mid_kernel<G, NB, 4, ACT>), grid, dim3(kMidThreads), 0, stream, a);
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
  a.tsplits = pre.tsplits = p.tsplits;
  a.splits = p.splits;
  a.wk = p.wk;
  a.chunks = (int)p.chunks;
  a.tp = (int)ceil_div(NB * (int64_t)a.N, kWideP);
  a.tq = (int)ceil_div(a.M, kWideQ);
  pre.M = a.M, pre.K = a.K, pre.mt = p.mt, pre.status = a.status;
  pre.ids = a.ids, pre.adapters = a.adapters, pre.R = a.R;
  if (NB == 1) {
    const int64_t tiles = ceil_div(a.M, kShrinkTile);
    const int64_t rows = std::min<int64_t>(a.M, kShrinkTile);
    // units of a tile: one for each 16 rows and one more for each adapter
    pre.units = (int)std::min(rows, ceil_div(rows, 16) + std::min<int64_t>(rows, a.adapters));
    pre.rtiles = (int)ceil_div(a.R, 16);
    if (a.adapters == 0) pre.units = pre.rtiles = pre.tsplits = 1;  // the ids are still checked
    pre.shrink_blocks = (int)std::min(kMaxPreBlocks, tiles * pre.units * pre.rtiles * pre.tsplits);
  }
  const int64_t sb = pre.shrink_blocks;
  if (p.kind == kWide) {
    hipLaunchKernelGGL((pre_kernel<G, kPreF16>), dim3((unsigned)(sb + std::min(kMaxPreBlocks, a.M))),
                       dim3(kPreThreads), 0, stream, pre);
    a.x = pre.xo;
  } else if (p.kind == kMid) {
    const int64_t units = p.chunks * 16 * p.mt * (a.K / G) * 4;
    hipLaunchKernelGGL((pre_kernel<G, kPreFrag>),
                       dim3((unsigned)(sb + std::min<int64_t>(4096, ceil_div(units, kPreThreads)))),
                       dim3(kPreThreads), 0, stream, pre);
    a.x = pre.xo;
  } else if (sb) {
    hipLaunchKernelGGL((pre_kernel<G, kPreNone>), dim3((unsigned)sb), dim3(kPreThreads), 0, stream, pre);
  }
  launch_product<G, NB, ACT>(p, a, stream);
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

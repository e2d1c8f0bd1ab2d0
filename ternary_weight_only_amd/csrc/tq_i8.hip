// tq_i8.hip -- 8-bit rows times packed ternary weights, by themselves and
// grouped by expert.
//
//   v[m,n]   = s_x[m] sum_g s[n,g] sum_{j<G} q[m,gG+j] c[n,gG+j]
//   out[m,n] = act(v[m,n] + bias[n]) + residual[m,n]
// With experts, rows offsets[e] .. offsets[e+1] - 1 meet the weights (and
// bias) of expert e; row m's q and s_x are those of row rows[m] where rows are
// given.
//
// A group's inner sum is a whole number below 2^15, made exactly by the 8-bit
// matrix cores, so the fp16 scale is never rounded into a code; the sum over
// groups is fp32.  The five codes of a byte come from a table in LDS, four in a
// dword and the fifth beside them, and dwords of four consecutive codes are put
// together from them: q is read as it lies in memory.
//
// Three kernels multiply:
//   few_kernel    few rows (of each expert).  Each lane decodes whole units of 128
//                 codes in registers.
//   tile_kernel   more: each block decodes its weight rows into LDS, where its
//                 rows of q use them.
//   part_kernel   many, of 128-groups: the same with q in two parts of six bits
//                 (made by parts_kernel), whose matrix instructions leave floats.
// Where K is split, join_kernel adds the splits' sums and applies the epilogue.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tq_ffn.h"
#include "tq_internal.h"
#include "tq_mm.h"

namespace tq {
namespace {

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4_c;
typedef __attribute__((address_space(3))) const f32x4 lds_f32x4_c;
typedef __attribute__((address_space(3))) const uint32_t lds_u32_c;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

template <int V>
struct Int {
  static constexpr int value = V;
};

struct I8Args {
  const int8_t *q;          // [sources,K]
  const float *qs;          // [sources]
  const uint8_t *packed;    // [E,N,K/G,B]
  const uint16_t *scales;   // [E,N,K/G]
  const void *bias;         // [E,N] or null
  const void *residual;     // [T,N] or null, of out's type
  void *out;                // [T,N]
  const int32_t *offsets;   // [E+1], null without experts
  const int32_t *rows;      // [T] or null
  int64_t T, sources;
  int N, K, E;
  bool bias32, out32, vec;  // vec: eight columns at a time are aligned
  int act;
  float *partial;           // [splits][T][N] where splits > 1
  uint8_t *parts;           // of q, where it is taken in parts
  int splits;
  int wk, wt;               // few: waves of a tile, tiles of a set
  int tp;                   // tile: tiles of weight rows
  int units;                // at most, of offsets that rise within 0 .. T
  int32_t *status;
};

// ---------------------------------------------------------------------------
// decoding
// ---------------------------------------------------------------------------

constexpr uint32_t kBad = 0x00FF0000u;  // in the second dword of invalid bytes' entries

// 256 entries of 8 bytes, COPIES times, as tq_ternary.h lays its table out:
// codes 0 .. 3 as bytes; code 4 in bytes 0 and 3 of the second dword, whose
// byte 2 marks invalid bytes.
template <uint32_t COPIES>
struct Codes {
  static constexpr uint32_t kStride = 8 * COPIES, kBytes = 256 * kStride;
  uint32_t at;

  __device__ __forceinline__ Codes(uint32_t base, int lane) : at(base + 8u * ((uint32_t)lane & (COPIES - 1u))) {}

  __device__ static __forceinline__ void build(lds_bytes *table, int tid, int threads) {
    constexpr uint32_t kParts = 2, kPer = COPIES / 2 / kParts;  // 16-byte stores a thread
    static_assert(kPer >= 1, "");
    const uint32_t part = (uint32_t)tid % kParts;
    for (uint32_t e = (uint32_t)tid / kParts; e < 256u; e += (uint32_t)threads / kParts) {
      uint32_t lo = 0, v = e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo |= ((v % 3u - 1u) & 0xFFu) << (8 * i);
        v /= 3u;
      }
      const uint32_t c4 = (v % 3u - 1u) & 0xFFu;
      const u32x2 entry = e >= 243u ? u32x2{0u, kBad} : u32x2{lo, c4 | c4 << 24};
      const u32x4 two{entry.x, entry.y, entry.x, entry.y};
#pragma unroll
      for (uint32_t k = 0; k < kPer; ++k)
        *(lds_u32x4 *)(table + e * kStride + 16u * (part + kParts * ((k + (e >> 1)) % kPer))) = two;
    }
  }

  __device__ __forceinline__ u32x2 read(lds_bytes *smem, uint32_t word, int i) const {
    if constexpr (COPIES == 32)  // `at` is below 256: byte 0 the lane, byte 1 the byte
      return *(lds_u32x2_c *)(smem + __builtin_amdgcn_perm(word, at, 0x0C0C0400u + 0x100u * (uint32_t)i));
    else
      return *(lds_u32x2_c *)(smem + (((word >> (8 * i)) & 0xFFu) * kStride + at));
  }
};

// The dwords of codes that begin in the first, second, third and fourth of
// four consecutive bytes a, b, c, d (the first byte's own codes 0 .. 3 are a.x).
__device__ __forceinline__ uint32_t join_ab(u32x2 a, u32x2 b) { return __builtin_amdgcn_alignbyte(b.x, a.y, 3); }
__device__ __forceinline__ uint32_t join_bc(u32x2 b, u32x2 c) {
  return __builtin_amdgcn_perm(c.x, __builtin_amdgcn_alignbyte(b.y, b.x, 3), 0x05040100u);
}
__device__ __forceinline__ uint32_t join_cd(u32x2 c, u32x2 d) {
  return __builtin_amdgcn_perm(d.x, __builtin_amdgcn_alignbyte(c.y, c.x, 2), 0x04020100u);
}
__device__ __forceinline__ uint32_t join_d(u32x2 d) { return __builtin_amdgcn_alignbyte(d.y, d.x, 1); }

// Keeps the OR of entries' second dwords where it is written.
__device__ __forceinline__ void settle(uint32_t &flags) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(flags));
#endif
}

// The 26 bytes of a unit (128 codes, one group or two) as two loads bring
// them: bytes 0 .. 15 and 10 .. 25.
struct Unit {
  u32x4 a, b;
  uint32_t scale;  // fp16, or two
};

// The entry of byte i of the group that starts at byte OFF of a unit.
template <int G, int OFF, class L>
__device__ __forceinline__ u32x2 unit_entry(lds_bytes *smem, const L &lut, const Unit &u, int i) {
  const int at = OFF + i;
  return at < 16 ? lut.read(smem, u.a[at >> 2], at & 3) : lut.read(smem, u.b[(at - 10) >> 2], (at - 10) & 3);
}

// All codes of the group that starts at byte OFF of a unit, in order.
template <int G, int OFF, class L>
__device__ __forceinline__ void decode_unit(lds_bytes *smem, const L &lut, const Unit &u, uint32_t (&d)[G / 4],
                                            uint32_t &flags) {
#pragma unroll
  for (int p = 0; p < G / 20; ++p) {
    const u32x2 a = unit_entry<G, OFF>(smem, lut, u, 4 * p), b = unit_entry<G, OFF>(smem, lut, u, 4 * p + 1);
    const u32x2 c = unit_entry<G, OFF>(smem, lut, u, 4 * p + 2), e = unit_entry<G, OFF>(smem, lut, u, 4 * p + 3);
    flags |= a.y | b.y | c.y | e.y;
    d[5 * p] = a.x;
    d[5 * p + 1] = join_ab(a, b);
    d[5 * p + 2] = join_bc(b, c);
    d[5 * p + 3] = join_cd(c, e);
    d[5 * p + 4] = join_d(e);
    settle(flags);
  }
  constexpr int P = G / 20;  // 8 codes are left of 128, 4 of 64
  const u32x2 a = unit_entry<G, OFF>(smem, lut, u, 4 * P);
  flags |= a.y;
  d[5 * P] = a.x;
  if constexpr (G == 128) {
    const u32x2 b = unit_entry<G, OFF>(smem, lut, u, 4 * P + 1);
    flags |= b.y;
    d[5 * P + 1] = join_ab(a, b);
  }
  settle(flags);
}

__device__ __forceinline__ float f16_value(uint32_t bits) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// experts' rows
// ---------------------------------------------------------------------------

// Up to `rows` rows of one expert's segment (at most 2^30 rows in all, so that
// their numbers fit int, and in scalar registers).
struct Segment {
  int e;      // -1: no such unit
  int a, b;   // its rows
  int unit;   // which of its units
};

// Segment e, forced into 0 .. T and to follow its own start, so that offsets
// of any value lead to no access out of range.
__device__ __forceinline__ void bounds_of(const I8Args &A, int e, int &a, int &b) {
  a = min(max(A.offsets[e], 0), (int)A.T);
  b = min(max(A.offsets[e + 1], a), (int)A.T);
}

// Units of `rows` rows in all segments before lane's of the 64 from e0 on, and
// its own; returns those of the 64.
__device__ __forceinline__ int scan_units(const I8Args &A, int e0, int rows, int &a, int &b, int &before, int &own) {
  const int lane = threadIdx.x & 63, e = e0 + lane;
  a = b = 0;
  if (e < A.E) bounds_of(A, e, a, b);
  own = (b - a + rows - 1) / rows;
  int sum = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(sum, o);
    if (lane >= o) sum += v;
  }
  before = sum - own;
  return __builtin_amdgcn_readlane(sum, 63);
}

__device__ __forceinline__ int count_units(const I8Args &A, int rows) {
  if (!A.offsets) return ((int)A.T + rows - 1) / rows;
  int a, b, before, own, total = 0;
  for (int e0 = 0; e0 < A.E && total < A.units; e0 += 64) total += scan_units(A, e0, rows, a, b, before, own);
  return min(total, A.units);
}

// Unit `u` in the order of the experts; by whole waves, the same in every lane.
__device__ __forceinline__ Segment find_unit(const I8Args &A, int rows, int u) {
  if (!A.offsets) return Segment{(int64_t)u * rows < A.T ? 0 : -1, 0, (int)A.T, u};
  int a, b, before, own;
  for (int e0 = 0; e0 < A.E; e0 += 64) {
    const int total = scan_units(A, e0, rows, a, b, before, own);
    if (u < total) {
      const int j = __builtin_ctzll(__ballot(before <= u && u < before + own));
      return Segment{e0 + j, __builtin_amdgcn_readlane(a, j), __builtin_amdgcn_readlane(b, j),
                     u - __builtin_amdgcn_readlane(before, j)};
    }
    u -= total;
  }
  return Segment{-1, 0, 0, 0};
}

// Where row m of the product is read: -1 for a row index out of range.
__device__ __forceinline__ int64_t source_of(const I8Args &A, int64_t m) {
  if (!A.rows) return m;
  const int r = A.rows[m];
  return r >= 0 && r < A.sources ? r : -1;
}

// ---------------------------------------------------------------------------
// the epilogue
// ---------------------------------------------------------------------------

__device__ __forceinline__ float activate(float v, int act) {
  if (act == kActSilu) return act_value<kActSilu>(v);
  if (act == kActGelu) return act_value<kActGelu>(v);
  if (act == kActRelu2) return v > 0.f ? v * v : (v <= 0.f ? 0.f : v);  // NaN stays
  return v;
}

__device__ __forceinline__ float bias_of(const I8Args &A, int e, int n) {
  const int64_t at = (int64_t)e * A.N + n;
  return A.bias32 ? ((const float *)A.bias)[at] : bf16_to_f32(((const uint16_t *)A.bias)[at]);
}

template <int C>
__device__ __forceinline__ void activate_all(float (&v)[C], int act) {
  if (act == kActNone) return;
  if (act == kActRelu2) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = activate(v[c], kActRelu2);
  } else if (act == kActSilu) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = activate(v[c], kActSilu);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = activate(v[c], kActGelu);
  }
}

// What results need, in scalar registers: left to itself the compiler loads the
// kernel's arguments again for every row, one after another.
struct Result {
  typedef __attribute__((address_space(1))) char byte;
  uint64_t residual, out;
  int N, act, out32, vec;

  __device__ __forceinline__ explicit Result(const I8Args &A)
      : residual((uint64_t)A.residual), out((uint64_t)A.out), N(A.N), act(A.act), out32(A.out32), vec(A.vec) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+s"(residual), "+s"(out), "+s"(N), "+s"(act), "+s"(out32), "+s"(vec));
#endif
  }

  template <class T>
  __device__ __forceinline__ __attribute__((address_space(1))) T *at(uint64_t base, int64_t i) const {
    return (__attribute__((address_space(1))) T *)(byte *)base + i;
  }

  // Column n of row m, scaled and with its bias.
  __device__ __forceinline__ void put(int64_t m, int n, float v) const {
    const int64_t i = m * N + n;
    float w[1] = {v};
    activate_all(w, act);
    if (residual) w[0] += out32 ? *at<const float>(residual, i) : bf16_to_f32(*at<const uint16_t>(residual, i));
    if (out32)
      *at<float>(out, i) = w[0];
    else
      *at<uint16_t>(out, i) = f32_to_bf16(w[0]);
  }

  // Eight columns, all there and aligned to 16 bytes (vec), and their residual's
  // eight.
  struct Eight {
    u32x4 a, b;
  };
  __device__ __forceinline__ Eight residual8(int64_t m, int n) const {
    const int64_t i = m * N + n;
    Eight r{};
    if (out32) {
      r.a = *at<const u32x4>(residual, i / 4);
      r.b = *at<const u32x4>(residual, i / 4 + 1);
    } else {
      r.a = *at<const u32x4>(residual, i / 8);
    }
    return r;
  }
  template <bool RES>
  __device__ __forceinline__ void put8(int64_t m, int n, float scale, const float (&bias)[8], f32x4 lo, f32x4 hi,
                                       const Eight &r) const {
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = fmaf(c < 4 ? lo[c] : hi[c - 4], scale, bias[c]);
    activate_all(v, act);
    if constexpr (RES)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        v[c] += __uint_as_float(out32 ? (c < 4 ? r.a[c & 3] : r.b[c & 3])
                                      : c & 1 ? r.a[c >> 1] & 0xFFFF0000u : r.a[c >> 1] << 16);
    const int64_t i = m * N + n;
    if (out32) {
      *at<f32x4>(out, i / 4) = f32x4{v[0], v[1], v[2], v[3]};
      *at<f32x4>(out, i / 4 + 1) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *at<u32x4>(out, i / 8) = u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    }
  }
};

// A split's sums of columns n .. n + 7 of a row, those below N.
__device__ __forceinline__ void store_sums(float *p, int n, int N, f32x4 lo, f32x4 hi) {
  if (N % 8 == 0) {
    *(f32x4 *)p = lo;
    *(f32x4 *)(p + 4) = hi;
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (n + c < N) p[c] = c < 4 ? lo[c] : hi[c - 4];
  }
}

// The splits' sums, in order, and the epilogue.  Blocks stride over the rows,
// threads over the columns.
__global__ __launch_bounds__(256) void join_kernel(const I8Args A) {
  const int64_t tn = A.T * A.N;
  const Result result(A);
  for (int64_t m = blockIdx.y; m < A.T; m += gridDim.y) {
    int e = 0;
    if (A.offsets) {  // the expert whose segment has m: the last one that starts at or before it
      int lo = -1, hi = A.E;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.offsets[mid] <= m)
          lo = mid;
        else
          hi = mid;
      }
      if (lo < 0 || m >= A.offsets[lo + 1]) continue;  // of no segment: left as it was
      e = lo;
    }
    const int64_t src = source_of(A, m);
    const float scale = src < 0 ? 0.f : A.qs[src];
    for (int n = (int)blockIdx.x * 256 + threadIdx.x; n < A.N; n += (int)gridDim.x * 256) {
      float v = 0.f;
      const float *p = A.partial + m * A.N + n;
#pragma unroll 4
      for (int s = 0; s < A.splits; ++s) v += p[s * tn];
      result.put(m, n, fmaf(v, scale, A.bias ? bias_of(A, e, n) : 0.f));
    }
  }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

constexpr int few_waves(int copies) { return copies == 32 ? 16 : 8; }  // of a block, at most

template <int MB, int COPIES>
struct FewRoom {
  static constexpr int kRows = 4 * MB, kWaves = few_waves(COPIES);
  static constexpr uint32_t kTable = Codes<COPIES>::kBytes, kSums = kWaves * MB * 256;
  static constexpr uint32_t kX = COPIES == 32 ? (159u << 10) - kTable - kSums : 32u << 10;
};

// A unit is up to 4 MB rows of q (of one expert); a block takes one split of K
// and sets of wt tiles of 16 weight rows, wk waves a tile.  Lane (l, q) decodes
// unit q of a quad (512 codes) of weight row l, so its bytes are two wide loads
// and the four lanes of a row read 104 neighbouring ones; a unit's loads are
// asked for when the one before it has been decoded, two units in turn.  (As
// compiled they do not stay on their way: `fetch` selects on the scale that it has
// just asked for and so waits for all of it, with G = 64 right behind the loads,
// with G = 128 in one half of a pair or both.)  The matrix cores sum over the four
// lanes of a row,
// which have different groups here: so of the 16 columns, four are given to
// each row of q, column 4 i + j with row i's part of unit j and zeros elsewhere,
// and a result is a row's sum over one unit, exact, which is then scaled.  (Four
// rows of q a matrix instruction instead of 16; the instructions are far from
// bounding it.)
//
// What bounds it: with few matrices the chain before the first sum, launch, q and
// the table into LDS, about 6 us (8 tokens, eight experts of [3584,1024], 10.8 us;
// 7 rows of [14336,4096] 12.0 us where the bytes alone take 2.7); with many a
// load's latency in every quad: 32 tokens, sixteen experts of [4096,14336], 72 to
// 82 us, 2.5 to 2.8 TB/s of packed bytes (of copy's 5.2; 76 us without decode and
// products, 70 without loads).  16 rows of [14336,4096] 15.5 us, with G = 64 19.4
// (few_kernel<64, 4, 32> spills 21 registers).
template <int G, int MB, int COPIES>
__global__ __launch_bounds__(64 * few_waves(COPIES)) void few_kernel(const I8Args A) {
  typedef Codes<COPIES> L;
  typedef FewRoom<MB, COPIES> Room;
  constexpr int B = bytes_per_group(G), GU = 128 / G;  // groups of a unit
  constexpr uint32_t kXOff = Room::kTable, kSumOff = kXOff + Room::kX, kZeroOff = kSumOff + Room::kSums;
  __shared__ __align__(16) unsigned char smem_raw[kZeroOff + 128];
  __shared__ float row_scale[Room::kRows];
  __shared__ int64_t row_source[Room::kRows];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6;
  // the blocks are shared among the units that there are (whose number the host,
  // which gives every one that may be a block, does not know)
  const int wk = A.wk, wt = A.wt, kw = wv % wk, tw = wv / wk;
  const int tiles = (A.N + 15) / 16, sets = (tiles + wt - 1) / wt;
  const int units = count_units(A, Room::kRows);
  const int bpu = max(1, min(sets, (int)gridDim.x / max(1, units * A.splits)));
  const int split = (int)(blockIdx.x % A.splits);
  const int b0 = (int)(blockIdx.x / A.splits % bpu);
  const Segment seg = find_unit(A, Room::kRows, (int)(blockIdx.x / A.splits / bpu));
  if (A.offsets && blockIdx.x == 0 && A.status)
    for (int e = tid; e < A.E; e += threads)
      if (A.offsets[e] < 0 || A.offsets[e + 1] < A.offsets[e] || A.offsets[e + 1] > A.T)
        atomicOr(A.status, kDevBadSegment);
  if (seg.e < 0) return;
  const int m0 = seg.a + seg.unit * Room::kRows, M = min(seg.b - m0, Room::kRows);
  const int nG = A.K / G, nU = (nG + GU - 1) / GU, nQ = (nU + 3) / 4;
  // (at most 4096 quads and as many splits: the products fit)
  const int u0 = 4 * (nQ * split / A.splits), u1 = min(nU, 4 * (nQ * (split + 1) / A.splits));
  const int steps = b0 < sets ? (sets - b0 + bpu - 1) / bpu : 0;
  const int quads = (u1 - u0 + 3) / 4, batches = (quads + wk - 1) / wk;
  const uint8_t *packed = A.packed + (int64_t)seg.e * A.N * nG * B;
  const uint16_t *scales = A.scales + (int64_t)seg.e * A.N * nG;

  auto tile_row = [&](int j) { return ((b0 + j * bpu) * wt + tw) * 16; };
  int fj = 0, fk = 0;  // step and batch of the next request
  auto fetch = [&](Unit &f) {
    // rows past N read row N - 1 (their results go nowhere), units past the last
    // read it with scales 0
    const int64_t n = min(tile_row(fj) + l, A.N - 1);
    const int u = u0 + 4 * (kw + wk * fk) + q, g = GU * min(u, u1 - 1);
    uint32_t sc;
    if constexpr (G == 128) {
      const int64_t at = n * nG + g;
      const uint8_t *p = packed + at * B;
      __builtin_memcpy(&f.a, p, 16);
      __builtin_memcpy(&f.b, p + 10, 16);
      sc = scales[at];
    } else if (nG > 1) {
      // of an odd number of groups the last unit is the last two, the first of which belongs to the unit before
      const int64_t at = n * nG + min(g, nG - 2);
      const uint8_t *p = packed + at * B;
      __builtin_memcpy(&f.a, p, 16);
      __builtin_memcpy(&f.b, p + 10, 16);
      __builtin_memcpy(&sc, scales + at, 4);
      if (g + 1 == nG) sc &= 0xFFFF0000u;
    } else {  // a row is one group: 13 bytes, the unit's first
      const uint8_t *p = packed + n * B;
      u32x2 v, w;
      __builtin_memcpy(&v, p, 8);
      __builtin_memcpy(&w, p + 5, 8);
      f.a = u32x4{v.x, v.y, __builtin_amdgcn_alignbyte(w.y, w.x, 3), w.y >> 24};
      f.b = u32x4{0u, 0u, 0u, 0u};
      sc = scales[n];
    }
    f.scale = u < u1 ? sc : 0u;
    if (++fk == batches) {
      fk = 0;
      ++fj;
    }
  };
  Unit f0, f1;
  fetch(f0);
  fetch(f1);
  L::build(smem, tid, threads);
  if (tid < 8) *(lds_u32x4 *)(smem + kZeroOff + 16 * tid) = u32x4{0u, 0u, 0u, 0u};
  if (tid < Room::kRows) {
    const int64_t src = tid < M ? source_of(A, m0 + tid) : -1;
    if (src < 0 && tid < M && b0 == 0 && split == 0 && A.status) atomicOr(A.status, kDevBadRow);
    row_source[tid] = src;
    row_scale[tid] = src < 0 ? 0.f : A.qs[src];
  }
  __syncthreads();
  // q of the split, a row after another; of the 16-byte chunks of a unit the
  // halves are exchanged in units 2 and 3 of a quad, so that four rows' four
  // units fall into different banks
  const uint32_t ld = 512u * (uint32_t)quads + 16u;
  {
    const int chunks = (min(A.K, 128 * u1) - 128 * u0) / 16;
    const bool odd = GU == 2 && (nG & 1) && nG > 1 && u1 == nU;  // the last unit: the last two groups
    for (int o = tid; o < M * chunks; o += threads) {
      const int r = o / chunks, c = o - r * chunks;
      const int64_t src = row_source[r];
      u32x4 v{0u, 0u, 0u, 0u};
      if (src >= 0) v = *(const u32x4 *)(A.q + src * A.K + 128 * (int64_t)u0 + 16 * c);
      uint32_t to = (uint32_t)c;
      if (odd && c >= chunks - 4) to += 4;  // its second half
      *(lds_u32x4 *)(smem + kXOff + r * ld + 16u * (to ^ ((to >> 2) & 4u))) = v;
      if (odd && c >= chunks - 4)
        *(lds_u32x4 *)(smem + kXOff + r * ld + 16u * ((uint32_t)c ^ (((uint32_t)c >> 2) & 4u))) = u32x4{0u, 0u, 0u, 0u};
    }
  }
  __syncthreads();

  const L lut(0, lane);
  const Result result(A);
  const int qc = l & 3, mi = l >> 2;  // this lane's column: unit, row
  uint32_t flags = 0;
  f32x4 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  int j = 0, k = 0;
  // row m of the unit, column n
  auto put = [&](int m, int n, float v) {
    if (A.splits > 1)
      A.partial[((int64_t)split * A.T + m0 + m) * A.N + n] = v;
    else
      result.put(m0 + m, n, fmaf(v, row_scale[m], A.bias ? bias_of(A, seg.e, n) : 0.f));
  };
  auto work = [&](Unit &f) {
    const int quad = kw + wk * k;
    if (tile_row(j) < A.N && quad < quads) {
      uint32_t d[GU][G / 4];
      decode_unit<G, 0>(smem, lut, f, d[0], flags);
      if constexpr (GU == 2) decode_unit<G, 13>(smem, lut, f, d[1], flags);
      // the scales of this lane's results: rows 4 q + r, unit qc
      float s[GU][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t sc = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (16 * qc + 4 * q + r), (int)f.scale);
        s[0][r] = f16_value(sc);
        if constexpr (GU == 2) s[1][r] = f16_value(sc >> 16);
      }
      fetch(f);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        if (4 * b >= M) break;
        const uint32_t x0 = kXOff + (uint32_t)(4 * b + mi) * ld + 512u * (uint32_t)quad + 128u * (uint32_t)q;
        const uint32_t swap = 64u * (uint32_t)(q >> 1);
        const uint32_t xa = qc == q ? x0 + swap : kZeroOff, xb = qc == q ? x0 - swap : kZeroOff;
#pragma unroll
        for (int h = 0; h < GU; ++h) {
          i32x4 sum{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < G / 16; ++i) {
            const int st = h * (G / 16) + i;  // of the unit's eight steps
            const uint32_t *w = d[h] + 4 * i;
            const u32x4 x = *(lds_u32x4_c *)(smem + (st < 4 ? xa : xb) + 16u * (uint32_t)st);
            sum = mfma_i8(u32x4{w[0], w[1], w[2], w[3]}, x, sum);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[b][r] = fmaf(s[h][r], (float)sum[r], acc[b][r]);
        }
      }
    } else {
      fetch(f);
    }
    if (++k < batches) return;
    k = 0;
    // the tile's last batch: the units' sums (four lanes); lane (l, q) then has
    // weight row 4 q + qc of row mi of each four
    if (wk > 1) __syncthreads();  // the sums before have been read
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      float mine = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[b][r];
        v += __shfl_xor(v, 1);
        v += __shfl_xor(v, 2);
        mine = qc == r ? v : mine;
        acc[b][r] = 0.f;
      }
      if (wk > 1) {
        *(lds_float *)(smem + kSumOff + 4u * (uint32_t)((b * waves + wv) * 64 + lane)) = mine;
      } else {
        const int n = tile_row(j) + 4 * q + qc;
        if (4 * b + mi < M && n < A.N) put(4 * b + mi, n, mine);
      }
    }
    if (wk > 1) {  // the waves' sums, in order
      __syncthreads();
      for (int o = tid; o < wt * MB * 64; o += threads) {  // [tile][row of q][column]
        const int ts = o / (MB * 64), m = o / 16 % (4 * MB), c = o & 15;
        const int n = ((b0 + j * bpu) * wt + ts) * 16 + c;
        if (m >= M || n >= A.N) continue;
        const uint32_t at = (uint32_t)((m >> 2) * waves + ts * wk) * 64 + (uint32_t)(16 * (c >> 2) + 4 * (m & 3) + (c & 3));
        float v = 0.f;
        for (int w = 0; w < wk; ++w) v += *(lds_float *)(smem + kSumOff + 4u * (at + 64u * (uint32_t)w));
        put(m, n, v);
      }
    }
    ++j;
  };
  const int total = steps * batches;
  for (int t = 0; t < total; t += 2) {
    work(f0);
    if (t + 1 < total) work(f1);
  }
  if ((flags & kBad) && A.status) atomicOr(A.status, kDevInvalidByte);
}

// ---------------------------------------------------------------------------
// more rows
// ---------------------------------------------------------------------------

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

// 16 bytes a lane from base + off (uniform, and a lane's) straight into LDS at
// dst + 16 lane, counted by no one but the waits written below (as dma16 in
// tq_mm.h, with 32 bits of offset).
__device__ __forceinline__ void dma16_from(const void *base, uint32_t off, lds_bytes *dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"((uint32_t)dst), "v"(off), "s"(base));
#endif
}

// The same value, known only here: what follows from it is computed here, not
// ahead of a loop around, where it would hold registers.
__device__ __forceinline__ uint32_t known_here(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
  return v;
}

// Slot rows are 128 bytes of k; chunk c of row r sits at c ^ this, so that the
// 16 rows and four chunks of an operand read fall into different banks.
__device__ __forceinline__ uint32_t swap_of(uint32_t r) { return (r >> 1) & 7u; }

// A tile of results: expert, first weight row, first row of q and how many, and
// which tile and split (each row of q is looked at by one of them).
struct Tile {
  int e, n0, m0, M, ip, split;
};

// Matrix tiles of rows of q that finish_tile takes at once, and LDS that it uses.
template <int P, int Q, int WP>
__host__ __device__ constexpr int finish_once() {
  return Q / (P / 32 / WP) / 16 < 2 || WP == 1 ? 1 : 2;
}
template <int P, int Q, int WP>
__host__ __device__ constexpr uint32_t finish_room() {
  return P / 32 * finish_once<P, Q, WP>() * 16 * (P / WP) * 4;
}

// What a tile's end needs, the scales of its rows of q and the bias of its weight
// rows, on their way since its beginning: a value a thread.
template <int P, int Q>
__device__ __forceinline__ float end_value(const I8Args &A, const Tile t, int tid) {
  static_assert(Q <= P, "");
  float v = 0.f;
  if (tid >= P) {
    if (A.bias && t.n0 + tid - P < A.N) v = bias_of(A, t.e, t.n0 + tid - P);
  } else if (tid < min(Q, t.M)) {
    const int64_t src = source_of(A, t.m0 + tid);
    if (src >= 0)
      v = A.qs[src];
    else if (t.ip == 0 && t.split == 0 && A.status)
      atomicOr(A.status, kDevBadRow);
  }
  return v;
}

template <int P, int Q>
__device__ __forceinline__ void put_end(lds_bytes *ends, int tid, float v) {
  if (tid < Q || tid >= P) *(lds_float *)(ends + 4u * (uint32_t)(tid < Q ? tid : tid - P + Q)) = v;
}

// Results go through this wave's part of LDS, kOnce tiles of 16 rows of q at
// a time, [row][weight row], and leave in runs of a wave's weight rows; chunk
// c of a row sits at c ^ row % 16.  (Loops that stay loops: unrolled, the
// epilogue was most of the kernel's code and its fetching took 10 us.)
template <int P, int Q, int WP>
__device__ __forceinline__ void finish_tile(const I8Args &A, f32x4 (&acc)[P / WP / 16][Q / (P / 32 / WP) / 16],
                                            lds_bytes *smem, uint32_t ends_off, int wv, const Tile t) {
  constexpr int WQ = P / 32 / WP, TP = P / WP / 16, TQ = Q / WQ / 16;
  const int wp = wv / WQ, wq = wv % WQ;
  constexpr int W = P / WP, kOnce = finish_once<P, Q, WP>(), kLanes = W / 8, kEach = 64 / kLanes;  // lanes of a row, rows at once
  static_assert(TQ % kOnce == 0 && W % 64 == 0 && TP % 4 == 0, "");
  const int lane = lane_here(), l = lane & 15, q = lane >> 4;
  lds_bytes *room = smem + (uint32_t)(wv * (kOnce * 16 * W * 4));
  // where column l of row 4 q would be but for its chunk of four
  const uint32_t mine = (uint32_t)(wv * (kOnce * 16 * W * 4)) + 16u * (uint32_t)(q * W) + 64u * (uint32_t)q + 4u * (uint32_t)(l & 3);
  const int nw = t.n0 + wp * W + 8 * (lane % kLanes);
  // a lane's row's scale (handed over below), and its columns' bias
  static_assert(Q / WQ <= 64, "a row a lane");
  lds_bytes *ends = smem + ends_off;
  const float own = *(lds_float *)(ends + 4u * (uint32_t)(wq * (Q / WQ) + min(lane, Q / WQ - 1)));
  float bias[8];
#pragma unroll
  for (int c = 0; c < 8; ++c)
    bias[c] = *(lds_float *)(ends + 4u * (uint32_t)(Q + wp * W + 8 * (lane % kLanes) + c));
  const Result result(A);
  const int64_t mw = t.m0 + wq * (Q / WQ);
  float *sums = A.splits > 1 ? A.partial + ((int64_t)t.split * A.T + mw) * A.N + nw : nullptr;
#pragma unroll 1
  for (int part = 0; part < TQ / kOnce; ++part) {
#pragma unroll
    for (int b = 0; b < TQ; ++b)
      if (b / kOnce == part)
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            lds_bytes *to = smem + ((mine + 16u * ((uint32_t)(l >> 2) ^ (uint32_t)r)) ^ 64u * (uint32_t)a) + 4u * (uint32_t)(r * W);
#pragma unroll
            for (int c = 0; c < TP / 4; ++c)
              *(lds_float *)(to + 256u * (uint32_t)c + 64u * (uint32_t)(b % kOnce * W)) = acc[4 * c + a][b][r];
          }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const uint32_t c = 2u * (uint32_t)(lane % kLanes);
    // rows k on of this part, this lane's; `each` gets (row of the wave, its sums)
    auto rows_of = [&](int k, auto each) __attribute__((always_inline)) {
      const int i = k + lane / kLanes, r = 16 * kOnce * part + i;
      lds_bytes *from = room + 4u * (uint32_t)(i * W);
      const f32x4 lo = *(lds_f32x4_c *)(from + 16u * (c ^ (uint32_t)(i & 15)));
      const f32x4 hi = *(lds_f32x4_c *)(from + 16u * ((c + 1u) ^ (uint32_t)(i & 15)));
      const float scale = __shfl(own, r);
      if (wq * (Q / WQ) + r < t.M && nw < result.N) each(r, scale, lo, hi);
    };
    // loops by themselves: a load in one would make every pass wait for the
    // stores of the pass before, as the second one's residual does, column after
    // column (2048 rows of [14337,4096] in bf16 184 us, 242 with a residual; of
    // [14336,4096], in the others, 170 and 173)
    if (sums) {
#pragma unroll 1
      for (int k = 0; k < 16 * kOnce; k += kEach)
        rows_of(k, [&](int r, float, f32x4 lo, f32x4 hi) { store_sums(sums + (int64_t)r * result.N, nw, result.N, lo, hi); });
    } else if (!result.vec) {
#pragma unroll 1
      for (int k = 0; k < 16 * kOnce; k += kEach)
        rows_of(k, [&](int r, float scale, f32x4 lo, f32x4 hi) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (nw + j < result.N) result.put(mw + r, nw + j, fmaf(j < 4 ? lo[j] : hi[j - 4], scale, bias[j]));
        });
    } else if (!result.residual) {
#pragma unroll 2
      for (int k = 0; k < 16 * kOnce; k += kEach)
        rows_of(k, [&](int r, float scale, f32x4 lo, f32x4 hi) {
          result.put8<false>(mw + r, nw, scale, bias, lo, hi, Result::Eight{});
        });
    } else {
      constexpr int kAhead = 4;  // rows whose residuals are requested together (in bf16 one after another, as compiled)
      static_assert(16 * kOnce % (kAhead * kEach) == 0, "");
#pragma unroll 1
      for (int k = 0; k < 16 * kOnce; k += kAhead * kEach) {
        Result::Eight res[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int r = 16 * kOnce * part + k + j * kEach + lane / kLanes;
          res[j] = wq * (Q / WQ) + r < t.M && nw < result.N ? result.residual8(mw + r, nw) : Result::Eight{};
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          rows_of(k + j * kEach, [&](int r, float scale, f32x4 lo, f32x4 hi) {
            result.put8<true>(mw + r, nw, scale, bias, lo, hi, res[j]);
          });
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// P weight rows by Q rows of q, stages of 128 k; 2 P threads, their waves WP by
// WQ, the tile kept with weight rows along a lane's four results.  Two LDS slots
// of q and two of codes.  While stage s is multiplied, a row of TQ matrix tiles
// after another, a wave
//   - reads the next row's weights, and behind the last row the q of stage
//     s + 1, which landed before this stage began;
//   - scales and adds the row before;
//   - decodes its codes of s + 1, two threads a weight row, 64 codes each;
//   - requests q of s + 2, whose slot this stage's q has left, and bytes of s + 2.
// (With G = 64 the requests of a stage are waited for within it: load_raw selects
// on the scale that it asks for, and of the bytes that a thread holds the second
// eight are first looked at behind the requests of q, which drains those.)
//
// What bounds it: short K.  A tile takes 5 to 8 us beside its stages (offsets, row
// indices, first bytes and decode, results), a stage of 128 x 64 0.8 us alone on
// its CU and 1.1 with another, with G = 64 1.5 and 1.7 (the waits above, and twice
// the sums): 2000 rows of 32 experts of [3584,1024] with G = 64 52 to 58 us (46 with
// 128), about half of it in stages; 333 rows of [1024,3584], K in five, 18.2 us.  In
// a stage the vector unit (two instructions a result and group, and the decode) has
// the longest part, which is why larger tiles of 128-groups go to part_kernel.
template <int G, int P, int Q, int WP, int COPIES>
__global__ __launch_bounds__(2 * P) __attribute__((amdgpu_waves_per_eu(2, P == 256 || Q > 64 ? 2 : 4)))
void tile_kernel(const I8Args A) {
  typedef Codes<COPIES> L;
  constexpr int NT = 2 * P, WQ = NT / 64 / WP, TP = P / WP / 16, TQ = Q / WQ / 16;
  constexpr int B = bytes_per_group(G), GS = 128 / G;
  constexpr uint32_t kPSlot = P * 128, kQSlot = Q * 128, kSSlot = 2 * P * 4;
  constexpr uint32_t kQOff = 2 * kPSlot, kSOff = kQOff + 2 * kQSlot, kLutOff = kSOff + 2 * kSSlot;
  constexpr int kLoads = Q * 8 / NT;
  static_assert(P % 64 == 0 && TP >= 4 && finish_room<P, Q, WP>() <= kSOff, "");
  constexpr uint32_t kEndOff = kLutOff + L::kBytes;
  __shared__ __align__(16) unsigned char smem_raw[kEndOff + 4 * (P + Q)];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), wp = wv / WQ, wq = wv % WQ;
  const int nG = A.K / G, S = (A.K + 127) / 128;
  const L lut(kLutOff, lane);
  if (A.offsets && blockIdx.x == 0 && A.status)
    for (int e = tid; e < A.E; e += NT)
      if (A.offsets[e] < 0 || A.offsets[e + 1] < A.offsets[e] || A.offsets[e + 1] > A.T)
        atomicOr(A.status, kDevBadSegment);
  uint32_t flags = 0;
  // (T N is at most 2^40, E N 2^34 and a tile has 2^13 results or more: their number
  // fits, and only fewer than 2^24 are split)
  const int tiles = A.splits == 1 ? 0 : count_units(A, Q) * A.tp;
  for (int work = (int)blockIdx.x;; work += (int)gridDim.x) {
    // the same for the block: kept in scalar registers
    auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    const int split = A.splits == 1 || tiles == 0 ? 0 : scalar((int)((uint32_t)work / (uint32_t)tiles)), t = work - split * tiles;
    if (split >= A.splits) break;
    const int unit = scalar((int)((uint32_t)t / (uint32_t)A.tp)), ip = t - unit * A.tp;
    if (unit >= A.units) break;  // (offsets that overlap make more)
    const Segment seg = find_unit(A, Q, unit);
    if (seg.e < 0) break;
    // stages are counted from the split's first
    // (S is at most 2^14)
    const int s0 = A.splits == 1 ? 0 : scalar(S * split / A.splits);
    const int S1 = A.splits == 1 ? S : scalar(S * (split + 1) / A.splits) - s0;
    const int n0 = ip * P, m0 = seg.a + seg.unit * Q, M = min(seg.b - m0, Q);
    const Tile tile{seg.e, n0, m0, M, ip, split};

    // q: this thread's chunks of a slot, as bytes from the first of A.q (where
    // rows are given: 32 bits reach all of them) or of this tile; rows past the
    // last read it
    uint32_t from[kLoads];
    uint32_t upper = 0;  // which of them are in the second half of a stage
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t at = (uint32_t)(i * NT + tid), r = at >> 3, c = (at & 7u) ^ swap_of(r);
      const int row = min((int)r, M - 1);
      from[i] = known_here((A.rows ? (uint32_t)max(source_of(A, m0 + row), (int64_t)0) : (uint32_t)row) * (uint32_t)A.K + 16u * c);
      upper |= (c >> 2) << i;
    }
    const int8_t *qbase = A.q + (A.rows ? (int64_t)0 : (int64_t)m0 * A.K) + 128 * (int64_t)s0;
    auto request = [&](int s, uint32_t slot, int i) __attribute__((always_inline)) {
      s = min(s, S1 - 1);  // past the end the last one again, unused
      // where the second half is past the row, the first again: its codes are 0
      const uint32_t back = G == 64 && 128 * (s0 + s) + 128 > A.K && (upper >> i & 1) ? 64u : 0u;
      dma16_from(qbase + 128 * s, from[i] - back,
                 smem + kQOff + slot + 16u * (uint32_t)(i * NT + 64 * wv));
    };

    // codes: this thread's are 64 hf .. 64 hf + 63 of row dr; hf is a wave's.
    // Of a 128-group they are in bytes 0 .. 13 or 12 .. 25, whose 17 dwords of
    // codes are this thread's but the last, or but the first.
    const int hf = wv / (NT / 128), dr = tid % P;
    const int64_t first = ((int64_t)seg.e * A.N + n0) * nG;
    const uint32_t row = (uint32_t)min(dr, A.N - 1 - n0) * (uint32_t)nG;  // rows past N read row N - 1
    const uint32_t boff = known_here(row * B + (G == 128 && hf ? 10u : 0u));
    // G = 128: the second thread of a row has no use for the scale; its wave's
    // lanes read one and put it where no one looks (a branch in the loop costs more)
    const uint32_t voff = known_here(GS == 2 || hf == 0 ? 2u * row : 0u);
    u32x4 raw;  // bytes as `byte_at` finds them
    uint32_t scale;
    constexpr int kBytes = G == 128 ? 14 : 13;
    auto load_raw = [&](int s) __attribute__((always_inline)) {
      s = s0 + min(s, S1 - 1);
      const int g = G == 128 ? s : min(2 * s + hf, nG - 1);
      const uint8_t *bytes = A.packed + (first + g) * B;
      // the scale first: whoever has waited for the bytes has all
      const uint32_t sc = *(const uint16_t *)((const uint8_t *)(A.scales + first + g) + voff);
      if constexpr (G == 128) {
        __builtin_memcpy(&raw, bytes + boff, 16);
      } else {
        u32x2 lo, hi;
        __builtin_memcpy(&lo, bytes + boff, 8);
        __builtin_memcpy(&hi, bytes + boff + 5, 8);
        raw = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
      scale = G == 128 || 2 * s + hf < nG ? sc : 0u;
    };
    // byte i of this thread's, as (dword, byte of it)
    auto entry = [&](int i) __attribute__((always_inline)) {
      if (G == 128) return lut.read(smem, raw[i >> 2], i & 3);
      return i < 8 ? lut.read(smem, raw[i >> 2], i & 3) : lut.read(smem, raw[2 + ((i - 5) >> 2)], (i - 5) & 3);
    };
    // bytes 12 .. 25 of a group, to where 0 .. 13 are
    auto align_raw = [&]() __attribute__((always_inline)) {
      if constexpr (G == 128) {
        const uint32_t by = hf ? 2u : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = known_here(raw[i]);  // not waited for earlier
#pragma unroll
        for (int i = 0; i < 3; ++i) raw[i] = __builtin_amdgcn_alignbyte(raw[i + 1], raw[i], by);
        raw[3] = __builtin_amdgcn_alignbyte(0u, raw[3], by);
      }
    };
    u32x2 e[4];  // entries of a piece
    uint32_t d[17];
    auto look = [&](auto pc) __attribute__((always_inline)) {
      constexpr int I = 4 * decltype(pc)::value;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (I + k < kBytes) e[k] = entry(I + k);
    };
    auto join = [&](auto pc) __attribute__((always_inline)) {
      constexpr int p = decltype(pc)::value;
      if constexpr (p < 3) {
        flags |= e[0].y | e[1].y | e[2].y | e[3].y;
        d[5 * p] = e[0].x;
        d[5 * p + 1] = join_ab(e[0], e[1]);
        d[5 * p + 2] = join_bc(e[1], e[2]);
        d[5 * p + 3] = join_cd(e[2], e[3]);
        d[5 * p + 4] = join_d(e[3]);
      } else {
        flags |= e[0].y;
        d[15] = e[0].x;
        if constexpr (G == 128) {
          flags |= e[1].y;
          d[16] = join_ab(e[0], e[1]);
        }
      }
      settle(flags);
    };
    // 16 codes (chunk c of this thread's four), once piece c is joined
    // where they go; slots are changed by their bit
    uint32_t put = known_here(128u * (uint32_t)dr + 16u * ((4u * (uint32_t)hf) ^ swap_of((uint32_t)dr)));
    uint32_t sput = known_here(kSOff + 4u * (uint32_t)(hf * P + dr));
    auto piece = [&](auto pc) __attribute__((always_inline)) {
      constexpr int D = 4 * decltype(pc)::value;
      join(pc);
      u32x4 v{d[D], d[D + 1], d[D + 2], d[D + 3]};
      if constexpr (G == 128)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = hf ? d[D + i + 1] : v[i];
      *(lds_u32x4 *)(smem + (put ^ 16u * decltype(pc)::value)) = v;
    };
    auto store_scale = [&]() __attribute__((always_inline)) {
      *(lds_float *)(smem + sput) = f16_value(scale);
    };

    f32x4 acc[TP][TQ];
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (work != (int)blockIdx.x) __syncthreads();  // the tile before is done with LDS
    load_raw(0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) request(0, 0, i);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) request(1, kQSlot, i);
    const float end = end_value<P, Q>(A, tile, tid);
    if (work == (int)blockIdx.x) {  // the table, while those are on their way
      L::build(smem + kLutOff, tid, NT);
      __syncthreads();
    }
    align_raw();
    look(Int<0>{}), piece(Int<0>{}), look(Int<1>{}), piece(Int<1>{});
    look(Int<2>{}), piece(Int<2>{}), look(Int<3>{}), piece(Int<3>{});
    store_scale();
    put_end<P, Q>(smem + kEndOff, tid, end);
    put ^= kPSlot;
    sput ^= kSSlot;
    load_raw(1);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    const uint32_t pr = (uint32_t)(wp * (P / WP) + l), qr = (uint32_t)(wq * (Q / WQ) + l);
    // rows 16 apart have the same exchange; the second half of a stage is 64 bytes
    // on, exchanged or not
    uint32_t pat = 128u * pr + 16u * ((uint32_t)q ^ swap_of(pr));
    uint32_t qat = kQOff + 128u * qr + 16u * ((uint32_t)q ^ swap_of(qr));
    uint32_t sat = kSOff + 4u * (uint32_t)(wp * (P / WP) + l);
    static_assert(kQOff % (2 * kQSlot) == 0 && kSOff % (2 * kSSlot) == 0, "a slot's bit");
    u32x4 qf[2][TQ], pf[2];
    float sc[GS];
    i32x4 sum[TQ];  // of a group: of both halves of a stage, or (G = 64) of one
    auto read_q = [&](int h) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < TQ; ++b) qf[h][b] = *(lds_u32x4_c *)(smem + (qat ^ 64u * h) + 2048u * (uint32_t)b);
    };
    auto read_p = [&](int a, int h) __attribute__((always_inline)) {
      pf[h] = *(lds_u32x4_c *)(smem + (pat ^ 64u * h) + 2048u * (uint32_t)a);
    };
    auto read_s = [&](int a) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < GS; ++h) sc[h] = *(lds_float *)(smem + sat + 4u * (uint32_t)(h * P + 16 * a));
    };
    auto multiply = [&](int h) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < TQ; ++b) sum[b] = mfma_i8(qf[h][b], pf[h], h < GS ? i32x4{0, 0, 0, 0} : sum[b]);
    };
    auto add = [&](int a, int h) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < TQ; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[a][b][r] = fmaf(sc[h], (float)sum[b][r], acc[a][b][r]);
    };
    read_q(0);
    read_q(1);
    qat ^= kQSlot;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // q of stage 0 has left its slot
    read_p(0, 0);
    read_p(0, 1);
    read_s(0);
    constexpr int kLate = TP > 4 ? 1 : 0;  // rows between a stage's begin and the first codes
    uint32_t here = 0;                     // the slot of this stage's q
    for (int s = 0; s < S1; ++s) {
#pragma unroll
      for (int a = 0; a < TP; ++a) {
        __builtin_amdgcn_sched_barrier(0);
        // waits for the bytes requested a stage ago, so before other requests (with
        // G = 64 for the first eight)
        if (kLate == 0 && a == 0) align_raw(), look(Int<0>{});
        // operands are read as soon as those that they replace have been used
        multiply(0);
        if (a + 1 < TP) read_p(a + 1, 0);
        if (a == TP - 1) read_q(0);  // of the next stage (past the end: what the slot happens to hold)
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (GS == 2) add(a, 0);
        multiply(1);
        if (a + 1 < TP) read_p(a + 1, 1);
        if (a == TP - 1) read_q(1);
        __builtin_amdgcn_sched_barrier(0);
        if (kLate == 1 && a == 0) align_raw(), look(Int<0>{});
        if (a == kLate) piece(Int<0>{}), look(Int<1>{});
        if (a == 0)
#pragma unroll
          for (int i = 0; i < kLoads; ++i) request(s + 2, here, i);
        if (a == kLate + 1) piece(Int<1>{}), look(Int<2>{});
        if (a == kLate + 2) {
          piece(Int<2>{}), look(Int<3>{});
          store_scale();
          load_raw(s + 2);
        }
        if (a == kLate + 3) piece(Int<3>{});
        __builtin_amdgcn_sched_barrier(0);
        if (a + 1 < TP) add(a, GS - 1), read_s(a + 1);
      }
      here ^= kQSlot;
      qat ^= kQSlot;
      pat ^= kPSlot;
      put ^= kPSlot;
      sat ^= kSSlot;
      sput ^= kSSlot;
      __builtin_amdgcn_sched_barrier(0);
      // q of s + 2 has landed: only the bytes and the scale of s + 2, requested
      // behind it, may still be on their way
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(G == 128 ? 2 : 3) : "memory");
      read_p(0, 0);
      read_p(0, 1);
      add(TP - 1, GS - 1);
      read_s(0);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // nothing is on its way into LDS

    finish_tile<P, Q, WP>(A, acc, smem, kEndOff, wv, tile);
  }
  if ((flags & kBad) && A.status) atomicOr(A.status, kDevInvalidByte);
}

// ---------------------------------------------------------------------------
// more rows, groups of 128
// ---------------------------------------------------------------------------

// |q| = 16 h + l with h <= 7 and l <= 15 (16 of -128): with q's sign, 2 h and
// l / 8 are numbers of the 6-bit formats (3 exponent and 2 mantissa bits; 2 and
// 3), codes -1, 0 and 1 of the 4-bit one, and a group's sum of products, an
// eighth of a whole number below 2^15, is exact in the fp32 of the matrix cores.
// They do 128 codes of both parts in the time of 128 8-bit ones (7.5 ns a SIMD for
// each of the two instructions), but leave a float (no conversion, of 128 a thread
// and group) and halve the codes' place and reading in LDS.
//
// Parts of q: [K/128][T + pad][192], a row's 128 codes as twelve 16-byte chunks:
// chunk 4 p + (j ^ (row / 4 % 4)) is lane j's (k 32 j .. 32 j + 31) first 128 bits
// of its 192 of 2 h (p = 0), of l / 8 (p = 1), and the last 64 of both (p = 2,
// exchanged for odd j).  So the 16 rows and four chunks of an operand read fall
// into different banks, and a tile's stage is one run of memory.
constexpr int kPartBytes = 192, kPartPad = 256;  // of a row and group; rows behind the last

__host__ __device__ constexpr int64_t part_bytes(int64_t T, int64_t K) { return (K / 128 * T + kPartPad) * kPartBytes; }

// Four bytes of six bits each, together: sums of products with 1 and 64.
__device__ __forceinline__ uint32_t six_bits(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_udot4(v, 0x00004001u, __builtin_amdgcn_udot4(v, 0x40010000u, 0u, false) << 12, false);
#else
  return 0;
#endif
}

// A thread a lane's 32 codes of a row: rows given by index are gathered here.
// Bound by memory (read once, written 1.5 times): 2048 rows of 4096 7.7 us.
__global__ __launch_bounds__(256) void parts_kernel(const I8Args A) {
  const int nG = A.K / 128, j = threadIdx.x & 3;
  for (int64_t m = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 2); m < A.T; m += (int64_t)gridDim.x * 64) {
    const int64_t src = source_of(A, m);
    for (int g = blockIdx.y; g < nG; g += gridDim.y) {
      u32x4 in[2] = {};
      if (src >= 0) {
        const u32x4 *from = (const u32x4 *)(A.q + src * A.K + 128 * g + 32 * j);
        in[0] = from[0];
        in[1] = from[1];
      }
      uint32_t hi[6], lo[6], h24[4], l24[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = in[half][i], sign = x & 0x80808080u, one = sign >> 7;
          const uint32_t mag = (x ^ ((one << 8) - one)) + one;  // by bytes: 0 .. 128
          const uint32_t top = mag >> 7 & 0x01010101u;          // of 128
          const uint32_t l = (mag & 0x0F0F0F0Fu) + (top << 4), h = (mag >> 4 & 0x0F0F0F0Fu) - top;
          // 2 h, h = 0 .. 7: the formats' bits, bytes chosen by h
          const uint32_t code = __builtin_amdgcn_perm(0x1B1A1918u, 0x16141000u, h);
          h24[i] = six_bits(code | sign >> 2);
          l24[i] = six_bits(l | sign >> 2);
        }
#pragma unroll
        for (int w = 0; w < 3; ++w) {
          hi[3 * half + w] = h24[w] >> (8 * w) | h24[w + 1] << (24 - 8 * w);
          lo[3 * half + w] = l24[w] >> (8 * w) | l24[w + 1] << (24 - 8 * w);
        }
      }
      u32x4 *to = (u32x4 *)(A.parts + ((int64_t)g * A.T + m) * kPartBytes) + (j ^ (int)(m >> 2 & 3));
      to[0] = u32x4{hi[0], hi[1], hi[2], hi[3]};
      to[4] = u32x4{lo[0], lo[1], lo[2], lo[3]};
      to[8] = j & 1 ? u32x4{lo[4], lo[5], hi[4], hi[5]} : u32x4{hi[4], hi[5], lo[4], lo[5]};
    }
  }
}

constexpr uint32_t kBadNibbles = 0x80000000u;

// 256 entries of a dword, COPIES times: a byte's five codes in four bits each,
// and the mark of invalid bytes.
template <uint32_t COPIES>
struct Nibbles {
  static constexpr uint32_t kStride = 4 * COPIES, kBytes = 256 * kStride;
  uint32_t at;

  __device__ __forceinline__ Nibbles(uint32_t base, int lane) : at(base + 4u * ((uint32_t)lane & (COPIES - 1u))) {}

  __device__ static __forceinline__ void build(lds_bytes *table, int tid, int threads) {
    for (uint32_t e = (uint32_t)tid; e < 256u; e += (uint32_t)threads) {
      uint32_t codes = 0, v = e;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        codes |= (0x20Au >> (4 * (v % 3u)) & 0xFu) << (4 * i);  // -1, 0, 1
        v /= 3u;
      }
      const uint32_t w = e >= 243u ? kBadNibbles : codes;
#pragma unroll
      for (uint32_t k = 0; k < COPIES / 4; ++k)
        *(lds_u32x4 *)(table + e * kStride + 16u * ((k + e) % (COPIES / 4))) = u32x4{w, w, w, w};
    }
  }

  __device__ __forceinline__ uint32_t read(lds_bytes *smem, uint32_t word, int i) const {
    return *(lds_u32_c *)(smem + (((word >> (8 * i)) & 0xFFu) * kStride + at));
  }
};

struct Part {  // a lane's 32 numbers of six bits
  u32x4 a;
  u32x2 b;
};

// FORMAT of the part: 3 (2 h), 2 (l / 8)
template <int FORMAT>
__device__ __forceinline__ f32x4 mfma_parts(const Part &x, u32x4 codes, f32x4 c) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 w{(int)codes.x, (int)codes.y, (int)codes.z, (int)codes.w, 0, 0, 0, 0};
  const i32x8 v{(int)x.a.x, (int)x.a.y, (int)x.a.z, (int)x.a.w, (int)x.b.x, (int)x.b.y, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, w, c, FORMAT, 4, 0, 0, 0, 0);
}

// As tile_kernel, from the parts of q, a stage a group.  Here a wave has all the
// tile's weight rows and 32 rows of q, so that q is read from LDS once; its parts
// of the next stage are read along the way, not at the stage's end by all waves at
// once.
//
// What bounds it: a stage takes 2.0 to 2.2 us, 4770 cycles, of which the matrix
// cores have 2050, the vector unit 1800 and LDS 2400: two waves a SIMD (there are
// registers for no more) do not hide each other's waits.  Power holds the clock at
// 2.1 GHz (2.4 with zeros as q, in the same cycles).  2048 rows of [14336,4096]
// 159 us, 1.51 Pop/s (a library's plain 8-bit product of 8192^3 reaches 2.1, with
// nothing to decode or scale); eight experts of them, two a token, 386 to 405 us.
template <int P, int Q, int COPIES>
__global__ __launch_bounds__(2 * P) __attribute__((amdgpu_waves_per_eu(2, 2)))
void part_kernel(const I8Args A) {
  typedef Nibbles<COPIES> L;
  constexpr int NT = 2 * P, TP = P / 16, TQ = Q / (NT / 64) / 16, B = bytes_per_group(128);
  constexpr uint32_t kPSlot = P * 64, kQSlot = Q * kPartBytes, kSSlot = P * 4;
  constexpr uint32_t kSOff = 2 * kPSlot, kQOff = kSOff + 2 * kSSlot, kLutOff = kQOff + 2 * kQSlot;
  constexpr uint32_t kEndOff = kLutOff + L::kBytes, kRoom = kEndOff + 4 * (P + Q);
  constexpr int kLoads = kQSlot / 16 / NT, kStep = 2;  // rows of matrix tiles between pieces of the codes
  static_assert(P % 64 == 0 && TP % 4 == 0 && 5 * kStep < TP && 4 * TQ <= TP && kQSlot % (16 * NT) == 0 && Q <= kPartPad, "");
  static_assert(finish_room<P, Q, 1>() <= kLutOff && kRoom <= 160 << 10, "");
  __shared__ __align__(16) unsigned char smem_raw[kRoom];
  lds_bytes *smem = (lds_bytes *)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int S = A.K / 128;
  const L lut(kLutOff, lane);
  if (A.offsets && blockIdx.x == 0 && A.status)
    for (int e = tid; e < A.E; e += NT)
      if (A.offsets[e] < 0 || A.offsets[e + 1] < A.offsets[e] || A.offsets[e + 1] > A.T)
        atomicOr(A.status, kDevBadSegment);
  uint32_t flags = 0;
  const int tiles = A.splits == 1 ? 0 : count_units(A, Q) * A.tp;
  for (int work = (int)blockIdx.x;; work += (int)gridDim.x) {
    auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    const int split = A.splits == 1 || tiles == 0 ? 0 : scalar((int)((uint32_t)work / (uint32_t)tiles)), t = work - split * tiles;
    if (split >= A.splits) break;
    const int unit = scalar((int)((uint32_t)t / (uint32_t)A.tp)), ip = t - unit * A.tp;
    if (unit >= A.units) break;  // (offsets that overlap make more)
    const Segment seg = find_unit(A, Q, unit);
    if (seg.e < 0) break;
    const int s0 = A.splits == 1 ? 0 : scalar(S * split / A.splits);
    const int S1 = A.splits == 1 ? S : scalar(S * (split + 1) / A.splits) - s0;
    const int n0 = ip * P, m0 = seg.a + seg.unit * Q, M = min(seg.b - m0, Q);
    const Tile tile{seg.e, n0, m0, M, ip, split};

    // the stage's rows, those behind the tile's last too (the next group's or the
    // pad: all bits are numbers, and their results go nowhere)
    const uint8_t *qbase = A.parts + ((int64_t)s0 * A.T + m0) * kPartBytes;
    const int64_t qstep = A.T * kPartBytes;
    auto request = [&](const uint8_t *from, uint32_t slot, int i) __attribute__((always_inline)) {
      dma16_from(from + i * (16 * NT), 16u * (uint32_t)tid, smem + kQOff + slot + 16u * (uint32_t)(i * NT + 64 * wv));
    };
    // past the end the last stage again, unused
    auto stage_of = [&](int s) __attribute__((always_inline)) { return qbase + qstep * min(s, S1 - 1); };

    // codes: this thread's are 64 hf .. 64 hf + 63 of row dr, in bytes 0 .. 12 or
    // 12 .. 25 of the group; hf is a wave's
    const int hf = wv / (NT / 128), dr = tid % P;
    const int64_t first = ((int64_t)seg.e * A.N + n0) * S + s0;
    const uint32_t row = (uint32_t)min(dr, A.N - 1 - n0) * (uint32_t)S;  // rows past N read row N - 1
    const uint32_t boff = known_here(row * B + (hf ? 10u : 0u));
    // the second thread of a row has no use for the scale and puts it where the
    // first does (a branch in the loop costs more)
    const uint32_t voff = known_here(2u * row);
    u32x4 raw;
    uint32_t scale;
    auto load_raw = [&](int s) __attribute__((always_inline)) {
      s = min(s, S1 - 1);
      // the scale first: whoever has waited for the bytes has both
      scale = *(const uint16_t *)((const uint8_t *)(A.scales + first + s) + voff);
      __builtin_memcpy(&raw, A.packed + (first + s) * B + boff, 16);
    };
    auto align_raw = [&]() __attribute__((always_inline)) {  // bytes 12 .. 25 to where 0 .. 13 are
      const uint32_t by = hf ? 2u : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = known_here(raw[i]);  // not waited for earlier
#pragma unroll
      for (int i = 0; i < 3; ++i) raw[i] = __builtin_amdgcn_alignbyte(raw[i + 1], raw[i], by);
      raw[3] = __builtin_amdgcn_alignbyte(0u, raw[3], by);
    };
    uint32_t e[4];  // entries of a piece
    uint32_t w[9];  // all codes, 20 bits a byte
    auto look = [&](auto pc) __attribute__((always_inline)) {
      constexpr int I = 4 * decltype(pc)::value;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (I + k < 14) e[k] = lut.read(smem, raw[(I + k) >> 2], (I + k) & 3);
    };
    uint32_t put = known_here(64u * (uint32_t)dr + 16u * ((2u * (uint32_t)hf) ^ ((uint32_t)dr >> 2 & 3u)));
    uint32_t sput = known_here(kSOff + 4u * (uint32_t)dr);
    auto store = [&](int c) __attribute__((always_inline)) {  // 32 codes
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbit(w[4 * c + i + 1], w[4 * c + i], 16 * hf);
      *(lds_u32x4 *)(smem + (put ^ 16u * (uint32_t)c)) = v;
    };
    // entries 4 p .. of the bytes, and 32 codes once all of theirs are there
    auto piece = [&](auto pc) __attribute__((always_inline)) {
      constexpr int p = decltype(pc)::value, W = 5 * (p / 2);
      flags |= p < 3 ? e[0] | e[1] | e[2] | e[3] : e[0] | e[1];
      if constexpr (p == 0 || p == 2) {  // (the mark is in none of the bits taken)
        w[W] = (e[0] & 0xFFFFFu) | e[1] << 20;
        w[W + 1] = (e[1] >> 12 & 0xFFu) | e[2] << 8 | e[3] << 28;
        w[W + 2] = e[3] >> 4 & 0xFFFFu;
      } else {
        w[W + 2] |= e[0] << 16;
        w[W + 3] = (e[0] >> 16 & 0xFu) | e[1] << 4;
        if constexpr (p == 1) {
          w[W + 3] |= e[2] << 24;
          w[W + 4] = (e[2] >> 8 & 0xFFFu) | e[3] << 12;
        }
      }
      settle(flags);
      if constexpr (p == 1) {
        // the first 32 end in the fifth dword
        store(0);
      }
      if constexpr (p == 3) store(1);
    };
    auto store_scale = [&](int s) __attribute__((always_inline)) {
      *(lds_float *)(smem + sput) = s < S1 ? 8.f * f16_value(scale) : 0.f;  // sums are eighths
    };

    f32x4 acc[TP][TQ];
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (work != (int)blockIdx.x) __syncthreads();  // the tile before is done with LDS
    load_raw(0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) request(stage_of(0), 0, i);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) request(stage_of(1), kQSlot, i);
    const float end = end_value<P, Q>(A, tile, tid);
    if (work == (int)blockIdx.x) {  // the table, while those are on their way
      L::build(smem + kLutOff, tid, NT);
      __syncthreads();
    }
    align_raw();
    look(Int<0>{}), piece(Int<0>{}), look(Int<1>{}), piece(Int<1>{});
    look(Int<2>{}), piece(Int<2>{}), look(Int<3>{}), piece(Int<3>{});
    store_scale(0);
    put_end<P, Q>(smem + kEndOff, tid, end);
    put ^= kPSlot;
    sput ^= kSSlot;
    load_raw(1);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // operand reads: all weight rows, and this wave's of q
    const uint32_t qr = (uint32_t)(wv * (16 * TQ) + l);
    uint32_t pat = 64u * (uint32_t)l + 16u * ((uint32_t)q ^ ((uint32_t)l >> 2 & 3u));
    const uint32_t qat = kQOff + kPartBytes * qr + 16u * ((uint32_t)q ^ (((uint32_t)m0 + qr) >> 2 & 3u));
    const uint32_t qrest[2] = {qat + 128u + 8u * (uint32_t)(q & 1), qat + 128u + 8u * (uint32_t)(~q & 1)};
    uint32_t sat = kSOff + 4u * (uint32_t)l;
    static_assert(kPSlot % 1024 == 0 && kSOff % (2 * kSSlot) == 0, "a slot's bit");
    Part qf[2][2][TQ];  // of a stage and the next
    u32x4 pf[2];
    float sc[2];
    f32x4 sum[2][TQ];
    auto read_q = [&](int slot, int h, int b) __attribute__((always_inline)) {
      const uint32_t on = (uint32_t)slot * kQSlot + 16u * kPartBytes * (uint32_t)b;
      qf[slot][h][b].a = *(lds_u32x4_c *)(smem + qat + 64u * (uint32_t)h + on);
      qf[slot][h][b].b = *(lds_u32x2_c *)(smem + qrest[h] + on);
    };
    auto read_p = [&](int a) __attribute__((always_inline)) {
      pf[a & 1] = *(lds_u32x4_c *)(smem + pat + 1024u * (uint32_t)a);
      sc[a & 1] = *(lds_float *)(smem + sat + 64u * (uint32_t)a);
    };
    auto add = [&](int a) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < TQ; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[a][b][r] = fmaf(sc[a & 1], sum[a & 1][b][r], acc[a][b][r]);
    };
#pragma unroll
    for (int b = 0; b < TQ; ++b) read_q(0, 0, b), read_q(0, 1, b);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // q of stage 0 has left its slot
    read_p(0);
    auto stage = [&](auto slot_c, int s) __attribute__((always_inline)) {
      constexpr int slot = decltype(slot_c)::value;
      const uint8_t *from = stage_of(s + 2);
#pragma unroll
      for (int a = 0; a < TP; ++a) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < TQ; ++b) sum[a & 1][b] = mfma_parts<3>(qf[slot][0][b], pf[a & 1], f32x4{0.f, 0.f, 0.f, 0.f});
        __builtin_amdgcn_sched_barrier(0);
        if (a > 0) add(a - 1);
        if (a + 1 < TP) read_p(a + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < TQ; ++b) sum[a & 1][b] = mfma_parts<2>(qf[slot][1][b], pf[a & 1], sum[a & 1][b]);
        __builtin_amdgcn_sched_barrier(0);
        // q of the next stage, which landed before this one began
        if (a % 2 == 1 && a / 2 < 2 * TQ) read_q(1 - slot, a / 2 & 1, a / 4);
        if (a == 0) align_raw();
        if (a == 0)
#pragma unroll
          for (int i = 0; i < kLoads; ++i) request(from, slot * kQSlot, i);
        if (a == kStep) look(Int<0>{});
        if (a == 2 * kStep) piece(Int<0>{}), look(Int<1>{});
        if (a == 3 * kStep) piece(Int<1>{}), look(Int<2>{});
        if (a == 4 * kStep) {
          piece(Int<2>{}), look(Int<3>{});
          store_scale(s + 1);
          load_raw(s + 2);
        }
        if (a == 5 * kStep) piece(Int<3>{});
      }
      pat ^= kPSlot;
      put ^= kPSlot;
      sat ^= kSSlot;
      sput ^= kSSlot;
      __builtin_amdgcn_sched_barrier(0);
      // q of s + 2 has landed: only the bytes and the scale of s + 2, requested
      // behind it, may still be on their way
      asm volatile("s_waitcnt vmcnt(2) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      pf[0] = *(lds_u32x4_c *)(smem + pat);
      const float next = *(lds_float *)(smem + sat);
      add(TP - 1);
      sc[0] = next;
    };
    // of an odd number the last stage has scales of 0
    for (int s = 0; s < S1; s += 2) {
      stage(Int<0>{}, s);
      stage(Int<1>{}, s + 1);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // nothing is on its way into LDS

    finish_tile<P, Q, 1>(A, acc, smem, kEndOff, wv, tile);
  }
  if ((flags & kBadNibbles) && A.status) atomicOr(A.status, kDevInvalidByte);
}

// ---------------------------------------------------------------------------
// which kernel, and the workspace
// ---------------------------------------------------------------------------

constexpr int kFew = 0, kTile = 1;

struct Plan {
  int kind, mb, copies, wk, wt, splits, p, q;
  bool parts;  // tile: q in parts
  int64_t units, blocks;
};

uint32_t few_room(int mb, int copies) {
  if (copies == 8) return 32u << 10;
  return (159u << 10) - 65536u - (uint32_t)few_waves(copies) * mb * 256u;
}

// tile_kernel's tiles and what they take, in us: a tile before and behind its
// stages, and a stage where it is alone on a CU and where all `places` are taken.
// Measured with G = 128, the largest of part_kernel.  With G = 64 a stage takes
// 1.52 and 1.74, 1.78 and 2.08, 2.98 us, which the table leaves out: it chooses
// the same.  Of thirteen sizes with G = 64 its choice was the fastest to 2 % but
// for one (us, this choice, then each shape without splits in the table's order;
// [14336,4096]: 64 rows 32, of 49, 60, 109; 512 rows 75, of 104, 75, 110; 1024 rows
// 111, of 192, 143, 114; 2048 rows 238, of 368, 266, 242; 2000 rows of 32 experts
// of [3584,1024] 57, of 58, 56, 84; 8000 of them 127, of 145, 115, 128).
struct Shape {
  int p, q, places;
  double start, alone, full;
};
constexpr Shape kShapes[] = {{128, 64, 512, 6.4, 0.82, 1.10}, {128, 128, 512, 8.5, 1.05, 1.56}, {256, 256, 256, 13, 2.2, 2.2}};

// Of the shapes and the splits of K the cheapest.  Splits keep two stages, and
// their sums are written, read and joined in a launch more; parts of q are made in
// one more.
void plan_tiles(Plan &p, int64_t T, int64_t N, int64_t K, int G, int64_t used, bool grouped) {
  const int64_t stages = ceil_div(K, 128);
  double least = 1e30;
  int places = 0;
  for (const Shape &c : kShapes) {
    // units of an expert: on average its last is half full
    const int64_t units = grouped ? std::max(used, T / c.q + used / 2) : ceil_div(T, c.q);
    const int64_t tiles = units * ceil_div(N, c.p);
    for (int s = 1; s <= 16 && (s == 1 || (stages / s >= 2 && tiles * s < 1 << 24)); ++s) {
      const int64_t rounds = tiles * s / c.places, rest = tiles * s - rounds * c.places;
      // (333 rows of [1024,3584], 48 tiles: 5 splits 18.1 us, 4 18.6, 6 19.9, 7 20.4)
      const double last = rest == 0 ? 0 : 2 * rest <= c.places ? c.alone : c.full;
      const double cost = c.start * (rounds + (rest > 0)) + ceil_div(stages, s) * (rounds * c.full + last) +
                          (s > 1 ? 4.5 + (double)s * T * N * 8 / 5.2e6 : 0) +
                          (c.p == 256 && G == 128 ? 4 + (double)T * K * 2.5 / 5.2e6 : 0);
      if (cost < least) least = cost, p.p = c.p, p.q = c.q, p.splits = s, places = c.places;
    }
  }
  p.kind = kTile;
  // 2048 rows of [14336,4096] 160 us, 170 with 8-bit matrix instructions; 333 rows
  // of [1024,3584], in small tiles, 26 and 21
  p.parts = G == 128 && p.p == 256;
  p.units = grouped ? T / p.q + used : ceil_div(T, p.q);
  // blocks stay for more tiles, and keep their table: 2000 rows of 32 experts of
  // [3584,1024] 58 us with a block a tile, 56 so; eight experts of 2048 rows of
  // [14336,4096] 416 and 408
  p.blocks = std::min<int64_t>(ceil_div(N, p.p) * p.units * p.splits, places);
}

Plan plan_of(int64_t T, int64_t N, int64_t K, int G, int64_t E, bool grouped) {
  Plan p{};
  const int64_t used = grouped ? std::min(E, T) : 1;  // experts that have rows, at most
  const int64_t mean = ceil_div(T, std::max<int64_t>(used, 1));
  // few_kernel against tile_kernel, us: one matrix, 16 rows: [14336,4096] 16 and
  // 20, [3584,1024] 7.7 and 9.4; 24 rows: 25 and 22, 11 and 10.  16 experts of 8
  // rows on average: [4096,4096] 41 and 46, [3584,1024] 15 and 17; of 16: 53 and
  // 44, 25 and 18.
  if (mean > (grouped ? 8 : 16)) {
    plan_tiles(p, T, N, K, G, used, grouped);
    return p;
  }
  p.kind = kFew;
  const int64_t quads = ceil_div(K, 512), tiles = ceil_div(N, 16);
  // Rows of a unit.  Experts' numbers of rows differ, and one with more than a
  // unit's has its weights decoded again, while larger units hold more registers:
  // where there is much to decode four times the mean, else twice (us, 4, 8 and 16
  // rows a unit: 16 experts of [4096,14336], 4 rows on average 107, 101, 81; 8 of
  // them, 2 on average, 62, 43, 60; 32 of [3584,1024], 4 on average, 23, 20, 25; 8
  // of those, 2 on average, 7.6, 8.2, 9.6)
  const int64_t want = !grouped ? mean : (used * tiles * quads >= 50000 ? 4 : 2) * mean;
  p.mb = want <= 4 ? 1 : want <= 8 ? 2 : 4;
  const int64_t rows = 4 * p.mb;
  p.units = grouped ? T / rows + used : 1;
  // the large table (no two lanes of a read in a bank; one block a CU) where a CU
  // has many quads: one row, [14336,4096] 9.9 us, 10.8 with the small one;
  // [3584,1024] 5.8 and 5.5
  p.copies = used * tiles * quads >= 4096 || rows * (512 * quads + 16) > few_room(p.mb, 8) ? 32 : 8;
  const int waves = few_waves(p.copies);
  const int64_t most = (few_room(p.mb, p.copies) / rows - 16) / 512;  // quads whose q fits
  p.splits = (int)ceil_div(quads, most);
  const int64_t q = ceil_div(quads, p.splits), all = used * tiles * p.splits;
  // as many waves a tile as fill the card once (16 a CU), and as many tiles a
  // block as leave every CU one (one row, [14336,4096], waves by tiles: 4 x 4 9.9
  // us, 8 x 2 10.8, 2 x 4 10.4, 4 x 1 23; [3584,1024]: 2 x 1 5.5, 1 x 1 12)
  p.wk = (int)std::max<int64_t>(1, std::min<int64_t>({q, waves, 4096 / all}));
  p.wt = (int)std::max<int64_t>(1, std::min<int64_t>(waves / p.wk, ceil_div(all, 256)));
  const int64_t sets = ceil_div(tiles, p.wt), blocks = p.mb == 4 ? 256 : 1024;
  p.blocks = p.units * p.splits * std::max<int64_t>(1, std::min<int64_t>(sets, blocks / (p.units * p.splits)));
  if (grouped) p.blocks = std::max(p.blocks, std::min(p.units * p.splits * sets, blocks));
  // (many experts of rows so long that q's take many splits: more blocks than a
  // launch has; tiles go round)
  if (p.blocks >= int64_t(1) << 22) plan_tiles(p, T, N, K, G, used, grouped);
  return p;
}

template <int G>
void launch(const Plan &p, const I8Args &a, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  if (p.kind == kFew) {
    const dim3 block(64 * p.wk * p.wt);
    auto go = [&](auto small, auto big) {
      if (p.copies == 8)
        hipLaunchKernelGGL(small, grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL(big, grid, block, 0, stream, a);
    };
    switch (p.mb) {
      case 1: go(few_kernel<G, 1, 8>, few_kernel<G, 1, 32>); break;
      case 2: go(few_kernel<G, 2, 8>, few_kernel<G, 2, 32>); break;
      default: go(few_kernel<G, 4, 8>, few_kernel<G, 4, 32>); break;
    }
  } else if (p.parts) {
    const int64_t rows = ceil_div(a.T, 64), groups = a.K / 128;
    const unsigned y = (unsigned)std::min<int64_t>(groups, 1024);
    hipLaunchKernelGGL(parts_kernel, dim3((unsigned)std::min<int64_t>(rows, 64), y), dim3(256), 0, stream, a);
    hipLaunchKernelGGL((part_kernel<256, 256, 16>), grid, dim3(512), 0, stream, a);
  } else if (p.p == 256) {
    if constexpr (G == 64) hipLaunchKernelGGL((tile_kernel<64, 256, 256, 2, 8>), grid, dim3(512), 0, stream, a);
  } else if (p.q == 128) {
    hipLaunchKernelGGL((tile_kernel<G, 128, 128, 2, 4>), grid, dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((tile_kernel<G, 128, 64, 2, 8>), grid, dim3(256), 0, stream, a);
  }
  if (a.splits > 1)
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(a.N, 256), 64), (unsigned)std::min<int64_t>(a.T, 65535)),
                       dim3(256), 0, stream, a);
}

}  // namespace

void i8_plan(int64_t T, int64_t N, int64_t K, int G, int64_t E, int64_t *plan) {
  const Plan p = plan_of(T, N, K, G, E ? E : 1, E > 0);
  const bool few = p.kind == kFew;
  plan[0] = few ? 0 : p.parts ? 2 : 1;
  plan[1] = p.splits;
  plan[2] = few ? 4 * p.mb : p.p;
  plan[3] = few ? p.copies : p.q;
  plan[4] = few ? p.wk : 0;
  plan[5] = few ? p.wt : 0;
  plan[6] = p.blocks;
}

int64_t gemm_i8_workspace(int64_t T, int64_t N, int64_t K, int G, int64_t E, bool grouped) {
  const Plan p = plan_of(T, N, K, G, E, grouped);
  return (p.parts ? part_bytes(T, K) : 0) + (p.splits > 1 ? (p.splits * T * N * 4 + 15) / 16 * 16 : 0);
}

void launch_gemm_i8(const int8_t *q, const float *qs, const uint8_t *packed, const uint16_t *scales,
                    const int32_t *offsets, int64_t E, const int32_t *rows, int64_t sources, const void *bias,
                    bool bias32, int act, const void *residual, int64_t T, int64_t N, int64_t K, int G, void *out,
                    bool out32, void *workspace, int32_t *status, hipStream_t stream) {
  const Plan p = plan_of(T, N, K, G, E, offsets != nullptr);
  I8Args a{};
  a.q = q;
  a.qs = qs;
  a.packed = packed;
  a.scales = scales;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.offsets = offsets;
  a.rows = rows;
  a.T = T;
  a.sources = sources;
  a.N = (int)N;
  a.K = (int)K;
  a.E = (int)E;
  a.bias32 = bias32;
  a.out32 = out32;
  auto at16 = [](const void *v) { return (uintptr_t)v % 16 == 0; };
  a.vec = N % 8 == 0 && at16(out) && at16(residual);
  a.act = act;
  a.parts = (uint8_t *)workspace;
  a.partial = (float *)(a.parts + (p.parts ? part_bytes(T, K) : 0));
  a.splits = p.splits;
  a.wk = p.wk;
  a.wt = p.wt;
  a.tp = p.kind == kTile ? (int)ceil_div(N, p.p) : 0;
  a.units = (int)p.units;
  a.status = status;
  if (G == 64)
    launch<64>(p, a, stream);
  else
    launch<128>(p, a, stream);
}

}  // namespace tq

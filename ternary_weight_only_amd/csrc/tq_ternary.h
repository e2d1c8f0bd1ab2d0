// tq_ternary.h -- decoding base-3 bytes into matrix operands, and the order
// of the terms of a group that goes with it.
//
// A group of G codes is ceil(G/5) bytes of five (format: include/tq.h).  Its
// whole bytes are dealt to the lanes or threads that build an operand, and the
// G % 5-ish left-over codes of the last byte (G = 64: byte 12, codes 60..63) or
// two (G = 128: bytes 24 and 25, codes 120..127) are dealt out singly, so that
// everyone holds 32 (or 16) codes without straddling a byte:
//   quarter q (few, mid), G = 128: bytes 6q .. 6q+5 and left-over codes 2q, 2q+1
//                           G = 64:  bytes 3q .. 3q+2 and left-over code q
//   eighth e (wide): bytes 3e .. 3e+2 and left-over code e (G = 64: e < 4)
// Codes become 16-bit floats two at a time by one v_perm of bytes: a table in
// LDS gives, for each byte value, the high bytes of its five codes' floats,
// whose low bytes are zero (bf16: 2c, +-2 = 0xC000, 0x4000; f16: c, +-1 =
// 0xBC00, 0x3C00).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_mm.h"

namespace tq {

template <int V>
struct Int {
  static constexpr int value = V;
};

constexpr int kLutBf16 = 0, kLutF16 = 1;
constexpr uint32_t kBadFlag = 0xFF00u;  // in the second dword of invalid bytes' entries

// The table: 256 entries of 8 bytes, COPIES times, copy i read by lanes i,
// i + COPIES, ...  32 copies (64 KB): the 32 lanes of each half of an 8-byte
// read touch all 64 banks once whatever the bytes are, and an entry's 256
// bytes make its address one v_perm of the byte and the lane's offset.  Fewer
// copies leave LDS to other uses; lanes that share one then meet in a bank
// now and then.
template <int KIND, uint32_t COPIES>
struct Lut {
  static constexpr uint32_t kStride = 8 * COPIES, kBytes = 256 * kStride;
  uint32_t at;  // LDS byte of this lane's copy of entry 0

  __device__ __forceinline__ Lut(uint32_t base, int lane)
      : at(base + 8u * ((uint32_t)lane & (COPIES - 1u))) {}

  __device__ static __forceinline__ void build(lds_bytes *table, int tid, int threads) {
    constexpr uint32_t neg = KIND == kLutBf16 ? 0xC0u : 0xBCu, pos = KIND == kLutBf16 ? 0x40u : 0x3Cu;
    constexpr uint32_t kParts = 2, kPer = COPIES / 2 / kParts;  // 16-byte stores a thread
    const uint32_t part = (uint32_t)tid % kParts;
    for (uint32_t e = (uint32_t)tid / kParts; e < 256u; e += (uint32_t)threads / kParts) {
      uint32_t h[5], v = e;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const uint32_t d = v % 3u;
        v /= 3u;
        h[i] = d == 0u ? neg : (d == 2u ? pos : 0u);
      }
      const u32x2 entry = e >= 243u ? u32x2{0u, kBadFlag}
                                    : u32x2{h[0] | (h[1] << 8) | (h[2] << 16) | (h[3] << 24), h[4]};
      const u32x4 two{entry.x, entry.y, entry.x, entry.y};
#pragma unroll
      for (uint32_t k = 0; k < kPer; ++k)  // neighbouring entries start at different banks
        *(lds_u32x4 *)(table + e * kStride + 16u * (part + kParts * ((k + (e >> 1)) % kPer))) = two;
    }
  }

  // The entry of byte `i` of `word`.
  __device__ __forceinline__ u32x2 read(lds_bytes *smem, uint32_t word, int i) const {
    if constexpr (COPIES == 32)  // `at` is below 256: byte 0 the lane, byte 1 the byte
      return *(lds_u32x2_c *)(smem + __builtin_amdgcn_perm(word, at, 0x0C0C0400u + 0x100u * (uint32_t)i));
    else
      return *(lds_u32x2_c *)(smem + (((word >> (8 * i)) & 0xFFu) * kStride + at));
  }
};

// Codes 0, 1 and 2, 3 of an entry; code 4 of entries a and b.
__device__ __forceinline__ uint32_t pair01(u32x2 e) { return __builtin_amdgcn_perm(e.x, e.x, 0x010C000Cu); }
__device__ __forceinline__ uint32_t pair23(u32x2 e) { return __builtin_amdgcn_perm(e.x, e.x, 0x030C020Cu); }
__device__ __forceinline__ uint32_t pair44(u32x2 a, u32x2 b) {
  return __builtin_amdgcn_perm(b.y, a.y, 0x040C000Cu);
}

// High bytes of a group's left-over codes, code i in byte i.
template <int G, class L>
__device__ __forceinline__ u32x2 leftover_pool(lds_bytes *smem, const L &lut, uint32_t tail,
                                               uint32_t &flags) {
  const u32x2 a = lut.read(smem, tail, 0);
  flags |= a.y;
  if constexpr (G == 64) return u32x2{a.x, 0u};
  const u32x2 b = lut.read(smem, tail, 1);
  flags |= b.y;
  return u32x2{a.x, __builtin_amdgcn_perm(b.x, a.y, 0x06050400u)};
}

// Quarter q of a group: 4 (G = 64: 2) fragments of eight codes, d[4 s ..].
// order_quarter lists the codes in the same order.
template <int G, class L>
__device__ __forceinline__ void decode_quarter(lds_bytes *smem, const L &lut, uint32_t w0, uint32_t w1,
                                               uint32_t tail, int q, uint32_t (&d)[G / 8],
                                               uint32_t &flags) {
  if constexpr (G == 128) {
    u32x2 e[6];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = lut.read(smem, w0, i);
#pragma unroll
    for (int i = 0; i < 2; ++i) e[4 + i] = lut.read(smem, w1, i);
    const u32x2 pool = leftover_pool<G>(smem, lut, tail, flags);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const u32x2 a = e[2 * p], b = e[2 * p + 1];
      flags |= a.y | b.y;
      d[5 * p] = pair01(a);
      d[5 * p + 1] = pair23(a);
      d[5 * p + 2] = pair01(b);
      d[5 * p + 3] = pair23(b);
      d[5 * p + 4] = pair44(a, b);
    }
    d[15] = __builtin_amdgcn_perm(pool.y, pool.x, 0x010C000Cu + 0x02000200u * (uint32_t)q);
  } else {
    const u32x2 a = lut.read(smem, w0, 0), b = lut.read(smem, w0, 1),
                c = lut.read(smem, w0, 2);
    const u32x2 pool = leftover_pool<G>(smem, lut, tail, flags);
    flags |= a.y | b.y | c.y;
    d[0] = pair01(a);
    d[1] = pair23(a);
    d[2] = pair01(b);
    d[3] = pair23(b);
    d[4] = pair44(a, b);
    d[5] = pair01(c);
    d[6] = pair23(c);
    d[7] = __builtin_amdgcn_perm(pool.x, c.y, 0x040C000Cu + 0x01000000u * (uint32_t)q);
  }
}

// The 16-bit x values of quarter q of the group at xg (4-byte aligned), in the
// order of decode_quarter.
template <int G>
__device__ __forceinline__ void order_quarter(const uint16_t *xg, int q, u32x4 (&f)[G / 32]) {
  uint32_t d[G / 8];
  auto lo_hi = [](uint32_t a, uint32_t b) {  // low half of a, high half of b
    return __builtin_amdgcn_perm(b, a, 0x07060100u);
  };
  auto hi_lo = [](uint32_t a, uint32_t b) {  // high half of a, low half of b
    return __builtin_amdgcn_perm(b, a, 0x05040302u);
  };
  if constexpr (G == 128) {
    const uint32_t *p = (const uint32_t *)(xg + 30 * q);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t w0 = p[5 * i], w1 = p[5 * i + 1], w2 = p[5 * i + 2], w3 = p[5 * i + 3],
                     w4 = p[5 * i + 4];
      d[5 * i] = w0;
      d[5 * i + 1] = w1;
      d[5 * i + 2] = hi_lo(w2, w3);
      d[5 * i + 3] = hi_lo(w3, w4);
      d[5 * i + 4] = lo_hi(w2, w4);
    }
    d[15] = *(const uint32_t *)(xg + 120 + 2 * q);
  } else {
    const uint16_t *p = xg + 15 * q;  // odd offsets: 16-bit loads
    auto two = [&](int i, int j) { return (uint32_t)p[i] | (uint32_t)p[j] << 16; };
    d[0] = two(0, 1);
    d[1] = two(2, 3);
    d[2] = two(5, 6);
    d[3] = two(7, 8);
    d[4] = two(4, 9);
    d[5] = two(10, 11);
    d[6] = two(12, 13);
    d[7] = (uint32_t)p[14] | (uint32_t)xg[60 + q] << 16;
  }
#pragma unroll
  for (int s = 0; s < G / 32; ++s) f[s] = u32x4{d[4 * s], d[4 * s + 1], d[4 * s + 2], d[4 * s + 3]};
}

// Eighth e of a group: the 16 codes of three bytes (in `word`) and left-over
// code e, times the scale (twice, packed), as f16: exact, codes are -1, 0, 1.
template <class L>
__device__ __forceinline__ void decode_eighth(lds_bytes *smem, const L &lut, uint32_t word, u32x2 left,
                                              uint32_t e, uint32_t scale2, u32x4 &c0, u32x4 &c1,
                                              uint32_t &flags) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const u32x2 a = lut.read(smem, word, 0), b = lut.read(smem, word, 1),
              c = lut.read(smem, word, 2);
  flags |= a.y | b.y | c.y;
  const uint32_t one = __builtin_amdgcn_perm(left.y, left.x, 0x0C0C0C00u + e);
  const f16x2 s = __builtin_bit_cast(f16x2, scale2);
  auto times = [&](uint32_t v) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v) * s); };
  c0 = u32x4{times(pair01(a)), times(pair23(a)), times(__builtin_amdgcn_perm(one, a.y, 0x040C000Cu)),
             times(pair01(b))};
  c1 = u32x4{times(pair23(b)), times(pair44(b, c)), times(pair01(c)), times(pair23(c))};
}

// Where in its group element j of eighth e comes from.
template <int G>
__device__ __forceinline__ int eighth_source(int e, int j) {
  constexpr int at[16] = {0, 1, 2, 3, 4, -1, 5, 6, 7, 8, 9, 14, 10, 11, 12, 13};
  return j == 5 ? (G == 128 ? 120 : 60) + e : 15 * e + at[j];
}

}  // namespace tq

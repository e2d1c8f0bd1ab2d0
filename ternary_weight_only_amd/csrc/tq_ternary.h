// tq_ternary.h -- decoding base-3 bytes into matrix operands, and the order
// of the terms of a group that goes with it.
//
// A group of G codes is ceil(G/5) bytes of five (format: include/tq.h).  Codes
// become f16 two at a time by one v_perm of bytes -- a table in LDS gives, for
// each byte value, the high bytes of its five codes' floats, whose low bytes
// are zero (+-1 = 0xBC00, 0x3C00) -- and are multiplied by their group's
// fp16 scale, which is exact.  Two orders of the codes:
//   group order (few_kernel, mid_kernel: a lane holds whole groups): bytes in
//     pairs, codes 0 1 | 2 3 | 5 6 | 7 8 | 4 9 of each pair's ten, then the
//     last G % 10 codes as they are;
//   eighth order (wide_kernel: eight, or for G = 64 four, threads share a
//     group): thread e has bytes 3e .. 3e+2 and one of the codes that are left
//     over, 120 + e (G = 64: 60 + e).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_internal.h"
#include "tq_mm.h"

namespace tq {

template <int V>
struct Int {
  static constexpr int value = V;
};

constexpr uint32_t kBadFlag = 0xFF00u;  // in the second dword of invalid bytes' entries

// The table: 256 entries of 8 bytes, COPIES times, copy i read by lanes i,
// i + COPIES, ...  32 copies (64 KB): the 32 lanes of each half of an 8-byte
// read touch all 64 banks once whatever the bytes are, and an entry's 256
// bytes make its address one v_perm of the byte and the lane's offset.  Fewer
// copies leave LDS to other uses; lanes that share one then meet in a bank
// now and then.
template <uint32_t COPIES>
struct Lut {
  static constexpr uint32_t kStride = 8 * COPIES, kBytes = 256 * kStride;
  uint32_t at;  // LDS byte of this lane's copy of entry 0

  __device__ __forceinline__ Lut(uint32_t base, int lane)
      : at(base + 8u * ((uint32_t)lane & (COPIES - 1u))) {}

  __device__ static __forceinline__ void build(lds_bytes *table, int tid, int threads) {
    constexpr uint32_t neg = 0xBCu, pos = 0x3Cu;
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

// BYTES consecutive bytes as two loads bring them, whatever their place: of
// 26, bytes 0 .. 15 and 10 .. 25; of 13, bytes 0 .. 7 and 5 .. 12.
template <int BYTES>
struct Bytes;
template <>
struct Bytes<26> {
  u32x4 a, b;
};
template <>
struct Bytes<13> {
  u32x2 a, b;
};

template <int BYTES>
__device__ __forceinline__ Bytes<BYTES> load_bytes(const uint8_t *p) {
  Bytes<BYTES> w;
  __builtin_memcpy(&w.a, p, sizeof(w.a));
  __builtin_memcpy(&w.b, p + (BYTES - (int)sizeof(w.b)), sizeof(w.b));
  return w;
}

// The entry of byte i (a constant once unrolled).
template <int BYTES, class L>
__device__ __forceinline__ u32x2 entry_of(lds_bytes *smem, const L &lut, const Bytes<BYTES> &w, int i) {
  constexpr int kLoad = sizeof(w.a);
  const bool first = i < kLoad;
  const int at = first ? i : i - BYTES + kLoad;
  return lut.read(smem, first ? w.a[at >> 2] : w.b[at >> 2], at & 3);
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t scaled(uint32_t pair, f16x2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, pair) * s);
}

// Keeps the OR of entries' second dwords where it is written: left to itself
// the compiler gathers them at the end and keeps every entry until then.
__device__ __forceinline__ void settle(uint32_t &flags) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(flags));
#endif
}

// Scaled codes of byte pairs [P0, P1) of the group that starts at byte OFF of
// w, in group order: dwords 5 P0 .. of d; with TAIL the last G % 10 codes follow.
template <int G, int P0, int P1, bool TAIL, int OFF, int BYTES, class L>
__device__ __forceinline__ void decode_group(lds_bytes *smem, const L &lut, const Bytes<BYTES> &w, f16x2 s,
                                             uint32_t (&d)[G / 2], uint32_t &flags) {
#pragma unroll
  for (int p = P0; p < P1; ++p) {
    const u32x2 a = entry_of(smem, lut, w, OFF + 2 * p), b = entry_of(smem, lut, w, OFF + 2 * p + 1);
    flags |= a.y | b.y;
    d[5 * p] = scaled(pair01(a), s);
    d[5 * p + 1] = scaled(pair23(a), s);
    d[5 * p + 2] = scaled(pair01(b), s);
    d[5 * p + 3] = scaled(pair23(b), s);
    d[5 * p + 4] = scaled(pair44(a, b), s);
    settle(flags);
  }
  if constexpr (TAIL) {
    const u32x2 a = entry_of(smem, lut, w, OFF + G / 10 * 2);
    flags |= a.y;
    constexpr int D = G / 10 * 5;
    d[D] = scaled(pair01(a), s);
    d[D + 1] = scaled(pair23(a), s);
    if constexpr (G == 128) {
      const u32x2 b = entry_of(smem, lut, w, OFF + 25);
      flags |= b.y;
      d[D + 2] = scaled(__builtin_amdgcn_perm(b.x, a.y, 0x040C000Cu), s);  // code 4 of a, 0 of b
      d[D + 3] = scaled(__builtin_amdgcn_perm(b.x, b.x, 0x020C010Cu), s);  // codes 1, 2 of b
    }
  }
}

// Where in its group code i of the group order comes from.
template <int G>
__device__ __forceinline__ int group_source(int i) {
  constexpr int at[10] = {0, 1, 2, 3, 5, 6, 7, 8, 4, 9};
  return i < G / 10 * 10 ? i / 10 * 10 + at[i % 10] : i;
}

// x as f16 times 2^shift.
__device__ __forceinline__ _Float16 f16_of(uint32_t bf16, int shift) {
  return (_Float16)ldexpf(bf16_to_f32(bf16), shift);
}

// The power of two that brings the largest finite magnitude `top` (bf16 bits
// without sign) to [2^14, 2^15): a bf16 value's eight bits fit f16's eleven,
// so every element down to 2^-32 of the largest is exact in f16.  A smaller
// one is off by at most 2^-40 of it; what the sums lose by that is added where
// it counts (lost_part in tq_glu.hip).
__device__ __forceinline__ int f16_shift(uint32_t top) {
  int exponent;  // top is in [2^(exponent - 1), 2^exponent)
  (void)frexpf(bf16_to_f32(top), &exponent);
  return top ? 15 - exponent : 0;
}

// Of some bf16 values, as bits without sign: the largest that is finite and
// the smallest that is not 0, two values a step in packed 16-bit operations.
// A span is one word, {largest, ~smallest}, and joins by its halves' maxima.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
struct SpanOf {
  u16x2 top{0, 0};           // less 0x7F80 modulo 2^16: the finite ones from 0x8080 on, Inf and NaN below
  u16x2 low{0xFFFF, 0xFFFF};  // less one: 0 is the largest

  __device__ __forceinline__ void take(u32x4 v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u16x2 b = __builtin_bit_cast(u16x2, v[j] & 0x7FFF7FFFu);
      top = __builtin_elementwise_max(top, b - (u16x2){0x7F80, 0x7F80});
      low = __builtin_elementwise_min(low, b - (u16x2){1, 1});
    }
  }
  __device__ __forceinline__ uint32_t word() const {
    const u16x2 t{top.x, (uint16_t)~low.x}, l{top.y, (uint16_t)~low.y};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(t, l));
  }
};
__device__ __forceinline__ uint32_t span_join(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t span_wave(uint32_t s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) s = span_join(s, (uint32_t)__shfl_xor((int)s, o));
  return s;
}
__device__ __forceinline__ uint32_t span_top(uint32_t s) {
  const uint32_t t = s & 0xFFFFu;
  return t > 0x8080u ? t - 0x8080u : 0u;
}
// Whether some may be inexact in f16 times 2^f16_shift(top): the last bit of
// one with exponent field f is worth 2^(f - top's field + 7), f16's 2^-24.
__device__ __forceinline__ bool span_loses(uint32_t s) {
  const uint32_t smallest = (~s >> 16) + 1u;  // 2^16: none
  return max(smallest >> 7, 1u) + 31u < span_top(s) >> 7;
}

// What a finite bf16 value has that f16_of leaves out (exact), and of eight the
// magnitudes' sum; 0 of an Inf or NaN.
__device__ __forceinline__ float lost_of(uint32_t bf16, int shift) {
  const float v = bf16_to_f32(bf16);
  return (bf16 & 0x7FFFu) < 0x7F80u ? v - ldexpf((float)f16_of(bf16, shift), -shift) : 0.f;
}
__device__ __forceinline__ float lost_of(u32x4 v, int shift) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum += fabsf(lost_of((j & 1 ? v[j / 2] >> 16 : v[j / 2]) & 0xFFFFu, shift));
  return sum;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Eighth e of a group is the 16 codes of three bytes (in `word`) and left-over
// code e.  Its entries:
struct Eighth {
  u32x2 a, b, c;
};
template <class L>
__device__ __forceinline__ Eighth look_up_eighth(lds_bytes *smem, const L &lut, uint32_t word) {
  return Eighth{lut.read(smem, word, 0), lut.read(smem, word, 1), lut.read(smem, word, 2)};
}
// Its codes times the scale (twice, packed), as f16: exact, codes are -1, 0, 1.
__device__ __forceinline__ void decode_eighth(const Eighth &t, u32x2 left, uint32_t e, uint32_t scale2,
                                              u32x4 &c0, u32x4 &c1, uint32_t &flags) {
  flags |= t.a.y | t.b.y | t.c.y;
  const uint32_t one = __builtin_amdgcn_perm(left.y, left.x, 0x0C0C0C00u + e);
  const f16x2 s = __builtin_bit_cast(f16x2, scale2);
  c0 = u32x4{scaled(pair01(t.a), s), scaled(pair23(t.a), s),
             scaled(__builtin_amdgcn_perm(one, t.a.y, 0x040C000Cu), s), scaled(pair01(t.b), s)};
  c1 = u32x4{scaled(pair23(t.b), s), scaled(pair44(t.b, t.c), s), scaled(pair01(t.c), s),
             scaled(pair23(t.c), s)};
}

// Where in its group element j of eighth e comes from.
template <int G>
__device__ __forceinline__ int eighth_source(int e, int j) {
  constexpr int at[16] = {0, 1, 2, 3, 4, -1, 5, 6, 7, 8, 9, 14, 10, 11, 12, 13};
  return j == 5 ? (G == 128 ? 120 : 60) + e : 15 * e + at[j];
}

}  // namespace tq

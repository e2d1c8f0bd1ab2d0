// tq_mm.h -- the matrix-core product shared by the gated feed-forward and
// adapter kernels of gfx950: a BP x BQ tile of
//   C[q,p] = sum_k P[p,k] Q[q,k]
// per block, four or eight waves, k in stages of 32.
//
// The tile is kept in registers with p along the four consecutive rows a lane
// of v_mfma_f32_16x16x32 holds, so a lane's results are contiguous in an
// output row.  Both operands pass through rings of LDS slots, a stage a slot:
//   * memory -> LDS without registers (buffer loads with the lds modifier),
//     kRing - 1 stages ahead;
//   * LDS -> registers one stage ahead: while the MFMAs of stage s run, the
//     fragments of s + 1 replace those just used, so the matrix cores find
//     their operands ready after the barrier that ends the stage.
// One barrier a stage.  The one that ends stage s says that stage s + 2 has
// landed for every wave (each waits for its own loads first), and that every
// wave has used the fragments of stage s, so all reads of its slot are done
// and stage s + 1 may request stage s + kRing into it.
//
// An operand is stored in memory either with k contiguous (kRows: row r at
// r * ld) or with its rows contiguous (kCols: k at k * ld), which the
// gradients need.  Slots mirror memory, 64 bytes a row or 2 R bytes a k, with
// 16-byte (kRows) or 32-byte (kCols) units exchanged so that a fragment read
// touches every LDS bank once; kCols fragments are read with the transposing
// ds_read_b64_tr_b16 (lane i of 16 supplies k = i / 4, columns 4 (i % 4)..+3
// and receives column i, four k).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_ffn.h"

namespace tq {

typedef __attribute__((address_space(3))) unsigned char lds_bytes;
typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8_c;
typedef __attribute__((address_space(3))) const u32x2 lds_u32x2_c;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kKS = 32;    // k per stage
constexpr int kRing = 5;   // LDS slots of a streamed operand: 5 x 32 KB are a CU's 160 KB
constexpr uint32_t kNoRow = 0x80000000u;  // past every range: such a load writes zeros

constexpr int kRows = 0, kCols = 1;  // operand storage

// Loads at a scalar address, plus a lane's offset, plus a scalar one: no lane
// holds or adds 64-bit addresses.  Any alignment; zeros past `bytes`.
struct Scalar {
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ explicit Scalar(const void *base, uint32_t bytes = 0x7FFFFFFFu)
      : rs(__builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000)) {}
  __device__ __forceinline__ uint32_t load4(uint32_t off, int at) const {
    return __builtin_amdgcn_raw_buffer_load_b32(rs, (int)off, at, 0);
  }
  __device__ __forceinline__ uint32_t load2(uint32_t off, int at) const {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)off, at, 0);
  }
  __device__ __forceinline__ uint32_t load1(uint32_t off, int at) const {
    return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, (int)off, at, 0);
  }
#else
  __device__ explicit Scalar(const void *, uint32_t = 0) {}
  __device__ uint32_t load4(uint32_t, int) const { return 0; }
  __device__ uint32_t load2(uint32_t, int) const { return 0; }
  __device__ uint32_t load1(uint32_t, int) const { return 0; }
#endif
};

// Unit exchange of a kCols slot: the 32-byte unit u of k sits at u ^ this.
__device__ __forceinline__ uint32_t cols_swz(uint32_t k) { return (k & 3u) | ((k >> 1) & 4u); }

// Exchange of the 16-byte chunks of row r in a kRows slot: chunk c sits at
// c ^ this.  A wave's b128 read goes through LDS in quarters made of lanes
// 0-3, 12-15, 20-23, 24-27 (and so on): rows of one quarter's four groups
// carry exchanges 0, 1 and, a chunk apart, 2, 3, so that the 16 chunks fall
// into 16 different 16-byte bank groups.  (An exchange by r / 4 alone made
// every such read take twice its time.)
__device__ __forceinline__ uint32_t rows_swz(uint32_t r) { return (0u - (r >> 2)) & 3u; }

// Byte offset of 16-byte chunk c (0..3) of row r in a kRows slot.
__device__ __forceinline__ uint32_t rows_at(uint32_t r, uint32_t c) {
  return 64u * r + 16u * (c ^ rows_swz(r));
}

// 16 bytes a lane from base + off straight into LDS at dst + 16 lane (dst is
// uniform); past-range offsets write zeros.  Written as one instruction of
// inline assembly because the compiler, seeing LDS written by a load, waits
// for all of them before each transposing LDS read; the waits here are the
// kernels' own (vmcnt before the barrier of a stage).  It has no register
// results.
__device__ __forceinline__ void dma16(const void *base, lds_bytes *dst, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass knows no such registers
  const uint64_t b = (uint64_t)base;
  const u32x4 rs{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, 0x7FFFFFFFu, 0x00020000u};
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "{m0}"((uint32_t)dst), "v"(off), "s"(rs));
#endif
}

// The same load for a kernel whose LDS reads the compiler can tell apart from
// these writes; its own wait counts then include it.
__device__ __forceinline__ void dma16_tracked(const void *base, lds_bytes *dst, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass knows no 16-byte load into LDS
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, 0x7FFFFFFF, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0, 0);
#endif
}

// One operand's stream into its ring: R rows (columns of its slot), NT
// threads, two 16-byte loads a thread and stage.
template <int KIND, int R, int NT>
struct Stream {
  static constexpr int kLoads = 4 * R / NT;
  static constexpr int kSlot = R * kKS * 2;
  uint32_t off[kLoads];  // byte offset of this thread's chunk in stage 0, kNoRow if masked
  uint32_t krow[kLoads]; // kCols: its k within the stage

  // kRows: row_of(r) gives the memory row of slot row r, or -1.
  template <class F>
  __device__ __forceinline__ void init_rows(int tid, uint32_t ld, F row_of) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t e = (uint32_t)(i * NT + tid), r = e >> 2, c = (e & 3u) ^ rows_swz(r);
      const int64_t m = row_of((int)r);
      off[i] = m < 0 ? kNoRow : (uint32_t)m * ld * 2u + 16u * c;
    }
  }
  // kCols: columns c0.. of which `cols` exist (a multiple of 8).
  __device__ __forceinline__ void init_cols(int tid, uint32_t ld, int cols) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t e = (uint32_t)(i * NT + tid), k = e / (R / 8), c16 = e % (R / 8);
      const uint32_t c = 2u * ((c16 >> 1) ^ cols_swz(k)) + (c16 & 1u);
      krow[i] = k;
      off[i] = (int)(8u * c) < cols ? k * ld * 2u + 16u * c : kNoRow;
    }
  }
  // Request i of the stage at `base` into `slot`; k rows >= krem read as
  // zeros.
  __device__ __forceinline__ void load(int i, const void *base, lds_bytes *slot, uint32_t wave,
                                       int krem) const {
    uint32_t o = off[i];
    if constexpr (KIND == kCols)
      o = (int)krow[i] < krem ? o : kNoRow;
    else
      o = krem > 0 ? o : kNoRow;
    dma16(base, slot + 16u * ((uint32_t)(i * NT) + 64u * wave), o);
  }
};

// Fragment addresses of a wave's T 16-row blocks starting at slot row r0 (a
// multiple of 16 T).
template <int KIND, int R, int T>
struct Frags {
  static constexpr int kBases = KIND == kRows ? 1 : T;
  uint32_t at[kBases];
  __device__ __forceinline__ void init(int lane, int r0) {
    const uint32_t l = lane & 15, q = lane >> 4;
    if constexpr (KIND == kRows) {
      at[0] = rows_at((uint32_t)r0 + l, q);
    } else {
      const uint32_t k = 8u * q + (l >> 2);
#pragma unroll
      for (int a = 0; a < T; ++a)
        at[a] = k * (2u * R) + 32u * (((uint32_t)(r0 / 16 + a)) ^ cols_swz(k)) + 8u * (l & 3u);
    }
  }
  // Block a of the stage in the slot at byte `slot`.
  __device__ __forceinline__ bf16x8 read(lds_bytes *smem, uint32_t slot, int a) const {
    if constexpr (KIND == kRows) {
      return *(lds_bf16x8_c *)(smem + slot + at[0] + 1024u * a);
    } else {
      // cols_swz(k + 4) == cols_swz(k): k and k + 4 agree in bits 0, 1 and 3
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(smem + slot + at[a]));
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(smem + slot + at[a] + 8u * R));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Order for the scheduler: the MFMAs of one stage in rows of TQ, each row
// followed by the fragment reads that replace its operands (and, in the first
// half, the other operand's).
template <int PK, int QK, int TP, int TQ>
__device__ __forceinline__ void order_stage() {
#pragma unroll
  for (int a = 0; a < TP; ++a) {
    __builtin_amdgcn_sched_group_barrier(0x008, TQ, 0);                 // MFMA
    if (2 * a < TP)  // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x100, (2 * TQ / TP) * (QK == kRows ? 1 : 2), 0);
    __builtin_amdgcn_sched_group_barrier(0x100, PK == kRows ? 1 : 2, 0);
  }
}

__device__ __forceinline__ int next_slot(int slot) { return slot == kRing - 1 ? 0 : slot + 1; }

template <bool F16>
__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | (uint32_t)f32_to_bf16(b) << 16;
}

// Four values as bf16, at an 8-byte aligned address.
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v) {
  *(u32x2 *)p = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
}

// Exchanges the odd 16-lane rows of a with the even ones of b.
__device__ __forceinline__ void swap_rows(uint32_t &a, uint32_t &b) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
#endif
}

// Two neighbouring 16-row tiles of P as bf16: lane (l, h) holds rows 4 h ..
// 4 h + 3 of each; after the exchange eight rows in order, from row
// pack8_row(lane) of the two tiles' 32 on, so that a row of the output gets 64
// bytes at once.
__device__ __forceinline__ u32x4 pack8(f32x4 v, f32x4 w) {
  uint32_t d[4] = {pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(w[0], w[1]), pack2(w[2], w[3])};
  swap_rows(d[0], d[2]);
  swap_rows(d[1], d[3]);
  return u32x4{d[0], d[1], d[2], d[3]};
}
__device__ __forceinline__ int pack8_row(int lane) {
  const int h = lane >> 4;
  return 16 * (h & 1) + 8 * (h >> 1);
}

// Tile of block b of a launch: consecutive tiles run on one XCD (blocks go to
// the eight XCDs in turn), and 4 tiles of q by a run of p follow one another,
// so that the 32 CUs of an XCD share operand rows in its L2.
__device__ __forceinline__ void tile_of_block(int b, int total, int tp, int tq, int &ip, int &iq) {
  const int xcds = 8, q = total / xcds, r = total % xcds, x = b % xcds;
  const int t = x * q + (x < r ? x : r) + b / xcds;
  const int band = 4 * tp, g = t / band, rest = t - g * band;
  const int h = tq - 4 * g < 4 ? tq - 4 * g : 4;
  ip = rest / h;
  iq = 4 * g + rest - ip * h;
}

}  // namespace tq

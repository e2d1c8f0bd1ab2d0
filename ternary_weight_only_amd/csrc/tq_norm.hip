// tq_norm.hip -- the root-mean-square norm in front of a projection whose rows
// are held in 8 bits: the residual's addition, the norm and the rounding of
// each row, one pass over the data; and its gradients.
//
//   y[m,k] = x[m,k] + r[m,k]             (rounded to r's type; y = x without r)
//   rstd[m] = 1 / sqrt(sum_k y[m,k]^2 / K + eps)
//   t[m,k] = y[m,k] w[k],  top[m] = max_k |t[m,k]|
//   q[m,k] = round_half_even(127 t[m,k] / top[m]),  s[m] = top[m] rstd[m] / 127
//   h[m,k] = bf16(q[m,k] s[m])           (what training multiplies by)
//
// 1 / rms cancels in q, which is therefore exact: t of a bf16 y and w has 16
// bits, 127 t and q top have 23, so a quotient near a border is decided by a
// difference that fp32 holds without rounding.  With fp32 among the types the
// same is done in fp64 (39 bits; with both y and w fp32, 127 t has 55 and fp64
// decides).
//
// Backward, straight through the rounding (absmax clips nothing), n = y rstd:
//   dx = rstd (dh w - n mean_k(dh w n)) + dy,   dw[k] = sum_m dh[m,k] n[m,k]
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tq_ffn.h"
#include "tq_internal.h"

namespace tq {
namespace {

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Eight consecutive elements as loaded: bf16 in `a`, fp32 in both.
struct Raw8 {
  u32x4 a, b;
};

// Elements k .. k + 7 of a row of K (zeros past its end), any alignment that
// the type has.
__device__ __forceinline__ Raw8 load8(const void *row, bool f32, int k, int K) {
  Raw8 r{u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
  if (f32) {
    const uint32_t *p = (const uint32_t *)row + k;
    if (k + 8 <= K) {
      __builtin_memcpy(&r.a, p, 16);
      __builtin_memcpy(&r.b, p + 4, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) (i < 4 ? r.a : r.b)[i & 3] = p[i];
    }
  } else {
    const uint16_t *p = (const uint16_t *)row + k;
    if (k + 8 <= K) {
      __builtin_memcpy(&r.a, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) r.a[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  return r;
}

__device__ __forceinline__ float value8(const Raw8 &r, bool f32, int i) {
  const uint32_t wide = i < 4 ? r.a[i & 3] : r.b[i & 3];
  const uint32_t half = i & 1 ? r.a[i >> 1] & 0xFFFF0000u : r.a[i >> 1] << 16;
  return __uint_as_float(f32 ? wide : half);
}

// Eight values as the type, rounded to nearest even.
__device__ __forceinline__ void store8(void *row, bool f32, int k, int K, const float (&v)[8]) {
  if (f32) {
    float *p = (float *)row + k;
    if (k + 8 <= K) {
      __builtin_memcpy(p, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) p[i] = v[i];
    }
  } else {
    uint16_t *p = (uint16_t *)row + k;
    uint16_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = f32_to_bf16(v[i]);
    if (k + 8 <= K) {
      __builtin_memcpy(p, h, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) p[i] = h[i];
    }
  }
}

struct NormArgs {
  const void *x, *r, *w;     // r, w may be null
  bool x32, r32, w32;        // fp32, else bf16
  int64_t M, m0;             // rows, and the first of this launch
  int K;
  double eps;
  void *y;                   // written where r is given, in its type
  int8_t *q;                 // 8-bit rows and their scales,
  float *scales;
  uint16_t *h;               // or the values they stand for
  float *rstd;               // may be null
  int32_t *status;
};

// What a row's threads know of it.
struct Row {
  double top, inv;   // max |t| and 127 / it (0 where top is 0)
  float s;           // scale
  float rstd;
  bool bad;          // an Inf or NaN in it
};

// 127 t / top, rounded half to even, exactly where 127 t and n top fit the
// type: beside a border the remainder decides.
template <class F>
__device__ __forceinline__ int code_of(F t, F top, F inv) {
  const F f = t * inv;
  F n = sizeof(F) == 4 ? (F)rintf((float)f) : (F)rint((double)f);
  const F d = f > n ? f - n : n - f;
  if (d > (F)0.4999) {
    const F r = sizeof(F) == 4 ? (F)fmaf(-(float)n, (float)top, 127.f * (float)t)
                               : (F)fma(-(double)n, (double)top, 127.0 * (double)t);
    const F a = r < 0 ? -r : r, half = (F)0.5 * top;
    if (a > half || (a == half && ((int)n & 1))) n += r < 0 ? (F)-1 : (F)1;
  }
  return (int)n;
}

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double wave_add(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// Of magnitudes as bits: NaN above infinity above every number.
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}
__device__ __forceinline__ uint64_t wave_top(uint64_t v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const uint64_t u = (uint64_t)__shfl_xor((long long)v, o);
    v = u > v ? u : v;
  }
  return v;
}

// The sum and the largest of W waves' values, by every thread of them (W > 1:
// through `room`, a barrier).
template <int W, class F, class U>
__device__ __forceinline__ void join_waves(F &sum, U &top, unsigned char *room) {
  sum = wave_add(sum);
  top = wave_top(top);
  if constexpr (W > 1) {
    F *sums = (F *)room;
    U *tops = (U *)(room + W * sizeof(F));
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sums[wave] = sum;
      tops[wave] = top;
    }
    __syncthreads();
    sum = 0;
    top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      sum += sums[i];
      top = tops[i] > top ? tops[i] : top;
    }
  }
}

constexpr float kTopLow = 0x1p-60f, kTopHigh = 0x1p60f;   // top and the sum of squares that fp32 takes:
constexpr float kSumLow = 0x1p-80f, kSumHigh = 0x1p100f;  // no product or quotient near them leaves its range

__device__ __forceinline__ Row row_narrow(float sum, float top, int K, double eps) {
  Row row;
  row.rstd = 1.f / sqrtf(sum / (float)K + (float)eps);
  row.s = top * row.rstd / 127.f;
  row.top = top;
  row.inv = 127.f / top;
  row.bad = false;
  return row;
}
__device__ __forceinline__ Row row_wide(double sum, uint64_t bits, int K, double eps) {
  Row row;
  const double rstd = 1.0 / sqrt(sum / (double)K + eps);
  row.bad = bits >= 0x7FF0000000000000ull;
  row.top = __longlong_as_double((long long)bits);
  row.inv = row.top > 0.0 ? 127.0 / row.top : 0.0;
  row.rstd = (float)rstd;
  row.s = row.bad ? __uint_as_float(0x7FC00000u) : (float)(row.top > 0.0 ? row.top * rstd / 127.0 : 0.0);
  return row;
}

__device__ __forceinline__ uint64_t magnitude(double t) {
  return (uint64_t)__double_as_longlong(t) & 0x7FFFFFFFFFFFFFFFull;
}

// Eight codes as asked for.
__device__ __forceinline__ void put8(const NormArgs &A, int64_t m, int k, const int (&n)[8], float s) {
  if (A.q) {
    uint32_t d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      d[i] = ((uint32_t)n[4 * i] & 0xFFu) | ((uint32_t)n[4 * i + 1] & 0xFFu) << 8 |
             ((uint32_t)n[4 * i + 2] & 0xFFu) << 16 | (uint32_t)n[4 * i + 3] << 24;
    int8_t *p = A.q + m * A.K + k;
    if (k + 8 <= A.K) {
      __builtin_memcpy(p, d, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < A.K) p[i] = (int8_t)n[i];
    }
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)n[i] * s;
    store8(A.h + m * A.K, false, k, A.K, v);
  }
}

__device__ __forceinline__ void put_row(const NormArgs &A, int64_t m, const Row &row) {
  if (A.q) A.scales[m] = row.s;
  if (A.rstd) A.rstd[m] = row.rstd;
  if (row.bad && A.status) atomicOr(A.status, kDevNonfinite);
}

__device__ __forceinline__ int64_t stride_of(bool f32, int K) { return (int64_t)K * (f32 ? 4 : 2); }

// A row by W waves, kept in registers between the sums and the rounding:
// eights v T + t of it a thread (T = 64 W threads), V of them.  Four rows a
// block where a wave has one.  NARROW: all of bf16; a row whose sums leave what
// fp32 is good for, and every row otherwise, is summed and rounded in fp64.
// Bound by HBM at many rows: 4096 rows of 4096 bf16 with a residual, 134 MB, 23.9 us
// on the device (a copy that moves as much takes 25.9, other buffers each time: a
// part of either is still in the last cache); all in fp32, 235 MB, 44.3 a call
// (45.5 at a large copy's 5.16 TB/s).  Without a residual 24.1 of fp32 rows, whose
// sums and codes are fp64 (the bytes 19.5), and 15.2 of bf16 ones (13.0).  By latency
// at few (a row of 1024: 3.5 us, of a call's 10.4 on the host).
template <int V, int W, bool NARROW>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_kernel(const NormArgs A) {
  __shared__ __align__(16) unsigned char room[2][W * 16];
  constexpr int T = 64 * W;
  const int64_t m = A.m0 + (W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x);
  if (m >= A.M) return;
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const bool x32 = !NARROW && A.x32, r32 = !NARROW && A.r32, w32 = !NARROW && A.w32;
  const char *x = (const char *)A.x + m * stride_of(x32, A.K);
  const char *r = (const char *)A.r + m * stride_of(r32, A.K);
  Raw8 xr[V], rr[V], wr[V];
#pragma unroll
  for (int v = 0; v < V; ++v) xr[v] = load8(x, x32, 8 * (v * T + t), A.K);
  if (A.r)
#pragma unroll
    for (int v = 0; v < V; ++v) rr[v] = load8(r, r32, 8 * (v * T + t), A.K);
  if (A.w)
#pragma unroll
    for (int v = 0; v < V; ++v) wr[v] = load8(A.w, w32, 8 * (v * T + t), A.K);

  float y[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (A.r) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sum = value8(xr[v], x32, i) + value8(rr[v], r32, i);
        y[v][i] = r32 ? sum : bf16_to_f32(f32_to_bf16(sum));
      }
      store8((char *)A.y + m * stride_of(r32, A.K), r32, 8 * (v * T + t), A.K, y[v]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] = value8(xr[v], x32, i);
    }
  }
  auto weight = [&](int v, int i) { return A.w ? value8(wr[v], w32, i) : 1.f; };

  if constexpr (NARROW) {
    float sum = 0.f;
    uint32_t bits = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum = fmaf(y[v][i], y[v][i], sum);
        bits = max(bits, __float_as_uint(y[v][i] * weight(v, i)) & 0x7FFFFFFFu);
      }
    join_waves<W>(sum, bits, room[0]);
    const float top = __uint_as_float(bits);
    if (top > kTopLow && top < kTopHigh && sum > kSumLow && sum < kSumHigh) {  // no NaN either
      const Row row = row_narrow(sum, top, A.K, A.eps);
      if (t == 0) put_row(A, m, row);
      const float inv = (float)row.inv;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = 8 * (v * T + t);
        int n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = code_of(y[v][i] * weight(v, i), top, inv);
        if (k < A.K) put8(A, m, k, n, row.s);
      }
      return;
    }
  }
  double sum = 0.0;
  uint64_t bits = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = y[v][i];
      sum = fma(d, d, sum);
      const uint64_t b = magnitude(d * (double)weight(v, i));
      bits = b > bits ? b : bits;
    }
  join_waves<W>(sum, bits, room[1]);
  const Row row = row_wide(sum, bits, A.K, A.eps);
  if (t == 0) put_row(A, m, row);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int k = 8 * (v * T + t);
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      n[i] = row.bad ? 0 : code_of((double)y[v][i] * (double)weight(v, i), row.top, row.inv);
    if (k < A.K) put8(A, m, k, n, row.s);
  }
}

// Rows longer than registers hold: two passes, the second over y (or x) as the
// first left it, in fp64 whatever the types.
constexpr int kLongWaves = 16;
__global__ __launch_bounds__(64 * kLongWaves) void norm_long_kernel(const NormArgs A) {
  __shared__ __align__(16) unsigned char room[kLongWaves * 16];
  const int64_t m = A.m0 + blockIdx.x;
  const int t = threadIdx.x;
  const char *x = (const char *)A.x + m * stride_of(A.x32, A.K);
  const char *r = (const char *)A.r + m * stride_of(A.r32, A.K);
  char *y = (char *)A.y + m * stride_of(A.r32, A.K);
  double sum = 0.0;
  uint64_t bits = 0;
  for (int k = 8 * t; k < A.K; k += 8 * 64 * kLongWaves) {
    const Raw8 xr = load8(x, A.x32, k, A.K);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value8(xr, A.x32, i);
    if (A.r) {
      const Raw8 rr = load8(r, A.r32, k, A.K);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] += value8(rr, A.r32, i);
        if (!A.r32) v[i] = bf16_to_f32(f32_to_bf16(v[i]));
      }
      store8(y, A.r32, k, A.K, v);
    }
    Raw8 wr{};
    if (A.w) wr = load8(A.w, A.w32, k, A.K);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = v[i];
      sum = fma(d, d, sum);
      const uint64_t b = magnitude(A.w ? d * (double)value8(wr, A.w32, i) : d);
      bits = b > bits ? b : bits;
    }
  }
  join_waves<kLongWaves>(sum, bits, room);
  const Row row = row_wide(sum, bits, A.K, A.eps);
  if (t == 0) put_row(A, m, row);
  const bool from32 = A.r ? A.r32 : A.x32;
  const char *from = A.r ? y : x;  // each thread's own stores
  for (int k = 8 * t; k < A.K; k += 8 * 64 * kLongWaves) {
    const Raw8 yr = load8(from, from32, k, A.K);
    Raw8 wr{};
    if (A.w) wr = load8(A.w, A.w32, k, A.K);
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = value8(yr, from32, i);
      n[i] = row.bad ? 0 : code_of(A.w ? d * (double)value8(wr, A.w32, i) : d, row.top, row.inv);
    }
    put8(A, m, k, n, row.s);
  }
}

template <int V, int W>
void launch_norm(const NormArgs &A, bool narrow, int64_t rows, hipStream_t stream) {
  const unsigned blocks = (unsigned)(W == 1 ? ceil_div(rows, 4) : rows), threads = W == 1 ? 256 : 64 * W;
  if (narrow)
    norm_kernel<V, W, true><<<blocks, threads, 0, stream>>>(A);
  else
    norm_kernel<V, W, false><<<blocks, threads, 0, stream>>>(A);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

struct BackArgs {
  const uint16_t *dh;
  const void *y, *w, *dy;    // w, dy may be null
  bool y32, w32;             // dy and dx are of y's type
  const float *rstd;
  int64_t M;
  int K;
  void *dx;
  float *partial;            // [parts][K], null where no dw is wanted or blocks of columns make it
  float *mean;               // long rows: [M]
  int row_blocks;            // those behind them: blocks of columns
  void *dw;                  // theirs
};

constexpr int kBackWaves = 16;
constexpr int kBackParts = 256;     // most partial sums of dw a column
constexpr int kRegisterK = 16384;   // longest row that registers hold

constexpr int kBackColumns = 64;  // of a block of them

// dw of 64 columns over all rows: eight threads a row, eight columns each, 128 rows
// at a time; the threads of a wave, then the waves are added in order.
__device__ __forceinline__ void back_columns(const BackArgs &A, int block, float (&sums)[kBackWaves][kBackColumns]) {
  const int c = threadIdx.x & 7, wave = threadIdx.x >> 6, k = block * kBackColumns + 8 * c;
  float dw[8] = {};
  for (int64_t m = threadIdx.x >> 3; m < A.M && k < A.K; m += 8 * kBackWaves) {
    const Raw8 hr = load8(A.dh + m * A.K, false, k, A.K);
    const Raw8 yr = load8((const char *)A.y + m * stride_of(A.y32, A.K), A.y32, k, A.K);
    const float rstd = A.rstd[m];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = fmaf(value8(hr, false, i), value8(yr, A.y32, i) * rstd, dw[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = 8; o < 64; o <<= 1) dw[i] += __shfl_xor(dw[i], o);
    if ((threadIdx.x & 56) == 0) sums[wave][8 * c + i] = dw[i];
  }
  __syncthreads();
  const int n = block * kBackColumns + (int)threadIdx.x;
  if (threadIdx.x >= kBackColumns || n >= A.K) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kBackWaves; ++i) sum += sums[i][threadIdx.x];
  if (A.w32)
    ((float *)A.dw)[n] = sum;
  else
    ((uint16_t *)A.dw)[n] = f32_to_bf16(sum);
}

// A block: G rows at a time (kBackWaves waves, W a row), rows strided over the
// blocks; a thread keeps its columns' share of dw over all its rows, and the
// block's G groups add theirs in order.  4096 rows of 4096 bf16: 29.9 us, 4.5 TB/s
// (copy 5.2; a row loaded ahead, 30.7), and norm_back_sum_kernel 4.2.  At few rows
// (by_columns) blocks behind those of rows make dw: 333 rows of 3584 with fp32 5.5,
// latency.  Rows that are read twice (below): 1100 of 8193 in fp32 49.2 us a call, of
// 8192 33.2 (24.5 at a large copy's rate); 1024 of 14336 59.2 of 39.8.
template <int V, int W, bool NARROW>
__global__ __launch_bounds__(64 * kBackWaves) void norm_back_kernel(const BackArgs A) {
  constexpr int T = 64 * W, G = kBackWaves / W;
  __shared__ float dots[2][kBackWaves];
  __shared__ float sums[kBackWaves][kBackColumns];
  extern __shared__ float total[];  // [K], for dw where G > 1
  if ((int)blockIdx.x >= A.row_blocks) return back_columns(A, (int)blockIdx.x - A.row_blocks, sums);
  const int g = threadIdx.x / T, t = threadIdx.x % T, wave = threadIdx.x >> 6;
  const bool y32 = !NARROW && A.y32, w32 = !NARROW && A.w32;
  // The weight and a row stay in registers, but where there is no room for them
  // (two eights of fp32 a thread): then both are read again behind the mean.
  // (Without room the compiler moved a lane's values over the masked stores below
  // and put one back where no lane was on: wrong from a block's second row on.)
  constexpr bool kHold = NARROW || V == 1;
  auto weight = [&](int v) { return A.w ? load8(A.w, w32, 8 * (v * T + t), A.K) : Raw8{}; };
  Raw8 wr[V];
  if (kHold)
#pragma unroll
    for (int v = 0; v < V; ++v) wr[v] = weight(v);
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  const int64_t step = (int64_t)A.row_blocks * G;
  int turn = 0;
  // every group takes as many turns: the barrier below is the block's
  for (int64_t m0 = (int64_t)blockIdx.x * G; m0 < A.M; m0 += step, turn ^= 1) {
    const int64_t m = m0 + g;
    const bool in = m < A.M;
    const int64_t ms = in ? m : A.M - 1;
    const char *const dh = (const char *)(A.dh + ms * A.K);
    const char *const y = (const char *)A.y + ms * stride_of(y32, A.K);
    Raw8 hr[V], yr[V], dr[V];
    auto addend = [&](int v) { return load8((const char *)A.dy + ms * stride_of(y32, A.K), y32, 8 * (v * T + t), A.K); };
    if (kHold) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hr[v] = load8(dh, false, 8 * (v * T + t), A.K);
        yr[v] = load8(y, y32, 8 * (v * T + t), A.K);
      }
      if (A.dy)
#pragma unroll
        for (int v = 0; v < V; ++v) dr[v] = addend(v);
    }
    const float rstd = A.rstd[ms];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = 8 * (v * T + t);
      const Raw8 h = kHold ? hr[v] : load8(dh, false, k, A.K), yv = kHold ? yr[v] : load8(y, y32, k, A.K);
      const Raw8 wv = kHold ? wr[v] : weight(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = value8(h, false, i);
        dot = fmaf(A.w ? d * value8(wv, w32, i) : d, value8(yv, y32, i) * rstd, dot);
      }
    }
    dot = wave_add(dot);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) dots[turn][wave] = dot;
      __syncthreads();  // the other half is read by waves that are a turn behind, at most
      dot = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) dot += dots[turn][g * W + i];
    }
    const float mean = dot / (float)A.K;
    if (!in) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = 8 * (v * T + t);
      const Raw8 h = kHold ? hr[v] : load8(dh, false, k, A.K), yv = kHold ? yr[v] : load8(y, y32, k, A.K);
      const Raw8 wv = kHold ? wr[v] : weight(v);
      if (!kHold && A.dy) dr[v] = addend(v);
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = value8(h, false, i), n = value8(yv, y32, i) * rstd;
        dw[v][i] = fmaf(d, n, dw[v][i]);
        dx[i] = rstd * fmaf(-n, mean, A.w ? d * value8(wv, w32, i) : d);
        if (A.dy) dx[i] += value8(dr[v], y32, i);
      }
      if (k < A.K) store8((char *)A.dx + m * stride_of(y32, A.K), y32, k, A.K, dx);
    }
  }
  if (!A.partial) return;
  if constexpr (G == 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = 8 * (v * T + t);
      if (k < A.K) store8(A.partial + (int64_t)blockIdx.x * A.K, true, k, A.K, dw[v]);
    }
    return;
  }
  for (int turn = 0; turn < G; ++turn) {
    if (g == turn)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = 8 * (v * T + t) + i;
          if (k < A.K) total[k] = (turn ? total[k] : 0.f) + dw[v][i];
        }
    __syncthreads();
  }
  for (int k = threadIdx.x; k < A.K; k += 64 * kBackWaves) A.partial[(int64_t)blockIdx.x * A.K + k] = total[k];
}

// Longer rows: mean_k(dh w n) of each row first, then columns by blocks.
__global__ __launch_bounds__(64 * kBackWaves) void norm_back_mean_kernel(const BackArgs A) {
  __shared__ float dots[2][kBackWaves];
  int turn = 0;
  for (int64_t m = blockIdx.x; m < A.M; m += gridDim.x, turn ^= 1) {
    const float rstd = A.rstd[m];
    float dot = 0.f;
    for (int k = 8 * threadIdx.x; k < A.K; k += 8 * 64 * kBackWaves) {
      const Raw8 hr = load8(A.dh + m * A.K, false, k, A.K);
      const Raw8 yr = load8((const char *)A.y + m * stride_of(A.y32, A.K), A.y32, k, A.K);
      Raw8 wr{};
      if (A.w) wr = load8(A.w, A.w32, k, A.K);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = value8(hr, false, i);
        dot = fmaf(A.w ? d * value8(wr, A.w32, i) : d, value8(yr, A.y32, i) * rstd, dot);
      }
    }
    dot = wave_add(dot);
    if ((threadIdx.x & 63) == 0) dots[turn][threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.f;
      for (int i = 0; i < kBackWaves; ++i) sum += dots[turn][i];
      A.mean[m] = sum / (float)A.K;
    }
  }
}
constexpr int kColumns = 2048;  // of a block, eight a thread
__global__ __launch_bounds__(kColumns / 8) void norm_back_columns_kernel(const BackArgs A, int parts) {
  const int k = (int)blockIdx.x * kColumns + 8 * threadIdx.x, part = (int)blockIdx.y;
  if (k >= A.K) return;
  Raw8 wr{};
  if (A.w) wr = load8(A.w, A.w32, k, A.K);
  float dw[8] = {};
  for (int64_t m = part; m < A.M; m += parts) {
    const Raw8 hr = load8(A.dh + m * A.K, false, k, A.K);
    const Raw8 yr = load8((const char *)A.y + m * stride_of(A.y32, A.K), A.y32, k, A.K);
    Raw8 dr{};
    if (A.dy) dr = load8((const char *)A.dy + m * stride_of(A.y32, A.K), A.y32, k, A.K);
    const float rstd = A.rstd[m], mean = A.mean[m];
    float dx[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = value8(hr, false, i), n = value8(yr, A.y32, i) * rstd;
      dw[i] = fmaf(d, n, dw[i]);
      dx[i] = rstd * fmaf(-n, mean, A.w ? d * value8(wr, A.w32, i) : d);
      if (A.dy) dx[i] += value8(dr, A.y32, i);
    }
    store8((char *)A.dx + m * stride_of(A.y32, A.K), A.y32, k, A.K, dx);
  }
  if (A.partial) store8(A.partial + (int64_t)part * A.K, true, k, A.K, dw);
}

constexpr int kShare = kBackParts / 32;

// dw[k]: the blocks' sums, in order within each of 32 shares, then the shares'.
__global__ __launch_bounds__(1024) void norm_back_sum_kernel(const float *partial, int parts, int K, void *dw,
                                                            bool w32) {
  __shared__ float sums[32][33];
  const int c = threadIdx.x & 31, p0 = threadIdx.x >> 5, k = (int)blockIdx.x * 32 + c;
  float sum = 0.f;
  for (int p = p0; p < parts; p += 32 * kShare) {  // their loads together: the kernel is their latency
    float v[kShare];
#pragma unroll
    for (int i = 0; i < kShare; ++i) v[i] = k < K && p + 32 * i < parts ? partial[(int64_t)(p + 32 * i) * K + k] : 0.f;
#pragma unroll
    for (int i = 0; i < kShare; ++i) sum += v[i];
  }
  sums[p0][c] = sum;
  __syncthreads();
  if (p0 || k >= K) return;
  sum = 0.f;
  for (int p = 0; p < 32; ++p) sum += sums[p][c];
  if (w32)
    ((float *)dw)[k] = sum;
  else
    ((uint16_t *)dw)[k] = f32_to_bf16(sum);
}

// Waves of a row: eight elements a thread, sixteen in rows beyond 8192.
int waves_of_row(int K) { return K <= 512 ? 1 : K <= 1024 ? 2 : K <= 2048 ? 4 : K <= 4096 ? 8 : 16; }

int back_parts(int64_t M, int K) {
  if (K > kRegisterK) return (int)std::min<int64_t>(64, M);
  return (int)std::min<int64_t>(kBackParts, ceil_div(M, kBackWaves / waves_of_row(K)));
}

// Whether blocks of columns make dw beside the blocks of rows, reading dh and y
// again, in place of partial sums that a second launch adds.  On the device, us,
// so and with partial sums: 333 rows of 3584 5.5 and 9.3, 700 10.8 and 12.5, 1500
// 20.6 and 17.2; 700 rows of 14336 20.5 and 24.1, 1500 39 and 35; 1500 rows of 1024
// 7.6 and 10.7, 3000 16.2 and 12.8; a row of 4096 3.3 and 6.9.
bool by_columns(int64_t M, int64_t K) {
  return K <= kRegisterK && (M <= 1024 || (M <= 2048 && M * K <= 1 << 21));
}

template <int V, int W>
void launch_back(const BackArgs &A, bool narrow, int parts, hipStream_t stream) {
  parts += A.dw ? (int)ceil_div(A.K, kBackColumns) : 0;
  const size_t lds = A.partial && W < kBackWaves ? (size_t)A.K * 4 : 0;  // 16 KB at most
  if (narrow)
    norm_back_kernel<V, W, true><<<parts, 64 * kBackWaves, lds, stream>>>(A);
  else
    norm_back_kernel<V, W, false><<<parts, 64 * kBackWaves, lds, stream>>>(A);
}

}  // namespace

void launch_rms_norm(const void *x, bool x32, const void *r, bool r32, const void *w, bool w32, int64_t M,
                     int64_t K, double eps, int8_t *q, float *scales, uint16_t *h, void *y, float *rstd,
                     int32_t *status, hipStream_t stream) {
  NormArgs A{x, r, w, x32, r32, w32, M, 0, (int)K, eps, y, q, scales, h, rstd, status};
  const bool narrow = !x32 && !(r && r32) && !(w && w32);
  constexpr int64_t kRows = 1 << 20;  // of a launch: blocks times threads stay below 2^32
  for (; A.m0 < M; A.m0 += kRows) {
    const int64_t rows = std::min(kRows, M - A.m0);
    if (K <= 512)
      launch_norm<1, 1>(A, narrow, rows, stream);
    else if (K <= 1024)
      launch_norm<2, 1>(A, narrow, rows, stream);
    else if (K <= 2048)
      launch_norm<1, 4>(A, narrow, rows, stream);
    else if (K <= 4096)
      launch_norm<2, 4>(A, narrow, rows, stream);
    else if (K <= 8192)
      launch_norm<1, 16>(A, narrow, rows, stream);
    else if (K <= kRegisterK)
      launch_norm<2, 16>(A, narrow, rows, stream);
    else
      norm_long_kernel<<<(unsigned)rows, 64 * kLongWaves, 0, stream>>>(A);
  }
}

int64_t rms_norm_backward_workspace(int64_t M, int64_t K) {
  if (by_columns(M, K)) return 0;
  const int64_t sums = (int64_t)back_parts(M, (int)K) * K * 4;
  return (sums + (K > kRegisterK ? M * 4 : 0) + 15) / 16 * 16;
}

void launch_rms_norm_backward(const uint16_t *dh, const void *y, bool y32, const float *rstd, const void *w,
                              bool w32, const void *dy, int64_t M, int64_t K, void *dx, void *dw,
                              void *workspace, hipStream_t stream) {
  const int parts = M > 0 ? back_parts(M, (int)K) : 0;
  const bool columns = M > 0 && by_columns(M, K);
  const BackArgs A{dh, y, w, dy, y32, w32, rstd, M, (int)K, dx, dw && !columns ? (float *)workspace : nullptr,
                   (float *)workspace + (int64_t)parts * K, parts, columns ? dw : nullptr};
  const bool narrow = !y32 && !(w && w32);
  if (M > 0) {
    if (K <= 512)
      launch_back<1, 1>(A, narrow, parts, stream);
    else if (K <= 1024)
      launch_back<1, 2>(A, narrow, parts, stream);
    else if (K <= 2048)
      launch_back<1, 4>(A, narrow, parts, stream);
    else if (K <= 4096)
      launch_back<1, 8>(A, narrow, parts, stream);
    else if (K <= 8192)
      launch_back<1, 16>(A, narrow, parts, stream);
    else if (K <= kRegisterK)
      launch_back<2, 16>(A, narrow, parts, stream);
    else {
      norm_back_mean_kernel<<<(unsigned)std::min<int64_t>(M, 1 << 16), 64 * kBackWaves, 0, stream>>>(A);
      norm_back_columns_kernel<<<dim3((unsigned)ceil_div(K, kColumns), (unsigned)parts), kColumns / 8, 0,
                                 stream>>>(A, parts);
    }
  }
  if (dw && !columns) norm_back_sum_kernel<<<(unsigned)ceil_div(K, 32), 1024, 0, stream>>>((const float *)workspace, parts,
                                                                              (int)K, dw, w32);
}

}  // namespace tq

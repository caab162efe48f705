// The paged 4-bit cache: its layout and the device helpers shared by its kernels.
//
// A vector x (one head of one token, key or value) is held as d codes of 4 bits
// and one pair (s, m): x^ = m + s c. m is min(x) rounded down and s is
// (max(x) - m) / 15 rounded up to bf16, so every coordinate lies in [m, m + 15 s]
// and the nearest code is off by at most s / 2; c = (x - m) / s rounded to
// nearest, ties to even. bf16 rather than fp16 pairs: their range is float's, so
// that only a vector whose own range is no finite float has no pair (it reads as
// NaN), and what their 8 bits round away is taken up by the codes, which are formed
// against the rounded pair.
//
// Sixteen tokens of one KV head are one block of 16 d + 128 contiguous bytes (a
// multiple of 128): key code rows, value code rows, key pairs, value pairs. One
// bulk copy brings a block, or a run of them, into shared memory. The 16-byte
// chunks of a code row are permuted by an xor that depends on the row, so that
// the eight 16-byte rows of an ldmatrix fall into eight different bank groups
// without a copy that rearranges them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "../../include/sq.h"

namespace sq {
namespace kv4 {

constexpr int kBlk = 16;   // tokens of a block

__host__ __device__ constexpr int blk_bytes(int d) { return 16 * d + 128; }
__host__ __device__ constexpr int v_codes(int d) { return 8 * d; }     // offsets inside a block
__host__ __device__ constexpr int k_pairs(int d) { return 16 * d; }
__host__ __device__ constexpr int v_pairs(int d) { return 16 * d + 64; }
// Chunk p of row t of a code block holds chunk p ^ swz(t, d).
__host__ __device__ constexpr int swz(int t, int d) { return (t * d / 256) & (d / 32 - 1); }

// The cache as the kernels take it.
struct Pool {
  uint8_t* pages;
  const int32_t* table;
  int64_t n_pages;
  int64_t table_stride;
  int batch, per_row;      // sequences, pages a sequence may hold
  int n_kv, d;
  int page_shift;          // log2 of the page's tokens
  __device__ int64_t cap() const { return (int64_t)per_row << page_shift; }
  // First byte of head h's blocks in a page.
  __device__ uint8_t* head(int page, int h) const {
    return pages + (((int64_t)page * n_kv + h) << (page_shift - 4)) * blk_bytes(d);
  }
};

struct RopeArgs {
  const float* table;      // [n_pos][rot]: cosines of the rot / 2 pairs, then their sines; NULL: no rotation
  int64_t n_pos;
  int rot;                 // rotated coordinates, the first ones of a head
  int inter;               // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements, 16-byte aligned.
template <typename T> struct Vec8 { uint4 u[sizeof(T) / 2]; };
template <typename T> __device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = __ldg((const uint4*)p + i);
  return r;
}
template <typename T> __device__ __forceinline__ void unpack8(const Vec8<T>& r, float* x) {
  const T* e = (const T*)&r;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f<T>(e[i]);
}

// Two values rounded to T.
template <typename T> __device__ __forceinline__ void round2(float* a, float* b) {}
template <> __device__ __forceinline__ void round2<__half>(float* a, float* b) {
  const float2 f = __half22float2(__floats2half2_rn(*a, *b));
  *a = f.x;
  *b = f.y;
}
template <> __device__ __forceinline__ void round2<__nv_bfloat16>(float* a, float* b) {
  const float2 f = __bfloat1622float2(__floats2bfloat162_rn(*a, *b));
  *a = f.x;
  *b = f.y;
}

// Coordinates i0 .. i0+7 (x) of a head rotated by its position: y = a cos - b sin
// of a pair's first element, b cos + a sin of its second, each operation rounded
// to float once (no contraction: what a row of the cache holds must not depend on
// how the compiler fuses), then the sum rounded to T, as a model's own rotation
// in T leaves it. part: the eight coordinates rot / 2 away (not interleaved).
template <typename T>
__device__ __forceinline__ void rotate8(float* x, const float* part, int i0, const RopeArgs& r, int64_t pos) {
  if (i0 >= r.rot) return;
  const int h = r.rot >> 1;
  const float* row = r.table + pos * r.rot;
  if (r.inter) {
    const float4 c = __ldg((const float4*)(row + (i0 >> 1)));
    const float4 s = __ldg((const float4*)(row + h + (i0 >> 1)));
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      x[2 * j] = to_f<T>(from_f<T>(__fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j]))));
      x[2 * j + 1] = to_f<T>(from_f<T>(__fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j]))));
    }
  } else {
    const bool first = i0 < h;
    const float* cp = row + (first ? i0 : i0 - h);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 c = __ldg((const float4*)(cp + 4 * q));
      const float4 s = __ldg((const float4*)(cp + h + 4 * q));
      const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * q + j;
        const float own = __fmul_rn(x[i], cs[j]), other = __fmul_rn(part[i], sn[j]);
        x[i] = to_f<T>(from_f<T>(first ? __fsub_rn(own, other) : __fadd_rn(own, other)));
      }
    }
  }
}

// First element of the partner coordinates of i0 .. i0+7 (i0 itself where there is none).
__device__ __forceinline__ int partner(int i0, const RopeArgs& r) {
  if (i0 >= r.rot || r.inter) return i0;
  const int h = r.rot >> 1;
  return i0 < h ? i0 + h : i0 - h;
}

// float -> bf16 bits, rounded toward -inf, and (for x >= 0) toward +inf.
__device__ __forceinline__ uint32_t bf16_down(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u >> 16) + ((u >> 31) & ((u & 0xffffu) != 0u));
}
__device__ __forceinline__ uint32_t bf16_up(float x) { return (__float_as_uint(x) + 0xffffu) >> 16; }

// Two floats a register pair: one instruction does an operation on both.
typedef unsigned long long f2;                 // two floats
__device__ __forceinline__ f2 f2_of(uint32_t lo, uint32_t hi) { return (f2)lo | ((f2)hi << 32); }
__device__ __forceinline__ f2 f2_of(float lo, float hi) { return f2_of(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float f2_lo(f2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float f2_hi(f2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The power of two at or above x >= 0, within the floats whose reciprocals are normal too.
__device__ __forceinline__ float pow2_up(float x) {
  const uint32_t u = (__float_as_uint(x) + 0x7fffffu) & 0x7f800000u;
  return fminf(fmaxf(__uint_as_float(u), 0x1p-100f), 0x1p127f);
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The pair of a vector from its smallest and largest coordinate (NaN where one of
// them is); NaN for a vector that holds a value that is not finite (or whose range
// is not): the codes are then 0 and every coordinate reads as NaN.
__device__ __forceinline__ void make_pair(float mn, float mx, float* s, float* m, uint32_t* word) {
  const bool finite = fabsf(mn) < INFINITY && fabsf(mx) < INFINITY;
  uint32_t mb = bf16_down(mn);
  const float r = __fsub_rn(mx, __uint_as_float(mb << 16));
  uint32_t sb = 0;
  if (r > 0.0f) {
    // r / 15 as a division rounds it: Markstein's correction of the product with the rounded 1 / 15, which is exact
    // for this divisor (every significand is compared in tests/test_oracle_kv4.py; below FLT_MIN it is not used)
    const float y = 1.0f / 15.0f, q = __fmul_rn(r, y);
    sb = bf16_up(fmaxf(__fmaf_rn(__fmaf_rn(-15.0f, q, r), y, q), FLT_MIN));
  }
  if (!finite || !(r < INFINITY)) {
    mb = 0x7fc0u;
    sb = 0;
  }
  *m = __uint_as_float(mb << 16);
  *s = __uint_as_float(sb << 16);
  *word = sb | (mb << 16);
}

// Eight codes: (x - m) / s rounded to nearest, ties to even, exactly. The product
// with inv, 1 / s within 2^-23, rounded to an integer by an addition to 1.5 2^23, is within 2^-19
// of the quotient: its nearest integer is the quotient's or, beside a tie, the next.
// The remainder against s / 2, which one fused multiply-add gives, tells the two
// apart; few vectors have such a coordinate. s > 0.
__device__ __forceinline__ float reciprocal(float s) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(s));
  return y;
}
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ uint32_t codes8(const float* x, float m, float s, float inv) {
  const f2 m2 = f2_of(-m, -m), i2 = f2_of(inv, inv), r2 = f2_of(kRound, kRound), n2 = f2_of(-kRound, -kRound), s2 = f2_of(-s, -s);
  const float half = 0.5f * s;
  float c[8], rest[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const f2 e = f2_add(f2_of(x[i], x[i + 1]), m2);
    const f2 q = f2_add(f2_fma(e, i2, r2), n2);
    const f2 t = f2_fma(q, s2, e);
    c[i] = f2_lo(q);
    c[i + 1] = f2_hi(q);
    rest[i] = f2_lo(t);
    rest[i + 1] = f2_hi(t);
    near |= fabsf(rest[i]) >= half || fabsf(rest[i + 1]) >= half;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(rest[i]) > half || (fabsf(rest[i]) == half && ((int)c[i] & 1))) c[i] += rest[i] > 0.0f ? 1.0f : -1.0f;
  }
  // four codes are one number of 16 bits, exact in float
  const float lo = fmaf(fmaf(fmaf(c[3], 16.0f, c[2]), 16.0f, c[1]), 16.0f, c[0]) + kRound;
  const float hi = fmaf(fmaf(fmaf(c[7], 16.0f, c[6]), 16.0f, c[5]), 16.0f, c[4]) + kRound;
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

// Sequence of token i among cu[0 .. batch] (cu NULL: one token a sequence), or -1 (also where its offset is below 0).
__device__ __forceinline__ int row_of(const int32_t* cu, int batch, int64_t i, int32_t* off) {
  if (!cu) {
    *off = 0;
    return i < batch ? (int)i : -1;
  }
  int lo = 0, hi = batch;              // the last b with cu[b] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)__ldg(cu + mid) <= i) lo = mid; else hi = mid;
  }
  const int32_t a = __ldg(cu + lo), b = __ldg(cu + lo + 1);
  if (a < 0 || i < a || i >= b) return -1;
  *off = (int32_t)(i - a);
  return lo;
}

__device__ __forceinline__ void raise(uint32_t* flags, uint32_t bit) {
  if (flags) atomicOr(flags, bit);
}

}  // namespace kv4
}  // namespace sq

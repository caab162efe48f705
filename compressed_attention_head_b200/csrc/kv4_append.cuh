// Append to, and read back from, the paged 4-bit cache.
//
// Both are streams: d / 8 threads hold one vector, eight coordinates each, which
// is one 16-byte load of a 16-bit input and one 32-bit word of codes; the minimum
// and maximum go through d / 8 lanes. A key that is rotated by halves is read
// twice by its warp (its own eight coordinates and the partners'; the second read
// hits L1). No vector shares a byte with another, so nothing is read to be
// written back and tokens may come in any order.
#pragma once

#include "kv4.cuh"

namespace sq {
namespace kv4 {

constexpr int kStreamThreads = 256;

struct StreamArgs {
  const int32_t* cu;
  const int32_t* start;
  int64_t n_tok;
  int64_t ks_tok, ks_head, vs_tok, vs_head;   // strides of the caller's keys and values, in elements
  uint32_t* flags;
};

// Where a token's vectors go: the byte of head 0's block in its page (or -1) and its slot and position.
struct Place {
  int64_t at;
  int slot;
  int32_t pos;
};

__device__ __forceinline__ Place place_of(const Pool& c, const StreamArgs& a, int64_t n_pos, int64_t tok) {
  Place p{-1, 0, 0};
  int32_t off = 0;
  const int b = tok < a.n_tok ? row_of(a.cu, c.batch, tok, &off) : -1;
  if (b < 0) return p;
  const int64_t pos = (int64_t)__ldg(a.start + b) + off;
  if (pos < 0 || pos >= c.cap()) {
    raise(a.flags, SQ_FLAG_CAPACITY);
    return p;
  }
  if (n_pos >= 0 && pos >= n_pos) {
    raise(a.flags, SQ_FLAG_ROPE);
    return p;
  }
  const int page = __ldg(c.table + b * c.table_stride + (pos >> c.page_shift));
  if (page < 0 || page >= c.n_pages) {
    raise(a.flags, SQ_FLAG_PAGE);
    return p;
  }
  p.slot = (int)(pos & ((1 << c.page_shift) - 1));
  p.at = (int64_t)page;
  p.pos = (int32_t)pos;
  return p;
}

// kVecs vectors a thread group; the block's vectors are consecutive in
// (token, side, head) order, so a warp reads whole rows of the caller's tensors.
template <typename T, int D, int kVecs>
__global__ void __launch_bounds__(kStreamThreads)
k_append4(Pool c, RopeArgs r, const T* __restrict__ k, const T* __restrict__ v, StreamArgs a) {
  constexpr int TPV = D / 8, VPB = kStreamThreads / TPV, NV = VPB * kVecs;
  __shared__ Place places[NV + 1];
  const int per_tok = 2 * c.n_kv;
  const int64_t v0 = (int64_t)blockIdx.x * NV;
  const int64_t t0 = v0 / per_tok;
  const int n_here = (int)((v0 + NV - 1) / per_tok - t0) + 1;
  for (int i = threadIdx.x; i < n_here; i += kStreamThreads) places[i] = place_of(c, a, r.table ? r.n_pos : -1, t0 + i);
  __syncthreads();
  const int j = threadIdx.x % TPV, i0 = 8 * j;
  Vec8<T> own[kVecs], part[kVecs];
  int64_t dst[kVecs];
  int32_t pos[kVecs];
  int slot[kVecs];
  bool key[kVecs];
  const int pi = partner(i0, r);
#pragma unroll
  for (int n = 0; n < kVecs; ++n) {
    const int64_t vec = v0 + n * VPB + threadIdx.x / TPV;
    const int ti = (int)(vec / per_tok - t0);
    const int rem = (int)(vec - (t0 + ti) * per_tok);
    const Place p = places[ti];
    dst[n] = -1;
    key[n] = rem < c.n_kv;
    if (p.at < 0) continue;
    const int h = key[n] ? rem : rem - c.n_kv;
    const T* x = key[n] ? k + (t0 + ti) * a.ks_tok + h * a.ks_head : v + (t0 + ti) * a.vs_tok + h * a.vs_head;
    own[n] = load8<T>(x + i0);
    if (key[n] && pi != i0) part[n] = load8<T>(x + pi);
    dst[n] = (c.head((int)p.at, h) - c.pages) + (int64_t)(p.slot >> 4) * blk_bytes(D);
    pos[n] = p.pos;
    slot[n] = p.slot & 15;
  }
#pragma unroll
  for (int n = 0; n < kVecs; ++n) {
    // a vector's threads take this branch together; the shuffles name only them
    if (dst[n] < 0) continue;
    float x[8];
    unpack8<T>(own[n], x);
    if (key[n] && r.table) {
      float y[8];
      if (pi != i0) unpack8<T>(part[n], y);
      rotate8<T>(x, y, i0, r, pos[n]);
    }
    float mn = x[0], mx = x[0], bad = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mn = fminf(mn, x[i]);
      mx = fmaxf(mx, x[i]);
      bad = fmaf(x[i], 0.0f, bad);      // NaN as soon as one value is not finite
    }
    bool finite = bad == 0.0f;
    const unsigned lanes = TPV == 32 ? 0xffffffffu : ((1u << TPV) - 1u) << ((threadIdx.x & 31) / TPV * TPV);
#pragma unroll
    for (int o = 1; o < TPV; o <<= 1) {
      mn = fminf(mn, __shfl_xor_sync(lanes, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(lanes, mx, o));
    }
    finite = __all_sync(lanes, finite);
    float s, m;
    uint32_t word, w = 0;
    make_pair(mn, mx, finite, &s, &m, &word);
    const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
    if (s > 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= code4(x[i], m, s, inv) << (4 * i);
    }
    uint8_t* blk = c.pages + dst[n];
    const int t = slot[n], side = key[n] ? 0 : 1;
    *(uint32_t*)(blk + side * v_codes(D) + t * (D / 2) + (((j >> 2) ^ swz(t, D)) << 4) + ((j & 3) << 2)) = w;
    if (j == 0) *(uint32_t*)(blk + k_pairs(D) + side * 64 + t * 4) = word;
  }
}

// x^ = m + s c of the tokens of a call: the product is exact in float (8 + 4
// bits), the sum is rounded once, then to the output's type.
template <typename T, int D>
__global__ void __launch_bounds__(kStreamThreads)
k_read4(Pool c, T* __restrict__ ko, T* __restrict__ vo, StreamArgs a) {
  constexpr int TPV = D / 8, VPB = kStreamThreads / TPV;
  __shared__ Place places[VPB + 1];
  const int per_tok = 2 * c.n_kv;
  const int64_t v0 = (int64_t)blockIdx.x * VPB;
  const int64_t t0 = v0 / per_tok;
  const int n_here = (int)((v0 + VPB - 1) / per_tok - t0) + 1;
  for (int i = threadIdx.x; i < n_here; i += kStreamThreads) places[i] = place_of(c, a, -1, t0 + i);
  __syncthreads();
  const int j = threadIdx.x % TPV;
  const int64_t vec = v0 + threadIdx.x / TPV;
  const int ti = (int)(vec / per_tok - t0);
  const int rem = (int)(vec - (t0 + ti) * per_tok);
  const Place p = places[ti];
  if (p.at < 0) return;
  const int side = rem < c.n_kv ? 0 : 1, h = rem - side * c.n_kv, t = p.slot & 15;
  const uint8_t* blk = c.head((int)p.at, h) + (int64_t)(p.slot >> 4) * blk_bytes(D);
  const uint32_t w = *(const uint32_t*)(blk + side * v_codes(D) + t * (D / 2) + (((j >> 2) ^ swz(t, D)) << 4) + ((j & 3) << 2));
  const uint32_t pw = *(const uint32_t*)(blk + k_pairs(D) + side * 64 + t * 4);
  const float s = __uint_as_float(pw << 16), m = __uint_as_float(pw & 0xffff0000u);
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f<T>(fmaf((float)((w >> (4 * i)) & 15u), s, m));
  T* out = side ? vo + (t0 + ti) * a.vs_tok + h * a.vs_head : ko + (t0 + ti) * a.ks_tok + h * a.ks_head;
  const uint4* u = (const uint4*)e;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((uint4*)(out + 8 * j))[i] = u[i];
}

}  // namespace kv4
}  // namespace sq

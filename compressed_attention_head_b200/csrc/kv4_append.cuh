// Append to, and read back from, the paged 4-bit cache.
//
// Both are streams, bound by memory only when their instructions are few: a thread
// holds sixteen coordinates of a vector, eight of each half of the head (16-byte
// loads of a 16-bit input, one word of codes each). Rotated by halves over the whole
// head, the two are each other's partners under the same angles; any other rotation
// reads its partners from memory again. Minimum and maximum go through d / 16 lanes.
// The vectors of a block belong to whole tokens, whose places are looked up once,
// while the loads are on their way. No vector shares a byte with another, so nothing
// is read to be written back and tokens may come in any order.
//
// Measured (one B200): 32768 tokens of 8 KV heads at head_dim 128, fp16: the append 66
// us (170 MB, 2.6 TB/s), the read 36 us (170 MB, 4.7 TB/s). The instruction slots bound
// both (72 % of them used, 380 and 190 a sixteen coordinates); twice the vectors a
// thread saves a tenth of the instructions and loses more by the warps it costs.
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
  int* zero;                                  // counters that the kernel behind an append wants at 0, or NULL
  int n_zero;
};

// Where a token's vectors go: head 0's block (an offset into the pool, or -1), its row in that, its position.
struct Place {
  int64_t at;
  int row;
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
  p.row = (int)(pos & 15);
  p.at = c.head(page, 0) - c.pages + ((int)(pos & ((1 << c.page_shift) - 1)) >> 4) * blk_bytes(c.d);
  p.pos = (int32_t)pos;
  return p;
}

// How a block divides the vectors of its tokens: `toks` tokens of `heads` vectors
// (keys' heads, then values'), or a part of one token's.
struct Share {
  int toks, heads, parts;
  int next_tok, next_head;     // a thread's next vector is this many tokens and heads on (less `heads` where that is too many)
  __host__ __device__ static Share of(int per_tok, int vecs, int step) {
    Share s;
    s.parts = (per_tok + vecs - 1) / vecs;
    s.toks = s.parts > 1 ? 1 : vecs / per_tok;
    s.heads = s.parts > 1 ? vecs : per_tok;
    s.next_tok = step / s.heads;
    s.next_head = step % s.heads;
    return s;
  }
};
constexpr int kVecs = 2;                      // vectors a thread has in flight
template <int D> __host__ __device__ constexpr int vecs_of_block() { return kStreamThreads / (D / 16) * kVecs; }

// MODE 0: no rotation, 1: halves of the whole head, 2: any.
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kStreamThreads)
k_append4(Pool c, RopeArgs r, const T* __restrict__ k, const T* __restrict__ v, StreamArgs a, Share sh) {
  constexpr int TPV = D / 16, VPB = kStreamThreads / TPV, NV = VPB * kVecs;
  __shared__ Place places[NV];
  const int64_t t0 = (int64_t)blockIdx.x * sh.toks;
  const int j = threadIdx.x % TPV, g = threadIdx.x / TPV;
  Vec8<T> own[kVecs][2], part[MODE == 2 ? kVecs : 1][2];
  int tok[kVecs], head[kVecs];
  const int p0 = partner(8 * j, r), p1 = partner(D / 2 + 8 * j, r);
  const T *k0 = k + t0 * a.ks_tok, *v0 = v + t0 * a.vs_tok;
  const int toks = (int)min((int64_t)sh.toks, a.n_tok - t0), first = (int)blockIdx.y * sh.heads;
  int x_tok = g / sh.heads, x_head = g - x_tok * sh.heads;
#pragma unroll
  for (int n = 0; n < kVecs; ++n) {
    tok[n] = x_tok;
    head[n] = x_head + first;
    x_tok += sh.next_tok;
    x_head += sh.next_head;
    if (x_head >= sh.heads) {
      x_head -= sh.heads;
      ++x_tok;
    }
    if (tok[n] >= toks || head[n] >= 2 * c.n_kv) {
      tok[n] = -1;
      continue;
    }
    const bool key = head[n] < c.n_kv;
    const T* src = key ? k0 + tok[n] * a.ks_tok + head[n] * a.ks_head : v0 + tok[n] * a.vs_tok + (head[n] - c.n_kv) * a.vs_head;
    own[n][0] = load8<T>(src + 8 * j);
    own[n][1] = load8<T>(src + D / 2 + 8 * j);
    if (MODE == 2 && key) {
      part[n][0] = load8<T>(src + p0);
      part[n][1] = load8<T>(src + p1);
    }
  }
  for (int i = threadIdx.x; i < sh.toks; i += kStreamThreads) places[i] = place_of(c, a, MODE ? r.n_pos : -1, t0 + i);
  if (a.zero && blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.n_zero; i += kStreamThreads) a.zero[i] = 0;
  __syncthreads();
  const int head_bytes = blk_bytes(D) << (c.page_shift - 4);
#pragma unroll
  for (int n = 0; n < kVecs; ++n) {
    // a vector's threads take these branches together; the shuffles name only them
    if (tok[n] < 0) continue;
    const Place p = places[tok[n]];
    if (p.at < 0) continue;
    const bool key = head[n] < c.n_kv;
    float x[2][8];
    unpack8<T>(own[n][0], x[0]);
    unpack8<T>(own[n][1], x[1]);
    if (MODE == 1 && key) {
      const float4* row = (const float4*)(r.table + (int64_t)p.pos * D + 8 * j);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 cv = __ldg(row + q), sv = __ldg(row + D / 8 + q);
        const float cs[4] = {cv.x, cv.y, cv.z, cv.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ya = x[0][4 * q + e], yb = x[1][4 * q + e];
          x[0][4 * q + e] = __fsub_rn(__fmul_rn(ya, cs[e]), __fmul_rn(yb, sn[e]));
          x[1][4 * q + e] = __fadd_rn(__fmul_rn(yb, cs[e]), __fmul_rn(ya, sn[e]));
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        round2<T>(&x[0][e], &x[0][e + 1]);
        round2<T>(&x[1][e], &x[1][e + 1]);
      }
    }
    if (MODE == 2 && key) {
      float y[8];
      unpack8<T>(part[n][0], y);
      rotate8<T>(x[0], y, 8 * j, r, p.pos);
      unpack8<T>(part[n][1], y);
      rotate8<T>(x[1], y, D / 2 + 8 * j, r, p.pos);
    }
    float mn = x[0][0], mx = x[0][0];
#pragma unroll
    for (int e = 1; e < 15; e += 2) {
      mn = min_nan(mn, x[e >> 3][e & 7], x[(e + 1) >> 3][(e + 1) & 7]);
      mx = max_nan(mx, x[e >> 3][e & 7], x[(e + 1) >> 3][(e + 1) & 7]);
    }
    mn = min_nan(mn, x[1][7]);
    mx = max_nan(mx, x[1][7]);
    const unsigned lanes = ((1u << TPV) - 1u) << ((threadIdx.x & 31) / TPV * TPV);
#pragma unroll
    for (int o = 1; o < TPV; o <<= 1) {
      mn = min_nan(mn, __shfl_xor_sync(lanes, mn, o));
      mx = max_nan(mx, __shfl_xor_sync(lanes, mx, o));
    }
    float s, m;
    uint32_t word, w[2] = {0u, 0u};
    make_pair(mn, mx, &s, &m, &word);
    if (s > 0.0f) {
      const float inv = reciprocal(s);
      w[0] = codes8(x[0], m, s, inv);
      w[1] = codes8(x[1], m, s, inv);
    }
    const int side = key ? 0 : 1, t = p.row;
    uint8_t* blk = c.pages + p.at + (int64_t)(head[n] - side * c.n_kv) * head_bytes;
    uint8_t* row = blk + side * v_codes(D) + t * (D / 2) + ((j & 3) << 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) *(uint32_t*)(row + ((((j >> 2) + e * (D / 64)) ^ swz(t, D)) << 4)) = w[e];
    if (j == 0) *(uint32_t*)(blk + k_pairs(D) + side * 64 + t * 4) = word;
  }
}

// Eight coordinates of a word: x^ = m + s c, the product exact in float (8 + 4 bits),
// the sum rounded once, then to the output's type. (A code or'ed into 2^23 is 2^23 + c.)
template <typename T> __device__ __forceinline__ void values8(uint32_t w, float s, float m, T* out) {
  const f2 s2 = f2_of(s, s), m2 = f2_of(m, m), b2 = f2_of(-8388608.0f, -8388608.0f);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t a = (w >> (4 * i)) & 15u | 0x4b000000u, b = (w >> (4 * i + 4)) & 15u | 0x4b000000u;
    const f2 z = f2_fma(f2_add(f2_of(a, b), b2), s2, m2);
    y[i] = f2_lo(z);
    y[i + 1] = f2_hi(z);
  }
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f<T>(y[i]);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((uint4*)out)[i] = ((const uint4*)e)[i];
}

template <typename T, int D>
__global__ void __launch_bounds__(kStreamThreads)
k_read4(Pool c, T* __restrict__ ko, T* __restrict__ vo, StreamArgs a, Share sh) {
  constexpr int TPV = D / 16, VPB = kStreamThreads / TPV, NV = VPB * kVecs;
  __shared__ Place places[NV];
  const int64_t t0 = (int64_t)blockIdx.x * sh.toks;
  for (int i = threadIdx.x; i < sh.toks; i += kStreamThreads) places[i] = place_of(c, a, -1, t0 + i);
  __syncthreads();
  const int j = threadIdx.x % TPV, g = threadIdx.x / TPV;
  T *k0 = ko + t0 * a.ks_tok, *v0 = vo + t0 * a.vs_tok;
  uint32_t w[kVecs][2], pair[kVecs];
  int tok[kVecs], head[kVecs];
  const int head_bytes = blk_bytes(D) << (c.page_shift - 4), first = (int)blockIdx.y * sh.heads;
  int x_tok = g / sh.heads, x_head = g - x_tok * sh.heads;
#pragma unroll
  for (int n = 0; n < kVecs; ++n) {
    tok[n] = x_tok;
    head[n] = x_head + first;
    x_tok += sh.next_tok;
    x_head += sh.next_head;
    if (x_head >= sh.heads) {
      x_head -= sh.heads;
      ++x_tok;
    }
    if (tok[n] >= sh.toks || head[n] >= 2 * c.n_kv) tok[n] = -1;
    if (tok[n] < 0) continue;
    const Place p = places[tok[n]];
    if (p.at < 0) {
      tok[n] = -1;
      continue;
    }
    const int side = head[n] < c.n_kv ? 0 : 1, t = p.row;
    const uint8_t* blk = c.pages + p.at + (int64_t)(head[n] - side * c.n_kv) * head_bytes;
    const uint8_t* row = blk + side * v_codes(D) + t * (D / 2) + ((j & 3) << 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) w[n][e] = *(const uint32_t*)(row + ((((j >> 2) + e * (D / 64)) ^ swz(t, D)) << 4));
    pair[n] = *(const uint32_t*)(blk + k_pairs(D) + side * 64 + t * 4);
  }
#pragma unroll
  for (int n = 0; n < kVecs; ++n) {
    if (tok[n] < 0) continue;
    const float s = __uint_as_float(pair[n] << 16), m = __uint_as_float(pair[n] & 0xffff0000u);
    T* out = (head[n] < c.n_kv ? k0 + head[n] * a.ks_head + tok[n] * a.ks_tok
                               : v0 + (head[n] - c.n_kv) * a.vs_head + tok[n] * a.vs_tok) + 8 * j;
    values8<T>(w[n][0], s, m, out);
    values8<T>(w[n][1], s, m, out + D / 2);
  }
}

}  // namespace kv4
}  // namespace sq

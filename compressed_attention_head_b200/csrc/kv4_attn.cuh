// Attention of chunks of queries over the paged 4-bit cache: one block a (query
// token, query head), tiles of 128 keys; a thread forms one key's score, then one
// coordinate's sum over the tile. Online softmax in base 2, everything in float.
#pragma once

#include "kv4_decode.cuh"

namespace sq {
namespace kv4 {

constexpr int kPlainTile = 128;

template <typename T, typename TO, int D>
__global__ void __launch_bounds__(kPlainTile)
k_attn4_plain(Pool c, RopeArgs r, const T* __restrict__ q, TO* __restrict__ out, AttnArgs a) {
  __shared__ float qs[D], p[kPlainTile], ms[kPlainTile], ss[kPlainTile];
  __shared__ float red[4];
  __shared__ const uint8_t* vrow[kPlainTile];
  const int64_t tok = blockIdx.x;
  const int h = blockIdx.y, tid = threadIdx.x;
  int32_t off = 0;
  const int b = row_of(a.cu, c.batch, tok, &off);
  if (b < 0) return;
  TO* o = out + (tok * a.n_q + h) * D;
  int64_t pos = (int64_t)a.start[b] + a.len_off + off;
  if (pos >= c.cap() || pos >= a.max_ctx) {
    if (tid == 0) raise(a.flags, SQ_FLAG_SEQLEN);
    pos = min(c.cap(), a.max_ctx) - 1;
  }
  if (pos < -1 && tid == 0) raise(a.flags, SQ_FLAG_SEQLEN);
  const bool no_rope = r.table && pos >= r.n_pos;
  if (no_rope && tid == 0) raise(a.flags, SQ_FLAG_ROPE);
  if (pos < 0 || no_rope) {
    for (int i = tid; i < D; i += kPlainTile) o[i] = from_f<TO>(0.0f);
    if (a.lse && tid == 0) a.lse[tok * a.n_q + h] = -INFINITY;
    return;
  }
  if (tid < D / 8) {
    const T* x = q + tok * a.qs_tok + h * a.qs_head;
    float e[8], y[8];
    unpack8<T>(load8<T>(x + 8 * tid), e);
    if (r.table) {
      const int pi = partner(8 * tid, r);
      if (pi != 8 * tid) unpack8<T>(load8<T>(x + pi), y);
      rotate8<T>(e, y, 8 * tid, r, pos);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) qs[8 * tid + i] = e[i];
  }
  __syncthreads();
  const int64_t lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  float acc[2] = {0.0f, 0.0f}, top = -INFINITY, sum = 0.0f;
  const float f = a.scale * 1.4426950408889634f;
  for (int64_t t0 = lo; t0 <= pos; t0 += kPlainTile) {
    const int64_t t = t0 + tid;
    float sc = -INFINITY;
    const uint8_t* vr = nullptr;
    if (t <= pos) {
      const int page = c.table[b * c.table_stride + (t >> c.page_shift)];
      if (page >= 0 && page < c.n_pages) {
        const int slot = (int)(t & ((1 << c.page_shift) - 1)), tt = slot & 15;
        const uint8_t* blk = c.head(page, h / a.group) + (int64_t)(slot >> 4) * blk_bytes(D);
        float dot = 0.0f, qsum = 0.0f;
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t w = *(const uint32_t*)(blk + tt * (D / 2) + (((j >> 2) ^ swz(tt, D)) << 4) + ((j & 3) << 2));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot = fmaf((float)((w >> (4 * i)) & 15u), qs[8 * j + i], dot);
            qsum += qs[8 * j + i];
          }
        }
        const uint32_t kw = *(const uint32_t*)(blk + k_pairs(D) + tt * 4);
        const uint32_t vw = *(const uint32_t*)(blk + v_pairs(D) + tt * 4);
        sc = f * (__uint_as_float(kw << 16) * dot + __uint_as_float(kw & 0xffff0000u) * qsum);
        ss[tid] = __uint_as_float(vw << 16);
        ms[tid] = __uint_as_float(vw & 0xffff0000u);
        vr = blk + v_codes(D) + tt * (D / 2);
      } else {
        raise(a.flags, SQ_FLAG_PAGE);
      }
    }
    vrow[tid] = vr;
    float mx = sc;
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float nt = fmaxf(top, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = nt == -INFINITY ? 0.0f : nt;
    const float keep = exp2f(top - base);
    p[tid] = exp2f(sc - base);
    __syncthreads();
    sum *= keep;
    acc[0] *= keep;
    acc[1] *= keep;
    const int n = (int)min((int64_t)kPlainTile, pos - t0 + 1);
    for (int i = 0; i < n; ++i) {
      if (!vrow[i]) continue;
      const int tt = (int)((t0 + i) & 15);
      sum += p[i];
#pragma unroll
      for (int e = 0; e < (D + kPlainTile - 1) / kPlainTile; ++e) {
        const int x = tid + e * kPlainTile;
        if (x < D) {
          const uint8_t byte = vrow[i][(((x >> 5) ^ swz(tt, D)) << 4) + ((x & 31) >> 1)];
          const float code = (float)((x & 1) ? byte >> 4 : byte & 15);
          acc[e] += p[i] * fmaf(code, ss[i], ms[i]);
        }
      }
    }
    top = nt;
    __syncthreads();
  }
  const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
  for (int e = 0; e < (D + kPlainTile - 1) / kPlainTile; ++e)
    if (tid + e * kPlainTile < D) o[tid + e * kPlainTile] = from_f<TO>(acc[e] * inv);
  if (a.lse && tid == 0)
    a.lse[tok * a.n_q + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace kv4
}  // namespace sq

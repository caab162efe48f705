// Causal attention of chunks of queries over the paged 4-bit cache (tcgen05).
//
// Mathematics. A key is x^ = m + s c = (m + 8 s) + s (c - 8). s has 8 significant
// bits and c - 8 three, or is a power of two, so s (c - 8) is an fp16 number exactly
// once a power of two a tile puts s in range: the tile is unpacked into fp16 without
// a rounding. The rest, sum(q) (m + 8 s), is one more step of 16 along the product's
// k: three fp16 parts of sum(q) against m and against 8 s, both exact. A score is
// therefore what the cache holds, to float's roundings. For the values s (c - 8) is
// unpacked in the same way against the rounded probabilities, and sum p (m + 8 s) is
// kept in float beside the running sum: only the part that varies within a vector
// meets a rounded probability. For an fp16 or float output that is two fp16 parts, 21
// bits, and a second product of the same values; one part left fp16 outputs 1.3 times
// as far from the exact ones as their own rounding does. For a bf16 output, eight times
// coarser, it is one part of 11 bits.
//
// Split. A block takes one KV head, 128 / group tokens with their query heads as the
// rows of one accumulator (two of them up to head_dim 128) and 128 keys at a time.
// Eight warps a row tile hold the softmax, half a row a thread; eight unpack keys and
// values, 16 keys each; one issues the products. Scores and probabilities share tensor
// memory, probabilities are the A operand from there. With two row tiles one's
// softmax runs beside the other's products; with one (short chunks, head_dim 256)
// the scores of the next keys are formed meanwhile.
//
// The maximum a row refers to is raised, and its sums scaled, only when a score
// passes it by 2^4. Pieces: a small kernel first lists the units, longest first, and
// cuts those that would outlast an even share of all the work; the pieces of a cut one
// leave partial sums, and the piece that ends last joins them in their order.
//
// Measured (one B200): a causal prompt of 2048 tokens, 32 query heads, 8 KV heads,
// head_dim 128, fp16: 82 us, 422 TFLOP/s (72 with one part); 512 tokens of two
// sequences behind 12001 and 16385 others, 12 heads on 2, bf16: 165 us, 551 TFLOP/s.
// With one part 128 keys against two row tiles take about 5000 cycles where the
// products alone are 2176 and the exponentials 2048: a row tile's softmax (2500), the
// end of its sum and its next scores (2000) follow one another, and the other tile's
// fall beside them. The unpacked keys and values, the products' reads of them and the
// offsets' use 3200 of those cycles of shared memory. Two issuing warps that do not
// take turns were slower (190 us for the chunks: both softmaxes at once). Not to wait
// for the end of a sum before the next scores take its operand's place would save about
// a tenth; nothing orders the two products, so it is waited for.
#pragma once

#include "kv4_decode.cuh"

namespace sq {
namespace kv4 {
namespace pre {

constexpr int KT = 128;                       // keys of a tile
constexpr int M = 128;                        // rows of an accumulator
constexpr int kGroup = 128;                   // threads of a warp group
constexpr int kInfo = 4;                      // tiles whose factors are kept
constexpr float kSlack = 4.0f;                // log2 of what a probability may exceed 1 by
constexpr float kUp = 11.0f;                  // log2 of the probabilities' scale: 2^15 at most with the slack

// Thirty-two rows of 32 elements in shared memory, an odd number of 16-byte words apart: no two lanes meet in a bank.
template <typename E> __host__ __device__ constexpr int box_pitch() { return 32 * (int)sizeof(E) + 16; }
constexpr int kBox = 32 * box_pitch<float>();

template <int D> struct Cfg {
  static constexpr int NS = D == 256 ? 1 : 2;          // row tiles of a block
  // Warp groups: two softmax a row tile (each half of the keys: one warp a scheduler would wait for its own
  // latencies), two that unpack, one that issues.
  static constexpr int SOFT = 2 * NS, THREADS = (SOFT + 3) * kGroup;
  // Registers a thread: 896 x 72 or 640 x 96 in all, the softmax's from what the issuers give up.
  static constexpr int R_SOFT = NS == 2 ? 88 : 112, R_UNPACK = NS == 2 ? 56 : 104, R_MMA = NS == 2 ? 40 : 48;
  static constexpr int NKV = D == 256 ? 1 : 2;         // stages of unpacked keys and values
  static constexpr int MAIN = (D / 64) * 16384;        // 128 rows x D fp16, 64 coordinates a slab
  static constexpr int OP = MAIN + 4096;               // and the step that carries the offsets
  static constexpr int QIMG = OP + M * 4;              // an operand as it lies in memory: rows, and their score factors
  static constexpr int Q = 0;
  static constexpr int K = Q + NS * OP;
  static constexpr int V = K + NKV * OP;
  static constexpr int MEAN = V + NKV * MAIN;
  static constexpr int USED = MEAN + kInfo * KT * 4;
  // Boxes of the eight warps that write a row tile out: over its queries, where they fit.
  static constexpr int BOX = OP >= 8 * kBox ? Q : USED, BOX_STEP = OP >= 8 * kBox ? OP : 8 * kBox;
  static constexpr int ALL = BOX == Q ? USED : USED + NS * BOX_STEP;
  static constexpr int TOTAL = (ALL > 118784 ? ALL : 118784) + 1024;   // one block an SM: it takes all tensor memory
};

// One piece of work.
struct Unit {
  int64_t pos;         // position of the first token
  int row, hs;         // sequence, KV head x pass
  int tok, n;          // first token of the call, tokens
  int off;             // of the first token in its sequence
  int t0, nt;          // key tiles
  int slot;            // of the first piece's partial sums, -1: the whole of it
  int part, parts;     // which piece of how many
};
struct Head { int units, pad[3]; };

struct Shape {
  int gt, nsub, tpm, tpu;      // heads of a pass, passes, tokens of a row tile, of a unit
  int cap_units, cap_slots, sms;
  int64_t q_tiles;
};

struct Plan {
  Head* head;
  Unit* units;
  int* done;                   // pieces of a cut unit that are written, at its first slot
  float* parts;
  uint8_t* q;                  // query operands, [n_kv x nsub][row tiles] of Cfg::QIMG bytes
  int64_t q_tiles;             // row tiles a head
};

// Row tile of the token at `off` in a sequence whose first token is `tok`: every
// sequence starts a tile of its own, no two share one, and all are below n_tok / tpm + batch.
__device__ __forceinline__ int64_t row_tile(int64_t tok, int row, int off, int tpm) { return tok / tpm + row + off / tpm; }

__host__ __device__ inline size_t part_rows(int ns) { return (size_t)ns * M; }

// First and last key of a unit's tokens, empty when hi < lo.
__device__ __forceinline__ void unit_keys(const Pool& c, const RopeArgs& r, const AttnArgs& a, int64_t pos, int n,
                                          int64_t* lo, int64_t* hi) {
  const int64_t cap = c.cap();
  const int64_t first = min(pos, cap - 1);
  int64_t last = min(pos + n - 1, cap - 1);
  if (r.table) last = min(last, r.n_pos - 1);
  *hi = last;
  *lo = a.window > 0 && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
}

constexpr int kPlanThreads = 512;
constexpr int kListed = 2048;                 // units a head up to which they are sorted and may be cut

// One unit a head: its sequence, its place in it, its tiles.
struct Listed { int row, j, len; };

struct PlanSmem {
  int off[kPlanThreads + 1];                  // units before a sequence, of the sequences at hand
  Listed unit[kListed];
  int warp[kPlanThreads / 32];
  int hist[64], parts[33], least[33];
  unsigned long long tiles;
  int longest, cut, slots;
};

// Unit j of sequence row.
__device__ __forceinline__ Unit unit_of(const Pool& c, const AttnArgs& a, const Shape& s, int row, int j) {
  const int64_t t_lo = __ldg(a.cu + row), t_hi = min((int64_t)__ldg(a.cu + row + 1), a.n_tok);
  Unit w;
  w.tok = (int)(t_lo + (int64_t)j * s.tpu);
  w.n = (int)min((int64_t)s.tpu, t_hi - w.tok);
  w.off = w.tok - (int)t_lo;
  w.pos = (int64_t)__ldg(a.start + row) + w.off;
  w.row = row;
  return w;
}

// All units of all heads, longest first, cut where that makes the whole end sooner.
__device__ __forceinline__ void make_units(const Pool& c, const RopeArgs& r, const AttnArgs& a, const Shape& s, const Plan& p,
                                           PlanSmem& m) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = c.n_kv * s.nsub;
  if (tid < 64) m.hist[tid] = 0;
  if (tid < 33) {
    m.parts[tid] = 0;
    m.least[tid] = 0x7fffffff;
  }
  if (tid == 0) {
    m.tiles = 0;
    m.longest = m.slots = 0;
  }
  int64_t count = 0;                          // units a head
  unsigned long long tiles = 0;
  int longest = 0;
  for (int b0 = 0; b0 < c.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < c.batch) {
      const int64_t t_lo = __ldg(a.cu + b), t_end = __ldg(a.cu + b + 1), t_hi = min(t_end, a.n_tok);
      if (t_end < t_lo) raise(a.flags, SQ_FLAG_SEQLEN);   // sequences may name the same tokens, and units have no place
      if (t_lo >= 0 && t_hi > t_lo) {
        n = (int)((uint32_t)(t_hi - t_lo + s.tpu - 1) / (uint32_t)s.tpu);
        const int64_t start = __ldg(a.start + b), last = start + (t_hi - t_lo) - 1;
        uint32_t bits = 0;
        if (last >= c.cap() || start < 0) bits |= SQ_FLAG_SEQLEN;
        if (r.table && min(last, c.cap() - 1) >= r.n_pos) bits |= SQ_FLAG_ROPE;
        if (bits && a.flags) atomicOr(a.flags, bits);
      }
    }
    // units before each of these sequences
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) m.warp[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += m.warp[w];
    m.off[tid + 1] = inc;
    if (tid == 0) m.off[0] = 0;
    __syncthreads();
    const int here = m.off[kPlanThreads];
    for (int e = tid; e < here; e += kPlanThreads) {
      int lo_b = 0, hi_b = kPlanThreads;      // the sequence of unit e
      while (hi_b - lo_b > 1) {
        const int mid = (lo_b + hi_b) >> 1;
        if (m.off[mid] <= e) lo_b = mid; else hi_b = mid;
      }
      const int j = m.off[lo_b + 1] - 1 - e;  // the last tokens, which attend most, first
      Unit w = unit_of(c, a, s, b0 + lo_b, j);
      int64_t lo, hi;
      unit_keys(c, r, a, w.pos, w.n, &lo, &hi);
      const int len = hi < lo ? 0 : (int)(hi / KT - lo / KT) + 1;
      tiles += len;
      longest = max(longest, len);
      if (count + e < kListed) {
        m.unit[count + e] = Listed{b0 + lo_b, j, len};
      }
      if (count + here > kListed) {
        // Too many to sort; so many share the work well enough as they come. (Those listed before are written below.)
        w.t0 = (int)(lo / KT);
        w.nt = len;
        w.slot = -1;
        for (int h = 0; h < heads; ++h) {
          w.hs = h;
          const int64_t at = (count + e) * heads + h;
          if (at < s.cap_units) p.units[at] = w;
        }
      }
    }
    count += here;
  }
  atomicAdd(&m.tiles, tiles);
  atomicMax(&m.longest, longest);
  __syncthreads();
  const bool sorted = count <= kListed;
  if (!sorted) {
    // the listed ones that came with earlier sequences
    for (int e = tid; e < kListed; e += kPlanThreads) {
      const Listed l = m.unit[e];
      Unit w = unit_of(c, a, s, l.row, l.j);
      int64_t lo, hi;
      unit_keys(c, r, a, w.pos, w.n, &lo, &hi);
      w.t0 = (int)(lo / KT);
      w.nt = l.len;
      w.slot = -1;
      for (int h = 0; h < heads; ++h) {
        w.hs = h;
        const int64_t at = (int64_t)e * heads + h;
        if (at < s.cap_units) p.units[at] = w;
      }
    }
    if (tid == 0) {
      p.head->units = (int)min(count * heads, (int64_t)s.cap_units);
    }
    return;
  }
  // ---- where to cut: an even share of the tiles, or more by up to twice, or nowhere (candidate 32)
  const int n_units = (int)count;
  const int share = max(4, (int)((m.tiles * heads + s.sms - 1) / s.sms));
  longest = max(1, m.longest);
  auto candidate = [&](int i) { return i == 32 ? longest : min(longest, share + (share * i + 15) / 16); };
  for (int i = lane; i < 33; i += 32) {
    const int cut = candidate(i);
    int parts = 0, least = 0x7fffffff;
    for (int e = warp; e < n_units; e += kPlanThreads / 32) {
      const int len = m.unit[e].len, n = len > cut ? (len + cut - 1) / cut : 1;
      parts += n;
      least = min(least, len / n);
    }
    atomicAdd(&m.parts[i], parts);
    atomicMin(&m.least[i], least);
  }
  __syncthreads();
  if (warp == 0) {
    // Pieces run longest first on `sms` places: up to that many, the longest ends last; beyond, the last to begin
    // ends within its own length of the even share. A piece costs about two tiles besides.
    auto ends = [&](int i) {
      const int cut = candidate(i), n = m.parts[i] * heads, waves = (n + s.sms - 1) / s.sms;
      return (n <= s.sms ? cut : max(cut, share + m.least[i])) + 2 * waves;
    };
    const uint32_t best = __reduce_min_sync(0xffffffffu, (uint32_t)ends(lane) << 6 | (uint32_t)lane);
    const uint32_t uncut = (uint32_t)ends(32) << 6;            // a tie goes to no cut
    if (lane == 0) m.cut = uncut <= best ? longest : candidate(best & 63u);
  }
  __syncthreads();
  // ---- the list by classes of length
  const int cut = m.cut;
  auto cls = [&](int len, int parts) { return 63 - (int)(((len + parts - 1) / parts) * 63.0f / cut); };
  for (int e = tid; e < n_units; e += kPlanThreads) {
    const int len = m.unit[e].len, parts = len > cut ? (len + cut - 1) / cut : 1;
    atomicAdd(&m.hist[cls(len, parts)], parts * heads);
  }
  __syncthreads();
  if (warp == 0) {                            // pieces before each class
    const int a0 = m.hist[2 * lane], a1 = m.hist[2 * lane + 1];
    int inc = a0 + a1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    m.hist[2 * lane] = inc - a0 - a1;
    m.hist[2 * lane + 1] = inc - a1;
    if (lane == 31) p.head->units = min(inc, s.cap_units);
  }
  __syncthreads();
  for (int x = tid; x < n_units * heads; x += kPlanThreads) {
    const int e = x / heads;
    const Listed l = m.unit[e];
    const int parts = l.len > cut ? (l.len + cut - 1) / cut : 1;
    int at = atomicAdd(&m.hist[cls(l.len, parts)], parts), slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&m.slots, parts);
      p.done[slot] = 0;                       // (there are places for all, whatever the offsets: see prefill_shape)
    }
    Unit w = unit_of(c, a, s, l.row, l.j);
    int64_t lo, hi;
    unit_keys(c, r, a, w.pos, w.n, &lo, &hi);
    w.hs = x - e * heads;
    w.slot = slot;
    w.parts = parts;
    int t = (int)(lo / KT);
    for (int i = 0; i < parts; ++i, ++at) {
      w.t0 = t;
      w.nt = l.len / parts + (i < l.len % parts ? 1 : 0);
      w.part = i;
      t += w.nt;
      if (at < s.cap_units) p.units[at] = w;
    }
  }
}

// Block 0 lists the units; the others turn, scale and lay out the queries, D / 16
// threads a row (eight coordinates of each half, as the append takes them) and two
// heads of a token at once, under the same angles: fp16, rows of a power of two
// each, 64 coordinates a 16 KB slab of swizzled lines, eight coordinates in the
// codes' order. Once a call, so that the pieces of a cut unit do not repeat it and a
// block's prologue is one bulk copy a row tile. MODE as in k_append4.
constexpr int kQHeads = 2;
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kPlanThreads, 2)
k_prepare4(Pool c, RopeArgs r, const T* __restrict__ q, AttnArgs a, Shape s, Plan p) {
  using C = Cfg<D>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    extern __shared__ __align__(16) uint8_t plan_smem[];
    make_units(c, r, a, s, p, *(PlanSmem*)plan_smem);
    return;
  }
  constexpr int TPR = D / 16;
  const int j = threadIdx.x % TPR, parts = (a.n_q + kQHeads - 1) / kQHeads;
  const int64_t items = a.n_tok * parts, step = (int64_t)(gridDim.x - 1) * (kPlanThreads / TPR);
  const int p0 = partner(8 * j, r), p1 = partner(D / 2 + 8 * j, r);
  for (int64_t x0 = (int64_t)(blockIdx.x - 1) * (kPlanThreads / TPR); x0 < items; x0 += step) {
    const int64_t v = x0 + threadIdx.x / TPR;
    const int64_t tok = v < items ? (items < 0x7fffffff ? (int64_t)((uint32_t)v / (uint32_t)parts) : v / parts) : 0;
    const int h0 = (int)(v - tok * parts) * kQHeads;
    int32_t off = 0;
    const int b = v < items ? row_of(a.cu, c.batch, tok, &off) : -1;
    if (__all_sync(0xffffffffu, b < 0)) continue;
    Vec8<T> own[kQHeads][2], part[MODE == 2 ? kQHeads : 1][2];
    const int nh = b < 0 ? 0 : min(kQHeads, a.n_q - h0);
#pragma unroll
    for (int n = 0; n < kQHeads; ++n)
      if (n < nh) {
        const T* src = q + tok * a.qs_tok + (int64_t)(h0 + n) * a.qs_head;
        own[n][0] = load8<T>(src + 8 * j);
        own[n][1] = load8<T>(src + D / 2 + 8 * j);
        if (MODE == 2) {
          part[n][0] = load8<T>(src + p0);
          part[n][1] = load8<T>(src + p1);
        }
      }
    const int64_t pos = b < 0 ? -1 : min((int64_t)__ldg(a.start + b) + off, c.cap() - 1);
    const bool live = pos >= 0 && !(MODE && pos >= r.n_pos);
    float cs[8], sn[8];
    if (MODE == 1 && live) {
      const float4* row = (const float4*)(r.table + pos * D + 8 * j);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        *(float4*)(cs + 4 * e) = __ldg(row + e);
        *(float4*)(sn + 4 * e) = __ldg(row + D / 8 + e);
      }
    }
    const int64_t tile = b < 0 ? 0 : row_tile(tok - off, b, off, s.tpm);
    const int row0 = off % s.tpm * s.gt;
#pragma unroll
    for (int n = 0; n < kQHeads; ++n) {
      float x[2][8];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e >> 3][e & 7] = 0.0f;
      if (n < nh && live) {
        unpack8<T>(own[n][0], x[0]);
        unpack8<T>(own[n][1], x[1]);
        if (MODE == 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float ya = x[0][e], yb = x[1][e];
            x[0][e] = __fsub_rn(__fmul_rn(ya, cs[e]), __fmul_rn(yb, sn[e]));
            x[1][e] = __fadd_rn(__fmul_rn(yb, cs[e]), __fmul_rn(ya, sn[e]));
          }
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            round2<T>(&x[0][e], &x[0][e + 1]);
            round2<T>(&x[1][e], &x[1][e + 1]);
          }
        }
        if (MODE == 2) {
          float y[8];
          unpack8<T>(part[n][0], y);
          rotate8<T>(x[0], y, 8 * j, r, pos);
          unpack8<T>(part[n][1], y);
          rotate8<T>(x[1], y, D / 2 + 8 * j, r, pos);
        }
      }
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e >> 3][e & 7]));
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^e with top 2^e in [2^6, 2^7): the sum over a head stays below 2^15 (-121 for the largest floats)
      int e2 = 0;
      if (top > 0.0f && top < INFINITY) e2 = min(100, 6 + 127 - (int)(__float_as_uint(top) >> 23));
      const float up = __int_as_float((127 + e2) << 23);
      float sum = 0.0f;
      uint32_t w[2][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2 hv = __floats2half2_rn(x[i >> 2][i & 3] * up, x[i >> 2][(i & 3) + 4] * up);
        const float2 f = __half22float2(hv);
        sum += f.x + f.y;
        w[i >> 2][i & 3] = *(const uint32_t*)&hv;
      }
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (n >= nh) continue;
      const int head = h0 + n, kvh = head / a.group, g = head - kvh * a.group, sub = g / s.gt, row = row0 + g - sub * s.gt;
      uint8_t* img = p.q + ((int64_t)(kvh * s.nsub + sub) * p.q_tiles + tile) * C::QIMG;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ch = j + e * TPR;
        *(uint4*)(img + (ch >> 3) * 16384 + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
      }
      if (j < 2) {
        // sum(q) in three parts, against the keys' m and 8 s
        const __half s0 = __float2half_rn(sum);
        const float d1 = sum - __half2float(s0);
        const __half s1 = __float2half_rn(d1), s2 = __float2half_rn(d1 - __half2float(s1));
        const __half2 a0 = __halves2half2(s0, s1), a1 = __halves2half2(s2, s0), a2 = __halves2half2(s1, s2);
        *(uint4*)(img + C::MAIN + (row >> 3) * 256 + j * 128 + (row & 7) * 16) =
            j ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(*(const uint32_t*)&a0, *(const uint32_t*)&a1, *(const uint32_t*)&a2, 0u);
        if (j) *(float*)(img + C::OP + 4 * row) = a.scale * 1.4426950408889634f * __int_as_float((127 - e2) << 23);
      }
    }
  }
}

// ---------------------------------------------------------------- tensor memory, packed floats
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// The registers of a load may be used behind this.
__device__ __forceinline__ void ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void ld_wait16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               ::"memory");
}
__device__ __forceinline__ void st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
// True in one lane of a converged warp. A warp that issues its products under this,
// and stays converged otherwise, keeps the operands' descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// Registers a thread of this warp group (multiples of 8), which together stay within what the block started with.
template <int N> __device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Descriptors of an operand in shared memory: keys and queries (coordinates run
// along k, 64 of a row's in a 128-byte swizzled line), their last step (no swizzle,
// 16-byte rows of 8 by 8 cores), values (coordinates run along n, tokens along k).
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t swizzle) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)swizzle << 61;
}

// Eight codes of a word, centred and scaled: 16 bytes in the order 0 4 1 5 2 6 3 7,
// which the queries follow for the keys and the epilogue undoes for the values. A
// code or'ed into the low bits of fp16 1024 is 1024 + c; both operations are exact.
__device__ __forceinline__ uint4 unpack_codes(uint32_t w, __half2 s, __half2 s16) {
  const uint32_t x = w >> 8;
  const uint32_t u0 = (w & 0x000f000fu) | 0x64006400u, u1 = (w & 0x00f000f0u) | 0x64006400u;
  const uint32_t u2 = (x & 0x000f000fu) | 0x64006400u, u3 = (x & 0x00f000f0u) | 0x64006400u;
  const __half2 lo = __float2half2_rn(-1032.0f), hi = __float2half2_rn(-1152.0f);
  const __half2 r0 = __hmul2(__hadd2(*(const __half2*)&u0, lo), s);
  const __half2 r1 = __hmul2(__hadd2(*(const __half2*)&u1, hi), s16);
  const __half2 r2 = __hmul2(__hadd2(*(const __half2*)&u2, lo), s);
  const __half2 r3 = __hmul2(__hadd2(*(const __half2*)&u3, hi), s16);
  return make_uint4(*(const uint32_t*)&r0, *(const uint32_t*)&r1, *(const uint32_t*)&r2, *(const uint32_t*)&r3);
}

// What the softmax needs to know of a tile of keys.
struct Info {
  float kf;              // score factor
  float vref;            // reference step of the values so far
  uint32_t ok[4];        // keys that exist
};

// Bits of the 32 keys from `from` on that are among a row's [lo, hi] and exist.
__device__ __forceinline__ uint32_t keys_kept(uint32_t ok, int from, int lo, int hi) {
  const int x = lo - from, y = hi - from;
  ok &= x <= 0 ? 0xffffffffu : (x > 31 ? 0u : 0xffffffffu << x);
  return ok & (y >= 31 ? 0xffffffffu : (y < 0 ? 0u : 0xffffffffu >> (31 - y)));
}

// A thread's share of a tile: a row's scores against 64 keys, 64 columns of tensor
// memory from t_s on. Their largest:
__device__ __forceinline__ float row_max(uint32_t t_s) {
  uint32_t x[32], y[32];
  ld32(t_s, x);
  ld32(t_s + 32, y);
  ld_wait(x);
  ld_wait(y);
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    m0 = fmaxf(m0, fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
    m1 = fmaxf(m1, fmaxf(__uint_as_float(y[e]), __uint_as_float(y[e + 1])));
  }
  return fmaxf(m0, m1);
}
// The same of the keys that the row attends (few tiles: short code rather than fast). ok: two words.
__device__ __forceinline__ float row_max_edge(uint32_t t_s, const uint32_t* ok, int key0, int lo, int hi) {
  float m = -INFINITY;
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t x[16];
    ld16(t_s + 16 * ch, x);
    const uint32_t keep = keys_kept(ok[ch >> 1], key0 + 32 * (ch >> 1), lo, hi) >> (16 * (ch & 1));
    ld_wait16(x);
#pragma unroll
    for (int e = 0; e < 16; ++e) m = (keep >> e) & 1u ? fmaxf(m, __uint_as_float(x[e])) : m;
  }
  return m;
}

struct Sums { f2 l, m; };
// A step's operand of the values' product: the probabilities of 16 keys in 8 columns of tensor memory, and for an fp16
// or float output what that rounding left of them in 8 more.
template <bool FINE> __host__ __device__ constexpr int prob_cols() { return FINE ? 16 : 8; }
// Two probabilities of it. The first part has a float's upper 11 bits (fp16's own below 2^-14), the second the rest.
template <bool FINE> __device__ __forceinline__ void put_probs(uint32_t* pk, int at, float p0, float p1) {
  if constexpr (FINE) {
    const float h0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u), h1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
    const f2 rest = f2_add(f2_of(p0, p1), f2_of(-h0, -h1));
    pk[at] = dec::pack_h2(h0, h1);
    pk[at + 8] = dec::pack_h2(f2_lo(rest), f2_hi(rest));
  } else {
    pk[at] = dec::pack_h2(p0, p1);
  }
}
template <bool FINE> __device__ __forceinline__ void store_probs(uint32_t t_s, const uint32_t* pk) {
  if constexpr (FINE) st16(t_s, pk);
  else sm100::tmem_st8(t_s, pk);
}
// Scores to probabilities 2^(s fk + nb), which take the place of the first half of
// them, or of all; the sums grow by their sum and their sum with the offsets. The sums
// and roundings of 16 keys are written beside the exponentials of the next 16.
template <bool FINE>
__device__ __forceinline__ Sums row_probs(uint32_t t_s, float fk, float nb, const float* mean, Sums sum) {
  const f2 fk2 = f2_of(fk, fk), nb2 = f2_of(nb, nb);
  uint32_t s[2][16];
  float p[16];
  ld16(t_s, s[0]);
#pragma unroll
  for (int ch = 0; ch <= 4; ++ch) {
    uint32_t* x = s[ch & 1];
    uint32_t pk[prob_cols<FINE>()];
    if (ch < 4) {
      ld_wait16(x);
      if (ch < 3) ld16(t_s + 16 * (ch + 1), s[(ch + 1) & 1]);
    }
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      if (ch > 0) {
        const ulonglong2 mu = *(const ulonglong2*)(mean + 16 * (ch - 1) + e);
        const f2 pa = f2_of(p[e], p[e + 1]), pb = f2_of(p[e + 2], p[e + 3]);
        sum.l = f2_add(sum.l, pa);
        sum.m = f2_fma(pa, mu.x, sum.m);
        sum.l = f2_add(sum.l, pb);
        sum.m = f2_fma(pb, mu.y, sum.m);
        put_probs<FINE>(pk, e / 2, p[e], p[e + 1]);
        put_probs<FINE>(pk, e / 2 + 1, p[e + 2], p[e + 3]);
      }
      if (ch < 4) {
        const f2 ta = f2_fma(f2_of(x[e], x[e + 1]), fk2, nb2), tb = f2_fma(f2_of(x[e + 2], x[e + 3]), fk2, nb2);
        p[e] = dec::ex2(f2_lo(ta));
        p[e + 1] = dec::ex2(f2_hi(ta));
        p[e + 2] = dec::ex2(f2_lo(tb));
        p[e + 3] = dec::ex2(f2_hi(tb));
      }
    }
    if (ch > 0) store_probs<FINE>(t_s + prob_cols<FINE>() * (ch - 1), pk);
  }
  return sum;
}
template <bool FINE>
__device__ __forceinline__ Sums row_probs_edge(uint32_t t_s, float fk, float nb, const float* mean, Sums sum,
                                               const uint32_t* ok, int key0, int lo, int hi) {
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t x[16], pk[prob_cols<FINE>()];
    ld16(t_s + 16 * ch, x);
    const uint32_t keep = keys_kept(ok[ch >> 1], key0 + 32 * (ch >> 1), lo, hi) >> (16 * (ch & 1));
    ld_wait16(x);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const bool k0 = (keep >> e) & 1u, k1 = (keep >> (e + 1)) & 1u;
      const float t0 = fmaf(__uint_as_float(x[e]), fk, nb), t1 = fmaf(__uint_as_float(x[e + 1]), fk, nb);
      const float m0 = mean[16 * ch + e], m1 = mean[16 * ch + e + 1];
      const float p0 = dec::ex2(k0 ? t0 : -INFINITY), p1 = dec::ex2(k1 ? t1 : -INFINITY);
      const f2 p = f2_of(p0, p1);
      sum.l = f2_add(sum.l, p);
      sum.m = f2_fma(p, f2_of(k0 ? m0 : 0.0f, k1 ? m1 : 0.0f), sum.m);
      put_probs<FINE>(pk, e / 2, p0, p1);
    }
    store_probs<FINE>(t_s + prob_cols<FINE>() * ch, pk);
  }
  return sum;
}
// Scales N of a row's sums in tensor memory.
template <int N> __device__ __forceinline__ void row_scale(uint32_t t_o, float f) {
  const f2 f2v = f2_of(f, f);
#pragma unroll 1
  for (int ch = 0; ch < N / 32; ++ch) {
    uint32_t x[32];
    ld32(t_o + 32 * ch, x);
    ld_wait(x);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const f2 y = f2_fma(f2_of(x[e], x[e + 1]), f2v, 0ull);
      x[e] = (uint32_t)y;
      x[e + 1] = (uint32_t)(y >> 32);
    }
    st16(t_o + 32 * ch, x);
    st16(t_o + 32 * ch + 16, x + 16);
  }
  sm100::tmem_wait_st();
}

// The rows of a box, each to where the lane of its number says (or nowhere).
template <typename E> __device__ __forceinline__ void unbox(const uint8_t* box, E* to) {
  constexpr int P = 2 * (int)sizeof(E);                // 16-byte words of a row
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int it = 0; it < P; ++it) {
    const int row = (32 * it + lane) / P, w = (32 * it + lane) % P;
    uint4* dst = (uint4*)__shfl_sync(0xffffffffu, (unsigned long long)to, row);
    if (dst) dst[w] = *(const uint4*)(box + row * box_pitch<E>() + 16 * w);
  }
}

// Joins the pieces of a cut unit in their order, a warp a row, by the block that wrote the last of them.
template <typename TO, int D>
__device__ __forceinline__ void join_unit(const Plan& plan, const Unit& u, TO* __restrict__ out, const AttnArgs& a, const Shape& sh,
                                          int h0, int nh, int rows, int warp, int warps) {
  constexpr int NS = Cfg<D>::NS;
  constexpr int R = 4;                        // rows at once: their reads are on the way together
  const int lane = threadIdx.x & 31;
  const float2* ml = (const float2*)(plan.parts + (size_t)sh.cap_slots * part_rows(NS) * D);
  for (int row0 = warp; row0 < rows; row0 += R * warps) {
    int64_t at[R], first[R];
    float top[R], l[R], o[R][D / 32];
#pragma unroll
    for (int n = 0; n < R; ++n) {
      const int row = row0 + n * warps, i = row / M, wt = row % M, ti = i * sh.tpm + wt / sh.gt, hh = wt % sh.gt;
      at[n] = row < rows && wt < sh.tpm * sh.gt && ti < u.n && hh < nh ? (int64_t)(u.tok + ti) * a.n_q + h0 + hh : -1;
      first[n] = (int64_t)u.slot * part_rows(NS) + (at[n] < 0 ? 0 : row);
      top[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[n][e] = 0.0f;
    }
    // lane p has piece p's maximum and sum
    for (int p = lane; p < u.parts; p += 32)
#pragma unroll
      for (int n = 0; n < R; ++n) top[n] = fmaxf(top[n], __ldcg(ml + first[n] + p * (int64_t)part_rows(NS)).x);
#pragma unroll
    for (int n = 0; n < R; ++n)
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], x));
    for (int p0 = 0; p0 < u.parts; p0 += 32) {
      float f[R];
#pragma unroll
      for (int n = 0; n < R; ++n) {
        const float2 x = p0 + lane < u.parts ? __ldcg(ml + first[n] + (p0 + lane) * (int64_t)part_rows(NS)) : make_float2(-INFINITY, 0.0f);
        f[n] = x.x == -INFINITY ? (x.y == 0.0f ? 0.0f : 1.0f) : dec::ex2(x.x - top[n]);
        float y = f[n] * x.y;
#pragma unroll
        for (int z = 16; z > 0; z >>= 1) y += __shfl_xor_sync(0xffffffffu, y, z);
        l[n] += y;
      }
      const int here = min(32, u.parts - p0);
#pragma unroll 2
      for (int p = 0; p < here; ++p)
#pragma unroll
        for (int n = 0; n < R; ++n) {
          const float fp = __shfl_sync(0xffffffffu, f[n], p);
          const float* src = plan.parts + (first[n] + (p0 + p) * (int64_t)part_rows(NS)) * D + lane;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) o[n][e] = fmaf(fp, __ldcg(src + 32 * e), o[n][e]);
        }
    }
#pragma unroll
    for (int n = 0; n < R; ++n) {
      if (at[n] < 0) continue;
      const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) out[at[n] * D + 32 * e + lane] = from_f<TO>(l[n] == 0.0f ? 0.0f : o[n][e] * inv);
      if (a.lse && lane == 0) a.lse[at[n]] = l[n] == 0.0f ? -INFINITY : (top[n] + (log2f(l[n]) - kUp)) * 0.69314718055994531f;
    }
  }
}

template <typename TO, int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
k_prefill4(Pool c, RopeArgs r, TO* __restrict__ out, AttnArgs a, Shape sh, Plan plan) {
  using C = Cfg<D>;
  constexpr int NS = C::NS, NKV = C::NKV;
  constexpr bool FINE = !dec::is_bf16<TO>();     // probabilities in two parts
  constexpr int kUnpack = C::SOFT * 4, kIssuer = kUnpack + 8;        // first unpacking warp, the one that issues
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t b_q, b_fin, b_s[2], b_p[2], b_o[NS], b_kf[NKV], b_ke[NKV], b_vf[NKV], b_ve[NKV], b_i[kInfo];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ Info s_info[kInfo];
  __shared__ uint2 s_red[2][8];
  __shared__ float s_max[NS][2][2][M];           // a half row's largest score, tiles taking turns
  __shared__ float2 s_sum[NS][2][M];
  uint8_t* smem = smem_raw + ((1024u - (sm100::smem_u32(smem_raw) & 1023u)) & 1023u);   // (kept a shared address)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int units = plan.head->units;
  const Unit u = plan.units[blockIdx.x];       // (asked for together with their number: there is a place for each block)
  if ((int)blockIdx.x >= units) return;
  const int ns = u.n > sh.tpm ? NS : 1, nt = u.nt;
  if (warp == kIssuer) sm100::tmem_alloc(&s_tmem, 512);
  if (tid == 0) {
    sm100::mbar_init(&b_q, 1);
    sm100::mbar_init(&b_fin, 1);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&b_s[i], 1);
      sm100::mbar_init(&b_p[i], 2 * kGroup);
    }
    for (int i = 0; i < NS; ++i) sm100::mbar_init(&b_o[i], 1);
    for (int i = 0; i < NKV; ++i) {
      sm100::mbar_init(&b_kf[i], 2 * kGroup);
      sm100::mbar_init(&b_ke[i], 1);
      sm100::mbar_init(&b_vf[i], 2 * kGroup);
      sm100::mbar_init(&b_ve[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) sm100::mbar_init(&b_i[i], 2 * kGroup);
    sm100::fence_mbar_init();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int64_t cap = c.cap();
  const int kvh = u.hs / sh.nsub, h0 = kvh * a.group + (u.hs % sh.nsub) * sh.gt;
  const int nh = min(sh.gt, (kvh + 1) * a.group - h0);

  if (warp < kUnpack) {
    set_regs_up<C::R_SOFT>();
    // ------------------------------------------------------------ softmax and outputs: half a row a thread
    const int i = warp >> 3, half = (warp >> 2) & 1, wt = tid & 127;
    if (i < ns) {
      const int ti = i * sh.tpm + wt / sh.gt, hh = wt % sh.gt;
      const bool is_row = wt < sh.tpm * sh.gt && ti < u.n && hh < nh;
      // keys [lo, hi] of the row; rows that are none take any, so that they ask for no masks
      int lo = 0, hi = 0x7fffffff;
      if (is_row) {
        const int64_t p = min(u.pos + ti, cap - 1);
        hi = p < 0 || (r.table && p >= r.n_pos) ? -1 : (int)p;
        lo = a.window > 0 && p - a.window + 1 > 0 ? (int)(p - a.window + 1) : 0;
      }
      const int w_lo = __reduce_max_sync(0xffffffffu, lo), w_hi = __reduce_min_sync(0xffffffffu, hi);
      const int64_t tile = (int64_t)u.hs * plan.q_tiles + row_tile(u.tok - u.off, u.row, u.off, sh.tpm) + i;
      const float fq = is_row ? *(const float*)(plan.q + tile * C::QIMG + C::OP + 4 * wt) : 0.0f;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t t_o = tmem + lanes + 256 + i * D + half * (D / 2);
      float mref = -INFINITY, vref = 0.0f;
      Sums sum{0ull, 0ull};
      bool dead = false;
      // A warp whose wait gave up keeps meeting the others at their barriers, and does no more.
      for (int k = 0; k < nt; ++k) {
        const int sl = ns == 2 ? i : (k & 1);
        const uint32_t t_s = tmem + lanes + 128 * sl + 64 * half;
        const int ring = k % kInfo;
        dead = dead || !sm100::mbar_wait(&b_i[ring], (k / kInfo) & 1, a.flags);
        dead = dead || !sm100::mbar_wait(&b_s[sl], ns == 2 ? (k & 1) : ((k >> 1) & 1), a.flags);
        dead = __any_sync(0xffffffffu, dead);
        sm100::tc_fence_after();
        const Info& in = s_info[ring];
        const uint32_t ok[2] = {in.ok[2 * half], in.ok[2 * half + 1]};
        const int key0 = (u.t0 + k) * KT + 64 * half;
        const bool edge = (ok[0] & ok[1]) != 0xffffffffu || key0 < w_lo || key0 + 63 > w_hi;
        const float fk = fq * in.kf, nv = in.vref;
        const float* mean = (const float*)(smem + C::MEAN) + ring * KT + 64 * half;
        const float mine = dead ? -INFINITY : edge ? row_max_edge(t_s, ok, key0, lo, hi) : row_max(t_s);
        s_max[i][k & 1][half][wt] = mine;
        sm100::named_bar(1 + i, 2 * kGroup);
        const float top = fk * fmaxf(mine, s_max[i][k & 1][half ^ 1][wt]);
        if (dead) continue;
        if (__any_sync(0xffffffffu, (is_row && top > mref + kSlack) || nv != vref)) {
          float f = 1.0f;
          if (is_row && top > mref) {
            f = dec::ex2(mref - top);            // 0 the first time
            mref = top;
          }
          const f2 ff = f2_of(f, f);
          sum.l = f2_fma(sum.l, ff, 0ull);
          sum.m = f2_fma(sum.m, ff, 0ull);
          if (k > 0) {
            dead = __any_sync(0xffffffffu, !sm100::mbar_wait(&b_o[i], (k - 1) & 1, a.flags));
            if (dead) continue;
            sm100::tc_fence_after();
            row_scale<D / 2>(t_o, f * (vref / nv));
          }
          vref = nv;
        }
        const float nb = kUp - (mref == -INFINITY ? 0.0f : mref);
        sum = edge ? row_probs_edge<FINE>(t_s, fk, nb, mean, sum, ok, key0, lo, hi) : row_probs<FINE>(t_s, fk, nb, mean, sum);
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        sm100::mbar_arrive(&b_p[sl]);
      }
      // ---- outputs
      // (The end of the last sum: with two score buffers this row tile may be two sums behind its softmax, and a
      // parity of b_o would not tell them apart.)
      if (nt > 0 && !dead) dead = ns == 2 ? !sm100::mbar_wait(&b_o[i], (nt - 1) & 1, a.flags) : !sm100::mbar_wait(&b_fin, 0, a.flags);
      dead = __any_sync(0xffffffffu, dead);
      sm100::tc_fence_after();
      const float2 own = make_float2(f2_lo(sum.l) + f2_hi(sum.l), f2_lo(sum.m) + f2_hi(sum.m));
      s_sum[i][half][wt] = own;
      sm100::named_bar(1 + i, 2 * kGroup);
      if (!dead) {
        const float2 other = s_sum[i][half ^ 1][wt];
        const float l = own.x + other.x, mv = own.y + other.y;
        const float vf = vref * 0x1p-12f;
        const bool whole = u.slot < 0;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t at = (int64_t)(u.tok + ti) * a.n_q + h0 + hh;
        const int64_t pr = whole ? 0 : (int64_t)(u.slot + u.part) * part_rows(NS) + i * M + wt;
        // 32 coordinates of 32 rows at a time go through shared memory, so that they leave in whole lines: where
        // the row tile's queries lie, which nothing reads any more, or behind everything.
        uint8_t* box = smem + C::BOX + i * C::BOX_STEP + (warp & 7) * kBox;
        TO* wo = is_row ? out + at * D + half * (D / 2) : nullptr;
        float* po = is_row ? plan.parts + pr * D + half * (D / 2) : nullptr;
#pragma unroll 1
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t x[32];
          if (nt > 0) {
            ld32(t_o + 32 * ch, x);
            ld_wait(x);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0u;
          }
#pragma unroll
          for (int g = 0; g < 32; g += 8) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)                                   // (the codes' order undone)
              o[((e & 1) << 2) + (e >> 1)] = fmaf(__uint_as_float(x[g + e]), vf, mv);
            if (whole) {
              TO y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = from_f<TO>(l == 0.0f ? 0.0f : o[e] * inv);
#pragma unroll
              for (int e = 0; e < (int)sizeof(TO) / 2; ++e)
                *(uint4*)(box + lane * box_pitch<TO>() + g * sizeof(TO) + 16 * e) = ((const uint4*)y)[e];
            } else {
#pragma unroll
              for (int e = 0; e < 8; e += 4)
                *(float4*)(box + lane * box_pitch<float>() + (g + e) * 4) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          __syncwarp();
          if (whole) unbox(box, wo == nullptr ? nullptr : wo + 32 * ch);
          else unbox(box, po == nullptr ? nullptr : po + 32 * ch);
          __syncwarp();
        }
        if (is_row && half == 0) {
          if (whole) {
            if (a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (mref + (log2f(l) - kUp)) * 0.69314718055994531f;
          } else {
            float* ml = plan.parts + (size_t)sh.cap_slots * part_rows(NS) * D + pr * 2;
            ml[0] = mref;
            ml[1] = l;
          }
        }
      }
      // ---- the piece that is written last joins them all
      if (u.slot >= 0) {
        __threadfence();
        sm100::named_bar(4, 2 * ns * kGroup);
        if (tid == 0) s_last = atomicAdd(plan.done + u.slot, 1) == u.parts - 1;
        sm100::named_bar(4, 2 * ns * kGroup);
        if (s_last) {
          __threadfence();
          join_unit<TO, D>(plan, u, out, a, sh, h0, nh, ns * M, warp, 8 * ns);
        }
      }
    }
  } else if (warp < kIssuer) {
    // ------------------------------------------------------------ unpacking: a warp a block of 16 keys
    if constexpr (NS == 1) set_regs_up<C::R_UNPACK>(); else set_regs_down<C::R_UNPACK>();
    constexpr int NC = D / 64;                       // 16-byte chunks of a block's codes a lane, a side
    const int uw = warp - kUnpack;
    int64_t ulo, uhi;
    unit_keys(c, r, a, u.pos, u.n, &ulo, &uhi);
    const int64_t page_bytes = ((int64_t)c.n_kv << (c.page_shift - 4)) * blk_bytes(D);
    const uint8_t* head = c.pages + ((int64_t)kvh << (c.page_shift - 4)) * blk_bytes(D);
    const int32_t* table = c.table + u.row * c.table_stride;
    const int in_page = (1 << c.page_shift) - 1;
    // page numbers two tiles ahead, codes one tile ahead
    auto page_of = [&](int k) {
      const int64_t t = (int64_t)(u.t0 + k) * KT + 16 * uw;
      if (k >= nt || t + 15 < ulo || t > uhi) return -2;
      return max(-1, __ldg(table + (t >> c.page_shift)));
    };
    // (looked at when its codes are loaded, a tile after it was asked for)
    auto checked = [&](int page) {
      if (page == -1 || page >= c.n_pages) {
        if (lane == 0) raise(a.flags, SQ_FLAG_PAGE);
        return -2;
      }
      return page;
    };
    auto block_of = [&](int k, int pg) {
      const int t = ((u.t0 + k) * KT + 16 * uw) & in_page;
      return head + pg * page_bytes + (t >> 4) * blk_bytes(D);
    };
    // Lane l holds the pair of key l, or of value l - 16, and chunks l, l + 32, ... of the codes as they lie. Where
    // they go: row t, coordinates 32 q .. 32 q + 31 as four chunks of a swizzled line. The lanes that write into
    // slabs of 64 coordinates at once begin with different ones of the four, so that no two meet in a bank.
    uint32_t to[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int x = 32 * i + lane, t = x / (D / 32), q = (x % (D / 32)) ^ swz(t, D), row = 16 * uw + t;
      const int rot = D == 256 ? q >> 1 : D == 128 ? q & 2 : 0;
      to[i] = (q >> 1) * 16384 + row * 128 + (((((q & 1) << 2) ^ rot ^ row) & 7) << 4);
    }
    auto unpack = [&](uint32_t dst, const uint4* codes, uint32_t scales, int from) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t sc = __shfl_sync(0xffffffffu, scales, from + (32 * i + lane) / (D / 32));
        const __half2 s2 = __half2half2(__ushort_as_half((unsigned short)sc)), s16 = __half2half2(__ushort_as_half((unsigned short)(sc >> 16)));
        uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
        const int q = ((32 * i + lane) % (D / 32)) ^ swz((32 * i + lane) / (D / 32), D);
        if (D >= 128) {                              // words in the order e ^ rot
          const bool b1 = D == 128 ? (q & 2) != 0 : (q & 4) != 0, b0 = D == 256 && (q & 2) != 0;
          const uint32_t y0 = b1 ? w[2] : w[0], y1 = b1 ? w[3] : w[1], y2 = b1 ? w[0] : w[2], y3 = b1 ? w[1] : w[3];
          w[0] = b0 ? y1 : y0;
          w[1] = b0 ? y0 : y1;
          w[2] = b0 ? y3 : y2;
          w[3] = b0 ? y2 : y3;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) *(uint4*)(smem + ((dst + to[i]) ^ (e << 4))) = unpack_codes(w[e], s2, s16);
      }
    };
    uint4 kc[NC], vc[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) kc[i] = vc[i] = make_uint4(0, 0, 0, 0);
    uint32_t pair = 0;
    auto load_k = [&](int k, int page) {
      pair = 0;
      if (page >= 0) {
        const uint8_t* blk = block_of(k, page);
        const int64_t t = (int64_t)(u.t0 + k) * KT + 16 * uw + (lane & 15);
        if (t >= ulo && t <= uhi) pair = __ldg((const uint32_t*)(blk + k_pairs(D) + 4 * lane));
#pragma unroll
        for (int i = 0; i < NC; ++i) kc[i] = __ldg((const uint4*)blk + 32 * i + lane);
      }
    };
    auto load_v = [&](int k, int page) {
      if (page >= 0) {
        const uint4* src = (const uint4*)(block_of(k, page) + v_codes(D));
#pragma unroll
        for (int i = 0; i < NC; ++i) vc[i] = __ldg(src + 32 * i + lane);
      }
    };
    int pg = checked(page_of(0)), pg_v = pg, pg_next;
    load_k(0, pg);
    load_v(0, pg);
    pg_next = page_of(1);
    float sref = 0.0f;
    uint32_t vs_cur = 0, vs_next = 0;
    bool dead = false;
    // keys of tile k, then values of tile k - 1: each is unpacked while the products of the other run
    for (int k = 0; k <= nt; ++k) {
      if (k < nt) {
        const int st = k % NKV;
        const float s = __uint_as_float(pair << 16), m = __uint_as_float(pair & 0xffff0000u);
        const int64_t t = (int64_t)(u.t0 + k) * KT + 16 * uw + (lane & 15);
        const uint32_t ok = __ballot_sync(0xffffffffu, pg >= 0 && t >= ulo && t <= uhi) & 0xffffu;
        // largest offset and step of the keys, largest step of the values (what is NaN is not greater), as words
        const uint32_t kv = __float_as_uint(fmaxf(fabsf(m), fmaxf(8.0f * s, 0.0f))), vv = __float_as_uint(fmaxf(s, 0.0f));
        const uint32_t kt_w = __reduce_max_sync(0xffffffffu, lane < 16 ? kv : 0u);
        const uint32_t vt_w = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : vv);
        if (lane == 0) s_red[k & 1][uw] = make_uint2(kt_w, vt_w);
        sm100::named_bar(3, 2 * kGroup);
        const uint2 red = s_red[k & 1][lane & 7];
        const float kref = pow2_up(__uint_as_float(__reduce_max_sync(0xffffffffu, red.x)));
        sref = fmaxf(sref, pow2_up(__uint_as_float(__reduce_max_sync(0xffffffffu, red.y))));
        const float kmul = 0x1p13f / kref, vmul = 0x1p12f / sref;
        dead = dead || !sm100::mbar_wait(&b_ke[st], ((k / NKV) & 1) ^ 1, a.flags);
        const int ring = k % kInfo;
        if (lane == 0) {
          if (uw == 0) {
            s_info[ring].kf = kref * 0x1p-13f;
            s_info[ring].vref = sref;
          }
          ((unsigned short*)s_info[ring].ok)[uw] = (unsigned short)ok;
        }
        if (lane >= 16) ((float*)(smem + C::MEAN))[ring * KT + 16 * uw + lane - 16] = fmaf(8.0f, s, m);
        sm100::mbar_arrive(&b_i[ring]);
        const float sm = s * (lane < 16 ? kmul : vmul);
        vs_next = dec::pack_h2(sm, sm * 0.0625f);
        const uint32_t kop = C::K + st * C::OP;
        unpack(kop, kc, vs_next, 0);
        if (lane < 16) {
          const __half kmh = __float2half_rn(m * kmul), ks8 = __float2half_rn(8.0f * sm);
          const __half2 e0 = __half2half2(kmh), e1 = __halves2half2(kmh, ks8), e2 = __half2half2(ks8);
          uint8_t* ext = smem + kop + C::MAIN + (2 * uw + (lane >> 3)) * 256 + (lane & 7) * 16;
          *(uint4*)ext = make_uint4(*(const uint32_t*)&e0, *(const uint32_t*)&e1, *(const uint32_t*)&e2, 0u);
          *(uint4*)(ext + 128) = make_uint4(0u, 0u, 0u, 0u);
        }
        sm100::fence_async_smem();
        sm100::mbar_arrive(&b_kf[st]);
      }
      // ---- the next tile's keys are on their way while the values are unpacked
      if (k + 1 < nt) {
        pg = checked(pg_next);
        load_k(k + 1, pg);
        pg_next = page_of(k + 2);
      }
      if (k > 0) {
        const int v = k - 1, st = v % NKV;
        dead = dead || !sm100::mbar_wait(&b_ve[st], ((v / NKV) & 1) ^ 1, a.flags);
        __syncwarp();
        unpack(C::V + st * C::MAIN, vc, vs_cur, 16);
        sm100::fence_async_smem();
        sm100::mbar_arrive(&b_vf[st]);
        if (k < nt) load_v(k, pg_v);
      }
      vs_cur = vs_next;
      pg_v = pg;
    }
  } else {
    // ------------------------------------------------------------ products
    set_regs_down<C::R_MMA>();
    if (warp == kIssuer && nt > 0) {
      // Unrolled, with the addresses of the steps folded into the descriptors: a step is then issued within the
      // 64 cycles that it takes (128 rows x 128 x 16); in a rolled loop issuing one takes more than 200.
      const uint32_t base = sm100::smem_u32(smem);
      constexpr uint32_t id_s = sm100::idesc_f16(M, KT), id_o = sm100::idesc_f16(M, D) | (1u << 16);   // values: n-major
      bool dead = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        dead = __any_sync(0xffffffffu, dead || !sm100::mbar_wait(bar, parity, a.flags));
        sm100::tc_fence_after();
        return !dead;
      };
      auto scores = [&](int i, int k, bool last) {
        const uint32_t qa = base + C::Q + i * C::OP, ka = base + C::K + (k % NKV) * C::OP;
        const int sl = ns == 2 ? i : (k & 1);
        const uint32_t d = tmem + 128 * sl;
        const uint64_t qd = desc_of(qa, 16, 1024, 2), kd = desc_of(ka, 16, 1024, 2);
        const uint64_t qe = desc_of(qa + C::MAIN, 128, 256, 0), ke = desc_of(ka + C::MAIN, 128, 256, 0);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint64_t off = (uint64_t)((s >> 2) * 1024 + (s & 3) * 2);       // in units of 16 bytes
            sm100::mma_f16(d, qd + off, kd + off, id_s, s > 0 ? 1u : 0u);
          }
          sm100::mma_f16(d, qe, ke, id_s, 1u);
          sm100::mma_commit(&b_s[sl]);
          if (last) sm100::mma_commit(&b_ke[k % NKV]);
        }
        __syncwarp();
      };
      auto sums = [&](int i, int k, bool last) {
        const uint32_t va = base + C::V + (k % NKV) * C::MAIN;
        const uint32_t p = tmem + 128 * (ns == 2 ? i : (k & 1)), d = tmem + 256 + i * D;
        const uint64_t vd = desc_of(va, 16384, 1024, 2);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < KT / 16; ++s) {
            const uint32_t ps = p + 64 * (s >> 2) + prob_cols<FINE>() * (s & 3);
            sm100::mma_f16_ts(d, ps, vd + 128 * s, id_o, (s > 0 || k > 0) ? 1u : 0u);
            if constexpr (FINE) sm100::mma_f16_ts(d, ps + 8, vd + 128 * s, id_o, 1u);
          }
          sm100::mma_commit(&b_o[i]);
          if (last) sm100::mma_commit(&b_ve[k % NKV]);
        }
        __syncwarp();
      };
      if (elect_one()) {
        asm volatile("fence.proxy.async.global;" ::: "memory");
        sm100::mbar_expect_tx(&b_q, ns * C::OP);
        for (int i = 0; i < ns; ++i)
          sm100::bulk_load(smem + C::Q + i * C::OP,
                           plan.q + ((int64_t)u.hs * plan.q_tiles + row_tile(u.tok - u.off, u.row, u.off, sh.tpm) + i) * C::QIMG,
                           C::OP, &b_q);
      }
      __syncwarp();
      if (!wait(&b_q, 0)) sm100::mbar_wait(&b_q, 0, nullptr);      // given up: the copies are waited for once more
      // Scores may not take the place of probabilities before the product that reads those has ended: products
      // of different accumulators are not ordered among each other, so the end is waited for.
      if (ns == 1) {
        for (int k = 0; k < 2 && k < nt && wait(&b_kf[k % NKV], (k / NKV) & 1); ++k) scores(0, k, true);
        for (int k = 0; k < nt && !dead; ++k) {
          if (!wait(&b_p[k & 1], (k >> 1) & 1) || !wait(&b_vf[k % NKV], (k / NKV) & 1)) break;
          sums(0, k, true);
          if (k + 2 < nt) {
            if (!wait(&b_o[0], k & 1) || !wait(&b_kf[k % NKV], ((k + 2) / NKV) & 1)) break;
            scores(0, k + 2, true);
          }
        }
      } else if (wait(&b_kf[0], 0)) {
        // One row tile's sum and next scores, then the other's: so their softmaxes fall into opposite phases,
        // and each has the exponential units to itself.
        scores(0, 0, false);
        scores(1, 0, true);
        for (int k = 0; k < nt && !dead; ++k) {
          for (int i = 0; i < 2; ++i) {
            if (!wait(&b_p[i], k & 1) || !wait(&b_vf[k % NKV], (k / NKV) & 1)) break;
            sums(i % NS, k, i == 1);
            if (k + 1 < nt) {
              if (!wait(&b_o[i % NS], k & 1) || !wait(&b_kf[(k + 1) % NKV], ((k + 1) / NKV) & 1)) break;
              scores(i, k + 1, i == 1);
            }
          }
        }
      }
      // nothing of this block is in flight when it gives its tensor memory back
      if (elect_one()) sm100::mma_commit(&b_fin);
      __syncwarp();
      sm100::mbar_wait(&b_fin, 0, a.flags);
    }
    __syncwarp();
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    sm100::tc_fence_after();
    sm100::tmem_relinquish();
    sm100::tmem_dealloc(tmem, 512);
  }
}

}  // namespace pre
}  // namespace kv4
}  // namespace sq

// Attention of one query a sequence over the paged 4-bit cache.
//
// Mathematics. With q' = q 2^e (a power of two a head, so that fp16 holds it) and
// codes c, the score of token t is s_t (q . c_t) + m_t sum(q), and the output is
// sum_t (p_t s_t) (c_t - 8) + sum_t p_t (m_t + 8 s_t): the tensor cores multiply the
// codes themselves, and the pairs act on scores and probabilities, one token at a time,
// never on coordinates. A code of 4 bits masked out of its word in place is the fp16 subnormal
// c 2^-24 (bits 0-3) or 16 c 2^-24 (bits 4-7) in each half of the word: one AND makes
// two operands, exactly, and the 16 goes into q' or out of the sum. ldmatrix (for the
// values, its transposed form) lays the words out so that the two halves of a word are
// the two neighbours along k that mma.sync wants. The tensor cores cut a product by
// the exponents of its factors, and a subnormal's is that of 2^-14 however small it is:
// against fp16 queries, whose products have 15 bits, the keys' codes are shifted two
// places up first (log-sum-exps of short spans 0.3 times as far from the exact ones, for
// 1.1 of 49.3 us at 16 x 32768 tokens); bf16 queries' have 12.
//
// Softmax: one pass, base 2. Each warp keeps a reference maximum a head, raised
// when a score passes it by more than 2^4 (one vote a tile), and a reference step
// (a power of two over all value steps it has met), so that p s, scaled to at most
// 2^15, keeps fp16's full precision. Up to four query heads a KV head take every other
// column of the product, so that each lane has one head to score; up to eight take all.
//
// Roundings. For an fp16 or float output p s enters the product in two fp16 parts, 22
// bits (with up to four heads the second takes the columns between, with more it is a
// second product), and the 8 comes off the codes before it: a long context's sum is far
// smaller than its terms' common part, and the tensor cores cut what they add. For a
// bf16 output, eight times coarser, one part is enough, and 8 times the sum of the
// rounded p s, which one more product with ones gives, comes off the sum: the rounding
// (half a step, 2^-11) meets at most 8 of the 15 codes. It comes off every sixteen
// tiles: the tensor cores cut units of the sum so far, of which a long context leaves
// little (32768 near-equal weights at head_dim 256: outputs 1.44 times as far from the
// exact ones as their rounding when it comes off at the end, 1.01 times so, for 2 us
// of the 125).
//
// Work. The tiles of all (sequence, KV head) pairs form one line that the resident
// blocks (two an SM) share evenly, whatever the lengths; inside a block tile i goes
// to warp i mod 8. A warp brings its tiles by bulk copies into a ring of its own and
// meets the other warps only where a pair ends, to add up. Pairs cut by a block's
// end leave partial sums, which are joined in order, so that results do not depend on
// timing: by a second, overlapped launch, or, in a decode step of few blocks, where a
// launch costs more than it does, by the block that writes the last of them (the append
// before has cleared the counters for that).
//
// Measured (one B200): 64 x 4096 x 8 KV heads at head_dim 256, two query heads each:
// 125 to 131 us on different GPUs, 4.2 to 4.4 TB/s; 16 x 32768 x 2 at 128, six heads
// each: 50 us, 2.8 TB/s (4 us less with one part and the 8 off the sum, but an output
// half again as far from the exact one; what is left is 4 % over it, as the second part
// is added to the sum of the first and cut with it). 16 warps an SM (128 registers) use
// 56 % of the instruction slots and 56 % of the ALU that takes the codes apart, in
// turns: neither more warps of fewer registers nor two chains of products a tile were
// faster.
#pragma once

#include "kv4_append.cuh"
#include "sm100.cuh"

namespace sq {
namespace kv4 {

struct AttnArgs {
  const int32_t* cu;      // chunks: token offsets of the sequences; NULL: one query a sequence
  const int32_t* start;   // chunks: position of a sequence's first query; decode: see len_off
  int len_off;            // position of the query = start + len_off (-1: start holds lengths)
  int64_t n_tok;
  int64_t max_ctx;        // bound on the attended positions
  int64_t qs_tok, qs_head;
  int n_q, group, window;
  float scale;
  float* lse;
  uint32_t* flags;
  int* done;              // decode: pieces of a pair that are written, at the block it begins in, all 0
};

namespace dec {

constexpr int W = 8;                       // warps of a block
constexpr int kMaxHeads = 8;               // query heads of one pass over a KV head
constexpr float kSlack = 4.0f;             // log2 of what a probability may exceed 1 by
constexpr int kTake = 16;                  // tiles of a warp after which 8 times the weights' sum comes off its sums
constexpr float kTop = 2048.0f;            // 2^11: scale of p s / reference, at most 2^15 with the slack

template <int D> struct Cfg {
  static constexpr int NB = D == 256 ? 1 : 2;             // 16-token blocks of a tile
  static constexpr int TT = 16 * NB;
  static constexpr int STAGE = NB * blk_bytes(D);
  static constexpr int NST = D == 64 ? 4 : 2;             // tiles in a warp's ring
  static constexpr int QROW = 2 * D + 64;                 // bytes of a head's query operand (64 over: conflict-free)
  static constexpr bool QREG = D <= 128;                  // the query operand stays in registers
  static constexpr int MC = D == 64 ? 64 : 128;           // coordinates of a round of the sum over the warps
};

template <int D> struct Smem {
  static constexpr int RING = W * Cfg<D>::NST * Cfg<D>::STAGE;
  static constexpr int MERGE = W * kMaxHeads * Cfg<D>::MC * 4;
  static constexpr int Q = kMaxHeads * Cfg<D>::QROW;
  static constexpr int TOTAL = RING + MERGE + Q;
};

// One partial result: a pass's heads x D sums, then (max, sum) a head.
__host__ __device__ constexpr int part_floats(int d) { return kMaxHeads * (d + 2); }
struct Desc { int parts, row, hsub, pad; };       // parts 0: this block owns no cut pair

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t u) { return __half22float2(*(const __half2*)&u); }

// Two codes less 8: c 2^-24 or (odd nibbles) 16 c 2^-24, exact.
__device__ __forceinline__ uint32_t less_middle(uint32_t c, bool odd) {
  const uint32_t mid = odd ? 0x00800080u : 0x00080008u;
  const __half2 r = __hsub2(*(const __half2*)&c, *(const __half2*)&mid);
  return *(const uint32_t*)&r;
}

// Attended positions [lo, hi) of a row's query; hi = 0 where there is nothing to do.
struct Span { int lo, hi; };
__device__ __forceinline__ Span span_of(const Pool& c, const RopeArgs& r, const AttnArgs& a, int b, uint32_t* flags) {
  const int64_t lim = min(c.cap(), a.max_ctx);
  int64_t n = (int64_t)__ldg(a.start + b) + a.len_off + 1;
  uint32_t bits = 0;
  if (n > lim || n < 0) {
    bits = SQ_FLAG_SEQLEN;
    n = n < 0 ? 0 : lim;
  }
  if (r.table && n > r.n_pos) {
    bits |= SQ_FLAG_ROPE;
    n = 0;
  }
  if (bits && flags) atomicOr(flags, bits);
  Span s;
  s.hi = (int)n;
  s.lo = a.window > 0 && n > a.window ? (int)(n - a.window) : 0;
  return s;
}
template <int TT> __device__ __forceinline__ int tiles_of(Span s) {
  return s.hi > 0 ? (s.hi - 1) / TT - s.lo / TT + 1 : 0;
}

// The line: every pair's tiles (their count rounded up to `unit`) behind `pair`
// empty places, which stand for what a pair costs besides (its query, the sum over
// the warps: about as long as sixteen tiles); `line` places in all, `quota` a block.
constexpr int kPair = 16;
struct Plan {
  int64_t line;
  int quota, unit, pair;
  int row;                 // of the block's first place
  int64_t row_at;          // and where that row begins on the line
};

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) v += red[i];
  return v;
}

template <int TT>
__device__ Plan make_plan(const Pool& c, const RopeArgs& r, const AttnArgs& a, int per_row, int64_t* red) {
  __shared__ int s_row;
  __shared__ int64_t s_at;
  const int tid = threadIdx.x, lane = tid & 31;
  int64_t n = 0, padded = 0;                 // places of a line of either kind
  for (int b = tid; b < c.batch; b += 32 * W) {
    const int t = tiles_of<TT>(span_of(c, r, a, b, nullptr));
    n += t ? t + kPair : 0;
    padded += (t + W - 1) / W * W;
  }
  n = block_sum(n, red) * per_row;
  padded = block_sum(padded, red) * per_row;
  Plan p;
  // Few tiles: a block takes up to eight tiles of one pair, a warp one; no block crosses a pair.
  // Many: equal shares of the line.
  p.unit = padded <= (int64_t)gridDim.x * W ? W : 1;
  p.line = p.unit == W ? padded : n;
  p.quota = p.unit == W ? W : (int)((n + gridDim.x - 1) / gridDim.x);
  p.pair = p.unit == W ? 0 : kPair;
  const int64_t first = (int64_t)blockIdx.x * p.quota;
  if (tid == 0) s_row = -1;
  int64_t carry = 0;
  for (int b0 = 0; b0 < c.batch; b0 += 32 * W) {
    int64_t mine = 0;
    if (b0 + tid < c.batch) {
      const int t = tiles_of<TT>(span_of(c, r, a, b0 + tid, nullptr));
      mine = t ? (int64_t)((t + p.unit - 1) / p.unit * p.unit + p.pair) * per_row : 0;
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) red[tid >> 5] = inc;
    __syncthreads();
    int64_t before = carry;
    for (int i = 0; i < W; ++i) {
      if (i < (tid >> 5)) before += red[i];
      carry += red[i];
    }
    const int64_t at = before + inc - mine;
    if (mine > 0 && at <= first && first < at + mine) {
      s_row = b0 + tid;
      s_at = at;
    }
    if (carry > first) break;
  }
  __syncthreads();
  p.row = s_row;
  p.row_at = s_at;
  return p;
}

// A tile on the line: its pair (sequence, heads) and its place in that.
template <int D>
struct Cursor {
  int row, hsub, tile, nt;        // nt: the pair's tiles, rounded up
  int lo, hi;
  __device__ __forceinline__ void enter(const Pool& c, const RopeArgs& r, const AttnArgs& a, int unit) {
    const Span s = span_of(c, r, a, row, nullptr);
    lo = s.lo;
    hi = s.hi;
    nt = (tiles_of<Cfg<D>::TT>(s) + unit - 1) / unit * unit;
  }
  // Into the pairs behind this one, when its tiles are used up; `place` is the tile's, below `count`.
  __device__ __forceinline__ void carry(const Pool& c, const RopeArgs& r, const AttnArgs& a, const Plan& p, int per_row,
                                        int count, int* place) {
    while (tile >= nt && *place < count) {
      tile -= nt;
      *place += p.pair;
      if (++hsub == per_row) {
        hsub = 0;
        do {
          ++row;
          enter(c, r, a, p.unit);
        } while (nt == 0);
      }
    }
  }
  // First position of the tile.
  __device__ __forceinline__ int first() const { return (lo / Cfg<D>::TT + tile) * Cfg<D>::TT; }
};

// The sum of pieces p0, p0 + step, ... of the pair that block `begin` began, for its hh-th head; a warp's lanes have
// the coordinates 32 i + lane.
template <int D>
__device__ __forceinline__ void join_parts(const float* parts, int begin, int hh, int p0, int step, int n, float* top_out,
                                           float* l_out, float* o) {
  const int lane = threadIdx.x & 31;
  auto slot = [&](int p) { return parts + ((int64_t)2 * (begin + p) + (p == 0 ? 1 : 0)) * part_floats(D); };
  auto ml = [&](int p) { return p < n ? __ldcg((const float2*)(slot(p) + kMaxHeads * D + 2 * hh)) : make_float2(-INFINITY, 0.0f); };
  float top = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
  // a lane a piece: its maximum and sum
  for (int p = p0 + step * lane; p < n; p += 32 * step) top = fmaxf(top, ml(p).x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  for (int q = p0; q < n; q += 32 * step) {
    const float2 m = ml(q + step * lane);
    const float f = m.x == -INFINITY ? (m.y == 0.0f ? 0.0f : 1.0f) : ex2(m.x - top);
    l += f * m.y;
    const int here = min(32, (n - q + step - 1) / step);
#pragma unroll 4
    for (int p = 0; p < here; ++p) {
      const float fp = __shfl_sync(0xffffffffu, f, p);
      const float* src = slot(q + step * p) + hh * D + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(fp, __ldcg(src + 32 * i), o[i]);
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  *top_out = top;
  *l_out = l;
}

template <typename T> __host__ __device__ constexpr bool is_bf16() { return false; }
template <> __host__ __device__ constexpr bool is_bf16<__nv_bfloat16>() { return true; }

// JOIN: the block that writes a pair's last piece joins them (AttnArgs::done); else a kernel behind this one does.
template <typename T, typename TO, int D, bool PAIR, bool JOIN>
__global__ void __launch_bounds__(32 * W, 2)
k_decode4(Pool c, RopeArgs r, const T* __restrict__ q, TO* __restrict__ out, AttnArgs a, int nsub, float* parts,
          Desc* descs) {
  using C = Cfg<D>;
  constexpr int HS = PAIR ? 4 : 8;
  constexpr bool FINE = !is_bf16<TO>();         // weights in two parts
  constexpr int UP = is_bf16<T>() ? 0 : 2;      // places that the keys' codes are shifted up by
  constexpr int NC = D / 32;                    // 16-byte chunks of a code row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[W][C::NST];
  __shared__ uint32_t oks[W][C::NST];
  __shared__ int64_t red[W];
  __shared__ float s_q[kMaxHeads][2];           // a head's score factor, and sum(q') in units of the codes
  __shared__ float s_ml[W][kMaxHeads][4];       // a warp's maximum, sum, sum with the offsets
  __shared__ float s_head[kMaxHeads][4];        // the same of all warps
  __shared__ int s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;
  uint8_t* ring = smem + warp * C::NST * C::STAGE;
  float* merge = (float*)(smem + Smem<D>::RING);
  uint8_t* qop = smem + Smem<D>::RING + Smem<D>::MERGE;
  if (lane == 0) {
    for (int i = 0; i < C::NST; ++i) sm100::mbar_init(&bars[warp][i], 1);
    sm100::fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per_row = c.n_kv * nsub;
  const Plan plan = make_plan<C::TT>(c, r, a, per_row, red);
  asm volatile("griddepcontrol.wait;" ::: "memory");      // a decode step's append must be in the pool,
  asm volatile("fence.proxy.async.global;" ::: "memory"); // and its plain stores before the bulk copies that read them
  // rows with nothing to attend
  for (int b = blockIdx.x; b < c.batch; b += gridDim.x) {
    const Span s = span_of(c, r, a, b, tid == 0 ? a.flags : nullptr);
    if (s.hi > 0) continue;
    for (int i = tid; i < a.n_q * D; i += 32 * W) out[(int64_t)b * a.n_q * D + i] = from_f<TO>(0.0f);
    if (a.lse)
      for (int i = tid; i < a.n_q; i += 32 * W) a.lse[(int64_t)b * a.n_q + i] = -INFINITY;
  }
  const int64_t first = (int64_t)blockIdx.x * plan.quota;
  const int64_t last = min(first + plan.quota, plan.line);
  if (!JOIN && tid == 0) descs[blockIdx.x].parts = 0;
  if (first >= last) return;

  // ---- the warp's copies. Places are counted from the block's first one; a pair's tiles go round the warps.
  const int count = (int)(last - first);
  Cursor<D> ahead;
  ahead.row = plan.row;
  ahead.enter(c, r, a, plan.unit);
  const int64_t in_row = first - plan.row_at;
  ahead.hsub = (int)(in_row / (ahead.nt + plan.pair));
  ahead.tile = (int)(in_row % (ahead.nt + plan.pair)) - plan.pair;
  int seg = 0;                         // the place of the first tile of the pair at hand in this block
  if (ahead.tile < 0) {
    seg = -ahead.tile;
    ahead.tile = 0;
  }
  if (seg >= count) return;
  const int row0 = ahead.row, hsub0 = ahead.hsub, tile0 = ahead.tile;
  const int64_t page_bytes = ((int64_t)c.n_kv << (c.page_shift - 4)) * blk_bytes(D);
  const int in_page = (1 << c.page_shift) - 1;
  int next = seg + warp, t_next = 0;   // the place of the tile to copy next, and its first position
  const int32_t* table = nullptr;      // its sequence's pages, and its head's bytes in a page
  const uint8_t* head = nullptr;
  auto in_pair = [&]() {
    ahead.carry(c, r, a, plan, per_row, count, &next);
    if (next >= count) return;
    t_next = ahead.first() + 16 * lane;
    table = c.table + ahead.row * c.table_stride;
    head = c.pages + ((int64_t)(ahead.hsub / nsub) << (c.page_shift - 4)) * blk_bytes(D);
  };
  ahead.tile += warp;
  in_pair();
  // Lanes below NB: a 16-token block each, its page number asked for a tile before its copy.
  bool pf_has = false;                 // there is one
  int pf_page = -1;                    // -1: nothing of it to copy
  const uint8_t* pf_from = nullptr;
  auto look = [&]() {
    pf_page = -1;
    pf_has = next < count;
    if (lane < C::NB && pf_has && t_next < ahead.hi && t_next + 16 > ahead.lo) {
      const int page = __ldg(table + (t_next >> c.page_shift));
      pf_page = page < 0 ? 0x7fffffff : page;
      pf_from = head + ((t_next & in_page) >> 4) * blk_bytes(D);
    }
    next += W;
    ahead.tile += W;
    t_next += W * C::TT;
    if (ahead.tile >= ahead.nt) in_pair();
  };
  auto issue = [&](int st) {
    const bool ok = pf_page >= 0 && pf_page < c.n_pages;
    if (pf_page >= 0 && !ok) raise(a.flags, SQ_FLAG_PAGE);
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) {
      oks[warp][st] = mask;
      sm100::mbar_expect_tx(&bars[warp][st], __popc(mask) * blk_bytes(D));
    }
    __syncwarp();
    if (ok)
      sm100::bulk_load(ring + st * C::STAGE + lane * blk_bytes(D), pf_from + pf_page * page_bytes, blk_bytes(D),
                       &bars[warp][st]);
  };
  look();
#pragma unroll
  for (int i = 0; i < C::NST - 1; ++i) {
    issue(i);
    look();
  }

  // ---- fragment addresses inside a block
  const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4;
  const int vrow = (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;
  const uint32_t koff = krow * (D / 2) + ((kch ^ swz(krow, D)) << 4);
  const uint32_t voff = v_codes(D) + vrow * (D / 2) + ((vch ^ swz(vrow, D)) << 4);
  const uint32_t ring_u = sm100::smem_u32(ring);

  Cursor<D> at;                                  // the segment (pair) being summed, the same for all warps
  at.row = row0;
  at.enter(c, r, a, plan.unit);
  at.hsub = hsub0;
  at.tile = tile0;
  int stage = 0;
  uint32_t phase = 0;
  bool dead = false;
  int mine = seg + warp;

  while (seg < count) {
    const int seg_end = min(count, seg + (at.nt - at.tile));
    const int pos0 = at.first();                 // the segment's first position
    const int kvh = at.hsub / nsub, h0 = kvh * a.group + (at.hsub % nsub) * HS;
    const int nh = min(HS, (kvh + 1) * a.group - h0);
    // ---- the query operand: D / 8 threads a head
    __syncthreads();
    for (int base = 0; base < kMaxHeads * (D / 8); base += 32 * W) {
      const int i = base + tid, col = i / (D / 8), j = i % (D / 8);
      const int hh = PAIR ? ((col & 1) ? kMaxHeads : col >> 1) : col;      // (odd columns of pairs are empty)
      float x[8];
      if (hh < nh) {
        const T* src = q + (int64_t)at.row * a.qs_tok + (int64_t)(h0 + hh) * a.qs_head;
        unpack8<T>(load8<T>(src + 8 * j), x);
        if (r.table) {
          float y[8];
          const int pi = partner(8 * j, r);
          if (pi != 8 * j) unpack8<T>(load8<T>(src + pi), y);
          rotate8<T>(x, y, 8 * j, r, at.hi - 1);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
      }
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^e with top 2^e in [2^14, 2^15); queries that are zero or not finite are taken as they are. Not below 2^-100,
      // where the score factor, 2^(24 - e), would pass a float's range: queries of 2^116 and above overflow.
      int e2 = 0;
      if (top > 0.0f && top < INFINITY) e2 = max(-100, min(100, 14 - ilogbf(top)));
      const float up = ldexpf(1.0f, e2);
      float sum = 0.0f;
      uint32_t w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // coordinates p and p + 4 are the two halves of nibble p; odd nibbles come times 16
        const __half2 hv = __floats2half2_rn(x[p] * up, x[p + 4] * up);
        const float2 f = __half22float2(hv);
        sum += f.x + f.y;
        const __half2 hs = (p & 1) ? __hmul2(hv, __float2half2_rn(0.0625f)) : hv;
        w[p] = *(const uint32_t*)&hs;
      }
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (col < kMaxHeads) {
        *(uint4*)(qop + col * C::QROW + j * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        if (j == 0 && hh < HS) {
          s_q[hh][0] = a.scale * 1.4426950408889634f * ldexpf(1.0f, 24 - UP - e2);
          s_q[hh][1] = ldexpf(sum, UP - 24);
        }
      }
    }
    __syncthreads();
    // lane (g, cc): column g of the query operand
    const uint8_t* qsrc = qop + g * C::QROW + cc * 16;
    uint4 qf[C::QREG ? NC : 1];
    if constexpr (C::QREG) {
#pragma unroll
      for (int j = 0; j < NC; ++j) qf[j] = *(const uint4*)(qsrc + j * 64);
    }
    constexpr int NHL = PAIR ? 1 : 2;            // heads a lane scores: cc, or 2 cc and 2 cc + 1
    // nref: what is added to a score, minus the maximum referred to (+inf while there is none)
    float fq[NHL], fm[NHL], nref[NHL], lsum[NHL], msum[NHL];
#pragma unroll
    for (int i = 0; i < NHL; ++i) {
      const int hh = PAIR ? cc : 2 * cc + i;
      fq[i] = s_q[hh][0];
      fm[i] = s_q[hh][1];
      nref[i] = INFINITY;
      lsum[i] = msum[i] = 0.0f;
    }
    float sref = 0.0f, sinv = 0.0f;              // reference step, and kTop over it
    float acc[D / 16][4], tot[4];                // sums of p s c, and of the rounded p s
#pragma unroll
    for (int j = 0; j < 4; ++j) tot[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;

    while (mine < seg_end) {
      const int stop = FINE ? seg_end : min(seg_end, mine + kTake * W);
      for (; mine < stop; mine += W) {
        // the next copy goes into the stage that the tile before this one has left
        {
          int st = stage + C::NST - 1;
          st = st >= C::NST ? st - C::NST : st;
          __syncwarp();
          if (!dead && pf_has) {
            issue(st);
            look();
          }
        }
        if (!dead && __any_sync(0xffffffffu, !sm100::mbar_wait(&bars[warp][stage], (phase >> stage) & 1u, a.flags))) {
          // given up: no more copies, but those on their way (of the other stages too) are waited for, with a limit again
          dead = true;
#pragma unroll 1
          for (int i = 0; i < C::NST; ++i) sm100::mbar_wait(&bars[warp][i], (phase >> i) & 1u, nullptr);
        }
        phase ^= 1u << stage;
        const uint32_t sb = ring_u + stage * C::STAGE;
        const uint8_t* sp = ring + stage * C::STAGE;
        const uint32_t okm = dead ? 0u : oks[warp][stage];
        stage = stage + 1 == C::NST ? 0 : stage + 1;
        const int t0 = pos0 + (mine - seg) * C::TT;
        const bool edge = okm != (1u << C::NB) - 1u || t0 < at.lo || t0 + C::TT > at.hi;
        if (okm == 0) continue;
        // ---- scores
        float u[C::NB][2][NHL], t[C::NB][2][NHL], vs[C::NB][2], vm[C::NB][2];
        bool over = false;
#pragma unroll
        for (int n = 0; n < C::NB; ++n) {
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < NC; j += 2) {
            uint32_t w[4];
            ldsm4(sb + n * blk_bytes(D) + (koff ^ (j << 4)), w);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint4 b;
              if constexpr (C::QREG) b = qf[j + k];
              else b = *(const uint4*)(qsrc + (j + k) * 64);
              constexpr uint32_t even = 0x000f000fu << UP, odd = 0x00f000f0u << UP;
              const uint32_t x = w[2 * k] << UP, y = w[2 * k + 1] << UP, xs = w[2 * k] >> (8 - UP), ys = w[2 * k + 1] >> (8 - UP);
              mma(s, x & even, y & even, x & odd, y & odd, b.x, b.y);
              mma(s, xs & even, ys & even, xs & odd, ys & odd, b.z, b.w);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t kw = *(const uint32_t*)(sp + n * blk_bytes(D) + k_pairs(D) + (g + 8 * e) * 4);
            const uint32_t vw = *(const uint32_t*)(sp + n * blk_bytes(D) + v_pairs(D) + (g + 8 * e) * 4);
            const float ks = __uint_as_float(kw << 16), km = __uint_as_float(kw & 0xffff0000u);
            vs[n][e] = __uint_as_float(vw << 16);
            vm[n][e] = fmaf(8.0f, vs[n][e], __uint_as_float(vw & 0xffff0000u));
#pragma unroll
            for (int i = 0; i < NHL; ++i) {
              u[n][e][i] = fmaf(ks, s[2 * e + i], km * fm[i]);
              t[n][e][i] = fmaf(u[n][e][i], fq[i], nref[i]);
            }
          }
        }
        if (edge) {
#pragma unroll
          for (int n = 0; n < C::NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int p = t0 + 16 * n + 8 * e + g;
              if (p < at.lo || p >= at.hi || !((okm >> n) & 1u)) {
                vs[n][e] = vm[n][e] = 0.0f;
#pragma unroll
                for (int i = 0; i < NHL; ++i) u[n][e][i] = t[n][e][i] = -INFINITY;
              }
            }
        }
        // ---- the references
#pragma unroll
        for (int n = 0; n < C::NB; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            over |= vs[n][e] > sref;
#pragma unroll
            for (int i = 0; i < NHL; ++i) over |= t[n][e][i] > kSlack;
          }
        if (__any_sync(0xffffffffu, over)) {
          float st = 0.0f;
#pragma unroll
          for (int n = 0; n < C::NB; ++n) st = fmaxf(st, fmaxf(vs[n][0], vs[n][1]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) st = fmaxf(st, __shfl_xor_sync(0xffffffffu, st, o));
          float down = 1.0f;
          if (st > sref) {
            // the power of two at or above the step, kept where its reciprocal stays a float
            const float ns = fminf(pow2_up(st), 0x1p126f);
            down = sref / ns;
            sref = ns;
            sinv = kTop / ns;
          }
#pragma unroll
          for (int i = 0; i < NHL; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < C::NB; ++n) mx = fmaxf(mx, fmaxf(u[n][0][i], u[n][1][i]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx *= fq[i];
            float f = 1.0f;
            if (mx > -nref[i]) {
              f = ex2(-nref[i] - mx);            // 0 the first time
              nref[i] = -mx;
              lsum[i] *= f;
              msum[i] *= f;
            }
            f *= down;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (PAIR || (j & 1) == i) tot[j] *= f;
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (PAIR || (j & 1) == i) acc[m][j] *= f;
#pragma unroll
            for (int n = 0; n < C::NB; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) t[n][e][i] = u[n][e][i] == -INFINITY ? -INFINITY : fmaf(u[n][e][i], fq[i], nref[i]);
          }
        }
        // ---- probabilities, and the values' product
#pragma unroll
        for (int n = 0; n < C::NB; ++n) {
          uint32_t b[2], b2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float ps[2] = {0.0f, 0.0f};
            const float step = vs[n][e] * sinv;
#pragma unroll
            for (int i = 0; i < NHL; ++i) {
              const float p = ex2(t[n][e][i]);
              lsum[i] += p;
              msum[i] = fmaf(p, vm[n][e], msum[i]);
              ps[i] = p * step;
            }
            if constexpr (FINE && PAIR) {
              const float hi = __half2float(__float2half_rn(ps[0]));
              b[e] = movm(pack_h2(hi, ps[0] - hi));
            } else {
              const uint32_t hi = pack_h2(ps[0], ps[1]);
              b[e] = movm(hi);
              if constexpr (FINE) {
                const float2 f = unpack_h2(hi);
                b2[e] = movm(pack_h2(ps[0] - f.x, ps[1] - f.y));
              }
            }
          }
          if constexpr (!FINE) mma(tot, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, b[0], b[1]);
#pragma unroll
          for (int j = 0; j < NC; j += 2) {
            uint32_t w[4];
            ldsm4t(sb + n * blk_bytes(D) + (voff ^ (j << 4)), w);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const uint32_t mask = (p & 1) ? 0x00f000f0u : 0x000f000fu;
              const int sh = p < 2 ? 0 : 8;
              uint32_t a0 = (w[0] >> sh) & mask, a1 = (w[1] >> sh) & mask, a2 = (w[2] >> sh) & mask, a3 = (w[3] >> sh) & mask;
              if constexpr (FINE) {
                a0 = less_middle(a0, p & 1);
                a1 = less_middle(a1, p & 1);
                a2 = less_middle(a2, p & 1);
                a3 = less_middle(a3, p & 1);
              }
              mma(acc[2 * j + p], a0, a1, a2, a3, b[0], b[1]);
              if constexpr (FINE && !PAIR) mma(acc[2 * j + p], a0, a1, a2, a3, b2[0], b2[1]);
            }
          }
        }
      }
      if constexpr (!FINE) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[m][x] = fmaf(tot[x], (m & 1) ? -0x1p-17f : -0x1p-21f, acc[m][x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) tot[x] = 0.0f;
      }
    }

    // ---- the segment's sums of the eight warps
#pragma unroll
    for (int i = 0; i < NHL; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        lsum[i] += __shfl_xor_sync(0xffffffffu, lsum[i], o);
        msum[i] += __shfl_xor_sync(0xffffffffu, msum[i], o);
      }
      if (g == 0) {
        float* ml = s_ml[warp][PAIR ? cc : 2 * cc + i];
        ml[0] = -nref[i];
        ml[1] = lsum[i];
        ml[2] = msum[i];
      }
    }
    __syncthreads();
    float fw[NHL];
#pragma unroll
    for (int i = 0; i < NHL; ++i) {
      const int hh = PAIR ? cc : 2 * cc + i;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_ml[w][hh][0]);
      fw[i] = nref[i] == INFINITY ? (lsum[i] == 0.0f ? 0.0f : 1.0f) : ex2(-nref[i] - top);
      fw[i] *= sref / kTop;
    }
    if (tid < 8 * HS) {                          // a head's maximum, sum and shared part: eight lanes a head, a warp's each
      const float* ml = s_ml[tid & 7][tid >> 3];
      float top = ml[0];
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float f = ml[0] == -INFINITY ? (ml[1] == 0.0f ? 0.0f : 1.0f) : ex2(ml[0] - top);
      float l = f * ml[1], m = f * ml[2];
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        m += __shfl_xor_sync(0xffffffffu, m, o);
      }
      if ((tid & 7) == 0) {
        s_head[tid >> 3][0] = top;
        s_head[tid >> 3][1] = l;
        s_head[tid >> 3][2] = m;
      }
    }
    const bool starts = at.tile == 0, ends = seg + (at.nt - at.tile) <= count;
    float* slot = parts + ((int64_t)2 * blockIdx.x + (starts ? 1 : 0)) * part_floats(D);
    constexpr int MC = Cfg<D>::MC;               // coordinates of a round
#pragma unroll
    for (int r0 = 0; r0 < D; r0 += MC) {
      if (r0 > 0) __syncthreads();
#pragma unroll
      for (int jr = r0 / 64; jr < (r0 + MC) / 64; ++jr)
        // 64 coordinates: 64 jr + 4 g + p, and 32 further
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < NHL; ++i) {
            const int hh = PAIR ? cc : 2 * cc + i;
            float4 o4;
            float* o = (float*)&o4;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const float* x = acc[4 * jr + p];
              const float v = FINE && PAIR ? x[2 * half] + x[2 * half + 1] : x[2 * half + i], up = (p & 1) ? 0x1p20f : 0x1p24f;
              o[p] = v * up * fw[i];
            }
            *(float4*)(merge + (warp * HS + hh) * MC + 64 * jr - r0 + 32 * half + 4 * g) = o4;
          }
      __syncthreads();
      for (int i = tid; i < nh * (MC / 4); i += 32 * W) {
        const int hh = i / (MC / 4), x = (i % (MC / 4)) * 4, dim = r0 + x;
        const float l = s_head[hh][1], m = s_head[hh][2];
        float4 o = make_float4(m, m, m, m);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 y = *(const float4*)(merge + (w * HS + hh) * MC + x);
          o.x += y.x;
          o.y += y.y;
          o.z += y.z;
          o.w += y.w;
        }
        if (starts && ends) {
          const int64_t at_out = (int64_t)at.row * a.n_q + h0 + hh;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          TO y[4] = {from_f<TO>(o.x * inv), from_f<TO>(o.y * inv), from_f<TO>(o.z * inv), from_f<TO>(o.w * inv)};
          if (sizeof(TO) == 2) *(uint2*)(out + at_out * D + dim) = *(const uint2*)y;
          else *(uint4*)(out + at_out * D + dim) = *(const uint4*)y;
          if (a.lse && dim == 0) a.lse[at_out] = l == 0.0f ? -INFINITY : (s_head[hh][0] + log2f(l)) * 0.69314718055994531f;
        } else {
          *(float4*)(slot + hh * D + dim) = o;
          if (dim == 0) {
            slot[kMaxHeads * D + 2 * hh] = s_head[hh][0];
            slot[kMaxHeads * D + 2 * hh + 1] = l;
          }
        }
      }
    }
    if (!starts || !ends) {
      const int64_t begin = first + seg - at.tile;     // the pair's first place
      const int b0 = (int)(begin / plan.quota), pieces = (int)((begin + at.nt - 1) / plan.quota) - b0 + 1;
      if constexpr (!JOIN) {
        if (starts && tid == 0) descs[blockIdx.x] = Desc{pieces, at.row, at.hsub, 0};
      } else {
        // the block that writes the last piece joins them all, a warp a head
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(a.done + b0, 1) == pieces - 1;
        __syncthreads();
        if (s_last && warp < nh) {
          __threadfence();
          float top, l, o[D / 32];
          join_parts<D>(parts, b0, warp, 0, 1, pieces, &top, &l, o);
          const int64_t at_out = (int64_t)at.row * a.n_q + h0 + warp;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) out[at_out * D + 32 * i + lane] = from_f<TO>(l == 0.0f ? 0.0f : o[i] * inv);
          if (a.lse && lane == 0) a.lse[at_out] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
        }
      }
    }
    // ---- the next pair
    seg = seg_end + plan.pair;
    mine += plan.pair;
    if (seg < count) {
      at.tile = 0;
      if (++at.hsub == per_row) {
        at.hsub = 0;
        do {
          ++at.row;
          at.enter(c, r, a, plan.unit);
        } while (at.nt == 0);
      }
    }
  }
}

// Joins the partial sums of pairs that several blocks of k_decode4 share: block (i, h)
// those of the pair that block i began, for its h-th head.
template <typename TO, int D>
__global__ void __launch_bounds__(256)
k_join4(const float* __restrict__ parts, const Desc* __restrict__ descs, TO* __restrict__ out, AttnArgs a, int nsub,
        int hs) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Desc ds = descs[blockIdx.x];
  if (ds.parts == 0) return;
  const int kvh = ds.hsub / nsub, hh = blockIdx.y, h = kvh * a.group + (ds.hsub % nsub) * hs + hh;
  if (hh >= hs || h >= (kvh + 1) * a.group) return;
  __shared__ float s_m[8], s_l[8];
  __shared__ float s_o[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float top, l, o[D / 32];
  join_parts<D>(parts, blockIdx.x, hh, warp, 8, ds.parts, &top, &l, o);
  if (lane == 0) {
    s_m[warp] = top;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s_o[warp][32 * i + lane] = o[i];
  __syncthreads();
  const int x = threadIdx.x;
  if (x >= D) return;
  float all = -INFINITY, sum = 0.0f, v = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) all = fmaxf(all, s_m[w]);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = s_m[w] == -INFINITY ? (s_l[w] == 0.0f ? 0.0f : 1.0f) : ex2(s_m[w] - all);
    sum = fmaf(f, s_l[w], sum);
    v = fmaf(f, s_o[w][x], v);
  }
  const int64_t at = (int64_t)ds.row * a.n_q + h;
  out[at * D + x] = from_f<TO>(sum == 0.0f ? 0.0f : v / sum);
  if (a.lse && x == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (all + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace dec
}  // namespace kv4
}  // namespace sq

"""The paged 4-bit cache on the GPU against its oracle (float64).

What the cache holds is compared bit for bit: the rotation, the pair and the codes are defined operation
by operation (include/sq.h). Attention is compared under a bound that is added up per output value, in
units of the roundings that a kernel may make:

* score: the codes and the query (rounded to its type) are exact factors of exact products; a float sum of d
  of them, scaled, is off by at most delta = (d + 16) 2^-24 scale (s sum |q_i| c_i + |m| sum |q_i|), to which
  base-2 exponentials add 2^-20 of relative error: an error eps = delta + 2^-20 in every exponent;
* probabilities times value steps may be rounded to fp16 (half a step is 2^-11) against codes centred on 8:
  2^-11 sum_t p_t s_t max(|c_t - 8|, 1/2), plus fp16's smallest steps, at most 2^-30 of the largest s;
* both factors of the softmax (numerator, denominator): 2 eps sum_t p_t |x_t|;
* the output's own rounding: finfo(type).eps / 2 relative.
"""

import math

import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from compressed_attention_head_b200 import sq  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def rounder(dtype):
    return lambda y: torch.from_numpy(np.ascontiguousarray(y, dtype=np.float32)).to(dtype).float().numpy()


def make_table(need, seed, spare=2, per_row=None, shared=()):
    """(page table int32 [batch, per_row] with -1 past each sequence, pages in all)."""
    total = sum(need) + spare
    perm = np.random.default_rng(seed).permutation(total)
    table = np.full((len(need), per_row or max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    for b, src, p in shared:
        table[b, p] = table[src, p]
    return table, total


def random_pool(n_pages, n_kv, page, d, seed, device="cuda"):
    """A pool of random codes and pairs s in about 2^-4..2^0, m in about -8..8."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    p = torch.randint(0, 256, (n_pages, n_kv, page // 16, 16 * d + 128), generator=g, dtype=torch.uint8)
    shape = (n_pages, n_kv, page // 16, 32)
    s = (torch.rand(shape, generator=g) * 0.9 + 0.07).to(BF16)
    m = (torch.randn(shape, generator=g) * 0.5 - 7.5 * s.float()).to(BF16)
    p[..., 16 * d:] = torch.stack([s, m], -1).contiguous().view(torch.uint8).reshape(*shape[:3], 128)
    return p.to(device)


def rows_of(pool_np, table, b, head, n, page, side):
    got = [kv4.load(pool_np, table[b, t // page], head, t % page, side) for t in range(n)]
    d = (pool_np.shape[-1] - 128) // 16
    codes = np.stack([x[0] for x in got]) if n else np.zeros((0, d), np.uint8)
    return codes, np.array([x[1] for x in got], np.uint32), np.array([x[2] for x in got], np.uint32)


def check_attention(out, lse, q, pos, pool, table, page, n_q, n_kv, d, dtype, rope=None, inter=False, window=0,
                    scale=None, skip=None):
    """out [tokens, n_q, d], lse [tokens, n_q], q [tokens, n_q, d]; pos: list of (sequence, position) per token."""
    scale = scale or 1.0 / math.sqrt(d)
    pool_np, out, lse = pool.cpu().numpy(), out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
    step = torch.finfo(dtype).eps / 2
    q = q.float().cpu().numpy()
    cache = {}
    worst = 0.0
    for i, (b, p) in enumerate(pos):
        if b < 0:
            continue
        qr = kv4.rotate(q[i], rope, max(p, 0), inter, rounder(Q_TYPE[0])).astype(np.float64)
        lo = max(0, p - window + 1) if window else 0
        for h in range(n_q):
            g = h // (n_q // n_kv)
            key = (b, g)
            if key not in cache:
                n = max([pp for bb, pp in pos if bb == b]) + 1
                cache[key] = [rows_of(pool_np, table, b, g, n, page, side) for side in (0, 1)]
            (kc, ks, km), (vc, vs, vm) = cache[key]
            sel = np.arange(lo, p + 1) if p >= 0 else np.arange(0)
            if skip is not None:
                sel = sel[[t // page not in skip.get(b, ()) for t in sel]] if len(sel) else sel
            keys, vals = kv4.values(kc[sel], ks[sel], km[sel]), kv4.values(vc[sel], vs[sel], vm[sel])
            s64, m64, v64 = (kv4.bf16_value(x[sel]).astype(np.float64) for x in (ks, km, vs))
            o, l, spread = kv4.attend(qr[h], keys, vals, scale, v64[:, None] * np.maximum(np.abs(vc[sel] - 8.0), 0.5))
            if len(sel) == 0:
                assert not out[i, h].any() and (lse is None or lse[i, h] == -math.inf)
                continue
            aq = np.abs(qr[h])
            delta = float(((d + 16) * 2.0 ** -24 * scale * (s64 * (kc[sel] @ aq) + np.abs(m64) * aq.sum())).max())
            eps = delta + 2.0 ** -20
            _, _, size = kv4.attend(qr[h], keys, vals, scale, np.abs(vals))
            bound = step * np.abs(o) + 2.0 ** -11 * spread + 2.0 ** -30 * v64.max() + 2 * eps * size + 1e-30
            err = np.abs(out[i, h] - o)
            worst = max(worst, float((err / bound).max()))
            assert np.all(err <= bound), (i, b, p, h, float((err / bound).max()))
            if lse is not None:
                assert abs(lse[i, h] - l) <= eps + 2.0 ** -22 * abs(l) + 2.0 ** -22, (i, h, lse[i, h], l)
    return worst


Q_TYPE = [F16]


# ------------------------------------------------------------------ append and read
def append_oracle(pool_np, table, page, k, v, start, cu, rope, inter, dtype):
    for b in range(len(start)):
        lo, hi = (cu[b], cu[b + 1]) if cu is not None else (b, b + 1)
        for i in range(lo, hi):
            p = start[b] + i - lo
            kr = kv4.rotate(k[i].float().numpy(), rope, p, inter, rounder(dtype))
            for side, x in ((0, kr), (1, v[i].float().numpy())):
                c, sb, mb = kv4.quantize(x)
                for h in range(x.shape[0]):
                    kv4.store(pool_np, table[b, p // page], h, p % page, side, c[h], sb[h], mb[h])


@pytest.mark.parametrize("d,dtype,page,n_kv,rot,inter", [
    (64, F16, 16, 1, 64, False), (64, BF16, 32, 3, 32, True), (128, F16, 16, 2, 128, False), (128, BF16, 64, 1, 64, False),
    (128, F32, 16, 2, 128, True), (256, BF16, 16, 2, 256, False), (256, F16, 32, 1, 16, True), (256, F32, 128, 2, 0, False)])
def test_append_writes_the_defined_bytes_and_nothing_else(d, dtype, page, n_kv, rot, inter):
    start, cu = [5, 0, 40, 17], [0, 23, 23, 24, 61]               # an empty sequence, a single token, a padded tail
    n_tok = 66
    g = torch.Generator().manual_seed(d + page)
    qkv = torch.randn(n_tok, 3 * n_kv * d + 8, generator=g) * torch.exp(torch.randn(n_tok, 1, generator=g))
    qkv = qkv.to(dtype)
    k, v = (qkv[:, i * n_kv * d:(i + 1) * n_kv * d].unflatten(1, (n_kv, d)) for i in (1, 2))
    table, total = make_table([-(-(s + b - a) // page) for s, a, b in zip(start, cu, cu[1:])], 3)
    pool = torch.randint(0, 256, (total, n_kv, page // 16, 16 * d + 128), generator=g, dtype=torch.uint8)
    want = pool.numpy().copy()
    rope = kv4.rope_table(64, rot) if rot else None
    append_oracle(want, table, page, k, v, start, cu, rope, inter, dtype)
    dev = qkv.cuda()
    kd, vd = (dev[:, i * n_kv * d:(i + 1) * n_kv * d].unflatten(1, (n_kv, d)) for i in (1, 2))
    cache = sq.PagedKV4(pool.cuda(), torch.from_numpy(table).cuda(), n_kv, d, page)
    st, cud = torch.tensor(start, dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq.sq_kv4_append(cache, kd, vd, st, cud, rope=sq.Rope(torch.from_numpy(rope).cuda(), inter) if rot else None,
                     flags=flags)
    assert flags.item() == 0
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    ko = torch.full((n_tok, n_kv, d), 7.0, device="cuda", dtype=dtype)
    vo = torch.full((n_kv, n_tok, d), 7.0, device="cuda", dtype=dtype).transpose(0, 1)       # head-major rows
    sq.sq_kv4_read(cache, st, cud, ko, vo, flags)
    assert flags.item() == 0
    for b in range(4):
        for i in range(cu[b], cu[b + 1]):
            p = start[b] + i - cu[b]
            for side, got in ((0, ko), (1, vo)):
                for h in range(n_kv):
                    c, sb, mb = kv4.load(want, table[b, p // page], h, p % page, side)
                    x = torch.from_numpy(kv4.values(c, np.uint32(sb), np.uint32(mb))).float().to(dtype)
                    assert torch.equal(got[i, h].cpu(), x)
    assert (ko[cu[-1]:] == 7).all() and (vo[cu[-1]:] == 7).all()


def test_append_of_values_at_borders_and_not_finite():
    d, page = 64, 16
    g = torch.Generator().manual_seed(0)
    rows = [torch.zeros(d), torch.full((d,), -3.3), torch.arange(d) * 0.5, torch.arange(d) % 16 + 0.5 * (torch.arange(d) % 2),
            torch.randn(d, generator=g) * 1e-38, torch.randn(d, generator=g) * 1e38, 1000 + torch.randn(d, generator=g) * 1e-3,
            torch.cat([torch.tensor([math.inf]), torch.ones(d - 1)]), torch.cat([torch.tensor([math.nan]), torch.ones(d - 1)]),
            torch.cat([torch.tensor([-math.inf]), torch.ones(d - 1)]), torch.tensor([3.4e38, -3.4e38]).repeat(d // 2),
            torch.tensor([1e-45, 0.0]).repeat(d // 2), -torch.rand(d, generator=g)]
    x = torch.stack([r.float() for r in rows])[:, None]
    n = len(rows)
    for dtype in (F32, BF16, F16):
        y = x.to(dtype)
        table, total = make_table([1], 0)
        cache = sq.alloc_kv4(total, 1, d, page, torch.from_numpy(table).cuda())
        want = cache.pages.cpu().numpy().copy()
        append_oracle(want, table, page, y, y, [0], [0, n], None, False, dtype)
        sq.sq_kv4_append(cache, y.cuda(), y.cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                         torch.tensor([0, n], dtype=torch.int32).cuda())
        assert np.array_equal(cache.pages.cpu().numpy(), want), dtype


def test_append_skips_and_flags_what_it_cannot_place():
    d, page, n_kv = 128, 16, 1
    k = torch.randn(6, n_kv, d, device="cuda", dtype=F16)
    rope = sq.Rope(sq.rope_table(40, d))
    table = torch.tensor([[0, 1], [7, 1], [-1, 2], [3, 3], [4, 5], [5, 4]], dtype=torch.int32, device="cuda")
    start = torch.tensor([32, 3, 1, -1, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    want = {0: sq.SQ_FLAG_CAPACITY, 1: sq.SQ_FLAG_PAGE, 2: sq.SQ_FLAG_PAGE, 3: sq.SQ_FLAG_CAPACITY, 4: 0,
            5: sq.SQ_FLAG_CAPACITY}
    for row, bit in want.items():
        cache = sq.alloc_kv4(6, n_kv, d, page, table[row:row + 1])
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        sq.sq_kv4_append(cache, k[:1], k[:1], start[row:row + 1].clone(), rope=rope, flags=flags)
        assert flags.item() == bit
        assert bool(cache.pages.any()) == (bit == 0)
    cache = sq.alloc_kv4(6, n_kv, d, page, torch.arange(4, dtype=torch.int32, device="cuda")[None])
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    sq.sq_kv4_append(cache, k, k, torch.tensor([37], dtype=torch.int32, device="cuda"), cu, rope=rope, flags=flags)
    assert flags.item() == sq.SQ_FLAG_ROPE                          # positions 40.. have no row in the table
    ko, vo = torch.full_like(k, 9.0), torch.full_like(k, 9.0)
    sq.sq_kv4_read(cache, torch.tensor([37], dtype=torch.int32, device="cuda"), cu, ko, vo)
    assert not (vo[:3] == 9).all(-1).any() and not vo[3:].any()


def test_pools_beyond_four_gigabytes():
    d, page, n_kv = 128, 128, 8
    n_pages = (1 << 32) // sq.sq_kv4_page_bytes(n_kv, d, page) + 40
    pages = torch.empty(n_pages, n_kv, page // 16, 16 * d + 128, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[n_pages - 1, 3], [n_pages - 2, n_pages - 3]], dtype=torch.int32, device="cuda")
    cache = sq.PagedKV4(pages, table, n_kv, d, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(300, n_kv, d, generator=g, device="cuda").to(F16) for _ in range(2))
    cu = torch.tensor([0, 150, 300], dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    sq.sq_kv4_append(cache, k, v, start, cu)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    sq.sq_kv4_read(cache, start, cu, ko, vo)
    for x, y in ((k, ko), (v, vo)):
        span = x.float().amax(-1) - x.float().amin(-1)
        assert ((x.float() - y.float()).abs().amax(-1) <= span / 30 * 1.05 + 0.01).all()
    lens = torch.tensor([150, 150], dtype=torch.int32, device="cuda")
    q = torch.randn(2, n_kv, d, generator=g, device="cuda").to(F16)
    out = torch.empty(2, n_kv, d, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_workspace(2, n_kv, n_kv, d, 150), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_decode(cache, lens, q, 0.0, out, 150, ws)
    s = torch.einsum("bhd,bthd->bht", q.double(), ko.double().view(2, 150, n_kv, d)) / math.sqrt(d)
    ref = torch.einsum("bht,bthd->bhd", s.softmax(-1), vo.double().view(2, 150, n_kv, d))
    assert (out - ref).abs().max() < 5e-3


# ------------------------------------------------------------------ attention of single tokens
def decode_case(d, group, n_kv, dtype, out_dtype, page, lens, window=0, rot=0, inter=False, seed=0, max_ctx=None,
                skip=None, poison=False, q_scale=1.0):
    Q_TYPE[0] = dtype
    batch = len(lens)
    table, total = make_table([-(-n // page) for n in lens], seed)
    pool = random_pool(total, n_kv, page, d, seed)
    if poison:                                  # 0xff bytes (NaN pairs) in every place past the sequences' ends
        used = torch.zeros(total, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(n):
                used[table[b, t // page], t % page] = True
        pn = pool.view(total, n_kv, page // 16, 16 * d + 128)
        bad = ~used.view(total, page // 16, 16)
        pairs = pn[..., 16 * d:].view(torch.int32).view(total, n_kv, page // 16, 2, 16)
        pairs.masked_fill_(bad[:, None, :, None].cuda(), -1)
        for side in (0, 1):
            rows = pn[..., side * 8 * d:(side + 1) * 8 * d].view(total, n_kv, page // 16, 16, d // 2)
            rows.masked_fill_(bad[:, None, :, :, None].cuda(), 255)
    g = torch.Generator().manual_seed(seed + 1)
    n_q = group * n_kv
    wide = (torch.randn(batch, n_q + 2, d, generator=g) * q_scale).to(dtype).cuda()
    q = wide[:, 1:1 + n_q]
    rope = kv4.rope_table(max(lens + [1]), rot) if rot else None
    tab = torch.from_numpy(table).cuda()
    if skip:
        for b, ps in skip.items():
            for p in ps:
                tab[b, p] = total + 5
    cache = sq.PagedKV4(pool, tab, n_kv, d, page)
    max_ctx = max_ctx or max(lens + [1])
    out = torch.full((batch, n_q, d), 3.0, dtype=out_dtype, device="cuda")
    lse = torch.full((batch, n_q), 3.0, device="cuda")
    ws = torch.full((sq.sq_kv4_attn_workspace(batch, n_q, n_kv, d, max_ctx),), 255, dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq.sq_kv4_attn_decode(cache, torch.tensor(lens, dtype=torch.int32).cuda(), q, 0.0, out, max_ctx, ws,
                          rope=sq.Rope(torch.from_numpy(rope).cuda(), inter) if rot else None, window=window, lse=lse,
                          flags=flags)
    assert flags.item() == (sq.SQ_FLAG_PAGE if skip else 0)
    return check_attention(out, lse, q, [(b, n - 1) for b, n in enumerate(lens)], pool, table, page, n_q, n_kv, d,
                           out_dtype, rope, inter, window, skip=skip)


LENS = [1, 0, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,dtype,out_dtype,page", [(1, F16, F16, 16), (3, BF16, BF16, 32), (4, F16, F32, 64),
                                                        (5, BF16, F16, 16), (8, F16, BF16, 128), (11, BF16, F32, 32)])
def test_decode_lengths(d, group, dtype, out_dtype, page):
    decode_case(d, group, 2, dtype, out_dtype, page, LENS, rot=d if group % 2 else 0, inter=group == 3, poison=True)


@pytest.mark.parametrize("d,group,lens,window", [(128, 4, [1300, 700, 5, 0, 2049], 0), (64, 2, [3001], 0), (256, 2, [900, 1500], 0),
                                                 (128, 6, [700, 40, 1], 33), (64, 1, [500, 16], 1), (256, 8, [300, 257], 128),
                                                 (128, 1, [5000], 0), (128, 16, [800, 90], 0)])
def test_decode_longer_and_windows(d, group, lens, window):
    decode_case(d, group, 1, BF16 if group % 2 else F16, F16, 16 if window else 32, lens, window=window, rot=64, seed=4)


@pytest.mark.parametrize("q_scale", [1e-4, 30.0, 2000.0])
def test_decode_small_and_large_queries(q_scale):
    decode_case(128, 4, 1, BF16, F16, 16, [70, 300], q_scale=q_scale)


def test_decode_leaves_pages_outside_the_pool_out():
    decode_case(128, 4, 2, F16, F32, 16, [100, 40, 16], skip={0: (0, 3), 2: (0,)})
    decode_case(64, 2, 1, F16, F32, 64, [300, 70], skip={0: (1,), 1: (1,)})


def small_cache(d=128, n_kv=1, page=16, tokens=64, batch=1, seed=0):
    need = -(-tokens // page)
    table, total = make_table([need] * batch, seed)
    return sq.PagedKV4(random_pool(total, n_kv, page, d, seed), torch.from_numpy(table).cuda(), n_kv, d, page), table


def test_decode_cuts_and_flags_lengths():
    cache, _ = small_cache()
    ws = torch.empty(sq.sq_kv4_attn_workspace(1, 4, 1, 128, 64), dtype=torch.uint8, device="cuda")
    q = torch.randn(1, 4, 128, device="cuda", dtype=F16)
    outs = {}
    for n, ctx, bit in ((64, 64, 0), (65, 80, sq.SQ_FLAG_SEQLEN), (2 ** 31 - 1, 80, sq.SQ_FLAG_SEQLEN), (30, 30, 0),
                        (64, 30, sq.SQ_FLAG_SEQLEN), (-1, 64, sq.SQ_FLAG_SEQLEN), (-2 ** 31, 64, sq.SQ_FLAG_SEQLEN)):
        out, flags = torch.full((1, 4, 128), 9.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        sq.sq_kv4_attn_decode(cache, torch.tensor([n], dtype=torch.int32, device="cuda"), q, 0.0, out, ctx, ws, flags=flags)
        assert flags.item() == bit, n
        outs[n, ctx] = out
    assert torch.equal(outs[65, 80], outs[64, 64]) and torch.equal(outs[2 ** 31 - 1, 80], outs[64, 64])
    assert torch.equal(outs[64, 30], outs[30, 30])
    assert not outs[-1, 64].any() and not outs[-2 ** 31, 64].any()
    rope = sq.Rope(sq.rope_table(40, 128))
    out, lse = torch.full((1, 4, 128), 9.0, device="cuda"), torch.zeros(1, 4, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq.sq_kv4_attn_decode(cache, torch.tensor([41], dtype=torch.int32, device="cuda"), q, 0.0, out, 64, ws, rope=rope, lse=lse,
                          flags=flags)
    assert flags.item() == sq.SQ_FLAG_ROPE and not out.any() and (lse == -math.inf).all()


def test_not_finite_tokens_reach_only_the_rows_that_attend_them():
    cache, table = small_cache(tokens=64, batch=2)
    k = torch.randn(1, 1, 128, device="cuda", dtype=F16)
    k[0, 0, 5] = math.nan
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    row0 = sq.PagedKV4(cache.pages, cache.table[:1], 1, 128, 16)
    q = torch.randn(2, 4, 128, device="cuda", dtype=F16)
    ws = torch.empty(sq.sq_kv4_attn_workspace(2, 4, 1, 128, 64), dtype=torch.uint8, device="cuda")
    for kk, vv in ((k, torch.zeros_like(k)), (torch.zeros_like(k), k)):
        sq.sq_kv4_append(row0, kk, vv, one(40))
        for n, nan in ((40, False), (41, True), (64, True)):
            out = torch.empty(2, 4, 128, device="cuda")
            sq.sq_kv4_attn_decode(cache, torch.tensor([n, 64], dtype=torch.int32, device="cuda"), q, 0.0, out, 64, ws)
            assert bool(torch.isnan(out[0]).all()) == nan and not torch.isnan(out[1]).any()
            out = torch.empty(2, 4, 128, device="cuda")
            sq.sq_kv4_attn_decode(cache, torch.tensor([n, 64], dtype=torch.int32, device="cuda"), q, 0.0, out, 64, ws, window=8)
            assert bool(torch.isnan(out[0]).all()) == (n == 41) and not torch.isnan(out[1]).any()


# ------------------------------------------------------------------ chunks of queries
def prefill_case(d, group, n_kv, dtype, out_dtype, page, start, new, window=0, rot=0, inter=False, seed=0, tail=3):
    Q_TYPE[0] = dtype
    table, total = make_table([-(-(s + n) // page) for s, n in zip(start, new)], seed)
    pool = random_pool(total, n_kv, page, d, seed)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n_tok, n_q = int(cu[-1]) + tail, group * n_kv
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(n_tok, n_q, d, generator=g).to(dtype).cuda()
    rope = kv4.rope_table(max(s + n for s, n in zip(start, new)) + 1, rot) if rot else None
    cache = sq.PagedKV4(pool, torch.from_numpy(table).cuda(), n_kv, d, page)
    out = torch.full((n_tok, n_q, d), 3.0, dtype=out_dtype, device="cuda")
    lse = torch.full((n_tok, n_q), 3.0, device="cuda")
    ws = torch.full((sq.sq_kv4_attn_prefill_workspace(len(new), n_q, n_kv, d, n_tok),), 255, dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq.sq_kv4_attn_prefill(cache, torch.tensor(start, dtype=torch.int32).cuda(), torch.from_numpy(cu).cuda(), q, 0.0, out, ws,
                           rope=sq.Rope(torch.from_numpy(rope).cuda(), inter) if rot else None, window=window, lse=lse,
                           flags=flags)
    assert flags.item() == 0
    pos = [(b, start[b] + i) for b in range(len(new)) for i in range(new[b])] + [(-1, 0)] * tail
    check_attention(out, lse, q, pos, pool, table, page, n_q, n_kv, d, out_dtype, rope, inter, window)
    assert (out[cu[-1]:] == 3).all() and (lse[cu[-1]:] == 3).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,dtype,out_dtype,page", [(1, F16, F16, 16), (4, BF16, BF16, 32), (5, F16, F32, 16), (8, BF16, F16, 128)])
def test_prefill_ragged(d, group, dtype, out_dtype, page):
    prefill_case(d, group, 1, dtype, out_dtype, page, [0, 7, 0, 130, 31], [3, 0, 1, 20, 40], rot=d if group != 4 else 0,
                 inter=group == 5)


@pytest.mark.parametrize("d,group,start,new,window", [(128, 4, [0], [300], 0), (64, 2, [500], [150], 0), (256, 2, [0, 260], [140, 70], 0),
                                                      (128, 2, [100, 0], [130, 260], 17), (64, 8, [0], [129], 1),
                                                      (128, 1, [1000], [140], 600), (128, 16, [200], [20], 0)])
def test_prefill_longer_and_windows(d, group, start, new, window):
    prefill_case(d, group, 1, F16, F16, 16 if window else 64, start, new, window=window, rot=32, seed=9)


def test_prefill_takes_nothing_from_places_that_are_masked():
    """NaN in every place past a query's own position leaves its output what it was."""
    d, page, n = 128, 16, 150
    cache, _ = small_cache(d=d, page=page, tokens=n)
    cu, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 40], [60]))
    q = torch.randn(40, 4, d, device="cuda", dtype=F16)
    ws = torch.empty(sq.sq_kv4_attn_prefill_workspace(1, 4, 1, d, 40), dtype=torch.uint8, device="cuda")
    a, b = (torch.empty(40, 4, d, device="cuda", dtype=F16) for _ in range(2))
    sq.sq_kv4_attn_prefill(cache, start, cu, q, 0.0, a, ws)
    bad = torch.full((50, 1, d), math.nan, device="cuda", dtype=F16)
    sq.sq_kv4_append(cache, bad, bad, torch.tensor([100], dtype=torch.int32, device="cuda"),
                     torch.tensor([0, 50], dtype=torch.int32, device="cuda"))
    sq.sq_kv4_attn_prefill(cache, start, cu, q, 0.0, b, ws)
    assert torch.equal(a, b)
    sq.sq_kv4_append(cache, bad[:1], bad[:1], torch.tensor([80], dtype=torch.int32, device="cuda"))
    sq.sq_kv4_attn_prefill(cache, start, cu, q, 0.0, b, ws)
    assert torch.equal(a[:20], b[:20]) and torch.isnan(b[20:]).all()


def test_prefill_of_wrong_offsets_stays_in_bounds():
    """Offsets and starts that name no tokens of the call: nothing is written for them."""
    cache, _ = small_cache(batch=3)
    q = torch.randn(8, 4, 128, device="cuda", dtype=F16)
    ws = torch.empty(sq.sq_kv4_attn_prefill_workspace(3, 4, 1, 128, 8), dtype=torch.uint8, device="cuda")
    for cu, start, bit in (([0, 4, 2, 8], [0, 0, 0], None), ([0, 400, 500, 600], [0, 0, 0], None), ([-5, 2, 4, 8], [0, 0, 0], None),
                           ([0, 2, 4, 8], [-3, 0, 0], sq.SQ_FLAG_SEQLEN), ([0, 2, 4, 8], [0, 0, 62], sq.SQ_FLAG_SEQLEN),
                           ([0, 2, 4, 8], [0, 0, 2 ** 31 - 1], sq.SQ_FLAG_SEQLEN)):
        out = torch.full((8, 4, 128), 3.0, device="cuda", dtype=F16)
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        sq.sq_kv4_attn_prefill(cache, torch.tensor(start, dtype=torch.int32, device="cuda"),
                               torch.tensor(cu, dtype=torch.int32, device="cuda"), q, 0.0, out, ws, flags=flags)
        torch.cuda.synchronize()
        if bit is not None:
            assert flags.item() == bit


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,dtype,group", [(64, BF16, 2), (128, F16, 5), (256, BF16, 1)])
def test_prompt_then_steps_match_the_oracle(d, dtype, group):
    """Two prompts appended and attended, then four decode steps of the batch: every output against the oracle's
    attention over what the oracle's own append holds."""
    Q_TYPE[0] = dtype
    n_kv, page, prompts, steps = 2, 16, [21, 50], 4
    n_q = group * n_kv
    g = torch.Generator().manual_seed(11)
    rope = kv4.rope_table(80, d)
    r = sq.Rope(torch.from_numpy(rope).cuda())
    table, total = make_table([-(-(n + steps) // page) for n in prompts], 5)
    cache = sq.alloc_kv4(total, n_kv, d, page, torch.from_numpy(table).cuda())
    want = cache.pages.cpu().numpy().copy()
    cu = [0, prompts[0], sum(prompts)]
    qkv = torch.randn(sum(prompts), (n_q + 2 * n_kv), d, generator=g).to(dtype)
    cut = lambda t: (t[:, :n_q], t[:, n_q:n_q + n_kv], t[:, n_q + n_kv:])  # noqa: E731
    _, k, v = cut(qkv)
    append_oracle(want, table, page, k, v, [0, 0], cu, rope, False, dtype)
    q, k, v = cut(qkv.cuda())
    zero, cud = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    sq.sq_kv4_append(cache, k, v, zero, cud, rope=r)
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    out, lse = torch.empty(sum(prompts), n_q, d, dtype=dtype, device="cuda"), torch.empty(sum(prompts), n_q, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_prefill_workspace(2, n_q, n_kv, d, sum(prompts)), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_prefill(cache, zero, cud, q, 0.0, out, ws, rope=r, lse=lse)
    pos = [(b, i) for b in range(2) for i in range(prompts[b])]
    check_attention(out, lse, q, pos, cache.pages, table, page, n_q, n_kv, d, dtype, rope)
    ws = torch.empty(sq.sq_kv4_attn_workspace(2, n_q, n_kv, d, 80), dtype=torch.uint8, device="cuda")
    for i in range(steps):
        at = [n + i for n in prompts]
        qkv = torch.randn(2, n_q + 2 * n_kv, d, generator=g).to(dtype)
        _, k, v = cut(qkv)
        append_oracle(want, table, page, k, v, at, None, rope, False, dtype)
        q, k, v = cut(qkv.cuda())
        out, lse = torch.empty(2, n_q, d, dtype=dtype, device="cuda"), torch.empty(2, n_q, device="cuda")
        sq.sq_kv4_decode_step(cache, k, v, q, torch.tensor(at, dtype=torch.int32, device="cuda"), 0.0, out, 80, ws, rope=r,
                              lse=lse)
        assert np.array_equal(cache.pages.cpu().numpy(), want)
        check_attention(out, lse, q, [(0, at[0]), (1, at[1])], cache.pages, table, page, n_q, n_kv, d, dtype, rope)


def test_step_is_append_then_decode_and_shared_prefix_pages_are_read():
    d, page, n_kv, n_q = 128, 16, 2, 8
    table, total = make_table([3, 3, 3], 2, shared=((1, 0, 0), (1, 0, 1), (2, 0, 0)))
    pool = random_pool(total, n_kv, page, d, 3)
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(3, n_kv, d, generator=g, device="cuda").to(F16) for _ in range(2))
    q = torch.randn(3, n_q, d, generator=g, device="cuda").to(F16)
    pos = torch.tensor([40, 33, 20], dtype=torch.int32, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_workspace(3, n_q, n_kv, d, 48), dtype=torch.uint8, device="cuda")
    rope = sq.Rope(sq.rope_table(64, d))
    a = sq.PagedKV4(pool.clone(), torch.from_numpy(table).cuda(), n_kv, d, page)
    b = sq.PagedKV4(pool.clone(), torch.from_numpy(table).cuda(), n_kv, d, page)
    oa, ob = (torch.empty(3, n_q, d, device="cuda") for _ in range(2))
    sq.sq_kv4_decode_step(a, k, v, q, pos, 0.0, oa, 48, ws, rope=rope)
    sq.sq_kv4_append(b, k, v, pos, rope=rope)
    sq.sq_kv4_attn_decode(b, pos + 1, q, 0.0, ob, 48, ws, rope=rope)
    assert torch.equal(a.pages, b.pages) and torch.equal(oa, ob)


def test_graphs_that_share_a_workspace_and_other_streams():
    d, n_q = 128, 8
    cache, _ = small_cache(d=d, n_kv=2, tokens=1200, batch=3, seed=7)
    g = torch.Generator(device="cuda").manual_seed(0)
    q = [torch.randn(3, n_q, d, generator=g, device="cuda").to(F16) for _ in range(2)]
    lens = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([1200, 0, 700], [3, 1100, 900])]
    ws = torch.full((sq.sq_kv4_attn_workspace(3, n_q, 2, d, 1200),), 255, dtype=torch.uint8, device="cuda")
    eager = []
    for i in range(2):
        o = torch.empty(3, n_q, d, device="cuda")
        sq.sq_kv4_attn_decode(cache, lens[i], q[i], 0.0, o, 1200, ws)
        eager.append(o)
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        gr, o = torch.cuda.CUDAGraph(), torch.zeros(3, n_q, d, device="cuda")
        with torch.cuda.stream(side):
            sq.sq_kv4_attn_decode(cache, lens[i], q[i], 0.0, o, 1200, ws)
        torch.cuda.synchronize()
        assert torch.equal(o, eager[i])                              # the side stream's own result
        o.zero_()
        with torch.cuda.graph(gr):
            sq.sq_kv4_attn_decode(cache, lens[i], q[i], 0.0, o, 1200, ws)
        graphs.append(gr)
        outs.append(o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, e) for o, e in zip(outs, eager))
    lens[0].copy_(torch.tensor([5, 1200, 64], dtype=torch.int32))    # a replay follows the lengths on the device
    graphs[0].replay()
    ref = torch.empty(3, n_q, d, device="cuda")
    sq.sq_kv4_attn_decode(cache, lens[0], q[0], 0.0, ref, 1200, ws)
    assert torch.equal(outs[0], ref)


# ------------------------------------------------------------------ where the kernels' own divisions could go wrong
@pytest.mark.parametrize("d,n_kv,page,rot,inter", [(256, 20, 16, 256, False), (128, 3, 32, 48, False), (64, 35, 16, 64, True)])
def test_append_of_many_and_of_odd_head_counts(d, n_kv, page, rot, inter):
    """More vectors a token than a block holds, and numbers of them that do not divide it."""
    g = torch.Generator().manual_seed(d + n_kv)
    k, v = (torch.randn(19, n_kv, d, generator=g).to(BF16) for _ in range(2))
    start, cu = [3, 11], [0, 12, 19]
    table, total = make_table([1, 2], 1)
    pool = torch.zeros(total, n_kv, page // 16, 16 * d + 128, dtype=torch.uint8)
    want = pool.numpy().copy()
    rope = kv4.rope_table(32, rot)
    append_oracle(want, table, page, k, v, start, cu, rope, inter, BF16)
    cache = sq.PagedKV4(pool.cuda(), torch.from_numpy(table).cuda(), n_kv, d, page)
    st, cud = torch.tensor(start, dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
    sq.sq_kv4_append(cache, k.cuda(), v.cuda(), st, cud, rope=sq.Rope(torch.from_numpy(rope).cuda(), inter))
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    ko, vo = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    sq.sq_kv4_read(cache, st, cud, ko, vo)
    for b, i, h in ((0, 0, 0), (0, 11, n_kv - 1), (1, 6, n_kv // 2)):
        p = start[b] + i
        for side, got in ((0, ko), (1, vo)):
            c, sb, mb = kv4.load(want, table[b, p // page], h, p % page, side)
            x = torch.from_numpy(kv4.values(c, np.uint32(sb), np.uint32(mb))).float().to(BF16)
            assert torch.equal(got[cu[b] + i, h].cpu(), x)


def test_codes_beside_ties_are_those_of_the_exact_quotient():
    """Coordinates half a step from two codes, and one float beside that, over many steps."""
    d, page = 256, 16
    g = torch.Generator().manual_seed(0)
    rows = []
    for e in range(-40, 40, 5):
        s = float(torch.tensor((1 + torch.rand(1, generator=g).item()) * 2.0 ** e).to(BF16))
        x = np.arange(d, dtype=np.float64) % 15 * s + s / 2
        x = x.astype(np.float32)
        x[1::3] = np.nextafter(x[1::3], np.float32(np.inf))
        x[2::3] = np.nextafter(x[2::3], np.float32(-np.inf))
        x[0], x[1] = 0.0, np.float32(15 * s)
        rows.append(torch.from_numpy(x))
    x = torch.stack(rows)[:, None]
    table, total = make_table([1], 0)
    cache = sq.alloc_kv4(total, 1, d, page, torch.from_numpy(table).cuda())
    want = cache.pages.cpu().numpy().copy()
    append_oracle(want, table, page, x, -x, [0], [0, len(rows)], None, False, F32)
    sq.sq_kv4_append(cache, x.cuda(), (-x).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                     torch.tensor([0, len(rows)], dtype=torch.int32).cuda())
    assert np.array_equal(cache.pages.cpu().numpy(), want)


@pytest.mark.parametrize("d,group", [(64, 130), (128, 150), (256, 33)])
def test_groups_larger_than_a_row_tile(d, group):
    decode_case(d, group, 1, F16, F32, 16, [70, 0, 5], rot=32, seed=3)
    prefill_case(d, group, 1, F16, F32, 16, [40, 0], [6, 3], rot=32, seed=3)


@pytest.mark.parametrize("d", [64, 256])
def test_steps_and_offsets_of_unlike_sizes(d):
    """Pairs of one pool over forty powers of two: what is exact for each must not depend on its neighbours."""
    Q_TYPE[0] = F16
    page, n = 16, 200
    table, total = make_table([-(-n // page)], 5)
    pool = random_pool(total, 1, page, d, 5)
    pairs = pool[..., 16 * d:].contiguous().view(BF16).view(total, 1, 1, 2, 16, 2)
    e = torch.randint(-20, 21, (total, 1, 1, 2, 16, 1), generator=torch.Generator().manual_seed(2)).cuda()
    e[:, :, :, 0] -= 18                                   # keys' scores stay moderate
    pairs = (pairs.float() * torch.exp2(e.float())).to(BF16)
    pool[..., 16 * d:] = pairs.contiguous().view(torch.uint8).view(total, 1, 1, 128)
    cache = sq.PagedKV4(pool, torch.from_numpy(table).cuda(), 1, d, page)
    q = torch.randn(9, 3, d, generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    out, lse = torch.empty(9, 3, d, device="cuda"), torch.empty(9, 3, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_prefill_workspace(1, 3, 1, d, 9), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_prefill(cache, torch.tensor([n - 9], dtype=torch.int32).cuda(), torch.tensor([0, 9], dtype=torch.int32).cuda(),
                           q, 0.0, out, ws, lse=lse)
    check_attention(out, lse, q, [(0, n - 9 + i) for i in range(9)], pool, table, page, 3, 1, d, F32)
    out, lse = torch.empty(1, 3, d, device="cuda"), torch.empty(1, 3, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_workspace(1, 3, 1, d, n), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_decode(cache, torch.tensor([n], dtype=torch.int32).cuda(), q[:1], 0.0, out, n, ws, lse=lse)
    check_attention(out, lse, q[:1], [(0, n - 1)], pool, table, page, 3, 1, d, F32)


def test_prefill_of_thousands_of_sequences():
    """More units than are sorted: single tokens, two of every three sequences idle; the same as decode attention."""
    d, page, n_kv, batch = 64, 16, 1, 6500
    rng = np.random.default_rng(0)
    lens = rng.integers(1, 40, batch)
    new = np.where(np.arange(batch) % 3 == 0, 1, 0)
    table, total = make_table([3] * 64, 0)
    table = table[rng.integers(0, 64, batch)]                        # shared pages
    cache = sq.PagedKV4(random_pool(total, n_kv, page, d, 0), torch.from_numpy(table).cuda(), n_kv, d, page)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    start = torch.from_numpy(lens.astype(np.int32)).cuda()
    n_tok = int(new.sum())
    q = torch.randn(n_tok, 2, d, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(F16)
    out, lse = torch.empty(n_tok, 2, d, device="cuda"), torch.empty(n_tok, 2, device="cuda")
    ws = torch.full((sq.sq_kv4_attn_prefill_workspace(batch, 2, n_kv, d, n_tok),), 255, dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_prefill(cache, start, cu, q, 0.0, out, ws, lse=lse)
    rows = torch.from_numpy(np.flatnonzero(new)).cuda()
    one = sq.PagedKV4(cache.pages, cache.table[rows].contiguous(), n_kv, d, page)
    want, wl = torch.empty(n_tok, 2, d, device="cuda"), torch.empty(n_tok, 2, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_workspace(n_tok, 2, n_kv, d, 41), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_decode(one, (start[rows] + 1).contiguous(), q, 0.0, want, 41, ws, lse=wl)
    # both weights rounded (2 x 2^-11) against steps below 0.97 and codes at most 8 from their middle
    assert (out - want).abs().max() <= 2 * 2.0 ** -11 * 0.97 * 8 and (lse - wl).abs().max() <= 2.0 ** -16


@pytest.mark.parametrize("d,group,start,new,window", [
    (64, 2, [500], [150], 0), (128, 6, [6000, 4100], [30, 7], 0), (256, 2, [3000, 36, 700], [300, 60, 90], 1024),
    (128, 4, [0], [700], 0), (64, 1, [9000], [1], 0), (256, 8, [5000], [3], 0)])
def test_chunks_repeat_bit_for_bit(d, group, start, new, window):
    """Cut units, single row tiles and pairs of them, whatever the blocks' order: twelve runs are equal, and equal in a graph
    that shares their workspace with another."""
    page, n_kv = 16, 2
    table, total = make_table([-(-(s + n) // page) for s, n in zip(start, new)], 1)
    cache = sq.PagedKV4(random_pool(total, n_kv, page, d, 1), torch.from_numpy(table).cuda(), n_kv, d, page)
    st = torch.tensor(start, dtype=torch.int32).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    n_tok, n_q = sum(new), group * n_kv
    q = [torch.randn(n_tok, n_q, d, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").to(F16) for i in (0, 1)]
    ws = torch.full((sq.sq_kv4_attn_prefill_workspace(len(new), n_q, n_kv, d, n_tok),), 255, dtype=torch.uint8, device="cuda")
    first = []
    for i in (0, 1):
        for r in range(12):
            out, lse = torch.full((n_tok, n_q, d), 9.0, device="cuda"), torch.full((n_tok, n_q), 9.0, device="cuda")
            sq.sq_kv4_attn_prefill(cache, st, cu, q[i], 0.0, out, ws, window=window, lse=lse)
            if r == 0:
                first.append((out, lse))
            assert torch.equal(out, first[i][0]) and torch.equal(lse, first[i][1])
    graphs = []
    outs = [torch.zeros_like(first[0][0]) for _ in (0, 1)]
    for i in (0, 1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sq.sq_kv4_attn_prefill(cache, st, cu, q[i], 0.0, outs[i], ws, window=window)
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, f[0]) for o, f in zip(outs, first))


@pytest.mark.parametrize("batch,pos", [(1, [501]), (2, [1700, 60]), (5, [9000, 1, 4000, 77, 2500])])
def test_steps_in_a_graph_continue_a_sequence(batch, pos):
    """A captured step replayed over positions that advance on the device: the outputs of separate calls, of few blocks (which
    join by themselves) and of many."""
    d, page, n_kv, n_q, steps = 128, 16, 2, 12, 4
    table, total = make_table([-(-(p + steps) // page) for p in pos], 4)
    pool = random_pool(total, n_kv, page, d, 4)
    rope = sq.Rope(sq.rope_table(max(pos) + steps, d))
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(steps, batch, n_q + 2 * n_kv, d, generator=g, device="cuda").to(BF16)
    cut = lambda t: (t[:, n_q:n_q + n_kv], t[:, n_q + n_kv:], t[:, :n_q])  # noqa: E731
    a = sq.PagedKV4(pool.clone(), torch.from_numpy(table).cuda(), n_kv, d, page)
    b = sq.PagedKV4(pool.clone(), torch.from_numpy(table).cuda(), n_kv, d, page)
    ctx = max(pos) + steps
    ws = torch.full((sq.sq_kv4_attn_workspace(batch, n_q, n_kv, d, ctx),), 255, dtype=torch.uint8, device="cuda")
    at = torch.tensor(pos, dtype=torch.int32).cuda()
    x, out = qkv[0].clone(), torch.zeros(batch, n_q, d, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        sq.sq_kv4_decode_step(a, *cut(x), at, 0.0, out, ctx, ws, rope=rope)
        at.add_(1)
    at.copy_(torch.tensor(pos, dtype=torch.int32))
    a.pages.copy_(pool)
    for i in range(steps):
        x.copy_(qkv[i])
        gr.replay()
        want = torch.zeros_like(out)
        now = torch.tensor(pos, dtype=torch.int32).cuda() + i
        k, v, q = cut(qkv[i])
        sq.sq_kv4_append(b, k, v, now, rope=rope)
        ws2 = torch.empty_like(ws)
        sq.sq_kv4_attn_decode(b, now + 1, q, 0.0, want, ctx, ws2, rope=rope)
        assert torch.equal(a.pages, b.pages)
        # the join of a step and of a separate call sum in the same order, but scale with other roundings: a few of 2^-24
        assert (out - want).abs().max() <= 16 * 2.0 ** -24 * 16


def test_calls_of_two_streams_at_once():
    """Two chunks and two decodes on two streams, each with a workspace of its own, leave each other's outputs alone."""
    d, page, n_kv, n_q = 128, 16, 2, 8
    table, total = make_table([200, 200], 6)
    cache = sq.PagedKV4(random_pool(total, n_kv, page, d, 6), torch.from_numpy(table).cuda(), n_kv, d, page)
    st, cu = torch.tensor([3000, 2500], dtype=torch.int32).cuda(), torch.tensor([0, 100, 180], dtype=torch.int32).cuda()
    lens = torch.tensor([3200, 3100], dtype=torch.int32).cuda()
    q = torch.randn(180, n_q, d, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(F16)

    def run(out, one, wp, wd, stream=None):
        sq.sq_kv4_attn_prefill(cache, st, cu, q, 0.0, out, wp, stream=stream)
        sq.sq_kv4_attn_decode(cache, lens, q[:2], 0.0, one, 3200, wd, stream=stream)

    new = lambda: (torch.empty(180, n_q, d, device="cuda"), torch.empty(2, n_q, d, device="cuda"),  # noqa: E731
                   torch.empty(sq.sq_kv4_attn_prefill_workspace(2, n_q, n_kv, d, 180), dtype=torch.uint8, device="cuda"),
                   torch.empty(sq.sq_kv4_attn_workspace(2, n_q, n_kv, d, 3200), dtype=torch.uint8, device="cuda"))
    ref = new()
    run(*ref)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [new(), new()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, x in zip(streams, sets):
            run(*x, stream=s)
    torch.cuda.synchronize()
    for x in sets:
        assert torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1])


def test_offsets_below_zero_name_no_tokens():
    """A sequence whose first offset is below 0, however far: its rows stay as they were, the others' are right."""
    Q_TYPE[0] = F16
    d, page, n_kv, n_q = 128, 16, 1, 4
    cache, table = small_cache(d=d, n_kv=n_kv, page=page, batch=3)
    q = torch.randn(8, n_q, d, generator=torch.Generator().manual_seed(0)).to(F16).cuda()
    ws = torch.full((sq.sq_kv4_attn_prefill_workspace(3, n_q, n_kv, d, 8),), 255, dtype=torch.uint8, device="cuda")
    start = torch.tensor([5, 9, 20], dtype=torch.int32, device="cuda")
    for first in (-1, -200, -2 ** 31):
        cu = torch.tensor([first, 2, 5, 8], dtype=torch.int32, device="cuda")
        out = torch.full((8, n_q, d), 3.0, device="cuda")
        sq.sq_kv4_attn_prefill(cache, start, cu, q, 0.0, out, ws)
        pos = [(-1, 0)] * 2 + [(1, 9 + i) for i in range(3)] + [(2, 20 + i) for i in range(3)]
        check_attention(out, None, q, pos, cache.pages, table, page, n_q, n_kv, d, F32)
        assert (out[:2] == 3).all()
        before = cache.pages.clone()
        k = torch.randn(2, n_kv, d, device="cuda", dtype=F16)
        sq.sq_kv4_append(cache, k, k, start, torch.tensor([first, 2, 2, 2], dtype=torch.int32, device="cuda"))
        assert torch.equal(cache.pages, before)


# ------------------------------------------------------------------ weights of fp16 and float outputs
def near_uniform(d, n, n_q, seed=0):
    """Sixteen-token blocks of steps near 1 and offsets -7.5 steps, and queries so small that every weight is close to 1 / n."""
    pool = random_pool(-(-n // 16), 1, 16, d, seed, device="cpu")
    q = (torch.randn(n, n_q, d, generator=torch.Generator().manual_seed(seed + 1)) * 2.0 ** -11).to(F16)
    return pool, q


def weighted(pool_np, q, n, one_part=False):
    """Float64 outputs [n_q, d] of one query over the first n tokens of page after page, and what two-part weights may be off by
    (below); or the outputs with every weight times its step rounded once to fp16."""
    d = q.shape[-1]
    table = np.arange(len(pool_np))[None]
    (kc, ks, km), (vc, vs, vm) = (rows_of(pool_np, table, 0, 0, n, 16, side) for side in (0, 1))
    keys, vals = kv4.values(kc, ks, km), kv4.values(vc, vs, vm)
    s, m = kv4.bf16_value(vs).astype(np.float64), kv4.bf16_value(vm).astype(np.float64)
    x = q.astype(np.float64) @ keys.T / math.sqrt(d)
    p = np.exp(x - x.max(-1, keepdims=True))
    l = p.sum(-1, keepdims=True)
    mid = vc - 8.0
    if one_part:
        w = (p * s * 2048.0).astype(np.float16).astype(np.float64) / 2048.0
        return (w @ mid + (p * (m + 8 * s)) @ np.ones_like(mid)) / l
    aq = np.abs(q.astype(np.float64))
    delta = ((d + 16) * 2.0 ** -24 / math.sqrt(d) * (kv4.bf16_value(ks) * (aq @ kc.T) + np.abs(kv4.bf16_value(km)) * aq.sum(-1, keepdims=True))).max()
    p /= l
    spread, size = (p * s) @ np.abs(mid), p @ np.abs(vals)
    # 2^-21: two parts. Sums of the products: the tokens are one step of 16 along k (two of a tile), in one or two
    # products, whose 17 terms each may lose a unit of 2^-23 of the largest: 4 x 17 x 2^-23 < 2^-16. Then exponents
    # (delta and the 2^-20 of a base-2 exponential, in numerator and denominator), fp16's smallest steps, float sums.
    bound = (2.0 ** -21 + 2.0 ** -16) * spread + 2 * (delta + 2.0 ** -20) * size + n * 2.0 ** -32 * s.max() + (n + 8) * 2.0 ** -24 * size
    return p @ vals, bound


@pytest.mark.parametrize("d,n_q", [(64, 2), (128, 4), (256, 1), (64, 7), (128, 8), (256, 5)])
def test_fp16_and_float_outputs_take_their_weights_in_two_parts(d, n_q):
    """Outputs over sixteen near-equal weights, far nearer than weights of 11 bits could bring them: decode and chunks."""
    n = 16
    pool, q = near_uniform(d, n, n_q)
    pn, qn = pool.numpy(), q.float().numpy()
    want, bound = zip(*[weighted(pn, qn[i], i + 1) for i in range(n)])
    coarse = np.stack([weighted(pn, qn[i], i + 1, True) for i in range(n)])
    want, bound = np.stack(want), np.stack(bound)
    assert (np.abs(coarse - want) > bound)[8:].mean() > 0.5            # one part would be seen
    unit = np.abs(want.astype(np.float16).astype(np.float64) - want)   # of an exact result rounded once
    cache = sq.PagedKV4(pool.cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda(), 1, d, 16)
    one = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for out_dtype in (F32, F16):
        outs = []
        out = torch.empty(n, n_q, d, device="cuda", dtype=out_dtype)
        ws = torch.empty(sq.sq_kv4_attn_prefill_workspace(1, n_q, 1, d, n), dtype=torch.uint8, device="cuda")
        sq.sq_kv4_attn_prefill(cache, one([0]), one([0, n]), q.cuda(), 0.0, out, ws)
        outs.append(out)
        out = torch.empty(n, n_q, d, device="cuda", dtype=out_dtype)
        ws = torch.empty(sq.sq_kv4_attn_workspace(1, n_q, 1, d, n), dtype=torch.uint8, device="cuda")
        for i in range(n):
            sq.sq_kv4_attn_decode(cache, one([i + 1]), q[i:i + 1].cuda(), 0.0, out[i:i + 1], n, ws)
        outs.append(out)
        for out in outs:
            err = np.abs(out.double().cpu().numpy() - want)
            assert np.all(err <= bound + torch.finfo(out_dtype).eps / 2 * np.abs(want) + 2.0 ** -25)
            if out_dtype == F16:       # root mean squares: the rounding's own, and beside it at most the bound's
                assert np.sqrt((err ** 2).mean()) <= np.sqrt((unit ** 2).mean()) + np.sqrt((bound ** 2).mean())


# ------------------------------------------------------------------ chunks that raise flags
def guarded(shape, dtype, fill, room=256):
    """(a tensor of that fill inside a larger buffer, a function that says whether the buffer around it is as it was)."""
    n = math.prod(shape)
    room = room // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2 * room,), fill, dtype=dtype, device="cuda")
    return buf[room:room + n].view(shape), lambda: bool((buf[:room] == fill).all()) and bool((buf[room + n:] == fill).all())


def flagged_chunks(cache, table, page, q, start, cu, bit, pos, n_kv, rope=None, skip=None, window=0, like=None):
    """One call of chunk attention: its flags, the rows of `pos` against the oracle (position -1: zeros), rows that no sequence
    names (-1, 0) left alone, nothing written around outputs and workspace."""
    Q_TYPE[0] = q.dtype
    n_tok, n_q, d = q.shape
    out, out_ok = guarded((n_tok, n_q, d), F32, 3.0)
    lse, lse_ok = guarded((n_tok, n_q), F32, 3.0)
    ws, ws_ok = guarded((sq.sq_kv4_attn_prefill_workspace(len(start), n_q, n_kv, d, n_tok),), torch.uint8, 255)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq.sq_kv4_attn_prefill(cache, torch.tensor(start, dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), q,
                           0.0, out, ws, rope=None if rope is None else sq.Rope(torch.from_numpy(rope).cuda()), window=window,
                           lse=lse, flags=flags)
    assert flags.item() == bit
    assert out_ok() and lse_ok() and ws_ok()
    if pos is not None:
        check_attention(out, lse, q, pos, cache.pages, table, page, n_q, n_kv, d, F32, rope, window=window, skip=skip)
        left = [i for i, (b, _) in enumerate(pos) if b < 0]
        assert (out[left] == 3).all() and (lse[left] == 3).all()


def test_chunks_that_begin_before_position_zero_are_flagged():
    cache, table = small_cache(batch=2)
    q = torch.randn(6, 4, 128, generator=torch.Generator().manual_seed(0)).to(F16).cuda()
    for start, bit in ((-1, sq.SQ_FLAG_SEQLEN), (-2, sq.SQ_FLAG_SEQLEN), (0, 0)):
        pos = [(0, max(start + i, -1)) for i in range(3)] + [(1, 20 + i) for i in range(2)] + [(-1, 0)]
        flagged_chunks(cache, table, 16, q, [start, 20], [0, 3, 5], bit, pos, 1)
    flagged_chunks(cache, table, 16, q, [-7, 20], [0, 0, 5], 0, [(1, 20 + i) for i in range(5)] + [(-1, 0)], 1)   # no token there


def test_chunk_offsets_that_fall_are_flagged():
    """Falling offsets raise a flag and write nothing outside the call's rows; offsets past the rows, and sequences that begin
    below 0, name no rows."""
    cache, table = small_cache(batch=3)
    q = torch.randn(8, 4, 128, generator=torch.Generator().manual_seed(0)).to(F16).cuda()
    rows = lambda *r: [(b, p + i) for b, p, n in r for i in range(n)]  # noqa: E731
    flagged_chunks(cache, table, 16, q, [0, 5, 9], [0, 4, 2, 8], sq.SQ_FLAG_SEQLEN, None, 1)
    flagged_chunks(cache, table, 16, q, [0, 5, 9], [0, 3, 3, 1], sq.SQ_FLAG_SEQLEN, rows((0, 0, 3)) + [(-1, 0)] * 5, 1)
    flagged_chunks(cache, table, 16, q, [0, 5, 9], [0, 3, 400, 401], 0, rows((0, 0, 3), (1, 5, 5)), 1)
    flagged_chunks(cache, table, 16, q, [7, 5, 9], [-1, 3, 5, 8], 0, [(-1, 0)] * 3 + rows((1, 5, 2), (2, 9, 3)), 1)
    many, table = small_cache(batch=64, tokens=2048)      # 32 x 32 units, more than the 392 or so that there are places for
    q = torch.randn(2048, 4, 128, generator=torch.Generator().manual_seed(0)).to(F16).cuda()
    flagged_chunks(many, table, 16, q, [0] * 64, [0, 2048] * 32 + [0], sq.SQ_FLAG_SEQLEN, None, 1)


@pytest.mark.parametrize("d,group,start,new,page,window", [
    (128, 4, [100, 0, 16], [40, 30, 1], 16, 0), (64, 1, [5000], [7], 64, 0), (256, 2, [700, 300], [90, 5], 32, 0),
    (128, 2, [900], [70], 16, 130)])
def test_chunks_leave_pages_outside_the_pool_out(d, group, start, new, page, window):
    """Page numbers past the pool and below 0 inside the attended span, in units that are cut (few rows, many keys) and are not."""
    table, total = make_table([-(-(s + n) // page) for s, n in zip(start, new)], 3)
    pool = random_pool(total, 1, page, d, 3)
    skip = {0: (0, (start[0] + 3) // page - 1, (start[0] + 3) // page)} if not window else {0: ((start[0] + 3) // page - 2,)}
    wrong = table.copy()
    for b, pages in skip.items():
        for i, p in enumerate(pages):
            wrong[b, p] = (total, -1, 2 ** 31 - 1)[i % 3]
    cache = sq.PagedKV4(pool, torch.from_numpy(wrong).cuda(), 1, d, page)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.randn(cu[-1], group, d, generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    pos = [(b, start[b] + i) for b in range(len(new)) for i in range(new[b])]
    flagged_chunks(cache, table, page, q, start, cu, sq.SQ_FLAG_PAGE, pos, 1, skip=skip, window=window)


@pytest.mark.parametrize("d,n_pos,window", [(128, 50, 0), (64, 33, 0), (256, 50, 20), (128, 1, 0), (64, 50, 4)])
def test_chunks_past_the_rotation_table_give_zeros(d, n_pos, window):
    cache, table = small_cache(d=d, batch=2, tokens=80)
    start, cu = [30, 0], [0, 45, 75]
    q = torch.randn(76, 3, d, generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    pos = [(b, p if p < n_pos else -1) for b in (0, 1) for p in range(start[b], start[b] + cu[b + 1] - cu[b])] + [(-1, 0)]
    flagged_chunks(cache, table, 16, q, start, cu, sq.SQ_FLAG_ROPE, pos, 1, rope=kv4.rope_table(n_pos, d), window=window)


def test_chunks_past_the_pages_attend_to_what_they_hold():
    cache, table = small_cache(batch=2)
    q = torch.randn(10, 4, 128, generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    pos = [(0, min(60 + i, 63)) for i in range(8)] + [(1, 3), (1, 4)]
    flagged_chunks(cache, table, 16, q, [60, 3], [0, 8, 10], sq.SQ_FLAG_SEQLEN, pos, 1)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_near_the_largest_floats(d):
    """bf16 queries up to 2^127 (2^116 for single tokens) over keys so small that the scores are moderate."""
    Q_TYPE[0] = BF16
    page, n, up = 16, 60, 121
    table, total = make_table([-(-n // page)], 5)
    pool = random_pool(total, 1, page, d, 5)
    pairs = pool[..., 16 * d:].contiguous().view(BF16).view(total, 1, 1, 2, 16, 2).float()
    pairs[:, :, :, 0] *= 2.0 ** -(up - 1)                 # keys' steps from 2^-124 on
    cache = lambda pairs: sq.PagedKV4(torch.cat([pool[..., :16 * d], pairs.to(BF16).contiguous().view(torch.uint8).view(total, 1, 1, 128)], -1),  # noqa: E731
                                      torch.from_numpy(table).cuda(), 1, d, page)
    q = torch.randn(9, 3, d, generator=torch.Generator().manual_seed(1)).clamp(-3.9, 3.9)
    q[:, :, 0] = 3.9
    c, x = cache(pairs), (q * 2.0 ** (up + 4)).to(BF16).cuda()
    assert torch.isfinite(x).all() and x.float().amax() > 2.0 ** 126
    out, lse = torch.empty(9, 3, d, device="cuda"), torch.empty(9, 3, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_prefill_workspace(1, 3, 1, d, 9), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_prefill(c, torch.tensor([n - 9], dtype=torch.int32).cuda(), torch.tensor([0, 9], dtype=torch.int32).cuda(),
                           x, 2.0 ** -8, out, ws, lse=lse)
    check_attention(out, lse, x, [(0, n - 9 + i) for i in range(9)], c.pages, table, page, 3, 1, d, F32, scale=2.0 ** -8)
    pairs[:, :, :, 0] *= 2.0 ** 11
    c, x = cache(pairs), (q[:1] * 2.0 ** (up - 7)).to(BF16).cuda()
    assert 2.0 ** 115 < x.float().amax() < 2.0 ** 116
    out, lse = torch.empty(1, 3, d, device="cuda"), torch.empty(1, 3, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_workspace(1, 3, 1, d, n), dtype=torch.uint8, device="cuda")
    sq.sq_kv4_attn_decode(c, torch.tensor([n], dtype=torch.int32).cuda(), x, 2.0 ** -8, out, n, ws, lse=lse)
    check_attention(out, lse, x, [(0, n - 1)], c.pages, table, page, 3, 1, d, F32, scale=2.0 ** -8)


# ------------------------------------------------------------------ long contexts
@pytest.mark.parametrize("d,group,batch,n", [(64, 1, 296, 20000), (128, 4, 296, 16384), (128, 6, 32, 32768), (256, 2, 296, 32768),
                                             (128, 8, 296, 16000)])
def test_long_contexts_of_every_output_type(d, group, batch, n):
    """Near-equal weights over up to 32768 tokens, against float64: outputs are then far smaller than what sums to them, so
    that what the tensor cores cut of long sums would show. 296 sequences: one block a sequence, the longest sums."""
    page = 64
    g = torch.Generator(device="cuda").manual_seed(1)
    n_pages = -(-n // page)
    row = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    one = sq.alloc_kv4(n_pages, 1, d, page, row[None].clone())
    k = torch.randn(n_pages * page, 1, d, generator=g, device="cuda").to(F16)
    v = (torch.randn(n_pages * page, 1, d, generator=g, device="cuda") * 0.3).to(F16)
    start, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, n_pages * page], dtype=torch.int32, device="cuda")
    sq.sq_kv4_append(one, k, v, start, cu)
    ko, vo = (torch.empty(n_pages * page, 1, d, device="cuda") for _ in range(2))
    sq.sq_kv4_read(one, start, cu, ko, vo)                # one rounding of 2^-24 of what is held
    keys, vals = ko[:n, 0].double(), vo[:n, 0].double()
    step = ((vals.amax(-1) - vals.amin(-1)) / 14).amax().item()          # of the values, at most (all use 14 codes or more)
    cache = sq.PagedKV4(one.pages, row.expand(batch, -1).contiguous(), 1, d, page)
    q = (torch.randn(batch, group, d, generator=g, device="cuda") * 0.1).to(F16)
    scale, want, size = 1 / math.sqrt(d), [], []
    for b in range(batch):
        p = torch.softmax(q[b].double() @ keys.T * scale, -1)
        want.append(p @ vals)
        size.append(p @ vals.abs())
    want, size = torch.stack(want), torch.stack(size)
    aq = q.double().abs().sum(-1).amax().item()
    eps = (d + 16) * 2.0 ** -24 * scale * aq * keys.abs().amax().item() * 2 + 2.0 ** -20
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    ws = torch.empty(sq.sq_kv4_attn_workspace(batch, group, 1, d, n), dtype=torch.uint8, device="cuda")
    for dtype in (BF16, F16, F32):
        out = torch.empty(batch, group, d, dtype=dtype, device="cuda")
        sq.sq_kv4_attn_decode(cache, lens, q, 0.0, out, n, ws)
        err, unit = (out.double() - want).abs(), (want.to(dtype).double() - want)
        # A product adds sixteen tokens and cuts a unit of 2^-23 of the sum at hand, of its warp. bf16: codes of 7.5 in the
        # mean over at most sixteen tiles, and 8 times the weights beside them; else codes less 8, at most 4 in the mean,
        # over all the warp's tokens.
        cut = 2.0 ** -23 * (16 * (1 if d == 256 else 2) * 7.5 if dtype == BF16 else n / 128 * 4 * 2) * step
        near = (2.0 ** -11 if dtype == BF16 else 2.0 ** -21) * 4 * step       # weights of one part, and of two
        assert (err <= torch.finfo(dtype).eps / 2 * want.abs() + near + cut + 2 * eps * size).all()
        if dtype == BF16:             # beside the output's own rounding, which the cuts do not follow
            rms = lambda x: x.pow(2).mean().sqrt().item()  # noqa: E731
            assert rms(err) <= math.hypot(rms(unit), cut) * 1.02


@pytest.mark.parametrize("d,group,dtype", [(64, 4, F16), (128, 3, F16), (128, 6, F16), (256, 3, F16), (256, 8, F16), (128, 3, BF16)])
def test_log_sum_exps_of_short_spans_are_floats(d, group, dtype):
    """Decode over one to four tokens, where log-sum-exps are of the size of one score: within 2^-20 of them in the root mean
    square, as float sums of d products are with room (theirs: 2^-24 to 2^-23)."""
    page, batch, n = 16, 96, 48
    g = torch.Generator(device="cuda").manual_seed(d)
    table = torch.arange(batch * 3, dtype=torch.int32, device="cuda").view(batch, 3)
    cache = sq.alloc_kv4(batch * 3, 1, d, page, table)
    large = torch.ones(d, device="cuda")
    large[:: 32] = 6.0
    k = (torch.randn(batch * n, 1, d, generator=g, device="cuda") * large).to(dtype)
    start, cu = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.arange(0, batch * n + 1, n, dtype=torch.int32, device="cuda")
    sq.sq_kv4_append(cache, k, k, start, cu)
    keys, vals = (torch.empty(batch * n, 1, d, device="cuda") for _ in range(2))
    sq.sq_kv4_read(cache, start, cu, keys, vals)
    keys = keys.view(batch, n, d).double()
    q = (torch.randn(batch, group, d, generator=g, device="cuda") * math.sqrt(32 / 67)).to(dtype)
    ws = torch.empty(sq.sq_kv4_attn_workspace(batch, group, 1, d, n), dtype=torch.uint8, device="cuda")
    for window in (1, 2, 4):
        out, lse = torch.empty(batch, group, d, device="cuda"), torch.empty(batch, group, device="cuda")
        lens = torch.arange(batch, dtype=torch.int32, device="cuda") % (n - 4) + 4
        sq.sq_kv4_attn_decode(cache, lens, q, 0.0, out, n, ws, window=window, lse=lse)
        want = torch.stack([torch.logsumexp(q[b].double() @ keys[b, int(lens[b]) - window:int(lens[b])].T / math.sqrt(d), -1)
                            for b in range(batch)])
        rms = lambda x: x.pow(2).mean().sqrt().item()  # noqa: E731
        assert rms(lse.double() - want) <= 2.0 ** -20 * rms(want), window

"""Refusals of the paged 4-bit cache's entry points: they need no GPU."""

import copy
import ctypes
import pickle

import pytest
import torch

from compressed_attention_head_b200 import build as sqbuild
from compressed_attention_head_b200 import sq

AT = 1 << 20      # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return sq.lib()


def _cache(**kw):
    f = dict(pages=AT, table=AT, n_pages=8, table_stride=4, batch=2, pages_per_row=4, n_kv_heads=2, d=128,
             page_tokens=16)
    f.update(kw)
    return sq.sq_kv4_cache(*[f[n] for n, _ in sq.sq_kv4_cache._fields_])


def _rope(**kw):
    f = dict(table=AT, n_pos=64, rot_dim=128, interleaved=0)
    f.update(kw)
    return sq.sq_rope(*[f[n] for n, _ in sq.sq_rope._fields_])


def _stream_call(L, name, cache, k=AT, v=AT, dtype=sq.SQ_F16, strides=(256, 128, 256, 128), n=4, cu=None, start=AT,
                 rope=None, flags=None):
    args = [ctypes.byref(cache) if cache else None, k, v, dtype, *strides, n, cu, start]
    if name == "sq_kv4_append":
        args.append(ctypes.byref(rope) if rope else None)
    return getattr(L, name)(*args, flags, None)


BAD_CACHES = [dict(pages=0), dict(pages=AT + 8), dict(table=0), dict(table=AT + 2), dict(n_pages=0), dict(batch=0),
              dict(pages_per_row=0), dict(table_stride=3), dict(n_kv_heads=0), dict(page_tokens=8),
              dict(page_tokens=48), dict(page_tokens=2048), dict(pages_per_row=1 << 27, table_stride=1 << 27)]
BAD_ROPES = [dict(table=0), dict(table=AT + 4), dict(n_pos=0), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144)]


@pytest.mark.parametrize("name", ["sq_kv4_append", "sq_kv4_read"])
def test_stream_refusals(L, name):
    for bad in BAD_CACHES:
        assert _stream_call(L, name, _cache(**bad)) == sq.SQ_ERR_ARG, bad
    assert _stream_call(L, name, None) == sq.SQ_ERR_ARG
    assert _stream_call(L, name, _cache(d=96)) == sq.SQ_ERR_UNSUPPORTED
    assert _stream_call(L, name, _cache(), dtype=7) == sq.SQ_ERR_UNSUPPORTED
    for kw in (dict(k=None), dict(v=None), dict(k=AT + 2), dict(v=AT + 8), dict(strides=(255, 128, 256, 128)),
               dict(strides=(256, 4, 256, 128)), dict(strides=(-256, 128, 256, 128)), dict(n=-1), dict(start=None),
               dict(start=AT + 1), dict(cu=AT + 2), dict(flags=AT + 1)):
        assert _stream_call(L, name, _cache(), **kw) == sq.SQ_ERR_ARG, kw
    assert _stream_call(L, name, _cache(), k=None, v=None, n=0) == sq.SQ_OK


def test_append_rotation_refusals(L):
    for bad in BAD_ROPES:
        assert _stream_call(L, "sq_kv4_append", _cache(), rope=_rope(**bad)) == sq.SQ_ERR_ARG, bad
    assert _stream_call(L, "sq_kv4_append", _cache(d=64), rope=_rope()) == sq.SQ_ERR_ARG     # 128 of 64 coordinates


def _decode(L, cache, lens=AT, n_q=8, ctx=64, q=AT, dtype=sq.SQ_F16, strides=(1024, 128), rope=None, window=0, out=AT,
            od=sq.SQ_F16, lse=None, ws=AT, nws=1 << 40, flags=None):
    return L.sq_kv4_attn_decode(ctypes.byref(cache) if cache else None, lens, n_q, ctx, q, dtype, *strides,
                                ctypes.byref(rope) if rope else None, 0.0, window, out, od, lse, ws, nws, flags, None)


def _prefill(L, cache, cu=AT, start=AT, n_q=8, n=4, q=AT, dtype=sq.SQ_F16, strides=(1024, 128), rope=None, window=0,
             out=AT, od=sq.SQ_F16, lse=None, ws=AT, nws=1 << 40, flags=None):
    return L.sq_kv4_attn_prefill(ctypes.byref(cache) if cache else None, cu, start, n_q, n, q, dtype, *strides,
                                 ctypes.byref(rope) if rope else None, 0.0, window, out, od, lse, ws, nws, flags, None)


def _step(L, cache, k=AT, v=AT, q=AT, dtype=sq.SQ_F16, kv=(256, 128, 256, 128), strides=(1024, 128), pos=AT, n_q=8,
          ctx=64, rope=None, window=0, out=AT, od=sq.SQ_F16, lse=None, ws=AT, nws=1 << 40, flags=None):
    return L.sq_kv4_decode_step(ctypes.byref(cache) if cache else None, k, v, q, dtype, *kv, *strides, pos, n_q, ctx,
                                ctypes.byref(rope) if rope else None, 0.0, window, out, od, lse, ws, nws, flags, None)


COMMON = [dict(n_q=7), dict(n_q=0), dict(q=None), dict(q=AT + 2), dict(strides=(1020, 128)), dict(window=-1),
          dict(out=None), dict(out=AT + 4), dict(lse=AT + 2), dict(ws=None), dict(ws=AT + 8), dict(flags=AT + 2)]


@pytest.mark.parametrize("call", [_decode, _prefill, _step])
def test_attention_refusals(L, call):
    for bad in BAD_CACHES:
        assert call(L, _cache(**bad)) == sq.SQ_ERR_ARG, bad
    for bad in BAD_ROPES:
        assert call(L, _cache(), rope=_rope(**bad)) == sq.SQ_ERR_ARG, bad
    for kw in COMMON:
        assert call(L, _cache(), **kw) == sq.SQ_ERR_ARG, kw
    assert call(L, None) == sq.SQ_ERR_ARG
    assert call(L, _cache(d=32)) == sq.SQ_ERR_UNSUPPORTED
    assert call(L, _cache(), dtype=sq.SQ_F32) == sq.SQ_ERR_UNSUPPORTED
    assert call(L, _cache(), od=9) == sq.SQ_ERR_UNSUPPORTED
    assert call(L, _cache(), nws=0) == sq.SQ_ERR_WORKSPACE


def test_own_refusals_of_each_call(L):
    assert _decode(L, _cache(), lens=None) == sq.SQ_ERR_ARG
    assert _decode(L, _cache(), lens=AT + 2) == sq.SQ_ERR_ARG
    assert _decode(L, _cache(), ctx=0) == sq.SQ_ERR_ARG
    assert _prefill(L, _cache(), cu=None) == sq.SQ_ERR_ARG
    assert _prefill(L, _cache(), start=None) == sq.SQ_ERR_ARG
    assert _prefill(L, _cache(), n=-1) == sq.SQ_ERR_ARG
    assert _prefill(L, _cache(), n=0) == sq.SQ_OK
    assert _step(L, _cache(), k=None) == sq.SQ_ERR_ARG
    assert _step(L, _cache(), pos=None) == sq.SQ_ERR_ARG
    assert _step(L, _cache(), kv=(252, 128, 256, 128)) == sq.SQ_ERR_ARG


def test_sizes(L):
    assert L.sq_kv4_page_bytes(2, 128, 32) == 2 * 2 * (16 * 128 + 128)
    assert L.sq_kv4_page_bytes(8, 64, 16) == 8 * (16 * 64 + 128)
    for bad in ((0, 128, 16), (2, 96, 16), (2, 128, 8), (2, 128, 24), (2, 128, 2048)):
        assert L.sq_kv4_page_bytes(*bad) == 0
    assert L.sq_kv4_attn_workspace(4, 8, 2, 128, 100) > 0 and L.sq_kv4_attn_prefill_workspace(4, 8, 2, 128, 100) > 0
    for bad in ((0, 8, 2, 128, 100), (4, 7, 2, 128, 100), (4, 8, 2, 32, 100), (4, 8, 2, 128, 0)):
        assert L.sq_kv4_attn_workspace(*bad) == 0 and L.sq_kv4_attn_prefill_workspace(*bad) == 0


def test_binding_refuses_wrong_tensors():
    table = torch.zeros(2, 4, dtype=torch.int32)
    pages = torch.zeros(8, 2, 1, 16 * 128 + 128, dtype=torch.uint8)
    c = sq.PagedKV4(pages, table, 2, 128, 16)
    assert c.struct().table_stride == 4 and c.batch == 2
    for bad in (dict(pages=pages.float()), dict(pages=pages[:, :1]), dict(table=table.long()), dict(table=table[0]),
                dict(d=64), dict(page_tokens=32)):
        with pytest.raises(ValueError):
            sq.PagedKV4(**{**dict(pages=pages, table=table, n_kv=2, d=128, page_tokens=16), **bad})
    with pytest.raises(ValueError):
        sq.Rope(torch.zeros(4, 16, dtype=torch.float64))
    k = torch.zeros(2, 2, 128, dtype=torch.float16)
    start = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="current device"):            # host tensors never reach a kernel
        sq.sq_kv4_append(c, k, k, start)
    with pytest.raises(ValueError, match="current device"):
        sq.sq_kv4_attn_decode(c, start, k, 0.0, k, 64, torch.zeros(1 << 10, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sq.alloc_kv4(4, 2, 96, 16, table, device="cpu")


def test_page_tables_whose_rows_share_memory_are_refused():
    """A row stride below a row's length would be read past the table; wider rows and a single row are taken."""
    pages = torch.zeros(8, 2, 1, 16 * 128 + 128, dtype=torch.uint8)
    row = torch.arange(4, dtype=torch.int32)[None]
    make = lambda t: sq.PagedKV4(pages, t, 2, 128, 16)  # noqa: E731
    for bad in (row.expand(3, -1), torch.zeros(16, dtype=torch.int32).as_strided((3, 4), (2, 1)),
                torch.zeros(16, dtype=torch.int32).as_strided((2, 4), (3, 1))):
        with pytest.raises(ValueError, match="share memory"):
            make(bad)
        c = make(row)
        c.table = bad                                            # set later, refused by the next call
        with pytest.raises(ValueError, match="share memory"):
            c.ref()
    wide = torch.zeros(3, 10, dtype=torch.int32)
    for t, stride in ((row, 4), (row.expand(1, -1), 4), (row.expand(3, -1).contiguous(), 4), (wide[:, :4], 10), (wide[:, :1], 10),
                      (wide[:1, :4], 4), (torch.zeros(16, dtype=torch.int32).as_strided((1, 4), (1, 1)), 4)):
        s = make(t).struct()
        assert (s.table_stride, s.batch, s.pages_per_row) == (stride, t.shape[0], t.shape[1])


def test_descriptions_follow_tensors_that_change_in_place():
    """Same address, other shape, stride or type: the kept structures are made again, and refused where they do not fit."""
    table = torch.zeros(64, dtype=torch.int32)[:16].view(4, 4)
    pages = torch.zeros(8, 2, 1, 16 * 128 + 128, dtype=torch.uint8)
    c = sq.PagedKV4(pages, table, 2, 128, 16)
    assert c.described()[1].table_stride == 4 and c.ref() is c.ref()
    table.as_strided_((4, 4), (16, 1))
    assert c.described()[1].table_stride == 16
    table.as_strided_((4, 4), (0, 1))
    with pytest.raises(ValueError, match="share memory"):
        c.ref()
    table.as_strided_((4, 4), (4, 1))
    pages.resize_(4, 2, 1, 16 * 128 + 128)
    assert c.described()[1].n_pages == 4
    pages.as_strided_((2, 2, 1, 16 * 128 + 128), (16 * 128 + 128, 2 * (16 * 128 + 128), 16 * 128 + 128, 1))
    with pytest.raises(ValueError, match="contiguous"):
        c.ref()
    rope = sq.Rope(torch.zeros(16, 16))
    assert rope.described()[1].rot_dim == 16
    rope.table.as_strided_((16, 16), (1, 16))
    with pytest.raises(ValueError, match="contiguous"):
        rope.ref()


def test_strides_of_axes_of_one_element_are_not_asked_for():
    """A row or a head taken out of a wider tensor keeps a stride that nothing uses; others are passed on as they are."""
    wide = torch.zeros(5, 2 * 128 + 4, dtype=torch.float16)
    assert sq._kv4_heads("q", wide[:1, :256].unflatten(1, (2, 128)), 2, 128)[1:] == (0, 128)
    assert sq._kv4_heads("q", wide[:3, :256].unflatten(1, (2, 128)), 2, 128)[1:] == (260, 128)
    odd = torch.zeros(4096, dtype=torch.float16).as_strided((3, 1, 128), (256, 1, 1))
    assert sq._kv4_heads("k", odd, 1, 128)[1:] == (256, 0)
    assert sq._kv4_heads("k", odd[:0], 1, 128)[1:] == (0, 0)


def test_copies_of_a_cache_describe_their_own_tensors():
    """After a call has kept its structures too: shallow and deep copies, and pickles."""
    c = sq.PagedKV4(torch.zeros(8, 2, 1, 16 * 128 + 128, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32), 2, 128, 16)
    r = sq.Rope(torch.ones(16, 16), True)
    c.ref(), r.ref()
    for made in (copy.deepcopy((c, r)), pickle.loads(pickle.dumps((c, r)))):
        d, s = made
        assert d.described()[1].pages == d.pages.data_ptr() != c.pages.data_ptr() and d.n_kv == 2
        assert s.described()[1].table == s.table.data_ptr() != r.table.data_ptr() and s.interleaved
    d = copy.copy(c)
    d.table = d.table[:1]
    assert d.described()[1].batch == 1 and c.described()[1].batch == 2


def test_outputs_whose_rows_share_memory_are_refused():
    """Read back into an expanded or overlapping view would leave rows to whichever block wrote last."""
    x = torch.zeros(1 << 16, dtype=torch.float16)
    apart = lambda t: sq._kv4_apart("k_out", t.shape[0], t.shape[1], t.shape[2], *sq._kv4_heads("k_out", t, None, t.shape[2])[1:])  # noqa: E731
    good = [x[:6 * 2 * 64].view(6, 2, 64), x[:6 * 2 * 64].view(2, 6, 64).transpose(0, 1), x[:64 * 200].view(10, 20, 64)[:, 3:5],
            x.as_strided((6, 2, 64), (3 * 64, 64, 1)), x.as_strided((1, 2, 64), (1, 64, 1)), x.as_strided((6, 1, 64), (64, 0, 1)),
            x.as_strided((1, 1, 64), (0, 0, 1)), x.as_strided((0, 2, 64), (0, 64, 1)), x.as_strided((2, 6, 64), (64, 128, 1))]
    bad = [x[:128].view(1, 2, 64).expand(6, -1, -1), x[:384].view(6, 1, 64).expand(-1, 2, -1), x[:64].view(1, 1, 64).expand(6, 2, -1),
           x.as_strided((6, 2, 64), (64, 64, 1)), x.as_strided((6, 2, 64), (128, 32, 1)), x.as_strided((6, 2, 64), (96, 64, 1)),
           x.as_strided((6, 2, 64), (64, 128, 1)), x.as_strided((1, 2, 64), (0, 56, 1)), x.as_strided((3, 1, 64), (56, 0, 1))]
    for t in good:
        apart(t)
    for t in bad:
        with pytest.raises(ValueError, match="share no memory"):
            apart(t)
    rows = lambda t: [set(range(i * t.stride(0) + h * t.stride(1), i * t.stride(0) + h * t.stride(1) + t.shape[2]))  # noqa: E731
                      for i in range(t.shape[0]) for h in range(t.shape[1])]
    for t in good + bad:
        r = rows(t)
        assert (len(set().union(*r)) == sum(map(len, r))) == any(t is g for g in good)

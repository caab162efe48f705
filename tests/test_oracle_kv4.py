"""Pins of the paged 4-bit cache's oracle: the pair and code rules, the layout, the rotation."""

import math

import numpy as np
import pytest

from oracle import kv4


def test_bf16_rounding_is_directed():
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(2000) * 10.0 ** g.integers(-30, 30, 2000), [0.0, 1.0, -1.0, 1.5, -2.75]])
    x = x.astype(np.float32)
    down, up = kv4.bf16_value(kv4.bf16_bits(x, False)), kv4.bf16_value(kv4.bf16_bits(x, True))
    assert np.all(down <= x) and np.all(up >= x)
    assert np.all(up.astype(np.float64) - down <= np.abs(x) * 2.0 ** -7 + 1e-45)
    exact = (x.view(np.uint32) & 0xFFFF) == 0
    assert np.all(down[exact] == x[exact]) and np.all(up[exact] == x[exact])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_quantization_error_is_half_a_step(d):
    g = np.random.default_rng(d)
    x = (g.standard_normal((64, d)) * 10.0 ** g.integers(-6, 4, (64, 1)) + g.standard_normal((64, 1)) * 5).astype(np.float32)
    c, sb, mb = kv4.quantize(x)
    s = kv4.bf16_value(sb).astype(np.float64)
    # half a step, and the float32 rounding of x - m
    assert np.all(np.abs(kv4.values(c, sb, mb) - x) <= 0.5 * s[:, None] * (1 + 2.0 ** -20) + np.abs(x) * 2.0 ** -23)
    assert c.min() == 0 and c.max() == 15


def test_hand_worked_vector():
    x = np.array([0.0, 15.0] + [7.5, 6.5] * 31, np.float32)          # s = 1, m = 0; ties to even: 7.5 -> 8, 6.5 -> 6
    c, sb, mb = kv4.quantize(x)
    assert sb == 0x3F80 and mb == 0
    assert c[:4].tolist() == [0, 15, 8, 6]


def test_constant_and_non_finite_vectors():
    c, sb, mb = kv4.quantize(np.full(64, -2.5, np.float32))
    assert sb == 0 and kv4.bf16_value(mb) == -2.5 and not c.any()
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones(64, np.float32)
        x[7] = bad
        c, sb, mb = kv4.quantize(x)
        assert sb == 0 and mb == 0x7FC0 and not c.any() and np.isnan(kv4.values(c, sb, mb)).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_layout_round_trip_and_disjoint_places(d):
    g = np.random.default_rng(1)
    pages = np.zeros((2, 2, 2, kv4.block_bytes(d)), np.uint8)
    want = {}
    for page in range(2):
        for head in range(2):
            for slot in range(32):
                for side in range(2):
                    v = (g.integers(0, 16, d).astype(np.uint8), int(g.integers(0, 1 << 15)), int(g.integers(0, 1 << 16)))
                    kv4.store(pages, page, head, slot, side, *v)
                    want[page, head, slot, side] = v
    for key, (c, sb, mb) in want.items():
        got = kv4.load(pages, *key)
        assert np.array_equal(got[0], c) and got[1:] == (sb, mb)


def test_layout_by_hand():
    d = 128
    pages = np.zeros((1, 1, 1, kv4.block_bytes(d)), np.uint8)
    codes = np.zeros(d, np.uint8)
    codes[0], codes[1], codes[32] = 3, 5, 9
    kv4.store(pages, 0, 0, 2, 0, codes, 0x3F80, 0xC000)              # token 2: x(t) = 1, chunk 0 at place 1
    b = pages[0, 0, 0]
    assert b[2 * 64 + 16] == 3 | (5 << 4) and b[2 * 64] == 9
    assert b[16 * d + 8:16 * d + 12].tolist() == [0x80, 0x3F, 0x00, 0xC0]


def test_eight_rows_of_a_chunk_fill_eight_bank_groups():
    for d in (64, 128, 256):
        for t0 in (0, 8):
            for chunk in range(d // 32):
                at = [(t * (d // 2) + 16 * (chunk ^ ((t * d // 256) % (d // 32)))) % 128 // 16 for t in range(t0, t0 + 8)]
                assert sorted(at) == list(range(8))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(interleaved):
    g = np.random.default_rng(2)
    tab = kv4.rope_table(64, 32)
    q, k = g.standard_normal((1, 64)), g.standard_normal((1, 64))
    same = lambda y: y  # noqa: E731
    dots = [float((kv4.rotate(q, tab, p + 9, interleaved, same)[0].astype(np.float64)
                   * kv4.rotate(k, tab, p, interleaved, same)[0]).sum()) for p in (0, 5, 40)]
    assert max(dots) - min(dots) < 1e-4
    y = kv4.rotate(q, tab, 13, interleaved, same)[0]
    assert np.allclose(y[32:], q[0, 32:].astype(np.float32)) and math.isclose(
        float(np.linalg.norm(y)), float(np.linalg.norm(q)), rel_tol=1e-6)


def test_attention_against_dense_softmax():
    g = np.random.default_rng(3)
    q, k, v = g.standard_normal(64), g.standard_normal((37, 64)), g.standard_normal((37, 64))
    o, lse, b = kv4.attend(q, k, v, 0.125, np.abs(v))
    e = np.exp(0.125 * (k @ q))
    assert np.allclose(o, e @ v / e.sum()) and math.isclose(lse, math.log(e.sum())) and np.all(b >= np.abs(o))
    o, lse, _ = kv4.attend(q, k[:0], v[:0], 0.125)
    assert not o.any() and lse == -math.inf


def test_ranges_that_are_no_finite_float_read_as_nan():
    """Finite vectors up to the largest float, and those whose range or rounded minimum passes it."""
    top = float(np.finfo(np.float32).max)
    bf = 255 * 2.0 ** 120                                            # the largest bf16
    for lo, hi, held in ((0.0, top, True), (-bf, 0.0, True), (-bf / 2, bf / 2, True), (-top, 0.0, False), (-bf, bf, False),
                         (-bf, 2.0 ** 127, False), (top, top, True), (-bf, -bf, True)):
        x = np.full(64, lo, np.float32)
        x[1::2] = hi
        c, sb, mb = kv4.quantize(x)
        y = kv4.values(c, sb, mb)
        assert np.isnan(y).all() == (not held) and (held or (sb == 0 and mb == 0x7FC0 and not c.any())), (lo, hi)
        if held:
            assert np.all(np.abs(y - x) <= 0.5 * float(kv4.bf16_value(sb)) * (1 + 2.0 ** -20) + 2.0 ** -7 * abs(lo) * (lo == hi))


def test_corrected_product_is_the_rounded_quotient_by_fifteen():
    """r y, y the rounded 1 / 15, and one correction q + (r - 15 q) y, each rounded to 24 bits, give r / 15 rounded: for every
    significand, in whole numbers (exponents only shift them while r / 15 is normal)."""
    r = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    y = 8947849                                                      # of 2^-27: 1 / 15 rounded to 24 bits
    assert abs(y * 15 - (1 << 27)) * 2 < 15 and 1 << 23 <= y < 1 << 24
    assert np.float32(1) / np.float32(15) == np.float32(y * 2.0 ** -27)

    def nearest(x, by):                                              # x / 2^by, ties to even
        q, rest = x >> by, x & ((np.int64(1) << by) - 1)
        half = np.int64(1) << (by - 1)
        return q + ((rest > half) | ((rest == half) & (q & 1 == 1)))

    p = r * y                                                        # of 2^-27
    by = np.where(p < 1 << 47, 23, 24)
    q = nearest(p, by) << by                                         # of 2^-27, 24 bits
    assert np.all(q >> by <= 1 << 24)                                # a float
    rest = (r << 27) - 15 * q                                        # of 2^-27: a float, its low bits are 0
    bits = rest >> 23
    assert np.all(bits << 23 == rest) and np.abs(bits).max() < 1 << 24
    s = (q << 4) + bits * y                                          # of 2^-31: (q 2^-27) + (bits 2^-4)(y 2^-27)
    by = np.where(s < 1 << 51, 27, 28)
    got = nearest(s, by) << by                                       # of 2^-31
    # r / 15 to 24 bits: no tie can occur, as 15 is odd and r has 24 bits
    unit = np.where(r < 15 << 20, 4, 3)                              # r 2^unit / 15 in [2^23, 2^24)
    z = r << unit
    want = (z // 15 + (z % 15 > 7)) << (31 - unit)                   # of 2^-31
    assert np.array_equal(got, want)

"""Pins of oracle/cache_oracle.py: closed forms and brute force."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import cache_oracle as co


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_complex_numbers(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 16))
    pos = np.array([0, 1, 7, 100, -3])
    inv = 10000.0 ** (-np.arange(4) / 4.0)
    y, scale = co.qk_norm_rope(x, pos, inv, None, 0.0, interleaved)
    for t in range(5):
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
            z = (x[t, :, a] + 1j * x[t, :, b]) * np.exp(1j * pos[t] * inv[i])
            np.testing.assert_allclose(y[t, :, a], z.real, atol=1e-12)
            np.testing.assert_allclose(y[t, :, b], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.all(np.abs(y) <= scale + 1e-12)


def test_norm_has_unit_mean_square_and_rotation_keeps_it():
    rng = np.random.default_rng(1)
    x = 3.0 * rng.standard_normal((4, 3, 64))
    y, _ = co.qk_norm_rope(x, np.arange(4) * 1000, np.ones(32), np.ones(64), 0.0, False)
    np.testing.assert_allclose(np.mean(y * y, -1), 1.0, rtol=1e-12)


def test_far_positions_against_whole_numbers():
    """Angle p * 2 pi / m for whole p, m: the exact remainder p mod m."""
    m, p = 1000, 2147483647
    inv = np.array([2 * np.pi / m])
    x = np.zeros((1, 1, 8))
    x[..., 0] = 1.0
    y, _ = co.qk_norm_rope(x, [p], inv, None, 0.0, False)
    # 2 pi / m rounded to fp64: off by 2^-53 relative, p times that at most 3e-10 * p / 2^31
    np.testing.assert_allclose(y[0, 0, 0], np.cos(2 * np.pi * (p % m) / m), atol=1e-8 * 20)


def test_every_code_and_every_midpoint():
    scale = 0.75
    vals = [v * scale for v in co.E2M1] + [-v * scale for v in co.E2M1[1:]]
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    to = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]                # ties to the even code
    x = np.array(vals + [m * scale for m in mids])
    x = np.concatenate([x, np.zeros(32 - len(x))])
    code, s = co.q4_quantise(x)
    assert s[0] == scale
    np.testing.assert_array_equal(co.q4_value(code, s)[:15], vals)
    np.testing.assert_array_equal(co.q4_value(code, s)[15:22], np.array(to) * scale)


def test_nearest_by_fractions():
    rng = np.random.default_rng(2)
    x = co.round_bf16(rng.standard_normal(320)).reshape(10, 32)
    code, s = co.q4_quantise(x)
    v = co.q4_value(code, s)
    for row in range(10):
        f = Fraction(float(s[row, 0]))
        for i in range(32):
            got = abs(Fraction(float(v[row, i])) - Fraction(float(x[row, i])))
            best = min(abs(sg * f * Fraction(float(e)) - Fraction(float(x[row, i])))
                       for e in co.E2M1 for sg in (1, -1))
            assert got == best


def test_round_bf16():
    assert co.round_bf16(1.0 + 2.0 ** -8) == 1.0            # tie to even
    assert co.round_bf16(1.0 + 3 * 2.0 ** -8) == 1.0 + 2.0 ** -6
    assert co.round_bf16(-0.1) == -0.10009765625


def test_non_finite_and_tiny_groups():
    x = np.zeros((4, 32))
    x[0, 3] = np.inf
    x[1, 5] = np.nan
    x[2, 7] = 2.0 ** -127
    x[3, :] = 1.0
    code, s = co.q4_quantise(x)
    assert np.isnan(s[0, 0]) and np.isnan(s[1, 0]) and s[2, 0] == 0.0
    assert not code[:3].any() and np.all(co.q4_value(code, s)[3] == 6 * s[3, 0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 64])
def test_places_tile_the_page(d, bs):
    seen = set()
    for which in (0, 1):
        for off in range(bs):
            for dim in range(d):
                seen.add(co.q4_place(which, bs, d, off, dim))
            for g in range(d // 32):
                b = co.q4_scale_place(which, bs, d, off, g)
                seen |= {(b + k, sh) for k in (0, 1) for sh in (0, 4)}
    assert len(seen) == 2 * bs * d * 9 // 8
    assert max(b for b, _ in seen) == bs * d * 9 // 8 - 1


def test_reserve_release_round_trip():
    rng = np.random.default_rng(3)
    bs, n, blocks = 16, 6, 40
    table = np.full((n, 12), -1)
    length, free, count = np.zeros(n, int), rng.permutation(blocks), blocks
    seen = {}
    for step in range(8):
        new = rng.integers(0, 30, n)
        slots, cu, length2, count, table, bits = co.cache_reserve(new, length, table, free, count,
                                                                  bs, 300)
        used = slots[slots >= 0]
        assert len(set(used)) == len(used)
        for s in range(n):
            mine = slots[cu[s]:cu[s + 1]]
            assert (mine >= 0).all() if length2[s] > length[s] else (mine < 0).all()
            for x in mine[mine >= 0]:
                assert x not in seen
                seen[x] = s
        length = length2
    assert bits & 0x20                                      # forty blocks do not last eight steps
    held = sum(-(-x // bs) for x in length)
    assert count + held == blocks
    length, table, free, count, bits = co.cache_release(np.ones(n), length, table, free, count, bs)
    assert count == blocks and sorted(free) == list(range(blocks)) and (table == -1).all()
    assert bits == 0 and not length.any()


def test_decode_closed_forms():
    q = np.ones((4, 64))
    V = np.random.default_rng(4).standard_normal((2, 5, 64))
    out, lse = co.q4_decode_attention(q, np.zeros((2, 5, 64)), V)
    np.testing.assert_allclose(out, np.repeat(V.mean(1), 2, axis=0))
    np.testing.assert_allclose(lse, np.log(5.0))
    out, lse = co.q4_decode_attention(q, np.zeros((2, 0, 64)), V[:, :0])
    assert not out.any() and np.isneginf(lse).all()

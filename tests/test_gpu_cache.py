"""The operators around the 4-bit paged cache on the GPU, against
oracle/cache_oracle.py in fp64 (or in whole numbers, then equal).

Tolerances (u = 2^-24, fp32; a bf16 rounding is off by at most 2^-8 of the
value, half its eps; fp16 by 2^-11):

* rope: the sum of 128 squares is off by at most 128 u = 2^-17 relative, its
  root by half; rsqrt and three products add at most 6 u; cos and sin are off
  by at most 2^-22 (argument to 2^-25 of a half turn).  Together below 2^-17
  of |y1| + |y2|, then one bf16 rounding.
* rows: exact (codes, scales and the one rounding to bf16).
* attention: p (times V's scale) is rounded to fp16: 2^-11 of sum_j p_j |V_j|
  at most; fp32 sums, 2^x and logits add below 2^-13 of it for the logits of
  these tests (|logit| <= 2^7: 128 * 2^-23 * 2^7 / 8 is under 2^-13, u per
  addition); then one bf16 rounding.  The LSE has the logits' error alone.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from prefill_eviction_scoring_b200 import _lib, api
from prefill_eviction_scoring_b200 import workloads as wl

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ rope

def _check_rope(q, k, pos, inv, qw, kw, eps, interleaved, got):
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        ref, scale = co.qk_norm_rope(_f64(x), pos.cpu().numpy(), inv.numpy(),
                                     None if w is None else _f64(w), eps, interleaved)
        assert y.shape == x.shape and y.dtype == torch.bfloat16
        err = np.abs(_f64(y) - ref)
        assert np.all(err <= BF * np.abs(ref) + 2.0 ** -17 * scale + 1e-38), err.max()


@pytest.mark.parametrize("T", [1, 3, 130])
@pytest.mark.parametrize("heads", [(32, 8), (28, 4), (1, 1), (7, 1)])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 24), (64, 64), (64, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(T, heads, d, rot, interleaved):
    g = _gen(T + rot)
    q, k = _bf(g, T, heads[0], d), _bf(g, T, heads[1], d)
    pos = torch.randint(-5, 200000, (T,), generator=g, device="cuda", dtype=torch.int32)
    inv = api.rotary_inv_freq(rot, 500000.0)
    w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    for qw, kw in ((w[0], w[1]), (None, None)):
        got = api.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, eps=1e-5,
                               interleaved=interleaved)
        _check_rope(q, k, pos, inv, qw, kw, 1e-5, interleaved, got)


def test_rope_far_positions_and_large_frequencies():
    pos = _i32([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 123456789, 0, -1])
    g = _gen(1)
    q, k = _bf(g, 6, 4, 64), _bf(g, 6, 2, 64)
    for inv in (api.rotary_inv_freq(64, 10000.0), api.rotary_inv_freq(64, 10000.0) * 7.5,
                -api.rotary_inv_freq(64, 10000.0)):
        _check_rope(q, k, pos, inv, None, None, 0.0, False, api.qk_norm_rope(q, k, pos, inv))


@pytest.mark.parametrize("d", [64, 128])
def test_rope_views_and_in_place(d):
    T, Hq, Hkv = 37, 12, 3
    g = _gen(2)
    qkv = _bf(g, T, (Hq + 2 * Hkv) * d)
    q = qkv[:, :Hq * d].view(T, Hq, d)
    k = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    inv = api.rotary_inv_freq(d, 10000.0)
    w = (1 + 0.3 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    got = api.qk_norm_rope(q, k, pos, inv, q_weight=w[0], k_weight=w[1])
    _check_rope(q, k, pos, inv, w[0], w[1], 1e-6, False, got)
    v = qkv[:, (Hq + Hkv) * d:].clone()
    api.qk_norm_rope(q, k, pos, inv, q_weight=w[0], k_weight=w[1], out=(q, k))
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])
    assert torch.equal(qkv[:, (Hq + Hkv) * d:], v)
    # into a wider buffer: nothing between the rows is touched
    wide = torch.full((T, Hq * d + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    wide_k = torch.full((T, Hkv * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    src = _bf(g, T, Hq, d), _bf(g, T, Hkv, d)
    ref = api.qk_norm_rope(*src, pos, inv)
    api.qk_norm_rope(*src, pos, inv, out=(wide[:, :Hq * d].view(T, Hq, d),
                                          wide_k[:, :Hkv * d].view(T, Hkv, d)))
    assert torch.equal(wide[:, :Hq * d].reshape(T, Hq, d), ref[0])
    assert torch.equal(wide_k[:, :Hkv * d].reshape(T, Hkv, d), ref[1])
    assert (wide[:, Hq * d:] == 7).all() and (wide_k[:, Hkv * d:] == 7).all()


def test_rope_magnitudes_zero_rows_and_nan():
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    q[1] = 1e-20
    q[2] = 1e15
    q[3, 0] = float("nan")
    q[3, 1] = 1.0
    one = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, _ = api.qk_norm_rope(q, q, pos, api.rotary_inv_freq(128, 1e4), q_weight=one,
                              k_weight=one, eps=1e-6)
    assert not out[0].any() and torch.isnan(out[3, 0]).all()
    assert (out[2] == 1).all() and (out[3, 1] == 1).all()       # mean square 1 at position 0
    assert torch.isfinite(out[1]).all()


def test_rope_empty():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    out = api.qk_norm_rope(q, q, pos, api.rotary_inv_freq(64, 1e4))
    assert out[0].shape == (0, 4, 64)


# ------------------------------------------------------------------ block tables

def _reserve_case(seed, n, bs, width, num_blocks, hi, new_hi, held=True):
    rng = np.random.default_rng(seed)
    order = rng.permutation(num_blocks)
    length = rng.integers(0, hi + 1, n)
    new = rng.integers(0, new_hi + 1, n)
    table = np.full((n, width), -1)
    at = 0
    for s in range(n):
        nb = min(-(-length[s] // bs), width, num_blocks - at)
        length[s] = min(length[s], nb * bs)
        table[s, :nb] = order[at:at + nb]
        at += nb
    free = np.zeros(num_blocks, int)
    free[:num_blocks - at] = order[at:]
    return new, length, table, free, num_blocks - at


def _check_reserve(new, length, table, free, count, bs, max_new):
    want = co.cache_reserve(new, length, table, free, count, bs, max_new)
    for in_place in (False, True):
        t, l, c = _i32(table), _i32(length), _i32([count])
        status = _i32([0])
        slots, cu, l2, c2 = api.cache_reserve(_i32(new), l, t, _i32(free), c, block_size=bs,
                                              max_new=max_new, in_place=in_place, status=status)
        assert np.array_equal(slots.cpu().numpy(), want[0])
        assert np.array_equal(cu.cpu().numpy(), np.minimum(want[1], 2 ** 31 - 1))
        assert np.array_equal(l2.cpu().numpy(), want[2]) and int(c2) == want[3]
        assert np.array_equal(t.cpu().numpy(), want[4])
        assert int(status) == want[5]
        assert (l2 is l) == in_place and (in_place or np.array_equal(l.cpu().numpy(), length))


@pytest.mark.parametrize("n", [1, 31, 1025, 8192])
@pytest.mark.parametrize("bs", [16, 256])
def test_reserve_random(n, bs):
    for seed, (hi, new_hi, spare) in enumerate([(0, 40, 0), (300, 1, 5), (300, 70, -n // 3),
                                                (17, 17, -1), (0, 0, 0)]):
        width = (hi + new_hi) // bs + 1
        new, length, table, free, count = _reserve_case(
            seed, n, bs, width, max(1, n * width + spare), hi, new_hi)
        _check_reserve(new, length, table, free, count, bs, int(new.sum()) + 7)


def test_reserve_long_prompts_and_short_slot_map():
    new, length, table, free, count = _reserve_case(5, 5, 64, 2200, 9000, 0, 130000)
    new[2] = 131072
    for max_new in (int(new.sum()), int(new.sum()) + 1001, int(new[:3].sum()) + 5, 0, 3):
        _check_reserve(new, length, table, free, count, 64, max_new)


def test_reserve_refusals_and_bad_blocks():
    bs, width, blocks = 16, 4, 12
    table = np.full((8, width), -1)
    table[0, 0], table[1, 0], table[2, 0], table[7, 0] = 3, 99, -5, 4
    length = np.array([5, 5, 5, -1, 0, 0, 0, 16])
    new = np.array([1, 1, 1, 1, -2, 65, 64, 16])
    free = np.array([0, 1, 2, 5, 77, 7, 8, 9, 10, 11, 0, 0])
    _check_reserve(new, length, table, free, 10, bs, 200)
    # a count outside the list is cut to it
    _check_reserve(new, length, table, free, -3, bs, 200)
    _check_reserve(new, length, table, free, 99, bs, 200)
    # sums past 31 bits
    big = np.full(8, 2 ** 30)
    _check_reserve(big, np.zeros(8, int), table, free, 10, bs, 64)


def test_reserve_starved_keeps_order():
    """Five free blocks: the first asks 3, the second 4 (refused), the third
    1 (refused too: a later one does not overtake), the fourth none."""
    table = np.full((4, 6), -1)
    table[3, 0] = 5
    _check_reserve(np.array([48, 64, 1, 3]), np.array([0, 0, 0, 9]), table, np.arange(6), 5, 16,
                   200)


def test_reserve_without_slot_map():
    lib = _lib.load()
    new, length, table, free, count = _reserve_case(3, 9, 16, 6, 60, 30, 40)
    want = co.cache_reserve(new, length, table, free, count, 16, 1000)
    t = [_i32(x) for x in (new, length, table, free, [count])]
    st = lib.waits_cache_reserve(9, 16, 6, 60, 1000, *(x.data_ptr() for x in t), t[1].data_ptr(),
                                 t[4].data_ptr(), None, None, None,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert np.array_equal(t[1].cpu().numpy(), want[2]) and np.array_equal(t[2].cpu().numpy(), want[4])
    assert int(t[4]) == want[3]


@pytest.mark.parametrize("n,width", [(1, 3), (40, 37), (1500, 5), (8192, 2)])
def test_release(n, width):
    bs = 16
    rng = np.random.default_rng(n)
    _, length, table, free, count = _reserve_case(n, n, bs, width, n * width + 3, width * bs, 0)
    if n > 30:
        length[7] = -4
        length[9] = width * bs + 100
        table[11, 0], table[12, 0] = n * width + 3, -1
        length[11] = length[12] = 16
    for ended in (rng.integers(0, 2, n), np.ones(n, int), np.zeros(n, int)):
        want = co.cache_release(ended, length, table, free, count, bs)
        a = _i32(length), _i32(table), _i32(free), _i32([count])
        status = _i32([0])
        api.cache_release(_i32(ended), *a, block_size=bs, status=status)
        assert np.array_equal(a[0].cpu().numpy(), want[0])
        assert np.array_equal(a[1].cpu().numpy(), want[1])
        assert int(a[3]) == want[3]
        assert np.array_equal(a[2].cpu().numpy(), want[2])
        assert int(status) == want[4]


# ------------------------------------------------------------------ rows

def _pool(blocks, Hkv, bs, d, fill=0xA5):
    return torch.full((blocks, Hkv, bs * d * 9 // 8), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs,Hkv", [(16, 3), (64, 1), (256, 2)])
def test_append_bytes_and_read(d, bs, Hkv):
    blocks, n = 3, 29
    g = _gen(d + bs)
    K, V = _bf(g, n, Hkv, d) * 3, _bf(g, n, Hkv, d)
    K[0] = 0
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:n].int()
    slots[4] = -1
    slots[9] = blocks * bs          # past the pool
    slots[10] = 2 ** 31 - 1
    pool = _pool(blocks, Hkv, bs, d)
    want = pool.cpu().numpy().copy()
    status = _i32([0])
    api.q4_append(K, V, slots, pool, status=status)
    Kn, Vn = _f64(K), _f64(V)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < blocks * bs:
            co.q4_write(want, s, Kn[i], Vn[i], bs)
    assert np.array_equal(pool.cpu().numpy(), want)       # the written bytes, and only those
    assert int(status) == _lib.DEV_BAD_INDEX
    Kr, Vr = api.q4_read(pool, slots, d)
    ok = ((slots >= 0) & (slots < blocks * bs)).cpu().numpy()[:, None, None]
    for x, y in ((Kn, Kr), (Vn, Vr)):
        ref = co.round_bf16(co.q4_value(*co.q4_quantise(x)))
        assert np.array_equal(_f64(y), np.where(ok, ref, 0.0))


def test_append_every_bf16_value():
    """Every bf16 pattern quantised beside a group maximum that makes it land
    in, on and between the codes; non-finite and tiny groups among them."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16)
    rows = torch.empty((65536, 1, 64), dtype=torch.bfloat16, device="cuda")
    m = torch.tensor([1, 0.5, 0.25, 1.25, 1 / 3, 2.4, 0.8, 6.5, 13.0, 0.09], device="cuda")
    for j in range(64):
        rows[:, 0, j] = (x.float() * m[j % 10] * (-1.0) ** j).to(torch.bfloat16)
    rows[:, 0, 0] = x
    rows[:, 0, 32] = x
    pool = _pool(4096, 1, 16, 64)
    slots = torch.arange(65536, dtype=torch.int32, device="cuda")
    api.q4_append(rows, rows, slots, pool)
    K, V = api.q4_read(pool, slots, 64)
    ref = co.q4_value(*co.q4_quantise(_f64(rows)))
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(_f64(K)), ~fin)
    # products below the normal range round in bf16's subnormals: 2^-134 at most
    big = fin & (np.abs(ref) >= 2.0 ** -126)
    assert np.array_equal(_f64(K)[big], co.round_bf16(ref[big]))
    small = fin & ~big
    assert np.all(np.abs(_f64(K)[small] - ref[small]) <= 2.0 ** -134)
    assert torch.equal(K.view(torch.int16), V.view(torch.int16))


def test_append_strided_views():
    g = _gen(8)
    qkv = _bf(g, 21, 10 * 64)
    K, V = qkv[:, 4 * 64:6 * 64].view(21, 2, 64), qkv[:, 8 * 64:].view(21, 2, 64)
    slots = torch.arange(21, dtype=torch.int32, device="cuda") * 3
    a, b = _pool(4, 2, 16, 64), _pool(4, 2, 16, 64)
    api.q4_append(K, V, slots, a)
    api.q4_append(K.contiguous(), V.contiguous(), slots, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("d,Hkv,bs,B", [(128, 2, 16, 70), (64, 3, 64, 33), (128, 1, 256, 300)])
def test_compact(d, Hkv, bs, B):
    lens = (500, 0, 20, 301)
    lay = wl.random_layer(lens, Hkv, Hkv, d, seed=B, device="cuda")
    scores = torch.rand((Hkv, lay.total_tokens), generator=_gen(B), device="cuda")
    idx, kept = api.select(scores, lay.cu_seqlens, recent_budget=8, budget=B)
    width = -(-B // bs) + 1
    table = torch.randperm(4 * width + 2, generator=_gen(3), device="cuda")[:4 * width]
    table = table.int().view(4, width).contiguous()
    pool = _pool(4 * width + 2, Hkv, bs, d)
    want = pool.cpu().numpy().copy()
    status = _i32([0])
    api.q4_compact(lay.K, lay.V, lay.cu_seqlens, idx, kept, table, pool, status=status)
    Kn, Vn, ix = _f64(lay.K), _f64(lay.V), idx.cpu().numpy()
    cu, tb = lay.cu_seqlens.cpu().numpy(), table.cpu().numpy()
    for s in range(4):
        for j in range(int(kept[s])):
            rows = cu[s] + ix[s, :, j]
            co.q4_write(want, int(tb[s, j // bs]) * bs + j % bs, Kn[rows, np.arange(Hkv)],
                        Vn[rows, np.arange(Hkv)], bs)
    assert np.array_equal(pool.cpu().numpy(), want)
    assert int(status) == 0
    # bad indices and blocks: skipped and flagged, the rest written
    idx2, table2 = idx.clone(), table.clone()
    idx2[0, 0, 3], idx2[2, Hkv - 1, 0], idx2[3, 0, 1] = 500, -7, 2 ** 31 - 1
    table2[3, 0] = 4 * width + 2
    pool2 = _pool(4 * width + 2, Hkv, bs, d)
    api.q4_compact(lay.K, lay.V, lay.cu_seqlens, idx2, kept, table2, pool2, status=status)
    assert int(status) == _lib.DEV_BAD_INDEX
    same = (pool2 == pool).view(-1, bs * d * 9 // 8)
    assert torch.equal(pool2[table[0, 1].long()], pool[table[0, 1].long()])
    assert not same.all() and (pool2[table[3, 0].long()] == 0xA5).all()


# ------------------------------------------------------------------ attention

def _fill(g, lens, Hkv, d, bs, kmul=None, vmul=None, spare=5):
    """A pool whose slots hold random rows (NaN bytes elsewhere), its table,
    and the stored values of every sequence, [Hkv, n, d] fp64 each."""
    nseq, cap = len(lens), max(max(lens), 1)
    width = -(-cap // bs) + 1
    blocks = nseq * width + spare
    perm = torch.randperm(blocks, generator=g, device="cuda")[:nseq * width].int()
    table = perm.view(nseq, width).contiguous()
    pool = _pool(blocks, Hkv, bs, d, fill=0xFF)
    kv = []
    for s, n in enumerate(lens):
        K, V = _bf(g, n, Hkv, d), _bf(g, n, Hkv, d)
        if n and kmul is not None:
            K = (K.float() * kmul(s, n)).to(torch.bfloat16)
        if n and vmul is not None:
            V = (V.float() * vmul(s, n)).to(torch.bfloat16)
        j = torch.arange(n, device="cuda")
        slots = (table[s, j // bs] * bs + j % bs).int()
        if n:
            api.q4_append(K, V, slots, pool)
        kv.append([co.q4_value(*co.q4_quantise(_f64(x))).transpose(1, 0, 2) for x in (K, V)])
        table[s, -(-n // bs):] = -1
    return pool, table, kv


def _check_attend(q, pool, table, lens, kv, lse_tol=2.0 ** -13):
    status = _i32([0])
    out, lse = api.q4_decode_attention(q, pool, table, _i32(lens), with_lse=True, status=status)
    assert int(status) == 0
    o, l, qn = _f64(out), _f64(lse), _f64(q)
    for s, (K, V) in enumerate(kv):
        ref, rl = co.q4_decode_attention(qn[s], K, V)
        mag, _ = co.q4_decode_attention(qn[s], K, np.abs(V))
        err = np.abs(o[s] - ref)
        assert np.all(err <= BF * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * mag + 1e-37), \
            (s, (err / (mag + 1e-37)).max())
        fin = np.isfinite(rl)
        assert np.all(np.abs(l[s][fin] - rl[fin]) <= lse_tol)
        assert np.all(np.isneginf(l[s][~fin])) and not o[s][~fin].any()
    return out, lse


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 700, 255, 33]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (28, 4), (4, 4), (8, 1), (18, 2), (16, 1)])
@pytest.mark.parametrize("bs", [16, 64])
def test_attend_ragged(d, Hq, Hkv, bs):
    g = _gen(d + Hq + bs)
    pool, table, kv = _fill(g, LENS, Hkv, d, bs)
    _check_attend(_bf(g, len(LENS), Hq, d), pool, table, LENS, kv)


@pytest.mark.parametrize("nseq,n,bs", [(1, 5003, 16), (2, 12289, 256), (1, 1, 128), (300, 40, 32)])
def test_attend_lengths(nseq, n, bs):
    g = _gen(n)
    lens = [max(0, n - 7 * i) for i in range(nseq)]
    pool, table, kv = _fill(g, lens, 2, 128, bs)
    _check_attend(_bf(g, nseq, 8, 128), pool, table, lens, kv)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_rising_logits_and_mixed_scales(d):
    """Keys that grow along the cache (every tile raises the maximum), V rows
    and V groups over thirty powers of two."""
    g = _gen(17)
    lens = [900, 2100]

    def kmul(s, n):
        return (torch.arange(n, device="cuda")[:, None, None] / n) * 2.0

    def vmul(s, n):
        e = torch.randint(-15, 16, (n, 1, 1), generator=g, device="cuda").float()
        grp = torch.arange(d, device="cuda").view(1, 1, d) // 32
        return torch.exp2(e if s == 0 else -8.0 * grp + 0 * e)

    pool, table, kv = _fill(g, lens, 2, d, 16, kmul, vmul)
    _check_attend(_bf(g, 2, 14, d), pool, table, lens, kv)


@pytest.mark.parametrize("power", [-100, -30, -16, 16, 30, 100])
def test_attend_magnitudes_of_v(power):
    g = _gen(18)
    pool, table, kv = _fill(g, [200, 3], 1, 64, 32, None, lambda s, n: 2.0 ** power)
    _check_attend(_bf(g, 2, 4, 64), pool, table, [200, 3], kv)


@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_attend_magnitudes_of_q(power):
    """Queries and keys whose product is of ordinary size, far from it alone."""
    g = _gen(19)
    pool, table, kv = _fill(g, [200, 3], 1, 64, 32, lambda s, n: 2.0 ** -power)
    q = (_bf(g, 2, 4, 64).float() * 2.0 ** power).to(torch.bfloat16)
    _check_attend(q, pool, table, [200, 3], kv)


def test_attend_one_key_dominates():
    """A sink: one logit far above the rest, first, last and in the middle."""
    g = _gen(20)
    for at in (0, 333, 699):
        pool, table, kv = _fill(g, [700], 2, 128, 16, lambda s, n: torch.where(
            torch.arange(n, device="cuda") == at, 6.0, 0.3)[:, None, None])
        _check_attend(_bf(g, 1, 8, 128), pool, table, [700], kv)


def test_attend_bad_table_entries_are_left_out():
    g = _gen(21)
    bs, n = 16, 200
    pool, table, kv = _fill(g, [n, n], 2, 128, bs)
    table[0, 3], table[0, 12], table[1, 0] = -1, pool.shape[0], 2 ** 31 - 1
    keep = [np.ones(n, bool), np.ones(n, bool)]
    keep[0][48:64] = keep[0][192:] = False
    keep[1][:16] = False
    status = _i32([0])
    q = _bf(g, 2, 8, 128)
    out, lse = api.q4_decode_attention(q, pool, table, _i32([n, n]), True, status=status)
    assert int(status) == _lib.DEV_BAD_INDEX
    for s in range(2):
        K, V = (x[:, keep[s]] for x in kv[s])
        ref, rl = co.q4_decode_attention(_f64(q[s]), K, V)
        mag, _ = co.q4_decode_attention(_f64(q[s]), K, np.abs(V))
        assert np.all(np.abs(_f64(out[s]) - ref) <= BF * np.abs(ref) + 2.0 ** -10 * mag)
        assert np.all(np.abs(_f64(lse[s]) - rl) <= 2.0 ** -13)
    table[:] = -1
    out, lse = api.q4_decode_attention(q, pool, table, _i32([n, n]), True)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("entry", [-1, -2, -2 ** 31])
@pytest.mark.parametrize("columns", [2, 9000])
@pytest.mark.parametrize("n", [17, 32])
def test_attend_every_negative_table_entry_sets_the_status(entry, columns, n):
    g = _gen(23)
    pool, table, _ = _fill(g, [n], 1, 64, 16)
    wide = torch.full((1, columns), entry, dtype=torch.int32, device="cuda")
    wide[:, :2] = table[:, :2]
    status = _i32([0])
    q = _bf(g, 1, 2, 64)
    a = api.q4_decode_attention(q, pool, wide, _i32([n]), status=status)
    assert int(status) == 0                        # entries past the length are not looked at
    wide[0, 1] = entry
    b = api.q4_decode_attention(q, pool, wide, _i32([n]), status=status)
    assert int(status) == _lib.DEV_BAD_INDEX
    assert not torch.equal(a, b)
    c = api.q4_decode_attention(q, pool, wide, _i32([16]))
    assert torch.equal(b, c)


def test_attend_lengths_out_of_range_are_clamped():
    g = _gen(22)
    pool, table, kv = _fill(g, [64, 64], 2, 64, 16)
    table = table[:, :4].contiguous()
    q = _bf(g, 2, 4, 64)
    a = api.q4_decode_attention(q, pool, table, _i32([64, 0]))
    b = api.q4_decode_attention(q, pool, table, _i32([2 ** 31 - 1, -9]))
    assert torch.equal(a, b) and not b[1].any()


def test_attend_nan_in_a_used_row_stays_in_its_sequence():
    g = _gen(23)
    lens = [100, 100]
    pool, table, kv = _fill(g, lens, 2, 64, 16)
    V = _bf(g, 1, 2, 64)
    K = V.clone()
    V[0, 1, 40] = float("inf")                     # head 1, group 1 of one token
    api.q4_append(K, V, (table[0, 2] * 16 + 5).view(1), pool)
    out = api.q4_decode_attention(_bf(g, 2, 4, 64), pool, table, _i32(lens))
    assert torch.isnan(out[0, 2:, 32:]).all()
    assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()


def test_attend_is_deterministic_and_workspace_needs_no_clearing():
    g = _gen(24)
    lens = [3000, 17, 0, 4097]
    pool, table, kv = _fill(g, lens, 4, 128, 64)
    q = _bf(g, 4, 16, 128)
    n = max(16, api.q4_decode_workspace_bytes(pool, 4, 16, 128))
    runs = []
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        runs.append(api.q4_decode_attention(q, pool, table, _i32(lens), True, workspace=ws))
        runs.append(api.q4_decode_attention(q, pool, table, _i32(lens), True, workspace=ws))
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


# ------------------------------------------------------------------ together

def _flow(d, Hq, Hkv, bs, B, lens, steps, graph):
    """Prompt: rotate, compress, into the 4-bit cache; then decode steps."""
    nseq, T = len(lens), sum(lens)
    g = _gen(31)
    qkv = _bf(g, T, (Hq + 2 * Hkv) * d)
    q, k, v = (qkv[:, a * d:b * d].view(T, b - a, d) for a, b in
               ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
    pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lens])
    inv = api.rotary_inv_freq(d, 500000.0)
    w = (1 + 0.2 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
    qr, kr = api.qk_norm_rope(q, k, pos, inv, q_weight=w[0], k_weight=w[1])
    Ko, Vo, idx, kept, _ = api.compress(qr, kr, v.contiguous(), cu, sigmoid_a=1.0, window=16,
                                        recent_budget=8, budget=B)
    cache = api.Q4Cache(nseq, Hq, Hkv, d, num_blocks=nseq * (B // bs + 3), max_blocks=B // bs + 3,
                        block_size=bs)
    cache.compact(kr, v.contiguous(), cu, idx, kept)
    assert torch.equal(cache.cache_len, kept)
    step_in = [(_bf(g, nseq, (Hq + 2 * Hkv) * d), _i32(lens) + i) for i in range(steps)]
    one = torch.ones(nseq, dtype=torch.int32, device="cuda")
    x, p = step_in[0][0].clone(), step_in[0][1].clone()

    def step():
        a, b, c = (x[:, u * d:w_ * d].view(nseq, w_ - u, d) for u, w_ in
                   ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        a, b = api.qk_norm_rope(a, b, p, inv, q_weight=w[0], k_weight=w[1])
        slots, _ = cache.reserve(one, nseq)
        cache.append(b, c, slots)
        return a, b, c, cache.attend(a, with_lse=True)

    outs = []
    run = step
    if graph:
        # captured once; the replays advance the lengths on the device
        saved = [t.clone() for t in (cache.cache_len, cache.free_count, cache.block_table,
                                     cache.pool)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for t, old in zip((cache.cache_len, cache.free_count, cache.block_table, cache.pool),
                          saved):
            t.copy_(old)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            res = step()

        def run():
            cg.replay()
            return res
    for xi, pi in step_in:
        x.copy_(xi)
        p.copy_(pi)
        a, b, c, (o, l) = run()
        outs.append(tuple(t.clone() for t in (a, b, c, o, l)))
    assert cache.device_status() == 0
    return cache, (Ko, Vo, kept), outs


@pytest.mark.parametrize("d,Hq,Hkv,bs,B", [(128, 8, 2, 16, 64), (64, 14, 2, 64, 128)])
def test_prompt_then_decode(d, Hq, Hkv, bs, B):
    lens = (700, 40, 333)
    cache, (Ko, Vo, kept), outs = _flow(d, Hq, Hkv, bs, B, lens, 20, False)
    K, V = ([co.q4_value(*co.q4_quantise(_f64(t[s, :, :int(kept[s])]))) for s in range(3)]
            for t in (Ko, Vo))
    for a, b, c, o, l in outs:
        for s in range(3):
            K[s] = np.concatenate([K[s], co.q4_value(*co.q4_quantise(_f64(b[s])))[:, None]], 1)
            V[s] = np.concatenate([V[s], co.q4_value(*co.q4_quantise(_f64(c[s])))[:, None]], 1)
            ref, rl = co.q4_decode_attention(_f64(a[s]), K[s], V[s])
            mag, _ = co.q4_decode_attention(_f64(a[s]), K[s], np.abs(V[s]))
            assert np.all(np.abs(_f64(o[s]) - ref) <= BF * np.abs(ref) + 2.0 ** -10 * mag)
            assert np.all(np.abs(_f64(l[s]) - rl) <= 2.0 ** -13)
    assert np.array_equal(cache.cache_len.cpu().numpy(), kept.cpu().numpy() + 20)
    cache.release(_i32([0, 1, 1]))
    assert cache.cache_len.tolist()[1:] == [0, 0]
    held = -(-(int(kept[0]) + 20) // bs)
    assert int(cache.free_count) == cache.pool.shape[0] - held


def test_captured_steps_equal_eager_ones():
    args = (128, 8, 2, 16, 64, (700, 40, 333), 20)
    a, _, eager = _flow(*args, False)
    b, _, replayed = _flow(*args, True)
    for x, y in zip(eager, replayed):
        for t, u in zip(x, y):
            assert torch.equal(t, u)
    assert torch.equal(a.pool, b.pool) and torch.equal(a.block_table, b.block_table)


def test_compact_leaves_running_sequences_alone():
    lens = (100, 0, 60)
    lay = wl.random_layer(lens, 2, 2, 64, seed=3, device="cuda")
    idx, kept = api.select(torch.rand((2, 160), device="cuda"), lay.cu_seqlens, recent_budget=4,
                           budget=32)
    cache = api.Q4Cache(3, 4, 2, 64, num_blocks=9, max_blocks=4, block_size=16)
    cache.compact(lay.K, lay.V, lay.cu_seqlens, idx, kept)
    assert cache.cache_len.tolist() == [32, 0, 32]
    before = cache.pool.clone()
    cache.compact(lay.V, lay.K, lay.cu_seqlens, idx, kept)       # all hold tokens, or keep none
    assert cache.cache_len.tolist() == [32, 0, 32] and torch.equal(cache.pool, before)
    assert cache.device_status() == 0
    # a pool too small for the last one
    small = api.Q4Cache(3, 4, 2, 64, num_blocks=3, max_blocks=4, block_size=16)
    small.compact(lay.K, lay.V, lay.cu_seqlens, idx, kept)
    assert small.cache_len.tolist() == [32, 0, 0]
    assert small.device_status() == _lib.DEV_CACHE_FULL and small.device_status() == 0


def test_other_stream():
    """The calls run on the current stream."""
    g = _gen(40)
    pool, table, kv = _fill(g, [500, 77], 2, 128, 16)
    q = _bf(g, 2, 8, 128)
    lens = _i32([500, 77])
    ref = api.q4_decode_attention(q, pool, table, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = api.q4_decode_attention(q, pool, table, lens)
    s.synchronize()
    assert torch.equal(ref, got)


# ------------------------------------------------------------------ calls at the edges

@pytest.mark.parametrize("shift", [8, 16])
def test_rows_on_sixteen_bytes(shift):
    """Rows that start on 16 bytes but not on 32 take the narrower accesses."""
    g = _gen(50)
    buf = _bf(g, 40 * (2 * 128 + 8) + 64)
    K = buf[shift:].as_strided((40, 2, 128), (264, 128, 1))
    V = K.contiguous()
    assert (K.data_ptr() % 32 == 0) == (shift == 16)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    a, b = _pool(3, 2, 16, 128), _pool(3, 2, 16, 128)
    api.q4_append(K, V, slots, a)
    api.q4_append(V, V, slots, b)
    assert torch.equal(a, b)
    # read back through the C entry into outputs on 16 bytes
    ref, _ = api.q4_read(a, slots, 128)
    out = torch.full((2 * 40 * 256 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    c = _lib.Q4Cache(3, 16, 2, 128, a.data_ptr())
    k0, v0 = shift, shift + 40 * 256 + 8
    st = _lib.load().waits_q4_read(ctypes.byref(c), 40, slots.data_ptr(),
                                   out.data_ptr() + 2 * k0, out.data_ptr() + 2 * v0, None,
                                   torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for at in (k0, v0):
        assert torch.equal(out[at:at + 40 * 256].view(40, 2, 128), ref)
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[k0:k0 + 40 * 256] = rest[v0:v0 + 40 * 256] = False
    assert (out[rest] == 7).all()


@pytest.mark.parametrize("n", [148 * 8 * 32 // 8 + 5, 40000])
def test_read_many_rows(n):
    """Enough rows that a thread reads two back, with an odd number of them."""
    g = _gen(51)
    K, V = _bf(g, n, 1, 64), _bf(g, n, 1, 64)
    blocks = n // 256 + 1
    slots = torch.randperm(blocks * 256, generator=g, device="cuda")[:n].int()
    pool = _pool(blocks, 1, 256, 64)
    api.q4_append(K, V, slots, pool)
    Kr, Vr = api.q4_read(pool, slots, 64)
    for x, y in ((K, Kr), (V, Vr)):
        assert np.array_equal(_f64(y), co.round_bf16(co.q4_value(*co.q4_quantise(_f64(x)))))


@pytest.mark.parametrize("nseq,Hq,Hkv,d", [(33, 8, 2, 128), (32, 8, 2, 128), (700, 2, 1, 64),
                                           (60, 64, 4, 128), (200, 28, 4, 64), (90, 32, 8, 128)])
def test_attend_many_sequences(nseq, Hq, Hkv, d):
    """Many short items per CTA, empty ones among them, on both planning paths."""
    rng = np.random.default_rng(nseq)
    lens = rng.integers(0, 260, nseq).tolist()
    lens[nseq // 2] = 2500
    g = _gen(nseq)
    pool, table, kv = _fill(g, lens, Hkv, d, 16)
    _check_attend(_bf(g, nseq, Hq, d), pool, table, lens, kv)


def test_attend_all_empty():
    q = _bf(_gen(1), 40, 8, 64)
    for nseq in (1, 32, 40):
        out, lse = api.q4_decode_attention(q[:nseq].contiguous(), _pool(2, 2, 16, 64),
                                           _i32(np.full((nseq, 3), -1)), _i32([0] * nseq), True)
        assert not out.any() and torch.isneginf(lse).all()


def test_attend_nan_key():
    """A key that is not a number makes its head's sequence NaN, no other."""
    g = _gen(52)
    lens = [70, 70]
    pool, table, _ = _fill(g, lens, 2, 64, 16)
    K = _bf(g, 1, 2, 64)
    V = K.clone()
    K[0, 0, 3] = float("nan")
    api.q4_append(K, V, (table[1, 1] * 16).view(1), pool)
    out, lse = api.q4_decode_attention(_bf(g, 2, 4, 64), pool, table, _i32(lens), True)
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[1, :2]).all()
    assert torch.isfinite(out[1, 2:]).all() and torch.isfinite(out[0]).all()
    assert torch.isfinite(lse[1, 2:]).all() and torch.isfinite(lse[0]).all()


def test_attend_zero_query_and_zero_cache():
    """No logit differs: the output is the mean of V; zero V gives zeros."""
    g = _gen(53)
    pool, table, kv = _fill(g, [333], 1, 128, 16)
    out, lse = api.q4_decode_attention(torch.zeros((1, 4, 128), dtype=torch.bfloat16,
                                                   device="cuda"), pool, table, _i32([333]), True)
    ref = kv[0][1][0].mean(0)
    assert np.all(np.abs(_f64(out[0, 0]) - ref) <= BF * np.abs(ref) + 2.0 ** -10 * 3)
    assert np.allclose(_f64(lse), np.log(333.0), atol=2.0 ** -13)
    zero = torch.zeros_like(pool)
    out, lse = api.q4_decode_attention(_bf(g, 1, 4, 128), zero, table, _i32([333]), True)
    assert not out.any() and np.allclose(_f64(lse), np.log(333.0), atol=2.0 ** -13)


def test_pool_past_four_gigabytes():
    """Blocks whose bytes lie past 32 bits."""
    Hkv, d, bs = 8, 128, 256
    blocks = 2 ** 32 // (Hkv * bs * d * 9 // 8) + 40
    pool = torch.empty((blocks, Hkv, bs * d * 9 // 8), dtype=torch.uint8, device="cuda")
    g = _gen(54)
    n = 600
    K, V = _bf(g, n, Hkv, d), _bf(g, n, Hkv, d)
    table = _i32([[blocks - 1, 3, blocks - 20]])
    j = torch.arange(n, device="cuda")
    slots = (table[0, j // bs] * bs + j % bs).int()
    api.q4_append(K, V, slots, pool)
    Kr, Vr = api.q4_read(pool, slots, d)
    kv = []
    for x, y in ((K, Kr), (V, Vr)):
        val = co.q4_value(*co.q4_quantise(_f64(x)))
        assert np.array_equal(_f64(y), co.round_bf16(val))
        kv.append(val.transpose(1, 0, 2))
    _check_attend(_bf(g, 1, 32, d), pool, table, [n], [kv])


def test_rope_offsets_past_32_bits():
    stride = 2 ** 27
    g = _gen(55)
    T = 18
    big = torch.empty(stride * (T - 1) + 4 * 128, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((T, 4, 128), (stride, 128, 1))
    src = _bf(g, T, 4, 128)
    q.copy_(src)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    inv = api.rotary_inv_freq(128, 1e6)
    k = _bf(g, T, 2, 128)
    ref = api.qk_norm_rope(src, k, pos, inv)
    got = api.qk_norm_rope(q, k, pos, inv, out=(q, torch.empty_like(k)))
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    pool = _pool(2, 4, 16, 128)
    pool2 = pool.clone()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    api.q4_append(q, q, slots, pool)
    api.q4_append(ref[0], ref[0], slots, pool2)
    assert torch.equal(pool, pool2)


def test_two_caches_on_two_streams():
    """Calls with their own workspaces may overlap."""
    g = _gen(56)
    sides = [torch.cuda.Stream() for _ in range(2)]
    sets, refs = [], []
    for i in range(2):
        lens = [3000 + 100 * i, 17, 900]
        pool, table, kv = _fill(g, lens, 4, 128, 16)
        q = _bf(g, 3, 16, 128)
        sets.append((q, pool, table, _i32(lens)))
        refs.append(api.q4_decode_attention(*sets[-1], True))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got[i].append(api.q4_decode_attention(*sets[i], True))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, refs[i][0]) and torch.equal(lse, refs[i][1])


def test_two_graphs_share_a_workspace_in_turn():
    g = _gen(57)
    lens = [1500, 40]
    pool, table, kv = _fill(g, lens, 2, 64, 16)
    q = [_bf(g, 2, 8, 64) for _ in range(2)]
    ws = torch.empty(api.q4_decode_workspace_bytes(pool, 2, 8, 64), dtype=torch.uint8,
                     device="cuda")
    L = _i32(lens)
    ref = [api.q4_decode_attention(x, pool, table, L, True) for x in q]
    graphs, res = [], []
    for x in q:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            res.append(api.q4_decode_attention(x, pool, table, L, True, workspace=ws))
        graphs.append(cg)
    for _ in range(3):
        for cg in graphs:
            cg.replay()
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(ref, res):
        assert torch.equal(a, c) and torch.equal(b, d)
    # the lengths are read when the graph runs, not when it is captured
    L.copy_(_i32([3, 0]))
    graphs[0].replay()
    out, lse = api.q4_decode_attention(q[0], pool, table, _i32([3, 0]), True)
    assert torch.equal(res[0][0], out) and torch.equal(res[0][1], lse)


def test_captured_append_rope_reserve_release():
    g = _gen(58)
    cache = api.Q4Cache(4, 8, 2, 64, num_blocks=30, max_blocks=6, block_size=16)
    ref = api.Q4Cache(4, 8, 2, 64, num_blocks=30, max_blocks=6, block_size=16)
    new, ended = _i32([3, 0, 1, 5]), _i32([0, 1, 0, 0])
    K, V = _bf(g, 9, 2, 64), _bf(g, 9, 2, 64)
    cg = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(cg):
        slots, cu = cache.reserve(new, 9)
        cache.append(K, V, slots)
        cache.release(ended)
    for i in range(8):
        new.copy_(_i32([3, 0, 1, 5] if i % 2 else [2, 4, 3, 0]))
        ended.copy_(_i32([0, 1, 0, i == 5]))
        cg.replay()
        s, c = ref.reserve(new, 9)
        ref.append(K, V, s)
        ref.release(ended)
        assert torch.equal(slots, s) and torch.equal(cu, c)
    for name in ("pool", "block_table", "cache_len", "free_list", "free_count", "status"):
        assert torch.equal(getattr(cache, name), getattr(ref, name)), name


def test_refused_tensors():
    """What the binding refuses once tensors are on the GPU."""
    g = _gen(59)
    pool = _pool(4, 2, 16, 64)
    K = _bf(g, 5, 2, 64)
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    table, lens = _i32([[0, 1]]), _i32([20])
    q = _bf(g, 1, 4, 64)
    inv = api.rotary_inv_freq(64, 1e4)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    bad = [
        (lambda: api.q4_append(K, K, slots.long(), pool), "slot_map must be torch.int32"),
        (lambda: api.q4_append(K, K, slots[:4], pool), "slot_map"),
        (lambda: api.q4_append(K.float(), K, slots, pool), "K must be torch.bfloat16"),
        (lambda: api.q4_append(K, K[:, :1], slots, pool), "V must have K's shape"),
        (lambda: api.q4_append(K[:, :1].contiguous(), K[:, :1].contiguous(), slots, pool),
         "pool must have K's heads"),
        (lambda: api.q4_append(K.transpose(0, 1), K.transpose(0, 1), slots, pool), "contiguous"),
        (lambda: api.q4_append(K, K, slots, pool[:, :, :-8].contiguous()), "whole number of tokens"),
        (lambda: api.q4_append(K, K, slots, pool.view(4, -1)), "pool must be uint8"),
        (lambda: api.q4_append(K, K, slots, pool, status=slots), "status must hold one"),
        (lambda: api.q4_append(K, K, slots.cpu(), pool), "slot_map must be a CUDA tensor"),
        (lambda: api.q4_read(pool, slots.view(5, 1), 64), "slot_map"),
        (lambda: api.q4_decode_attention(q, pool, table.view(2, 1), lens), "block_table must be"),
        (lambda: api.q4_decode_attention(q, pool, table, lens.view(1, 1)), "cache_len"),
        (lambda: api.q4_decode_attention(q[0], pool, table, lens), "q must be"),
        (lambda: api.q4_decode_attention(q, pool, table, lens,
                                         workspace=torch.empty(99, device="cuda")), "workspace"),
        (lambda: api.qk_norm_rope(K, K[:4], pos, inv), "k must be"),
        (lambda: api.qk_norm_rope(K, K, pos[:4], inv), "positions"),
        (lambda: api.qk_norm_rope(K, K, pos, inv.float()), "inv_freq"),
        (lambda: api.qk_norm_rope(K, K, pos, inv.cuda()), "inv_freq"),
        (lambda: api.qk_norm_rope(K, K, pos, inv, q_weight=K[0, 0]), "come together"),
        (lambda: api.qk_norm_rope(K, K, pos, inv, out=(K, K[:, :1])), "out must have"),
        (lambda: api.cache_reserve(lens, lens, table, slots, slots, block_size=16, max_new=3),
         "free_count must hold one"),
        (lambda: api.cache_reserve(lens, lens, table, slots, slots[:1], block_size=16,
                                   max_new=-3), "max_new"),
    ]
    for call, text in bad:
        with pytest.raises(ValueError, match=text):
            call()
    for call, status in [
            (lambda: api.cache_reserve(lens, lens, table, slots, slots[:1], block_size=24,
                                       max_new=3), 3),
            (lambda: api.q4_decode_attention(q, pool, table, lens, workspace=torch.empty(
                16, dtype=torch.uint8, device="cuda")), 4),
            (lambda: api.q4_decode_attention(_bf(g, 1, 3, 64), pool, table, lens), 2),
            (lambda: api.q4_decode_attention(_bf(g, 1, 34, 64), pool, table, lens), 3),
            (lambda: api.qk_norm_rope(K, K, pos, api.rotary_inv_freq(128, 1e4)), 2),
            (lambda: api.qk_norm_rope(K, K, pos, inv * 1e13), 1),
            (lambda: api.qk_norm_rope(K, K, pos, inv, q_weight=K[0, 0], k_weight=K[0, 0],
                                      eps=-1.0), 1)]:
        with pytest.raises(_lib.WaitsError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()


def test_empty_calls():
    pool = _pool(2, 2, 16, 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int32, device="cuda")
    before = pool.clone()
    api.q4_append(none, none, slots, pool)
    K, V = api.q4_read(pool, slots, 64)
    assert K.shape == V.shape == (0, 2, 64) and torch.equal(pool, before)


@pytest.mark.parametrize("nseq,Hq,Hkv,d,hi", [
    (1, 32, 8, 128, 2500), (1, 16, 1, 128, 40), (2, 28, 4, 128, 3000), (3, 8, 2, 64, 6000),
    (7, 16, 8, 64, 700), (16, 16, 4, 128, 380), (60, 4, 2, 128, 700), (140, 3, 1, 64, 300)])
def test_attend_short_and_wide_tables(nseq, Hq, Hkv, d, hi):
    """A table that holds little has clusters of 1, 2, 4 or 8 CTAs per item,
    some without a tile of their own; a wide one of the same contents does
    not.  Both agree with the oracle."""
    rng = np.random.default_rng(hi)
    lens = rng.integers(0, hi + 1, nseq).tolist()
    lens[0] = hi
    if nseq > 2:
        lens[1], lens[2] = 0, 33
    g = _gen(hi + nseq)
    pool, table, kv = _fill(g, lens, Hkv, d, 16)
    q = _bf(g, nseq, Hq, d)
    wide = torch.full((nseq, 20000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    for t in (table, wide):
        a = _check_attend(q, pool, t, lens, kv)
        b = api.q4_decode_attention(q, pool, t, _i32(lens), True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("nseq,Hq,Hkv,d,hi", [
    (45, 32, 8, 128, 900), (310, 4, 1, 64, 90), (32, 48, 12, 64, 300), (100, 28, 4, 128, 500),
    (80, 64, 4, 128, 200), (330, 16, 1, 64, 260)])
def test_attend_many_short_items(nseq, Hq, Hkv, d, hi):
    """More than two short items per CTA, on tables too wide for clusters: a
    warp takes each by itself.  Empty sequences and pages that are missing
    among them."""
    rng = np.random.default_rng(nseq + hi)
    lens = rng.integers(0, hi + 1, nseq).tolist()
    lens[0], lens[3], lens[nseq - 1] = 0, hi, 1
    g = _gen(nseq + hi)
    pool, table, kv = _fill(g, lens, Hkv, d, 16)
    wide = torch.full((nseq, 9000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = _bf(g, nseq, Hq, d)
    a = _check_attend(q, pool, wide, lens, kv)
    b = api.q4_decode_attention(q, pool, wide, _i32(lens), True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide[3, 0] = pool.shape[0]                     # the first page of a long one is missing
    status = _i32([0])
    out, lse = api.q4_decode_attention(q, pool, wide, _i32(lens), True, status=status)
    assert int(status) == _lib.DEV_BAD_INDEX
    ref, rl = co.q4_decode_attention(_f64(q[3]), *(x[:, 16:] for x in kv[3]))
    mag, _ = co.q4_decode_attention(_f64(q[3]), kv[3][0][:, 16:], np.abs(kv[3][1][:, 16:]))
    assert np.all(np.abs(_f64(out[3]) - ref) <= BF * np.abs(ref) + 2.0 ** -10 * mag)
    assert np.all(np.abs(_f64(lse[3]) - rl) <= 2.0 ** -13)
    keep = [i for i in range(nseq) if i != 3]
    assert torch.equal(out[keep], a[0][keep]) and torch.equal(lse[keep], a[1][keep])

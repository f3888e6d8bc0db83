"""fp64 / whole-number restatement of the operators around the 4-bit paged
KV cache (``include/waits.h``: ``waits_qk_norm_rope``, ``waits_cache_reserve``,
``waits_cache_release``, ``waits_q4_*``).  Plain numpy, no code shared with
the CUDA path."""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def qk_norm_rope(x, positions, inv_freq, weight, eps, interleaved):
    """``x [T, H, d]`` -> the normalised, rotated rows in fp64 and the sum of
    magnitudes |y1| + |y2| of each output's pair (|y| where nothing turns).
    Angles in extended precision, so far positions keep 1e-9 of a radian."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * weight
    half = len(inv_freq)
    pos = np.asarray(positions, np.longdouble)[:, None]
    ang = np.mod(pos * np.asarray(inv_freq, np.longdouble)[None], 2 * np.arccos(np.longdouble(-1)))
    cos, sin = (f(ang).astype(np.float64)[:, None, :] for f in (np.cos, np.sin))
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out, scale = y.copy(), np.abs(y)
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    scale[..., a] = scale[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, scale


def cache_reserve(new_len, cache_len, table, free_list, free_count, block_size, max_new):
    """Returns (slot_map, cu_new, cache_len, free_count, table, bits): the
    sequences one after the other, with a stack."""
    n = len(new_len)
    table = np.array(table)
    length = np.array(cache_len)
    width, num_blocks = table.shape[1], len(free_list)
    left = min(max(int(free_count), 0), num_blocks)
    slots = np.full(max_new, -1, np.int64)
    cu = [0]
    bits, starved = 0, False
    for s in range(n):
        add, have_tokens = int(new_len[s]), int(length[s])
        at = cu[-1]
        cu.append(at + max(add, 0))
        if add < 0 or have_tokens < 0:
            bits |= 0x2
            continue
        if have_tokens + add > width * block_size or cu[-1] > max_new:
            bits |= 0x20
            continue
        have = -(-have_tokens // block_size)
        want = -(-(have_tokens + add) // block_size)
        if want > have and (starved or want - have > left):
            starved = True
            bits |= 0x20
            continue
        for logical in range(have, want):
            left -= 1
            table[s, logical] = free_list[left]
        for t in range(add):
            pos = have_tokens + t
            block = int(table[s, pos // block_size])
            if 0 <= block < num_blocks:
                slots[at + t] = block * block_size + pos % block_size
            else:
                bits |= 0x8
        length[s] = have_tokens + add
    return slots, np.array(cu), length, left, table, bits


def cache_release(ended, cache_len, table, free_list, free_count, block_size):
    """Returns (cache_len, table, free_list, free_count, bits)."""
    length, table, free = np.array(cache_len), np.array(table), np.array(free_list)
    num_blocks = len(free)
    count = min(max(int(free_count), 0), num_blocks)
    bits = 0
    for s in range(len(length)):
        if not ended[s]:
            continue
        blocks = -(-int(length[s]) // block_size)
        if length[s] < 0 or blocks > table.shape[1]:
            bits |= 0x2
            blocks = 0 if length[s] < 0 else table.shape[1]
        for j in range(blocks):
            b = table[s, j]
            if 0 <= b < num_blocks and count < num_blocks:
                free[count] = b
                count += 1
            else:
                bits |= 0x8
            table[s, j] = -1
        length[s] = 0
    return length, table, free, count, bits


def round_bf16(x):
    """fp64 -> the nearest bf16 value (ties to even), normal range."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def q4_quantise(x):
    """``x [..., d]`` -> (codes [..., d], scales [..., d / 32]).  The code
    whose value times the scale is nearest, the even one of two equally near
    ones; non-finite groups have a NaN scale, tiny ones scale 0."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.max(np.abs(g), axis=-1)
    finite = np.isfinite(top)
    scale = round_bf16(np.where(finite, top, 0.0) / 6.0)
    scale = np.where(scale < 2.0 ** -126, 0.0, scale)
    gap = np.abs(np.abs(np.where(finite[..., None], g, 0.0))[..., None]
                 - scale[..., None, None] * E2M1)
    # of two equally near codes, which are neighbours, the even one
    tie = gap == gap.min(axis=-1, keepdims=True)
    order = np.where(tie, np.arange(8) % 2, 2)
    code = order.argmin(axis=-1)
    code = np.where(np.signbit(g), code + 8, code)
    dead = (scale == 0.0) | ~finite
    code = np.where(dead[..., None], 0, code)
    return code.reshape(x.shape), np.where(finite, scale, np.nan)


def q4_value(code, scale):
    v = np.concatenate([E2M1, -E2M1])[code]
    with np.errstate(invalid="ignore"):
        return v * np.repeat(scale, 32, axis=-1)


def q4_place(which, block_size, d, off, dim):
    """(byte, shift) of a code in a page, which = 0 for K, 1 for V."""
    base = which * block_size * d * 9 // 16 + off * d // 2
    h = dim % 4 // 2
    if which == 0:
        return base + dim % 16 // 4 * (d // 8) + 2 * (dim // 16) + h, dim % 2 * 4
    return base + dim % 32 // 4 * (d // 16) + 2 * (dim // 32) + h, dim % 2 * 4


def q4_scale_place(which, block_size, d, off, group):
    """Byte of a bf16 scale in a page."""
    return which * block_size * d * 9 // 16 + block_size * d // 2 + off * d // 16 + 2 * group


def bf16_bits(x):
    """bf16 bit patterns of values that are bf16 numbers (NaN: 0x7fff)."""
    x = np.asarray(x, np.float64)
    bits = x.astype(np.float32).view(np.uint32) >> 16
    return np.where(np.isnan(x), 0x7FFF, bits)


def q4_write(pool, slot, K, V, block_size):
    """Quantise K, V ``[Hkv, d]`` into ``slot`` of pool uint8 ``[blocks, Hkv,
    bytes]``."""
    Hkv, d = K.shape
    block, off = slot // block_size, slot % block_size
    for which, x in enumerate((K, V)):
        code, scale = q4_quantise(x)
        sb = bf16_bits(scale)
        for dim in range(d):
            byte, shift = q4_place(which, block_size, d, off, dim)
            pool[block, :, byte] = (pool[block, :, byte] & (0xF0 >> shift)) | (code[:, dim] << shift)
        for g in range(d // 32):
            byte = q4_scale_place(which, block_size, d, off, g)
            pool[block, :, byte] = sb[:, g] & 255
            pool[block, :, byte + 1] = sb[:, g] >> 8


def q4_decode_attention(q, K, V):
    """``q [Hq, d]``, ``K, V [Hkv, n, d]`` -> (out [Hq, d], lse [Hq]) in fp64."""
    Hq, d = q.shape
    G = Hq // K.shape[0]
    out, lse = np.zeros((Hq, d)), np.full(Hq, -np.inf)
    if K.shape[1] == 0:
        return out, lse
    for h in range(Hq):
        x = K[h // G] @ q[h] / np.sqrt(d)
        top = x.max()
        p = np.exp(x - top)
        out[h] = p @ V[h // G] / p.sum()
        lse[h] = top + np.log(p.sum())
    return out, lse

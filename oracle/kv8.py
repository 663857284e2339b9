"""Oracle of the block-scaled 8-bit KV cache (append and attention).

The cache of one layer is codes uint8 [pages, 2, kv_heads, 64, dim] (E4M3,
keys then values) with scales float32 [pages, 2, kv_heads]: value = code *
scale. Everything is float64; the codes of an append are decided on x / scale,
exact for the power-of-two scales that an append chooses.
"""

import math

import numpy as np

from .fp8 import E4M3_MAX, bf16_bits_to_float64, e4m3_encode, e4m3_to_float64

PAGE = 64
MIN_EXP, MAX_EXP = -60, 120


def kv8_need_scale(amax):
    """The smallest power of two s with amax <= 448 s (exponent limited to
    [-60, 120]); 0 for amax = 0."""
    if not amax > 0:
        return 0.0
    e = MIN_EXP
    while e < MAX_EXP and E4M3_MAX * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def kv8_append(k_bits, v_bits, starts, lens, block_table, codes, scales):
    """New tokens (uint16 bf16 bits [T, kv_heads, dim]) into copies of codes
    and scales; returns (codes, scales, bad_len, bad_page)."""
    codes, scales = codes.copy(), scales.astype(np.float32).copy()
    x = np.stack([bf16_bits_to_float64(k_bits), bf16_bits_to_float64(v_bits)], 1)
    bad_len = bad_page = False
    for r, length in enumerate(lens):
        n = int(starts[r + 1]) - int(starts[r])
        if n <= 0:
            continue
        first = int(length) - n
        if first < 0:
            bad_len = True
            continue
        for b in range(first // PAGE, -(-int(length) // PAGE)):
            page = int(block_table[r, b]) if b < block_table.shape[1] else -1
            if not 0 <= page < codes.shape[0]:
                bad_page = True
                continue
            lo, hi = max(first, b * PAGE), min(int(length), (b + 1) * PAGE)
            had = lo - b * PAGE
            new = x[starts[r] + lo - first: starts[r] + hi - first]      # [m, 2, H, D]
            for side in range(2):
                for h in range(codes.shape[2]):
                    y = new[:, side, h]
                    a = np.abs(y[~np.isnan(y)]).max(initial=0.0)
                    old = float(scales[page, side, h]) if had else 0.0
                    s = max(old, kv8_need_scale(a))
                    s = s if s > 0 else 2.0 ** MIN_EXP
                    at = codes[page, side, h]
                    if had and s != old:
                        at[:had] = e4m3_encode(e4m3_to_float64(at[:had]) * np.float32(old / s))
                    at[had:had + hi - lo] = e4m3_encode((y / s).astype(np.float32))
                    scales[page, side, h] = s
    return codes, scales, bad_len, bad_page


def kv8_visible(lens, counts, bt_stride):
    """Positions each token sees: [(request, visible)] in token order, for
    requests whose last counts[r] positions are the tokens."""
    rows = []
    for r, (length, n) in enumerate(zip(lens, counts)):
        for i in range(int(n)):
            rows.append((r, min(max(int(length) - int(n) + 1 + i, 0), PAGE * bt_stride)))
    return rows


def kv8_attention(q_bits, rows, codes, scales, block_table, scale):
    """Attention of tokens q (uint16 bf16 bits [T, heads, dim]); rows[t] =
    (request, visible positions). Pages outside the pool are left out.

    Returns (out, lse, weight, reach, bad_page): weight [T, heads, dim] =
    sum_i p_i |v_i| and reach [T, heads] = max_i scale * sum_d |q_d k_id|, the
    magnitudes that error bounds are made of.
    """
    q = bf16_bits_to_float64(q_bits)
    t_n, heads, dim = q.shape
    hk = codes.shape[2]
    group = heads // hk
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    reach = np.zeros(q.shape[:2])
    bad = False
    kv_of = {}
    for t, (r, visible) in enumerate(rows):
        if visible <= 0:
            continue
        blocks = -(-visible // PAGE)
        if r not in kv_of or kv_of[r][0] < blocks:
            longest = max(v for rr, v in rows if rr == r)
            nb = -(-longest // PAGE)
            pages = block_table[r, :nb].astype(np.int64)
            good = (pages >= 0) & (pages < codes.shape[0])
            at = np.where(good, pages, 0)
            val = e4m3_to_float64(codes[at]) * scales[at].astype(np.float64)[..., None, None]
            kv_of = {r: (nb, val, good)}
        _, val, good = kv_of[r]
        keep = np.repeat(good[:blocks], PAGE)[:visible]
        bad |= not keep.all()
        for g in range(hk):
            k = val[:blocks, 0, g].reshape(-1, dim)[:visible][keep]
            v = val[:blocks, 1, g].reshape(-1, dim)[:visible][keep]
            if not len(k):
                continue
            qq = q[t, g * group:(g + 1) * group]
            s = scale * qq @ k.T
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p = p / l
            sl = slice(g * group, (g + 1) * group)
            out[t, sl] = p @ v
            weight[t, sl] = p @ np.abs(v)
            lse[t, sl] = (m + np.log(l))[:, 0]
            reach[t, sl] = (abs(scale) * np.abs(qq) @ np.abs(k).T).max(1)
    return out, lse, weight, reach, bad


def kv8_bounds(ref_out, ref_lse, weight, reach, dim, length):
    """Error bounds of a kernel that keeps scores, sums and accumulators in
    fp32 and rounds each softmax weight to 8 significant bits and the output
    to bf16 (half a step is 2^-8 of the value in both).

    A score is a dim-term fp32 sum: off by at most (dim + 8) 2^-24 * reach,
    which moves a weight (and the sum that divides it) by that factor each; a
    sum of `length` terms adds length * 2^-24; exp2 and log2 add a few 2^-22.
    """
    score = (dim + 8) * 2.0 ** -24 * reach
    rel = 2 * np.expm1(score) + 2 * length * 2.0 ** -24 + 2.0 ** -18
    out = 2.0 ** -8 * np.abs(ref_out) + (2.0 ** -8 + rel[..., None]) * 1.01 * weight + 1e-37
    lse = score + length * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(np.where(
        np.isfinite(ref_lse), ref_lse, 0.0))) + math.ulp(0.0)
    return out, lse

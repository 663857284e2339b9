"""Oracle of what a serving step does around the block-scaled 8-bit cache: norm
with rotation, attention of a tree of drafts, accepted drafts, attention mass
and eviction. Everything is float64 but for the scales of moved codes, whose
ratio is a float32 as the operators define it.
"""

import numpy as np

from .fp8 import bf16_bits_to_float64, e4m3_encode, e4m3_to_float64
from .topk import topk_per_row

PAGE = 64


# ------------------------------------------------------ norm and rotation
def qk_norm_rope(x_bits, w_bits, positions, inv_freq, eps, norm_dim, rot_start, interleaved):
    """One side (uint16 bf16 bits [T, heads, dim]; w_bits None: no norm).

    Returns (y, size): size [T, heads, dim] is the magnitude that a value's
    error goes by: |y| or, where it is turned, |u| + |v| of its pair.
    """
    x = bf16_bits_to_float64(x_bits).copy()
    if w_bits is not None and norm_dim:
        ms = (x[..., :norm_dim] ** 2).mean(-1, keepdims=True)
        x[..., :norm_dim] *= bf16_bits_to_float64(w_bits) / np.sqrt(ms + float(np.float32(eps)))
    size = np.abs(x)
    half = len(inv_freq)
    angle = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    cos, sin = np.cos(angle), np.sin(angle)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = a + rot_start, b + rot_start
        u, v = x[..., a].copy(), x[..., b].copy()
        c, s = cos[:, i, None], sin[:, i, None]
        x[..., a], x[..., b] = u * c - v * s, v * c + u * s
        size[..., a] = size[..., b] = np.abs(u) + np.abs(v)
    return x, size


# ------------------------------------------------------------ moved codes
def _place(codes, scales, pages, head_list, src):
    """In copies of one layer's arrays: position j of a request gets what
    position src[j] (ascending, src[j] >= j) held, for the given heads; `pages`
    are the request's."""
    old_codes, old_scales = codes.copy(), scales.copy()
    for b in range(-(-len(src) // PAGE)):
        lo, hi = b * PAGE, min(len(src), (b + 1) * PAGE)
        for side in range(2):
            for g in head_list:
                s = np.array([old_scales[pages[src[j] // PAGE], side, g] for j in range(lo, hi)],
                             np.float32)
                top = s.max()
                for j in range(lo, hi):
                    row = old_codes[pages[src[j] // PAGE], side, g, src[j] % PAGE]
                    ratio = np.float32(1 if s[j - lo] == top else s[j - lo] / top)
                    if ratio != 1:
                        row = e4m3_encode((e4m3_to_float64(row) * float(ratio)).astype(np.float32))
                    codes[pages[b], side, g, j % PAGE] = row
                scales[pages[b], side, g] = top


def kv8_accept(layers, block_table, lens, next_n, accepted):
    """layers: [(codes, scales)]; returns (layers, new_lens, flags)."""
    layers = [(c.copy(), s.copy()) for c, s in layers]
    num_pages = layers[0][0].shape[0]
    heads = range(layers[0][0].shape[2])
    new_lens, flags = [], set()
    for r, length in enumerate(int(x) for x in lens):
        new_lens.append(length)
        if length <= 0:
            continue
        row = [int(a) for a in accepted[r]]
        n = next((i for i, a in enumerate(row) if a < 0), len(row))
        bad = set()
        if length < next_n or length > PAGE * block_table.shape[1]:
            bad.add("len")
        if any(a >= next_n for a in row) or any(a >= 0 for a in row[n:]) or \
                any(row[i] <= row[i - 1] for i in range(1, n)):
            bad.add("idx")
        base = length - next_n
        if not bad and n:
            touched = {base // PAGE, (base + row[n - 1]) // PAGE}
            if any(not 0 <= block_table[r, b] < num_pages for b in touched):
                bad.add("page")
        flags |= bad
        if bad:
            continue
        new_lens[-1] = base + n
        if n == 0:
            continue
        first = base // PAGE
        pages = [int(p) for p in block_table[r, first:first + 2]]
        src = list(range(base % PAGE)) + [base % PAGE + a for a in row[:n]]
        for codes, scales in layers:
            _place(codes, scales, pages, heads, src)
    return layers, new_lens, flags


def kv8_evict(mass, budget, first, recent, codes, scales, block_table, lens, refs=None):
    """Returns (mass, codes, scales, new_lens, flags)."""
    mass, codes, scales = mass.copy(), codes.copy(), scales.copy()
    new_lens, flags = [], set()
    for r, length in enumerate(int(x) for x in lens):
        new_lens.append(length)
        if length <= budget:
            continue
        if length > PAGE * block_table.shape[1] or length > mass.shape[2]:
            flags.add("len")
            continue
        pages = [int(p) for p in block_table[r, :-(-length // PAGE)]]
        bad = set()
        if any(not 0 <= p < codes.shape[0] for p in pages):
            bad.add("page")
        if refs is not None and any(0 <= p < codes.shape[0] and refs[p] > 1
                                    for p in pages[:-(-budget // PAGE)]):
            bad.add("shared")
        flags |= bad
        if bad:
            continue
        new_lens[-1] = budget
        k = budget - first - recent
        for g in range(codes.shape[2]):
            best = []
            if k:
                row = mass[r, g][None, :].astype(np.float32)
                best = topk_per_row(row, np.array([first], np.int32),
                                    np.array([length - recent], np.int32), k)[0]
            src = [*range(first), *(first + int(b) for b in best), *range(length - recent, length)]
            _place(codes, scales, pages, [g], src)
            mass[r, g, :budget] = mass[r, g][src]
    return mass, codes, scales, new_lens, flags


# ------------------------------------------------- attention of the drafts
def tree_sees(masks_row, length, next_n, bt_stride):
    """[next_n, positions] bool: what the drafts of one request see."""
    n = min(max(int(length), 0), PAGE * bt_stride)
    base = int(length) - next_n
    sees = np.zeros((next_n, n), bool)
    for j in range(next_n):
        m = int(masks_row[j]) & (2 ** 64 - 1)
        for p in range(n):
            sees[j, p] = p < base or (p - base < next_n and bool(m >> (p - base) & 1))
    return sees


def _request(codes, scales, block_table, r, n, g, side):
    """(values [n, dim], in the pool [n]) of one side and head."""
    pages = block_table[r, :-(-n // PAGE)].astype(np.int64)
    good = (pages >= 0) & (pages < codes.shape[0])
    at = np.where(good, pages, 0)
    val = e4m3_to_float64(codes[at, side, g]) * scales[at, side, g].astype(np.float64)[:, None, None]
    return val.reshape(-1, codes.shape[4])[:n], np.repeat(good, PAGE)[:n]


def kv8_tree(q_bits, masks, codes, scales, block_table, lens, scale):
    """Attention of drafts q [R, n, heads, dim]; returns (out, lse, weight,
    reach) as kv8_attention does."""
    q = bf16_bits_to_float64(q_bits)
    reqs, n, heads, dim = q.shape
    group = heads // codes.shape[2]
    out, weight = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for r in range(reqs):
        sees = tree_sees(masks[r], lens[r], n, block_table.shape[1])
        if not sees.any():
            continue
        for h in range(heads):
            k, good = _request(codes, scales, block_table, r, sees.shape[1], h // group, 0)
            v, _ = _request(codes, scales, block_table, r, sees.shape[1], h // group, 1)
            for j in range(n):
                on = sees[j] & good
                if not on.any():
                    continue
                s = scale * k[on] @ q[r, j, h]
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[r, j, h] = p @ v[on] / l
                weight[r, j, h] = p @ np.abs(v[on]) / l
                lse[r, j, h] = m + np.log(l)
                reach[r, j, h] = (abs(scale) * np.abs(k[on]) @ np.abs(q[r, j, h])).max()
    return out, lse, weight, reach


# ------------------------------------------------------------------- mass
def kv8_mass(q_bits, lse, starts, codes, scales, block_table, lens, scale, mass):
    """Returns (mass, reach): reach [R, kv_heads] is the largest scale *
    sum_d |q_d k_id| + |lse| of a request and head."""
    q = bf16_bits_to_float64(q_bits)
    mass = mass.astype(np.float64).copy()
    hk = codes.shape[2]
    group = q.shape[1] // hk
    reach = np.zeros(mass.shape[:2])
    for r, raw in enumerate(int(x) for x in lens):
        a, b = int(starts[r]), int(starts[r + 1])
        length = min(max(raw, 0), PAGE * block_table.shape[1])
        if b <= a or length <= 0:
            continue
        base = raw - (b - a)
        mass[r, :, max(base, 0):length] = 0.0
        for g in range(hk):
            k, good = _request(codes, scales, block_table, r, length, g, 0)
            for t in range(a, b):
                n = min(max(base + 1 + t - a, 0), length)
                for h in range(g * group, (g + 1) * group):
                    if not n or np.isneginf(lse[t, h]):
                        continue
                    s = scale * k[:n] @ q[t, h]
                    mass[r, g, :n] += np.where(good[:n], np.exp(s - float(lse[t, h])), 0.0)
                    size = (abs(scale) * np.abs(k[:n][good[:n]]) @ np.abs(q[t, h])).max(initial=0.0)
                    reach[r, g] = max(reach[r, g], size + abs(float(lse[t, h])))
    return mass, reach

"""Attention mass where small elements of q carry the score: how exactly a row of few
is multiplied in 8-bit pieces. The bounds are checked on the CPU first, against pieces
that are one too few and against elements that are off."""

import numpy as np
import pytest
import torch

import oracle
from kv8_cases import DEV, Cache, bits

HEADS, DIM, LENS, COUNTS = 4, 64, [150, 80], [2, 1]
BIG = 8.0


def _inputs(lo, hi):
    """Element 0 of a row is its largest, BIG, and meets keys of 0; the others lie in
    [2^lo, 2^hi) of it, and `scale` makes scores of a few nats of them."""
    c = Cache(LENS, 1, DIM, 30, spread=1)
    c.codes[..., 0] = 0
    shape = (sum(COUNTS), HEADS, DIM)
    x = np.exp2(c.rng.uniform(lo, hi, shape)) * c.rng.choice([-1.0, 1.0], shape) * BIG
    q = torch.as_tensor(x).to(torch.bfloat16)
    q[..., 0] = BIG
    starts = np.concatenate([[0], np.cumsum(COUNTS)]).astype(np.int32)
    norm = np.sqrt((bits_to_float(q)[..., 1:] ** 2).sum(-1)).max()
    # codes are about N(0, 100) at a scale of 2^-8
    scale = float(np.float32(2.0 / (norm * 100 * 2.0 ** -8)))
    rows = oracle.kv8_visible(c.lens, COUNTS, c.table.shape[1])
    lse = oracle.kv8_attention(bits(q), rows, c.codes, c.scales, c.table, scale)[1].astype(np.float32)
    return c, q, starts, lse, scale


def bits_to_float(q):
    return oracle.bf16_bits_to_float64(bits(q))


def _mass(c, q_bits, lse, starts, scale):
    old = np.zeros((len(LENS), 1, 64 * c.table.shape[1]))
    return oracle.kv8_mass(q_bits, lse, starts, c.codes, c.scales, c.table, c.lens, scale, old)


def _bound(c, want, reach, scale, piece):
    """What a position's mass may be off by. A score: a sum of dim products in fp32, two
    roundings more and that of the lse, and for elements below 2^-19 of the largest
    2^-27 of that each, times the key. The exponential 2^-20 of itself, the sum of the rows a
    half step each."""
    tol = np.zeros(want.shape)
    for r in range(want.shape[0]):
        k = np.zeros(want.shape[2])
        for b in range(-(-c.lens[r] // 64)):
            page = c.table[r, b]
            value = oracle.e4m3_to_float64(c.codes[page, 0, 0]) * float(c.scales[page, 0, 0])
            k[64 * b:64 * b + 64] = np.abs(value).sum(-1)
        off = (DIM + 16) * 2.0 ** -24 * reach[r, 0] + (2.0 ** -27 * BIG * k * scale if piece else 0.0)
        tol[r, 0] = (np.expm1(off) + 2.0 ** -20 + 2.0 ** -20) * want[r, 0]
    return np.where(np.isfinite(tol), tol, 0.0)


def _pieces(q, n):
    """q as n E4M3 pieces under the row's power of two, as float64."""
    out = np.zeros_like(q)
    up = 2.0 ** (7 - np.floor(np.log2(np.abs(q).max(-1, keepdims=True))))
    rest = q * up
    for z in range(n):
        p = oracle.e4m3_to_float64(oracle.e4m3_encode((rest * 32.0 ** z).astype(np.float32)))
        out += p / 32.0 ** z
        rest = rest - p / 32.0 ** z
    return out / up


def _mass_of_values(c, q, lse, starts, scale):
    """The oracle's mass with q of any float64 values."""
    real = oracle.kv8_step.bf16_bits_to_float64
    oracle.kv8_step.bf16_bits_to_float64 = lambda x: x
    try:
        return _mass(c, q, lse, starts, scale)[0]
    finally:
        oracle.kv8_step.bf16_bits_to_float64 = real


RANGES = [(-19.0, -17.0, False), (-21.0, -19.0, True), (-19.0, -12.0, False), (-23.0, -21.0, True)]


@pytest.mark.parametrize("lo,hi,piece", RANGES)
def test_the_bound_tells_pieces_apart(lo, hi, piece):
    c, q, starts, lse, scale = _inputs(lo, hi)
    want, reach = _mass(c, bits(q), lse, starts, scale)
    tol = _bound(c, want, reach, scale, piece)
    x = bits_to_float(q)

    def worst(y):
        got = _mass_of_values(c, y, lse, starts, scale)
        return max(np.max(np.abs(got - want)[r, 0, :n] / tol[r, 0, :n]) for r, n in enumerate(LENS))
    three = _pieces(x, 3)
    assert worst(three) <= 1.0
    if not piece:
        assert (three == x).all()
    else:
        assert (three != x).any() and np.abs(three - x).max() <= 2.0 ** -27 * BIG
    assert worst(_pieces(x, 2)) > 2.0 and worst(_pieces(x, 1)) > 2.0
    half = x / 2
    half[..., 0] = x[..., 0]
    assert worst(half) > 2.0


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi,piece", RANGES)
def test_small_elements_carry_the_score(lo, hi, piece):
    from harness import ensure_built
    ds = ensure_built()
    c, q, starts, lse, scale = _inputs(lo, hi)
    want, reach = _mass(c, bits(q), lse, starts, scale)
    tol = _bound(c, want, reach, scale, piece)
    codes, scales, table, lens = c.device()
    mass = torch.zeros(want.shape, device=DEV)
    ds.kv8_mass(q.to(DEV), torch.as_tensor(lse).to(DEV), torch.as_tensor(starts).to(DEV), codes,
                scales, table, lens, scale, mass)
    got = mass.double().cpu().numpy()
    for r, n in enumerate(LENS):
        err = np.abs(got - want)[r, 0, :n] / tol[r, 0, :n]
        assert (err <= 1.0).all(), err.max()

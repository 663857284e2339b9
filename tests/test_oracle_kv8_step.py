"""Pins of oracle/kv8_step.py: closed forms, identities and the oracles that
were there."""

import numpy as np
import torch

import oracle


def _bits(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16) \
        .numpy().view(np.uint16)


def _cache(rng, pages, hk, d):
    x = torch.as_tensor(np.clip(rng.standard_normal((pages, 2, hk, 64, d)) * 100, -448, 448))
    codes = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    return codes, (2.0 ** rng.integers(-8, -5, (pages, 2, hk))).astype(np.float32)


def test_rotation_keeps_lengths_and_angles_between_positions():
    rng = np.random.default_rng(0)
    x = _bits(np.broadcast_to(rng.standard_normal((1, 1, 16)), (3, 1, 16)))
    y = _bits(np.broadcast_to(rng.standard_normal((1, 1, 16)), (3, 1, 16)))
    f = (100.0 ** (-np.arange(8) / 8)).astype(np.float32)
    for inter in (False, True):
        a, _ = oracle.qk_norm_rope(x, None, np.array([0, 5, 1005]), f, 0.0, 0, 0, inter)
        b, _ = oracle.qk_norm_rope(y, None, np.array([3, 8, 1008]), f, 0.0, 0, 0, inter)
        assert np.allclose(a[0], oracle.bf16_bits_to_float64(x)[0])
        assert np.allclose((a ** 2).sum(-1), (a[0] ** 2).sum())
        dots = (a * b).sum(-1)[:, 0]                 # a function of the difference alone
        assert np.allclose(dots, dots[0], atol=1e-9)
        # one pair turned by a quarter
        z, size = oracle.qk_norm_rope(x[:1], None, np.array([1]), np.full(8, np.pi / 2, np.float32),
                                      0.0, 0, 0, inter)
        v = oracle.bf16_bits_to_float64(x)[0, 0]
        u, w = (v[0::2], v[1::2]) if inter else (v[:8], v[8:])
        got = (z[0, 0, 0::2], z[0, 0, 1::2]) if inter else (z[0, 0, :8], z[0, 0, 8:])
        assert np.allclose(got[0], -w, atol=1e-6) and np.allclose(got[1], u, atol=1e-6)
        assert (size + 1e-12 >= np.abs(z)).all()


def test_norm_of_a_constant_row():
    x = _bits(np.full((2, 3, 24), -3.0))
    w = _bits(np.arange(16) / 8)
    y, _ = oracle.qk_norm_rope(x, w, np.zeros(2, int), np.zeros(0, np.float32), 0.0, 16, 0, False)
    assert np.allclose(y[..., :16], -np.arange(16) / 8) and (y[..., 16:] == -3).all()


def test_a_chain_is_causal_and_a_tree_is_its_paths():
    rng = np.random.default_rng(1)
    hk, d, n, length = 2, 64, 5, 90
    codes, scales = _cache(rng, 3, hk, d)
    table = np.array([[2, 0]], np.int32)
    q = _bits(rng.standard_normal((1, n, 4, d)))
    chain = np.array([[(1 << (j + 1)) - 1 for j in range(n)]], np.uint64)
    rows = oracle.kv8_visible([length], [n], 2)
    want = oracle.kv8_attention(q[0], rows, codes, scales, table, 0.1)
    got = oracle.kv8_tree(q, chain, codes, scales, table, [length], 0.1)
    for a, b in zip(got, want[:4]):
        assert np.allclose(a[0], b)
    # node 4 on the path 0-2-4: the same as the last of three accepted drafts
    tree = np.array([[1, 3, 5, 11, 21]], np.uint64)
    out, lse, _, _ = oracle.kv8_tree(q, tree, codes, scales, table, [length], 0.1)
    acc = np.array([[0, 2, 4]], np.int32)
    flat = np.full_like(scales, 2.0 ** -7)       # equal scales: nothing is rounded
    out, lse, _, _ = oracle.kv8_tree(q, tree, codes, flat, table, [length], 0.1)
    layers, new_lens, flags = oracle.kv8_accept([(codes, flat)], table, [length], n, acc)
    assert new_lens == [length - 2] and not flags
    alone = oracle.kv8_attention(q[0, 4:5], [(0, length - 2)], *layers[0], table, 0.1)
    assert np.allclose(out[0, 4], alone[0][0]) and np.allclose(lse[0, 4], alone[1][0])
    sees = oracle.tree_sees(tree[0], length, n, 2)
    assert sees[:, :length - n].all() and sees[3, length - n:].tolist() == [True, True, False, True,
                                                                          False]


def test_mass_of_all_rows_is_their_number_and_evicting_nothing_of_weight_keeps_attention():
    rng = np.random.default_rng(2)
    hk, d, length, n = 2, 64, 150, 3
    codes, scales = _cache(rng, 4, hk, d)
    table = np.array([[1, 3, 0]], np.int32)
    q = _bits(rng.standard_normal((n, 4, d)))
    rows = oracle.kv8_visible([length], [n], 3)
    lse = oracle.kv8_attention(q, rows, codes, scales, table, 0.2)[1]
    mass, _ = oracle.kv8_mass(q, lse, [0, n], codes, scales, table, [length], 0.2,
                              np.zeros((1, hk, 192)))
    assert np.allclose(mass.sum(-1), n * 2) and (mass[..., length:] == 0).all()
    again, _ = oracle.kv8_mass(q, lse, [0, n], codes, scales, table, [length], 0.2, mass)
    assert np.allclose(again[..., :length - n], 2 * mass[..., :length - n])
    assert np.allclose(again[..., length - n:], mass[..., length - n:])
    # keys of huge negative score have no mass: they go, and attention stays
    q1 = _bits(np.ones((1, 2, d)))
    codes[:, 0] = np.where(rng.random((4, hk, 64, 1)) < 0.5, 0x38, 0xF8)     # 1 or -256
    flat = np.full_like(scales, 1.0)
    one = oracle.kv8_attention(q1, [(0, length)], codes, flat, table, 1.0)
    mass, _ = oracle.kv8_mass(q1, one[1], [0, 1], codes, flat, table, [length], 1.0,
                              np.zeros((1, hk, 192)))
    keep = int(max((m > 0).sum() for m in mass[0])) + 1
    m2, c2, s2, new_lens, flags = oracle.kv8_evict(mass.astype(np.float32), keep, 0, 1, codes, flat,
                                                   table, [length])
    assert new_lens == [keep] and not flags
    cut = oracle.kv8_attention(q1, [(0, keep)], c2, s2, table, 1.0)
    assert np.allclose(cut[0], one[0]) and np.allclose(cut[1], one[1])
    assert np.allclose(m2[0, :, :keep].sum(-1), 1.0, rtol=1e-6)


def test_moved_codes_take_the_largest_scale():
    codes = np.zeros((2, 2, 1, 64, 64), np.uint8)
    codes[0] = 0x30                                  # 0.5
    codes[1] = 0x09                                  # 1.125 * 2^-6, odd mantissa
    scales = np.array([[[1.0], [1.0]], [[4.0], [0.25]]], np.float32)
    table = np.array([[0, 1]], np.int32)
    layers, new_lens, _ = oracle.kv8_accept([(codes, scales)], table, [70], 16, [[0, 12, 15]])
    c, s = layers[0]
    # base 54: drafts 12 and 15 lie in page 1 and come to slots 55 and 56 of page 0
    assert new_lens == [57] and s[0, 0, 0] == 4.0 and s[0, 1, 0] == 1.0
    val = oracle.e4m3_to_float64(c) * s[..., None, None]
    assert (val[0, 0, 0, :55] == 0.5).all() and (val[0, 0, 0, 55:57] == 4 * 1.125 * 2.0 ** -6).all()
    # values go to a coarser scale: 1.125 * 2^-8 is a tie between steps of 2^-9
    assert (val[0, 1, 0, 55:57] == 2.0 ** -8).all() and (c[0, 0, 0, 57:] == 0x30).all()


def test_shrink_gives_back_what_extend_took():
    refs, table, lens = [0] * 6, [[-1] * 4, [-1] * 4], [0, 0]
    a = oracle.pages_extend(refs, table, lens, [0, 1], [200, 70])
    b = oracle.pages_shrink(a[0], a[1], a[2], [0, 1, 0, 5], [64, 70, 3, 1])
    assert b[2] == [64, 70] and b[3] == {"row"} and sum(b[0]) == 3
    assert b[1][0] == [0, -1, -1, -1] and b[1][1] == a[1][1]
    assert oracle.pages_shrink(a[0], a[1], a[2], [0], [201])[3] == {"len"}

"""Pins of the oracle's block-scaled cache (oracle/kv8.py) and page operations
(oracle/pages.py), against closed forms and identities."""

import numpy as np
import torch

import oracle


def _bits(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16) \
        .numpy().view(np.uint16)


def test_need_scale_is_the_smallest_power_of_two_that_covers():
    for a in (1e-3, 0.5, 1.0, 1.75, 1.7578125, 448.0, 450.0, 3e4, 1e30):
        s = oracle.kv8_need_scale(a)
        assert np.log2(s) == np.rint(np.log2(s))
        assert a <= 448 * s and a > 448 * s / 2
    assert oracle.kv8_need_scale(0.0) == 0.0
    assert oracle.kv8_need_scale(1e-37) == 2.0 ** -60
    assert oracle.kv8_need_scale(np.inf) == 2.0 ** 120


def test_append_token_by_token_equals_at_once_while_codes_stay_normal():
    rng = np.random.default_rng(0)
    n, hk, d = 70, 2, 64
    k, v = (rng.choice([-1, 1], (n, hk, d)) * rng.uniform(1, 40, (n, hk, d)) for _ in range(2))
    kb, vb = _bits(k), _bits(v)
    bt = np.array([[2, 0]], np.int32)
    codes = np.full((3, 2, hk, 64, d), 0x7F, np.uint8)
    scales = np.full((3, 2, hk), 99.0, np.float32)
    once = oracle.kv8_append(kb, vb, [0, n], [n], bt, codes, scales)
    assert not once[2] and not once[3]
    c, s = codes, scales
    for t in range(n):
        c, s, _, _ = oracle.kv8_append(kb[t:t + 1], vb[t:t + 1], [0, 1], [t + 1], bt, c, s)
    assert np.array_equal(c, once[0]) and np.array_equal(s, once[1])
    # page 1 is nobody's: untouched; values are within half an E4M3 step
    assert (once[0][1] == 0x7F).all() and (once[1][1] == 99.0).all()
    val = oracle.e4m3_to_float64(once[0]) * once[1][..., None, None]
    got = val[2, 0].transpose(1, 0, 2)
    ref = oracle.bf16_bits_to_float64(kb)[:64]
    assert (np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref)).all()


def test_append_flags():
    codes, scales = np.zeros((2, 2, 1, 64, 64), np.uint8), np.ones((2, 2, 1), np.float32)
    kb = _bits(np.ones((3, 1, 64)))
    bt = np.array([[5], [1]], np.int32)
    c, s, bad_len, bad_page = oracle.kv8_append(kb, kb, [0, 1, 3], [1, 1], bt, codes, scales)
    assert bad_len and bad_page and np.array_equal(c, codes) and np.array_equal(s, scales)


def test_attention_uniform_and_single_and_empty():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 0x7F, (4, 2, 1, 64, 64)).astype(np.uint8)
    codes[3] = 0x7F                                    # never referenced
    scales = 2.0 ** rng.integers(-6, 2, (4, 2, 1)).astype(np.float64)
    bt = np.array([[2, 0], [1, 3]], np.int32)
    q = _bits(np.zeros((3, 2, 64)))
    rows = [(0, 100), (1, 1), (1, 0)]
    out, lse, weight, _, bad = oracle.kv8_attention(q, rows, codes, scales, bt, 0.125)
    val = oracle.e4m3_to_float64(codes) * scales[..., None, None]
    v = np.concatenate([val[2, 1, 0], val[0, 1, 0]])[:100]
    assert np.allclose(out[0], v.mean(0)) and np.allclose(lse[0], np.log(100))
    assert np.allclose(weight[0], np.abs(v).mean(0))
    assert np.array_equal(out[1, 0], val[1, 1, 0, 0]) and lse[1, 0] == 0
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all() and not bad


def test_attention_matches_torch_float64():
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 0x7F, (3, 2, 2, 64, 128)).astype(np.uint8)
    codes ^= (rng.integers(0, 2, codes.shape) << 7).astype(np.uint8)
    scales = 2.0 ** rng.integers(-9, -6, (3, 2, 2)).astype(np.float64)
    bt = np.array([[1, 2]], np.int32)
    q = _bits(rng.standard_normal((1, 6, 128)))
    out, lse, *_ = oracle.kv8_attention(q, [(0, 90)], codes, scales, bt, 0.1)
    val = torch.as_tensor(oracle.e4m3_to_float64(codes) * scales[..., None, None])[[1, 2]]
    k, v = (val[:, i].permute(1, 0, 2, 3).reshape(2, 128, 128)[:, :90].repeat_interleave(3, 0)
            for i in (0, 1))
    qq = torch.as_tensor(oracle.bf16_bits_to_float64(q))[0][:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(qq, k, v, scale=0.1)[:, 0]
    assert np.allclose(out[0], ref.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(lse[0], torch.logsumexp(0.1 * (qq @ k.mT)[:, 0], -1).numpy())


def test_visible_counts_are_causal_and_clamped():
    assert oracle.kv8_visible([5, 2, 200], [2, 3, 1], 2) == [
        (0, 4), (0, 5), (1, 0), (1, 1), (1, 2), (2, 128)]


def _consistent(refs, table, lens):
    count = [0] * len(refs)
    for row, length in zip(table, lens):
        for p in row[:-(-length // 64)]:
            count[p] += 1
    return count == [max(c, 0) for c in refs]


def test_page_operations_keep_the_counts():
    refs, table, lens = [0] * 12, [[-1] * 4 for _ in range(4)], [0] * 4
    refs, table, lens, fl = oracle.pages_extend(refs, table, lens, [2, 0], [130, 64])
    assert not fl and table[2][:3] == [0, 1, 2] and table[0][0] == 3 and lens == [64, 0, 130, 0]
    refs, table, lens, fl, copies = oracle.pages_fork(refs, table, lens, [2, 0], [1, 3])
    assert not fl and copies == [(2, 4)] and table[1][:3] == [0, 1, 4] and table[3][0] == 3
    assert refs[:5] == [2, 2, 1, 2, 1] and _consistent(refs, table, lens)
    refs, table, lens, fl = oracle.pages_free(refs, table, lens, [2, -1, 2])
    assert not fl and lens[2] == 0 and refs[:5] == [1, 1, 0, 2, 1]
    refs2, table2, fl, n, moves = oracle.pages_compact(refs, table, lens)
    assert n == 4 and moves == [(4, 2)] and not fl and _consistent(refs2, table2, lens)
    assert table2[1][:3] == [0, 1, 2] and refs2 == [1, 1, 1, 2] + [0] * 8


def test_page_operations_flag_what_they_skip():
    refs, table, lens = [1, 0, 0], [[0, -1], [-1, -1], [-1, -1]], [30, 0, 0]
    assert oracle.pages_fork(refs, table, lens, [0, 0, 9, 0], [1, 1, 2, 0])[3] == {"row"}
    assert oracle.pages_extend(refs, table, lens, [0, 1], [128, 128])[3] == {"nopage"}
    assert oracle.pages_extend(refs, table, lens, [0, 1], [20, 129])[3] == {"len"}
    assert oracle.pages_free(refs, [[7, -1]] + table[1:], lens, [0, 3])[3] == {"row", "page"}

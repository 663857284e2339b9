"""GPU tests of the norm of queries and keys with rotation against float64."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from harness import ensure_built
from kv8_cases import bits

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


def _freqs(rot, base=1e6):
    return torch.as_tensor(base ** (-np.arange(0, rot, 2) / max(rot, 1)), dtype=torch.float32)


def _bound(y, size, norm_dim):
    """fp32 before one rounding to bf16: the sum of squares loses at most
    norm_dim + 8 half steps (half of that in its root), the products a few more,
    and an angle off by 2^-22 turns plus sine and cosine's own 2^-22 move a value
    by at most 2^-19 of its pair. bf16 rounds by 2^-8 of the value."""
    e = size * ((norm_dim + 32) * 2.0 ** -24 + 2.0 ** -19)
    return e + 2.0 ** -8 * (np.abs(y) + e) + 1e-39


def _check(got, x, w, pos, freq, eps, norm_dim, rot_start, inter):
    y, size = oracle.qk_norm_rope(bits(x), None if w is None else bits(w), pos.cpu().numpy(),
                                  freq.cpu().numpy(), eps, norm_dim, rot_start, inter)
    err = np.abs(got.float().cpu().numpy() - y)
    assert (err <= _bound(y, size, norm_dim)).all(), err.max()


def _case(ds, tokens, heads, kv_heads, dim, rot, seed, norm_dim=None, rot_start=0, inter=False,
          weights="qk", max_pos=100000, eps=1e-6, pad=0, gain=1.0):
    rng = np.random.default_rng(seed)
    norm_dim = dim if norm_dim is None else norm_dim
    wide = (heads + 2 * kv_heads) * dim + pad
    x = torch.as_tensor(rng.standard_normal((tokens, wide)) * gain
                        * np.exp(rng.standard_normal((tokens, 1)))).to(torch.bfloat16).to(DEV)
    q = x[:, :heads * dim].unflatten(1, (heads, dim))
    k = x[:, heads * dim:(heads + kv_heads) * dim].unflatten(1, (kv_heads, dim)) if kv_heads else None
    pos = torch.as_tensor(rng.integers(-max_pos if max_pos > 1 << 30 else 0, max_pos, tokens),
                          dtype=torch.int32).to(DEV)
    freq = _freqs(rot).to(DEV)
    w = {s: torch.as_tensor(1 + 0.3 * rng.standard_normal(norm_dim)).to(torch.bfloat16).to(DEV)
         if s in weights and (s == "q" or kv_heads) else None for s in "qk"}
    before = x.clone()
    qo, ko = ds.qk_norm_rope(q, k, pos, freq, w["q"], w["k"], eps=eps, norm_dim=norm_dim,
                             rot_start=rot_start, interleaved=inter)
    torch.cuda.synchronize()
    assert torch.equal(x.view(torch.int16), before.view(torch.int16))
    for got, src, s in ((qo, q, "q"), (ko, k, "k")):
        if src is not None:
            assert got.is_contiguous() and got.shape == src.shape
            _check(got, src, w[s], pos, freq, eps, norm_dim, rot_start, inter)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot,norm_dim,rot_start", [
    (16, 16, 16, 0), (64, 64, 64, 0), (80, 32, 80, 48), (96, 96, 48, 0), (128, 128, 128, 0),
    (128, 64, 128, 64), (128, 16, 0, 8), (192, 64, 192, 128), (256, 256, 256, 0),
    (272, 48, 136, 40), (512, 0, 512, 0), (576, 64, 512, 512), (768, 768, 768, 0),
    (1024, 1024, 1024, 0),
])
def test_dims(ds, dim, rot, norm_dim, rot_start, inter):
    _case(ds, 5, 3, 2, dim, rot, seed=dim + rot, norm_dim=norm_dim, rot_start=rot_start, inter=inter,
          weights="qk" if norm_dim else "")


@pytest.mark.parametrize("tokens,heads,kv_heads", [(1, 1, 1), (1, 16, 2), (2, 7, 1), (3, 64, 8),
                                                   (33, 5, 0), (257, 28, 4), (1500, 1, 1),
                                                   (700, 128, 1), (1, 1024, 1024)])
def test_shapes(ds, tokens, heads, kv_heads):
    _case(ds, tokens, heads, kv_heads, 64 if heads > 200 else 128, 64, seed=tokens + heads)


@pytest.mark.parametrize("weights", ["", "q", "k"])
def test_sides_without_norm(ds, weights):
    _case(ds, 9, 4, 2, 128, 128, seed=3, weights=weights, pad=24)


def test_far_positions(ds):
    """Positions over the whole int32 range, both signs: the angle is exact."""
    _case(ds, 300, 2, 1, 128, 128, seed=4, max_pos=2 ** 31 - 1)
    _case(ds, 300, 2, 1, 64, 64, seed=5, max_pos=2 ** 31 - 1, inter=True)


def test_magnitudes_and_zero_rows(ds):
    _case(ds, 40, 2, 1, 128, 64, seed=6, gain=1e-18, eps=1e-6)
    _case(ds, 40, 2, 1, 128, 64, seed=7, gain=1e15, eps=0.0)
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([0, 7], dtype=torch.int32, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    q, k = ds.qk_norm_rope(x, None, pos, _freqs(64).to(DEV), w)
    assert k is None and (q == 0).all()


def test_non_finite_values_stay_in_their_row(ds):
    rng = np.random.default_rng(8)
    q = torch.as_tensor(rng.standard_normal((4, 6, 128))).to(torch.bfloat16).to(DEV)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    want, _ = ds.qk_norm_rope(q, None, pos, _freqs(128).to(DEV), w)
    q[1, 2, 5], q[3, 0, 127] = float("nan"), float("inf")
    got, _ = ds.qk_norm_rope(q, None, pos, _freqs(128).to(DEV), w)
    same = (got.view(torch.int16) == want.view(torch.int16)).all(-1).cpu()
    assert not same[1, 2] and not same[3, 0] and same.sum() == 22
    assert got[1, 2].isnan().all()


def test_a_row_does_not_depend_on_the_batch(ds):
    rng = np.random.default_rng(9)
    q = torch.as_tensor(rng.standard_normal((900, 12, 128))).to(torch.bfloat16).to(DEV)
    pos = torch.as_tensor(rng.integers(0, 50000, 900), dtype=torch.int32).to(DEV)
    w = torch.as_tensor(1 + 0.1 * rng.standard_normal(128)).to(torch.bfloat16).to(DEV)
    f = _freqs(128).to(DEV)
    whole, _ = ds.qk_norm_rope(q, None, pos, f, w)
    for lo, hi in ((0, 1), (5, 6), (100, 164), (17, 900)):
        part, _ = ds.qk_norm_rope(q[lo:hi], None, pos[lo:hi], f, w)
        assert torch.equal(part.view(torch.int16), whole[lo:hi].view(torch.int16))
    one, _ = ds.qk_norm_rope(q[:, 3:4], None, pos, f, w)
    assert torch.equal(one.view(torch.int16), whole[:, 3:4].view(torch.int16))


def test_in_place_and_strided_outputs(ds):
    rng = np.random.default_rng(10)
    x = torch.as_tensor(rng.standard_normal((50, 6 * 128))).to(torch.bfloat16).to(DEV)
    pos = torch.arange(50, dtype=torch.int32, device=DEV) * 9
    w, f = torch.ones(128, dtype=torch.bfloat16, device=DEV), _freqs(128).to(DEV)

    def parts(t):
        return t[:, :512].unflatten(1, (4, 128)), t[:, 512:640].unflatten(1, (1, 128))
    q, k = parts(x)
    want = ds.qk_norm_rope(q, k, pos, f, w, w)
    y = torch.zeros_like(x)
    ds.qk_norm_rope(q, k, pos, f, w, w, q_out=parts(y)[0], k_out=parts(y)[1])
    assert all(torch.equal(a, b) for a, b in zip(parts(y), want)) and (y[:, 640:] == 0).all()
    behind = x[:, 640:].clone()
    ds.qk_norm_rope(q, k, pos, f, w, w, q_out=q, k_out=k)
    assert all(torch.equal(a, b) for a, b in zip((q, k), want))
    assert torch.equal(x[:, 640:], behind)


def test_streams_and_graphs(ds):
    rng = np.random.default_rng(11)
    q = torch.as_tensor(rng.standard_normal((64, 8, 128))).to(torch.bfloat16).to(DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    w, f = torch.ones(128, dtype=torch.bfloat16, device=DEV), _freqs(128).to(DEV)
    want, _ = ds.qk_norm_rope(q, None, pos, f, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ds.qk_norm_rope(q, None, pos, f, w, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.qk_norm_rope(q, None, pos, f, w, q_out=out)
    pos += 1000
    g.replay()
    torch.cuda.synchronize()
    again, _ = ds.qk_norm_rope(q, None, pos, f, w)
    assert torch.equal(out, again) and not torch.equal(out, want)


def test_refusals(ds):
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((4, 1, 128), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    w, f = torch.ones(128, dtype=torch.bfloat16, device=DEV), _freqs(128).to(DEV)
    with pytest.raises(TypeError):
        ds.qk_norm_rope(q.float(), k, pos, f)
    with pytest.raises(TypeError):
        ds.qk_norm_rope(q, k, pos.long(), f)
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, k[:3], pos, f)
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, k, pos[:3], f)
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, k, pos, f, w[:64])
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, None, pos, f, k_weight=w)
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q.transpose(0, 1), None, pos, f)
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, None, pos, f, q_out=q[:2])
    with pytest.raises(ds.DSError, match="rot_start"):
        ds.qk_norm_rope(q, k, pos, f, rot_start=8)
    with pytest.raises(ds.DSError, match="head_dim=72"):
        ds.qk_norm_rope(torch.zeros((4, 2, 72), dtype=torch.bfloat16, device=DEV), None, pos, f[:8])
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, k, pos, f.cpu())
    e, _ = ds.qk_norm_rope(q[:0], None, pos[:0], f)
    assert e.shape == (0, 2, 128)


# 1 / (2 pi) to 60 digits, as a fraction.
_INV_2PI = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


def _angle(pos, freq):
    """pos * freq without its whole turns, exact to a float64's rounding."""
    turns = Fraction(int(pos)) * Fraction(float(freq)) * _INV_2PI
    return 2 * np.pi * float(turns - round(turns))


def _nearly_cancelling(angle):
    """(u, v) of 8 significant bits each whose u cos a - v sin a is near 0, so that
    no rounding of it hides the angle: the best of all pairs."""
    c, s = np.cos(angle), np.sin(angle)
    m = np.arange(128.0, 256.0)
    best = None
    for e in (-1, 0, 1):                       # |u / v| near |tan a|
        shift = 2.0 ** (np.floor(np.log2(abs(s / c))) + e)
        u, v = m[:, None] * shift, m[None, :]
        r = np.abs(u * abs(c) - v * abs(s)) / np.hypot(u, v)
        i, j = np.unravel_index(np.argmin(r), r.shape)
        if best is None or r[i, j] < best[0]:
            best = r[i, j], u[i, 0], v[0, j]
    _, u, v = best
    scale = 2.0 ** -np.floor(np.log2(max(u, v)))
    return u * scale, v * scale * np.sign(s * c)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("near,freqs", [
    (1 << 12, [1.0, 0.3, 1e-3]), (10 ** 6, [1.0, 0.73, 0.01]), (1 << 27, [1.0, 0.71, 0.049]),
    (1 << 30, [1.0, 0.649, 0.11]), ((1 << 31) - 50, [1.0, 0.649, 0.25, 0.0131]),
    ((1 << 31) - 50, [16.0, 11.3, 2.5])])
def test_angles_of_far_positions(ds, near, freqs, inter):
    """Pairs that the turn brings near 0: the angle is off by 2^-22 turns at most
    (2^-19.3 of the pair's length), sine and cosine, the products and their sum by four
    half steps of float32 (each 2^-24 of at most 1.5 lengths, and twice that for the
    functions), the result by one of bf16."""
    rng = np.random.default_rng(near & 0xFFFF)
    f = np.array(freqs * (8 // len(freqs) + 1), np.float32)[:8]
    pos = np.concatenate([near - rng.integers(0, 40, 32), -near + rng.integers(0, 40, 32)]).astype(np.int32)
    a = np.array([[_angle(p, x) for x in f] for p in pos])
    uv = np.array([[_nearly_cancelling(y) for y in row] for row in a])
    u, v = uv[..., 0], uv[..., 1]
    x = np.zeros((len(pos), 1, 16))
    iu, iv = (np.arange(0, 16, 2), np.arange(1, 16, 2)) if inter else (np.arange(8), np.arange(8, 16))
    x[:, 0, iu], x[:, 0, iv] = u, v
    q = torch.as_tensor(x).to(torch.bfloat16)
    assert (q.double().numpy() == x).all()
    got, _ = ds.qk_norm_rope(q.to(DEV), None, torch.as_tensor(pos).to(DEV), torch.as_tensor(f).to(DEV),
                             interleaved=inter)
    got = got.double().cpu().numpy()[:, 0]
    size = np.hypot(u, v)
    e = size * (2 * np.pi * 2.0 ** -22 + 2.0 ** -21)
    for at, y in ((iu, u * np.cos(a) - v * np.sin(a)), (iv, v * np.cos(a) + u * np.sin(a))):
        err = np.abs(got[:, at] - y)
        assert (err <= e + 2.0 ** -8 * (np.abs(y) + e)).all(), (err / size).max() / (2 * np.pi)
    assert np.median(np.abs(u * np.cos(a) - v * np.sin(a)) / size) <= 2.0 ** -16

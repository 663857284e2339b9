"""GPU tests of moved positions (accepted drafts, eviction) and of the pages
given back, against the oracle: codes as values, scales, mass and states exact."""

import numpy as np
import pytest
import torch

import oracle
from harness import ensure_built
from kv8_cases import Cache
from test_pages_gpu import FLAGS, State, _err, _i32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BITS = {**FLAGS, "idx": 1, "shared": 64}


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


def _same(codes, scales, want_codes, want_scales):
    a, b = (oracle.e4m3_to_float64(x) for x in (codes.cpu().numpy(), want_codes))
    assert np.array_equal(a, b, equal_nan=True)
    assert np.array_equal(scales.cpu().numpy(), want_scales, equal_nan=True)


def _paths(rng, reqs, next_n, width):
    out = np.full((reqs, width), -1, np.int32)
    for r in range(reqs):
        n = int(rng.integers(0, width + 1))
        out[r, :n] = np.sort(rng.choice(next_n, n, replace=False))
    return out


# ------------------------------------------------------------------ accept
def _accept(ds, lens, next_n, accepted, hk, dim, seed, layers=1, spread=3, odd_scales=False,
            bad=(), edit=None):
    c = Cache(lens, hk, dim, seed, spread=spread)
    if edit is not None:
        edit(c)
    for r, b, p in bad:
        c.table[r, b] = p
    host = []
    for i in range(layers):
        codes = np.roll(c.codes, i, -1)
        scales = c.scales * (c.rng.uniform(0.5, 2, c.scales.shape).astype(np.float32)
                             if odd_scales else 1)
        host.append((codes, scales.astype(np.float32)))
    dev = [(torch.as_tensor(a).to(DEV), torch.as_tensor(b).to(DEV)) for a, b in host]
    _, _, table, lens_d = c.device()
    err = _err()
    got = ds.kv8_accept(dev, table, lens_d, next_n, _i32(accepted), err_flag=err)
    torch.cuda.synchronize()
    want, new_lens, flags = oracle.kv8_accept(host, c.table, c.lens, next_n, np.asarray(accepted))
    assert got.tolist() == new_lens and lens_d.tolist() == c.lens
    for (codes, scales), (wc, ws) in zip(dev, want):
        _same(codes, scales, wc, ws)
    assert int(err) == sum(BITS[f] for f in flags)
    return flags


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("next_n", [1, 2, 8, 33, 64])
def test_accept(ds, next_n, dim):
    rng = np.random.default_rng(next_n + dim)
    lens = [next_n, next_n + 64, next_n + 63, next_n + 1, next_n + 40, 500 + next_n, 127, 128, 129]
    for width in sorted({1, next_n // 2 + 1, next_n}):
        assert not _accept(ds, lens, next_n, _paths(rng, len(lens), next_n, width), 3, dim, seed=width)


def test_accept_all_and_none(ds):
    n = 64
    acc = np.stack([np.arange(n), np.full(n, -1), np.arange(n)]).astype(np.int32)
    assert not _accept(ds, [100, 100, 64], n, acc, 2, 128, seed=1)


@pytest.mark.parametrize("odd", [False, True])
def test_accept_scales_that_grow(ds, odd):
    """Drafts from the second page whose scale is far above the first one's."""
    rng = np.random.default_rng(12)
    lens = list(range(70, 130, 4))
    for seed in range(3):
        assert not _accept(ds, lens, 48, _paths(rng, len(lens), 48, 20), 2, 64, seed=seed, spread=12,
                           odd_scales=odd)


def test_accept_many_layers_at_once(ds):
    rng = np.random.default_rng(13)
    for layers in (5, 16, 17, 40):
        assert not _accept(ds, [90, 200, 65], 16, _paths(rng, 3, 16, 8), 2, 64, seed=layers,
                           layers=layers)


def test_accept_leaves_and_flags(ds):
    ok = [0, 2, 5]
    assert _accept(ds, [100, 90], 8, [ok, [2, 2, -1]], 1, 64, 1) == {"idx"}
    assert _accept(ds, [100, 90], 8, [[3, 1, -1], ok], 1, 64, 2) == {"idx"}
    assert _accept(ds, [100, 90], 8, [[0, -1, 4], ok], 1, 64, 3) == {"idx"}
    assert _accept(ds, [100, 90], 8, [[0, 7, 8], ok], 1, 64, 4) == {"idx"}
    assert _accept(ds, [5, 90], 8, [ok, ok], 1, 64, 5) == {"len"}
    assert _accept(ds, [0, -3, 90], 8, [ok, ok, ok], 1, 64, 6) == set()
    assert _accept(ds, [100, 90], 8, [ok, ok], 1, 64, 7, bad=[(0, 1, -1)]) == {"page"}
    assert _accept(ds, [100, 90], 8, [ok, ok], 1, 64, 8, bad=[(1, 1, 10 ** 6)]) == {"page"}
    # the page in front of the drafts may be anything
    assert _accept(ds, [200, 90], 8, [ok, ok], 1, 64, 9, bad=[(0, 0, -1)]) == set()


# ------------------------------------------------------------------- evict
def _evict(ds, lens, budget, first, recent, hk, dim, seed, spread=3, odd_scales=False, mass=None,
           refs=None, bad=(), extra=0, capture=False, edit=None):
    c = Cache(lens, hk, dim, seed, spread=spread)
    if edit is not None:
        edit(c)
    for r, b, p in bad:
        c.table[r, b] = p
    if odd_scales:
        c.scales *= c.rng.uniform(0.5, 2, c.scales.shape).astype(np.float32)
    stride = 64 * c.table.shape[1] + extra
    m = np.exp(2 * c.rng.standard_normal((len(lens), hk, stride))).astype(np.float32)
    if mass is not None:
        m = mass(c.rng, m)
    codes, scales, table, lens_d = c.device()
    md = torch.as_tensor(m).to(DEV)
    err = _err()
    rd = None if refs is None else _i32(refs(c))
    args = (md, budget, first, recent, codes, scales, table, lens_d)
    if capture:
        got = torch.empty(len(lens), dtype=torch.int32, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ds.kv8_evict(*args, refcounts=rd, new_lens=got, err_flag=err)
        g.replay()
    else:
        got = ds.kv8_evict(*args, refcounts=rd, err_flag=err)
    torch.cuda.synchronize()
    wm, wc, ws, new_lens, flags = oracle.kv8_evict(m, budget, first, recent, c.codes, c.scales,
                                                   c.table, c.lens, None if rd is None else rd.tolist())
    assert got.tolist() == new_lens and lens_d.tolist() == c.lens
    _same(codes, scales, wc, ws)
    assert np.array_equal(md.cpu().numpy(), wm, equal_nan=True)
    assert int(err) == sum(BITS[f] for f in flags)
    return flags


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (1, 0, 1), (1, 1, 0), (64, 4, 16),
                                                 (65, 0, 64), (100, 2, 98), (129, 3, 0), (200, 0, 7)])
def test_evict(ds, budget, first, recent, dim):
    lens = [0, 1, budget, budget + 1, budget + 64, 300, 257, 64, 700, -5]
    assert not _evict(ds, lens, budget, first, recent, 2, dim, seed=budget + dim)


@pytest.mark.parametrize("reqs,hk,dim,lens,budget", [
    (1, 1, 128, 4000, 2500), (1, 8, 128, 2700, 1024), (3, 2, 64, 3000, 2111), (40, 8, 64, 200, 90)])
def test_evict_rounds_and_rankings(ds, reqs, hk, dim, lens, budget):
    """Budgets of several rounds, and batches that each ranking kernel serves."""
    rng = np.random.default_rng(reqs)
    ls = rng.integers(budget // 2, lens + 1, reqs)
    ls[0] = lens
    assert not _evict(ds, ls, budget, 4, 33, hk, dim, seed=reqs)


@pytest.mark.parametrize("odd", [False, True])
def test_evict_scales_that_grow(ds, odd):
    assert not _evict(ds, [900, 130], 111, 1, 9, 2, 64, seed=3, spread=14, odd_scales=odd)


def test_evict_ties_and_strange_mass(ds):
    def ties(rng, m):
        return rng.integers(0, 3, m.shape).astype(np.float32)

    def strange(rng, m):
        m[rng.random(m.shape) < 0.3] = np.nan
        m[rng.random(m.shape) < 0.1] = np.inf
        m[rng.random(m.shape) < 0.1] = -np.inf
        return m
    for f in (ties, strange, lambda rng, m: np.zeros_like(m), lambda rng, m: m * np.nan):
        assert not _evict(ds, [500, 100, 333], 90, 2, 20, 2, 64, seed=4, mass=f)


def test_evict_leaves_and_flags(ds):
    assert _evict(ds, [300, 200], 100, 0, 10, 2, 64, 5, bad=[(0, 4, -1)]) == {"page"}
    assert _evict(ds, [300, 200], 100, 0, 10, 2, 64, 6, bad=[(1, 0, 10 ** 6)]) == {"page"}

    def refs(c, page):
        r = np.zeros(c.pages, np.int32)
        r[c.table[c.table >= 0]] = 1
        r[page] += 1
        return r
    assert _evict(ds, [300, 200], 100, 0, 10, 2, 64, 7, refs=lambda c: refs(c, c.table[0, 1])) \
        == {"shared"}
    assert _evict(ds, [300, 200], 100, 0, 10, 2, 64, 7, refs=lambda c: refs(c, c.table[0, 2])) == set()
    # longer than the table
    c = Cache([300, 200], 1, 64, 8, extra_width=0)
    codes, scales, table, lens = c.device()
    lens[0] = 1000
    mass = torch.rand((2, 1, 320), device=DEV)
    before, err = codes.clone(), _err()
    got = ds.kv8_evict(mass, 250, 0, 10, codes, scales, table, lens, err_flag=err)
    assert got.tolist() == [1000, 200] and int(err) == 32 and torch.equal(codes, before)


def test_evict_wider_mass_and_capture(ds):
    assert not _evict(ds, [900, 150, 66], 60, 3, 9, 2, 128, seed=9, extra=4, capture=True)
    assert not _evict(ds, [3000], 1500, 3, 9, 2, 64, seed=10, extra=36, capture=True)


@pytest.mark.parametrize("value", [0.0, np.inf])
def test_codes_under_equal_scales_are_copied(ds, value):
    """Also where the scales have no quotient: pages that were never scaled, or lost."""
    def all_pages(c):
        c.scales[...] = value

    def some_pages(c):
        c.scales[c.rng.random(c.scales.shape) < 0.5] = 0.0
    rng = np.random.default_rng(14)
    for edit in (all_pages, some_pages):
        lens = [90, 120, 64, 300]
        assert not _accept(ds, lens, 40, _paths(rng, 4, 40, 20), 2, 64, seed=5, edit=edit)
        assert not _evict(ds, lens, 80, 2, 20, 2, 128, seed=6, edit=edit)


def test_accept_captured_and_two_evictions_at_once(ds):
    c = Cache([700, 900], 2, 64, 16)
    codes, scales, table, lens = c.device()
    acc = _i32([[0, 3, 7, -1], [2, -1, -1, -1]])
    want = (codes.clone(), scales.clone())
    new = ds.kv8_accept([want], table, lens, 8, acc)
    got = (codes.clone(), scales.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens2 = ds.kv8_accept([got], table, lens, 8, acc)
    g.replay()
    torch.cuda.synchronize()
    # (As bits: the scales of unused pages are NaN.)
    assert torch.equal(new, lens2) and torch.equal(got[0], want[0])
    assert torch.equal(got[1].view(torch.int32), want[1].view(torch.int32))
    mass = torch.rand((2, 2, 64 * table.shape[1]), device=DEV)

    def evict(kw):
        m, k, s = mass.clone(), codes.clone(), scales.clone()
        torch.cuda.synchronize()
        new = ds.kv8_evict(m, 300, 4, 50, k, s, table, lens, **kw)
        return m, k, s.view(torch.int32), new
    one = evict({})
    for _ in range(3):
        both = [evict(dict(stream=torch.cuda.Stream())) for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for b in both for x, y in zip(b, one))


# ------------------------------------------------------------------ shrink
@pytest.mark.parametrize("rows,new_lens", [
    ([0], [64]), ([0, 1, 2, 4], [0, 64, 0, 129]), ([4, -1, 0], [1, 7, 700]), ([3, 2], [0, 1]),
    ([0, 0], [65, 64]), ([9, 1], [5, 3]), ([0, 1], [701, -1]), ([0, 5], [640, -4]),
])
def test_shrink(ds, rows, new_lens):
    s = State(60, 12, [700, 64, 1, 0, 130, -4], seed=1, share=[(0, 4, 2)])
    refs, table, lens = s.device()
    err = _err()
    ds.pages_shrink(refs, table, lens, _i32(rows), _i32(new_lens), err_flag=err)
    s.check(*oracle.pages_shrink(s.refs, s.table, s.lens, rows, new_lens), err)


def test_shrink_flags_what_it_cannot_count(ds):
    s = State(10, 4, [200, 100], seed=2)
    s.table[0][2], s.table[0][3], s.refs[s.table[1][1]] = 77, -1, 0
    refs, table, lens = s.device()
    err = _err()
    ds.pages_shrink(refs, table, lens, _i32([0, 1]), _i32([64, 10]), err_flag=err)
    want = oracle.pages_shrink(s.refs, s.table, s.lens, [0, 1], [64, 10])
    assert want[3] == {"page"}
    s.check(*want, err)


def test_shrink_then_extend_gives_the_lowest_pages_again(ds):
    s = State(40, 8, [500, 200], seed=3)
    refs, table, lens = s.device()
    ds.pages_shrink(refs, table, lens, _i32([0, 1]), _i32([130, 64]))
    ds.pages_extend(refs, table, lens, _i32([1, 0]), _i32([256, 300]))
    a = oracle.pages_shrink(s.refs, s.table, s.lens, [0, 1], [130, 64])
    b = oracle.pages_extend(a[0], a[1], a[2], [1, 0], [256, 300])
    torch.cuda.synchronize()
    assert (refs.tolist(), table.tolist(), lens.tolist()) == (b[0], b[1], b[2])


def test_evictions_again_and_again(ds):
    """A cache at its budget that grows by a few tokens and is cut again, many times: each
    cut as the oracle's, and values no further off than one rounding in the normal
    range and half a step of the page's present scale, and of each smaller one, below it."""
    rng = np.random.default_rng(31)
    reqs, hk, heads, d, budget, first, recent, width = 2, 2, 4, 64, 150, 3, 30, 5
    pages = reqs * width
    table = _i32(rng.permutation(pages).reshape(reqs, width))
    codes = torch.zeros((pages, 2, hk, 64, d), dtype=torch.uint8, device=DEV)
    scales = torch.ones((pages, 2, hk), device=DEV)
    mass = torch.zeros((reqs, hk, 64 * width), device=DEV)
    lens = np.zeros(reqs, np.int64)
    exact = [[np.zeros((0, 2, d)) for _ in range(hk)] for _ in range(reqs)]
    need = np.zeros((2, hk))                  # largest scale that any token asked for
    cuts = 0
    for step in range(24):
        counts = [int(rng.integers(1, 9)) for _ in range(reqs)] if step else [150, 40]
        lens += counts
        n = sum(counts)
        # (Tokens of very different sizes: pages' scales differ, and grow.)
        x = rng.standard_normal((n, 2, hk, d)) * np.exp2(rng.uniform(-6, 6, (n, 2, hk, 1)))
        x = torch.as_tensor(x).to(torch.bfloat16)
        starts = _i32(np.concatenate([[0], np.cumsum(counts)]))
        dev_lens, dev_x = _i32(lens), x.to(DEV)
        ds.kv8_append(dev_x[:, 0], dev_x[:, 1], starts, table, dev_lens, codes, scales)
        q = torch.as_tensor(rng.standard_normal((n, heads, d))).to(torch.bfloat16).to(DEV)
        _, lse = ds.kv8_prefill(q, starts, codes, scales, table, dev_lens, 0.02)
        ds.kv8_mass(q, lse, starts, codes, scales, table, dev_lens, 0.02, mass)
        torch.cuda.synchronize()
        before = [t.cpu().numpy() for t in (mass, codes, scales, table)]
        got = ds.kv8_evict(mass, budget, first, recent, codes, scales, table, dev_lens)
        torch.cuda.synchronize()
        want = oracle.kv8_evict(before[0], budget, first, recent, before[1], before[2], before[3],
                                dev_lens.cpu().numpy())
        assert got.tolist() == want[3]
        assert np.array_equal(mass.cpu().numpy(), want[0]) and not np.isnan(want[0]).any()
        _same(codes, scales, want[1], want[2])
        host = x.double().numpy()
        top = np.maximum.reduce(np.abs(host).max(-1), axis=0) / 448
        need = np.maximum(need, np.exp2(np.ceil(np.log2(top))))
        at = 0
        for r in range(reqs):
            for g in range(hk):
                e = np.concatenate([exact[r][g], host[at:at + counts[r], :, g]])
                if lens[r] > budget:
                    k = budget - first - recent
                    best = oracle.topk_per_row(before[0][r, g][None], np.array([first], np.int32),
                                               np.array([lens[r] - recent], np.int32), k)[0]
                    e = e[[*range(first), *(first + int(b) for b in best),
                           *range(lens[r] - recent, lens[r])]]
                    cuts += 1
                exact[r][g] = e
            at += counts[r]
        lens = np.minimum(lens, budget)
    assert cuts >= 40
    held_codes, held_scales = codes.cpu().numpy(), scales.cpu().numpy()
    for r in range(reqs):
        for g in range(hk):
            for side in range(2):
                p = table[r].cpu().numpy()[:-(-int(lens[r]) // 64)]
                s = held_scales[p, side, g]
                assert (s <= need[side, g]).all()
                v = oracle.e4m3_to_float64(held_codes[p, side, g]) * s[:, None, None]
                v, s = v.reshape(-1, d)[:lens[r]], np.repeat(s, 64)[:lens[r], None]
                x = exact[r][g][:, side]
                assert (np.abs(v - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * s).all()


def test_evict_and_accept_with_many_heads(ds):
    assert not _evict(ds, [200, 130, 60], 70, 2, 10, 300, 64, seed=17)
    rng = np.random.default_rng(17)
    assert not _accept(ds, [90, 64 + 5, 64], 20, _paths(rng, 3, 20, 20), 300, 64, seed=18)

"""GPU tests of the attention of draft trees over the block-scaled cache, within
the bounds of the other attention calls, and of a whole speculative step."""

import math

import numpy as np
import pytest
import torch

import oracle
from harness import ensure_built
from kv8_cases import DEV, Cache, bits
from test_kv8_gpu import _close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


def _tree(rng, reqs, n):
    """Masks of random trees: node 0 the root, every other node an earlier parent."""
    masks = np.zeros((reqs, n), np.uint64)
    for r in range(reqs):
        for j in range(n):
            up = masks[r, rng.integers(0, j)] if j else np.uint64(0)
            masks[r, j] = up | np.uint64(1 << j)
    return masks


def _dev(masks):
    return torch.as_tensor(masks.view(np.int64)).to(DEV)


def _run(ds, c, masks, heads, scale=None, gain=2.5, q=None, bound_scale=None, **kw):
    n = masks.shape[1]
    scale = 1 / math.sqrt(c.dim) if scale is None else scale
    q = c.q(len(c.lens) * n, heads, gain) if q is None else q
    codes, scales, table, lens = c.device()
    out, lse = ds.kv8_tree_decode(q.to(DEV).view(len(c.lens), n, heads, c.dim), _dev(masks), codes,
                                  scales, table, lens, scale, **kw)
    qb = bits(q).reshape(len(c.lens), n, heads, c.dim)
    ref = oracle.kv8_tree(qb, masks, c.codes, c.scales, c.table, c.lens, scale)
    torch.cuda.synchronize()
    flat = [x.reshape(-1, *x.shape[2:]) for x in ref]
    _close(out.flatten(0, 1), lse.flatten(0, 1), (*flat, False), c.dim, max(c.lens + [1]))
    return out, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,kv_heads,group", [(1, 1, 1), (2, 2, 8), (5, 3, 7), (8, 2, 3), (13, 1, 16),
                                              (33, 2, 4), (64, 1, 2), (16, 2, 8), (43, 1, 6),
                                              (64, 2, 8), (64, 1, 12)])
def test_trees(ds, n, kv_heads, group, dim):
    c = Cache([n, n + 1, n + 63, n + 64, 200 + n, 0, 129 + n, n - 1, n + 100, -4], kv_heads, dim,
              seed=n + group)
    _run(ds, c, _tree(c.rng, len(c.lens), n), kv_heads * group)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [6, 16])
def test_masks_of_any_kind(ds, heads, dim):
    """No bit at all (the prefix alone, or nothing), bits of later nodes, bits that
    no node has, all of them."""
    n = 9
    c = Cache([n, 300, 70, 64 + n, 128], 2, dim, seed=3)
    masks = _tree(c.rng, 5, n)
    masks[:, 0] = 0
    masks[:, 3] = 0x100
    masks[:, 4] = np.uint64(0xFFFFFFFFFFFFFFFF)
    masks[:, 5] = np.uint64(0xFFFFFFFFFFFFFE00)
    out, lse = _run(ds, c, masks, heads)
    assert (out[0, 0] == 0).all() and torch.isneginf(lse[0, 0]).all()
    assert (out[0, 5] == 0).all() and torch.isneginf(lse[0, 5]).all()


@pytest.mark.parametrize("n,lens,dim", [
    (8, [5000, 1030, 1024, 2049 + 6], 128), (64, [2100, 1024 + 63, 1100], 128), (16, [40000], 128),
    (20, [9000, 1030, 1024, 1044, 2048 + 19, 8192 + 7], 128), (33, [3000, 1056, 64], 64),
    (41, [9000, 1030, 1024, 1065, 2048 + 19, 8192 + 7], 64)])
def test_long_contexts(ds, n, lens, dim):
    """Trees that begin, end and straddle where spans are cut."""
    c = Cache(lens, 1, dim, seed=n)
    _run(ds, c, _tree(c.rng, len(lens), n), 4)


@pytest.mark.parametrize("n,group", [(1, 8), (5, 8), (12, 3), (64, 1), (10, 8)])
def test_a_chain_is_decode(ds, n, group):
    """Up to 80 rows, bit for bit."""
    c = Cache([700, n, 64 + n, 1500, 3, 0], 2, 128, seed=n)
    masks = np.array([(1 << (j + 1)) - 1 for j in range(n)], np.uint64)
    masks = np.broadcast_to(masks, (6, n)).copy()
    codes, scales, table, lens = c.device()
    q = c.q(6 * n, 2 * group).to(DEV).view(6, n, 2 * group, 128)
    a = ds.kv8_decode(q, codes, scales, table, lens, 0.1)
    b = ds.kv8_tree_decode(q, _dev(masks), codes, scales, table, lens, 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,heads,d", [(6, 8, 128), (30, 8, 128), (30, 8, 64), (64, 12, 128)])
def test_nan_drafts_reach_only_who_sees_them(ds, n, heads, d):
    """A NaN key or value of draft 3: nodes that do not see it stay as they are."""
    hk, half = 2, heads // 2
    c = Cache([64 + n - 2, 1100], hk, d, seed=5)
    masks = _tree(c.rng, 2, n)
    codes, scales, table, lens = c.device()
    q = c.q(2 * n, heads).to(DEV).view(2, n, heads, d)
    want = ds.kv8_tree_decode(q, _dev(masks), codes, scales, table, lens, 0.1)
    for side in (0, 1):
        bad = codes.clone()
        for r in range(2):
            p = c.lens[r] - n + 3
            bad[c.table[r, p // 64], side, 1, p % 64, 17] = 0x7F
        out, lse = ds.kv8_tree_decode(q, _dev(masks), bad, scales, table, lens, 0.1)
        torch.cuda.synchronize()
        for r in range(2):
            for j in range(n):
                sees = bool(int(masks[r, j]) >> 3 & 1)
                assert torch.equal(out[r, j, :half], want[0][r, j, :half])     # kv head 0
                if sees:
                    assert out[r, j, half:, 17].isnan().all()
                else:
                    assert torch.equal(out[r, j, half:], want[0][r, j, half:])
                    assert torch.equal(lse[r, j], want[1][r, j])


@pytest.mark.parametrize("n", [10, 31])
def test_pages_outside_the_pool(ds, n):
    c = Cache([300, 100], 2, 64, seed=6)
    c.table[0, 2], c.table[0, 4], c.table[1, 0] = -1, 10 ** 6, -5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _run(ds, c, _tree(c.rng, 2, n), 4, err_flag=err)
    assert int(err) == ds.DEVERR_PAGE


@pytest.mark.parametrize("n", [7, 20])
def test_large_elements_of_q(ds, n):
    """Elements hundreds of times the others: what the 8-bit pieces lose is added."""
    c = Cache([500, 90], 1, 128, seed=7)
    q = c.q(2 * n, 4, gain=1.0)
    q[:, 1, 5] = 900.0
    codes = c.codes[:, 0]
    codes[..., 5] = 0
    _run(ds, c, _tree(c.rng, 2, n), 4, q=q)


@pytest.mark.parametrize("n,dim", [(5, 128), (12, 128), (12, 64), (40, 128)])
def test_bits_do_not_depend_on_the_batch(ds, n, dim):
    c = Cache([2500, 64, 900, 1300, 40], 2, dim, seed=8)
    masks = _tree(c.rng, 5, n)
    codes, scales, table, lens = c.device()
    q = c.q(5 * n, 16).to(DEV).view(5, n, 16, dim)
    whole = ds.kv8_tree_decode(q, _dev(masks), codes, scales, table, lens, 0.1)
    for r in range(5):
        one = ds.kv8_tree_decode(q[r:r + 1], _dev(masks[r:r + 1]), codes, scales,
                                 table[r:r + 1].contiguous(), lens[r:r + 1], 0.1)
        assert torch.equal(one[0][0], whole[0][r]) and torch.equal(one[1][0], whole[1][r])


@pytest.mark.parametrize("n", [5, 24])
def test_captured_and_on_two_streams(ds, n):
    """Both forms, replayed twice, and two calls at once."""
    c = Cache([2500, 64, 9000, 0], 2, 128, seed=15)
    masks = _dev(_tree(c.rng, 4, n))
    codes, scales, table, lens = c.device()
    q = c.q(4 * n, 16).to(DEV).view(4, n, 16, 128)

    def run(x, **kw):
        return ds.kv8_tree_decode(x, masks, codes, scales, table, lens, 0.1, **kw)
    want, other = run(q), run(-q)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a, b = run(q, stream=streams[0]), run(-q, stream=streams[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*a, *b), (*want, *other)))
    x = q.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(x)
    for y, ref in ((-q, other), (q, want)):
        x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, ref))


def test_refusals(ds):
    c = Cache([100], 2, 64, seed=9)
    codes, scales, table, lens = c.device()
    q = c.q(3, 4).to(DEV).view(1, 3, 4, 64)
    m = torch.ones((1, 3), dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        ds.kv8_tree_decode(q, m.int(), codes, scales, table, lens, 0.1)
    with pytest.raises(ValueError):
        ds.kv8_tree_decode(q, m[:, :2].contiguous(), codes, scales, table, lens, 0.1)
    with pytest.raises(TypeError):
        ds.kv8_tree_decode(q, None, codes, scales, table, lens, 0.1)
    big = torch.zeros((1, 65, 4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ds.DSError, match="next_n=65"):
        ds.kv8_tree_decode(big, torch.ones((1, 65), dtype=torch.int64, device=DEV), codes, scales,
                           table, lens, 0.1)


@pytest.mark.parametrize("capture", [False, True])
def test_a_speculative_step_then_eviction(ds, capture):
    """norm + rotation, extend, append, tree attention, accept, shrink; the mass of
    the accepted tokens; eviction; and decode over what is left, once eagerly and
    once as one captured graph."""
    rng = np.random.default_rng(10)
    reqs, n, heads, hk, d, budget = 3, 8, 8, 2, 64, 96
    i32 = dict(dtype=torch.int32, device=DEV)
    width, pages = 4, 16
    refs, table = torch.zeros(pages, **i32), torch.full((reqs, width), -1, **i32)
    lens = torch.zeros(reqs, **i32)
    codes = torch.full((pages, 2, hk, 64, d), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.ones((pages, 2, hk), device=DEV)
    rows, prompt = torch.arange(reqs, **i32), [100, 57, 130]
    ds.pages_extend(refs, table, lens, rows, torch.tensor(prompt, **i32))
    kv = torch.as_tensor(rng.standard_normal((sum(prompt), 2, hk, d))).to(torch.bfloat16).to(DEV)
    starts = torch.tensor([0, 100, 157, 287], **i32)
    ds.kv8_append(kv[:, 0], kv[:, 1], starts, table, lens, codes, scales)
    mass = torch.zeros((reqs, hk, 64 * width), device=DEV)
    q0 = torch.as_tensor(rng.standard_normal((287, heads, d))).to(torch.bfloat16).to(DEV)
    _, lse0 = ds.kv8_prefill(q0, starts, codes, scales, table, lens, 0.125)
    ds.kv8_mass(q0, lse0, starts, codes, scales, table, lens, 0.125, mass)

    x = torch.as_tensor(rng.standard_normal((reqs * n, (heads + 2 * hk) * d))).to(torch.bfloat16).to(DEV)
    w = torch.as_tensor(1 + 0.1 * rng.standard_normal(d)).to(torch.bfloat16).to(DEV)
    freq = torch.as_tensor(1e4 ** (-np.arange(0, d, 2) / d), dtype=torch.float32).to(DEV)
    masks = _tree(rng, reqs, n)
    path = [[j for j in range(n) if int(masks[r, m]) >> j & 1] for r, m in enumerate((7, 4, 0))]
    acc = np.full((reqs, n), -1, np.int32)
    for r, p in enumerate(path):
        acc[r, :len(p)] = p
    depth = torch.as_tensor([[bin(int(m)).count("1") - 1 for m in masks[r]] for r in range(reqs)], **i32)
    positions = (torch.tensor(prompt, **i32)[:, None] + depth).flatten().contiguous()
    full = torch.tensor([p + n for p in prompt], **i32)
    acc_d, masks_d = torch.as_tensor(acc).to(DEV), _dev(masks)
    took = torch.as_tensor(np.concatenate([[r * n + j for j in p] for r, p in enumerate(path)])).to(DEV)
    tree_starts = torch.arange(reqs + 1, **i32) * n
    took_starts = torch.tensor(np.cumsum([0] + [len(p) for p in path]), **i32)
    outs = {}

    def step():
        q, k = ds.qk_norm_rope(x[:, :heads * d].unflatten(1, (heads, d)),
                               x[:, heads * d:(heads + hk) * d].unflatten(1, (hk, d)), positions,
                               freq, w, w)
        v = x[:, (heads + hk) * d:].unflatten(1, (hk, d))
        ds.pages_extend(refs, table, lens, rows, full)
        ds.kv8_append(k, v, tree_starts, table, lens, codes, scales)
        out, lse = ds.kv8_tree_decode(q.view(reqs, n, heads, d), masks_d, codes, scales, table, lens,
                                      0.125)
        left = ds.kv8_accept([(codes, scales)], table, lens, n, acc_d)
        ds.pages_shrink(refs, table, lens, rows, left)
        q_took, lse_took = q[took], lse.flatten(0, 1)[took]
        ds.kv8_mass(q_took, lse_took, took_starts, codes, scales, table, lens, 0.125, mass)
        outs["before"] = [t.clone() for t in (codes, scales, table, lens, mass)]
        cut = ds.kv8_evict(mass, budget, 2, 20, codes, scales, table, lens, refcounts=refs)
        ds.pages_shrink(refs, table, lens, rows, cut)
        after, _ = ds.kv8_decode(q.view(reqs, n, heads, d)[:, :1].contiguous(), codes, scales, table,
                                 lens, 0.125)
        outs.update(out=out, q=q, lse=lse, lse_took=lse_took, after=after)
    if capture:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        g.replay()
    else:
        step()
    torch.cuda.synchronize()
    host = [t.cpu().numpy() for t in outs["before"]]
    assert host[3].tolist() == [p + len(a) for p, a in zip(prompt, path)]
    # the accepted path alone, as decode sees it after the move, is what the tree
    # gave for its last node (codes may be rounded once more where a scale grew)
    for r, p in enumerate(path):
        qb = bits(outs["q"]).reshape(reqs, n, heads, d)[r, p[-1]][None]
        want = oracle.kv8_attention(qb, [(r, int(host[3][r]))], host[0], host[1], host[2], 0.125)
        err = np.abs(outs["out"][r, p[-1]].float().cpu().numpy() - want[0][0])
        assert (err <= 2.0 ** -6 * want[2][0] + 1e-6).all()
    assert lens.tolist() == [min(budget, int(x)) for x in host[3]]
    held = [-(-int(x) // 64) for x in lens.tolist()]
    assert int((refs > 0).sum()) == sum(held) and int((table >= 0).sum()) == sum(held)
    e = oracle.kv8_evict(host[4], budget, 2, 20, host[0], host[1], host[2], host[3])
    assert e[3] == lens.tolist()
    assert np.array_equal(mass.cpu().numpy(), e[0])
    rows_seen = [(r, int(x)) for r, x in enumerate(lens.tolist())]
    qb = bits(outs["q"]).reshape(reqs, n, heads, d)[:, 0]
    want = oracle.kv8_attention(qb, rows_seen, e[1], e[2], table.cpu().numpy(), 0.125)
    err = np.abs(outs["after"][:, 0].float().cpu().numpy() - want[0])
    assert (err <= 2.0 ** -7 * want[2] + 1e-6).all()


def test_many_large_trees(ds):
    """Runs of tiles that end inside an item, empty requests among them; two streams."""
    rng = np.random.default_rng(11)
    lens = rng.integers(40, 3000, 40)
    lens[[3, 17, 18]] = 0
    c = Cache(lens, 2, 128, seed=11)
    masks = _tree(c.rng, 40, 32)
    codes, scales, table, ln = c.device()
    q = c.q(40 * 32, 16).to(DEV).view(40, 32, 16, 128)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = ds.kv8_tree_decode(q, _dev(masks), codes, scales, table, ln, 0.1, err_flag=err)
    md = _dev(masks)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [ds.kv8_tree_decode(q, md, codes, scales, table, ln, 0.1, stream=s) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert int(err) == 0
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for r in (0, 3, 7, 39):
        one = ds.kv8_tree_decode(q[r:r + 1], md[r:r + 1].contiguous(), codes, scales,
                                 table[r:r + 1].contiguous(), ln[r:r + 1], 0.1)
        assert torch.equal(one[0][0], want[0][r]) and torch.equal(one[1][0], want[1][r])


@pytest.mark.parametrize("dim,n,group", [(64, 24, 4), (64, 41, 8), (128, 24, 4), (64, 5, 4)])
@pytest.mark.parametrize("length", [600, 3000])
@pytest.mark.parametrize("gone", [0, 1, None])
def test_scores_too_low_for_a_reference_give_nan(ds, dim, n, group, length, gone):
    """Scores near -2^26 in every span, and the even or the odd pages outside the pool: the
    outputs are NaN as where all pages are there, never 0 with an lse of -inf."""
    c = Cache([length], 1, dim, seed=25)
    c.codes[c.table[0, :-(-length // 64)]] = 0x7E          # 448 everywhere
    c.scales[:] = 1.0
    if gone is not None:
        c.table[0, gone::2] = -1
    q = torch.full((1, n, group, dim), -8.0, dtype=torch.bfloat16, device=DEV)
    codes, scales, table, lens = c.device()
    masks = _dev(_tree(c.rng, 1, n))
    out, lse = ds.kv8_tree_decode(q, masks, codes, scales, table, lens, 2.0 ** 26 / (448 * 8 * dim))
    torch.cuda.synchronize()
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("dim", [64, 128])
def test_thousands_of_requests(ds, dim):
    """More units than the kernel that numbers them has threads; most requests are short,
    many empty. A request's outputs are those of a call of its own."""
    rng = np.random.default_rng(26)
    reqs, n, heads, pages = 3000, 12, 8, 40
    lens = rng.integers(-3, 200, reqs)
    lens[rng.integers(0, reqs, 40)] = rng.integers(1000, 2500, 40)
    codes = torch.as_tensor(rng.integers(0, 0x70, (pages, 2, 1, 64, dim)), dtype=torch.uint8).to(DEV)
    scales = torch.full((pages, 2, 1), 2.0 ** -7, device=DEV)
    table = torch.as_tensor(rng.integers(0, pages, (reqs, 40)), dtype=torch.int32).to(DEV)
    ln = torch.as_tensor(lens, dtype=torch.int32).to(DEV)
    masks = _dev(_tree(rng, reqs, n))
    q = torch.as_tensor(rng.standard_normal((reqs, n, heads, dim))).to(torch.bfloat16).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = ds.kv8_tree_decode(q, masks, codes, scales, table, ln, 0.1, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for r in [0, 1, reqs - 1, *rng.integers(0, reqs, 40), *np.argsort(lens)[-5:], *np.argsort(lens)[:3]]:
        a, b = ds.kv8_tree_decode(q[r:r + 1], masks[r:r + 1], codes, scales, table[r:r + 1].contiguous(),
                                  ln[r:r + 1], 0.1)
        assert torch.equal(a[0], out[r]) and torch.equal(b[0], lse[r])
        if lens[r] <= 0:
            assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()


@pytest.mark.parametrize("n,kv_heads,group", [(2, 1024, 1), (64, 200, 2), (3, 40, 25), (1, 1, 1024)])
def test_many_heads(ds, n, kv_heads, group):
    c = Cache([n + 70, n], kv_heads, 64, seed=27)
    _run(ds, c, _tree(c.rng, 2, n), kv_heads * group)

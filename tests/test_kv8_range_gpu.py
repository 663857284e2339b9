"""GPU tests of the block-scaled 8-bit cache where its numbers leave the usual
range: queries with one element far above the others, scores far below those
that matter, long contexts, key scales and tables at their limits.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from harness import ensure_built
from kv8_cases import DEV, Cache, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


def _both(ds, c, q, counts, scale, **kw):
    """(kernel, out, lse) of the last counts[r] (all equal) tokens by decode and
    by prefill."""
    codes, scales, table, lens = c.device()
    n, h = counts[0], q.shape[1]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    q = q.to(DEV)
    o, l = ds.kv8_decode(q.view(len(counts), n, h, c.dim), codes, scales, table, lens, scale, **kw)
    yield "decode", o.flatten(0, 1), l.flatten(0, 1)
    yield "prefill", *ds.kv8_prefill(q, starts, codes, scales, table, lens, scale, **kw)


def _ref(c, q, counts, scale):
    rows = oracle.kv8_visible(c.lens, counts, c.table.shape[1])
    return oracle.kv8_attention(bits(q), rows, c.codes, c.scales, c.table, scale)


def _close(out, lse, ref, dim, length, score=0.0):
    """Within oracle.kv8_bounds, for scores that are off by `score` [T, heads]
    more: that moves a weight, and the sum that divides it, by that factor."""
    ref_out, ref_lse, weight, reach, _ = ref
    tol, tol_lse = oracle.kv8_bounds(ref_out, ref_lse, weight, reach, dim, length)
    score = np.broadcast_to(score, ref_lse.shape)
    tol = tol + 1.01 * 2 * np.expm1(score)[..., None] * weight
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(o - ref_out) <= tol).all(), np.nanmax(np.abs(o - ref_out) / tol)
    fin = np.isfinite(ref_lse)
    assert np.array_equal(np.isneginf(l), ~fin)
    tol_lse = tol_lse + score
    assert (np.abs(l - ref_lse)[fin] <= tol_lse[fin]).all(), \
        np.nanmax(np.abs(l - ref_lse)[fin] / tol_lse[fin])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lift", [9, 14, 17, 20, 22])
@pytest.mark.parametrize("group,n", [(1, 1), (4, 3), (7, 3), (10, 3), (13, 3)])
def test_one_element_of_q_far_above_the_others(ds, group, n, lift, dim):
    """2^lift in one dim whose key codes are 0, in every other head: the other
    dims alone make the score.

    Decode's form of q may move a score by 2^-14 (of a power of two). Prefill holds
    q times a power of two, its largest at least 2^14, in f16, exact down to 2^-14
    and with half steps of 2^-25 below: 2^-39 of the row's largest for each."""
    c = Cache([700, 90, 1100], 2, dim, seed=80 + group)
    c.codes[:, 0, :, :, 5] = 0
    c.table[0, 2] = -1
    counts, heads, scale = [n] * 3, 2 * group, 1 / math.sqrt(dim)
    q = c.q(3 * n, heads)
    q[:, ::2, 5] = 2.0 ** lift
    q[0, 0, 5] *= -1.0
    ref = _ref(c, q, counts, scale)
    k = oracle.e4m3_to_float64(c.codes[:, 0]) * c.scales[:, 0, :, None, None].astype(np.float64)
    keys = np.nanmax(np.abs(k).sum(-1))
    top = q.abs().amax(-1).double().numpy()
    for name, out, lse in _both(ds, c, q, counts, scale):
        _close(out, lse, ref, dim, 1100,
               2.0 ** -14 if name == "decode" else 2.0 ** -39 * top * keys * scale)


@pytest.mark.parametrize("dim", [64, 128])
def test_such_a_row_changes_no_other(ds, dim):
    """Neither its neighbours' bits, nor its own where it stands alone."""
    c = Cache([700, 1500], 1, dim, seed=84)
    c.codes[:, 0, :, :, 5] = 0
    q = c.q(10, 7).to(DEV).view(2, 5, 7, dim)
    codes, scales, table, lens = c.device()
    want = ds.kv8_decode(q, codes, scales, table, lens, 0.1)
    far = q.clone()
    far[0, 3, 2, 5] = far[1, 0, 6, 5] = 2.0 ** 21
    got = ds.kv8_decode(far, codes, scales, table, lens, 0.1)
    torch.cuda.synchronize()
    same = torch.ones(2, 5, 7, dtype=torch.bool, device=DEV)
    same[0, 3, 2] = same[1, 0, 6] = False
    assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1][same], want[1][same])
    for r, j in ((0, 3), (1, 0)):
        one = ds.kv8_decode(far[r:r + 1, j:j + 1].contiguous(), codes, scales,
                            table[r:r + 1].contiguous(), lens[r:r + 1] - 4 + j, 0.1)
        assert torch.equal(one[0][0, 0], got[0][r, j]) and torch.equal(one[1][0, 0], got[1][r, j])


def _low_pages(c, low):
    """The pages that `low` lists, of every request, get one key: -448 in dim 0
    at a scale of 2^8, 0 elsewhere."""
    for r in range(len(c.lens)):
        for b in low:
            if b < c.table.shape[1] and c.table[r, b] >= 0:
                c.codes[c.table[r, b], 0] = 0
                c.codes[c.table[r, b], 0, :, :, 0] = 0xFE
                c.scales[c.table[r, b], 0] = 2.0 ** 8


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length,low", [
    (400, [0, 1]), (400, [0]), (400, [1]), (400, [0, 1, 2, 3, 4]), (400, [2, 3]), (150, [0, 1]),
    (2500, range(16)), (2500, range(16, 32)), (2500, range(39)), (2500, [0, 1, 16, 17, 32, 33]),
    (2500, range(20)),
])
def test_scores_far_below_add_nothing(ds, length, low, dim):
    """Pages whose scores are below -2^25, before, between and behind ordinary
    ones: weights of 0 beside them, as if the pages were not there. A row that
    sees no other score is NaN."""
    low = list(low)
    c = Cache([length, 77], 1, dim, seed=90)
    counts, heads = [60] * 2, 3
    c.lens[1] = 67                                    # (of the two pages it has)
    _low_pages(c, low)
    q = torch.as_tensor(c.rng.uniform(0.5, 2.0, (120, heads, dim)).astype(np.float32))
    q *= torch.as_tensor(c.rng.choice([-1.0, 1.0], (120, heads, dim)).astype(np.float32))
    q[..., 0] = 2.0 ** 12                             # (q in two pieces is exact: 2^-1 is left of it)
    q = q.to(torch.bfloat16)
    # Ordinary pages hold 0 in dim 0.
    for p in range(c.pages):
        if not (c.codes[p, 0, :, :, 0] == 0xFE).all():
            c.codes[p, 0, :, :, 0] = 0
    scale = 0.125
    assert 448 * 2.0 ** 8 * 2.0 ** 12 * scale > 2.0 ** 25
    rows = oracle.kv8_visible(c.lens, counts, c.table.shape[1])
    there = c.table.copy()
    there[:, [b for b in low if b < there.shape[1]]] = -1
    ref = oracle.kv8_attention(bits(q), rows, c.codes, c.scales, there, scale)
    only_low = np.array([v > 0 and all(b in low for b in range(-(-v // 64))) for _, v in rows])
    assert np.array_equal(only_low, np.isneginf(ref[1]).all(1))
    for _, out, lse in _both(ds, c, q, counts, scale):
        o, l = out.cpu(), lse.cpu()
        assert torch.isnan(o[only_low]).all() and torch.isnan(l[only_low]).all()
        _close(o[~only_low], l[~only_low], tuple(x[~only_low] for x in ref[:4]) + (False,), dim,
               length)


@pytest.mark.parametrize("dim", [64, 128])
def test_low_scores_in_chunks_and_cut_runs(ds, dim):
    """Items of very different lengths whose first 17 pages are low, so that
    rows are handed over before they have a reference: the bits are those of
    calls of one request each."""
    lens, counts = [3000, 40, 2900, 1129, 1500], [700, 40, 1, 129, 300]
    c = Cache(lens, 3, dim, seed=91)
    c.codes[:, 0, :, :, 0] = 0
    _low_pages(c, range(17))
    q = c.q(sum(counts), 12)
    q[..., 0] = 2.0 ** 12
    q = q.to(DEV)
    codes, scales, table, lens_d = c.device()
    starts = np.concatenate([[0], np.cumsum(counts)])
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = ds.kv8_prefill(q, torch.as_tensor(starts, **i32), codes, scales, table, lens_d, 0.125)
    torch.cuda.synchronize()
    seen = torch.zeros(len(q), dtype=torch.bool, device=DEV)
    for r, n in enumerate(counts):
        lo, hi = int(starts[r]), int(starts[r + 1])
        seen[lo:hi] = torch.arange(lens[r] - n + 1, lens[r] + 1, device=DEV) > 17 * 64
        o, l = ds.kv8_prefill(q[lo:hi], torch.tensor([0, n], **i32), codes, scales,
                              table[r:r + 1].contiguous(), lens_d[r:r + 1].contiguous(), 0.125)
        assert torch.equal(o.nan_to_num(7.0), out[lo:hi].nan_to_num(7.0))
        assert torch.equal(l.nan_to_num(7.0), lse[lo:hi].nan_to_num(7.0))
    assert torch.isfinite(lse[seen]).all() and torch.isfinite(out[seen].float()).all()
    assert torch.isnan(lse[~seen]).all() and torch.isnan(out[~seen].float()).all()


@pytest.mark.slow
def test_decode_of_more_than_2_31_tiles(ds):
    """2^28 positions (one page, 2^22 times) and 1024 heads: 2^31 tiles of 128
    positions. Every page adds the same, so the outputs are those of one page and
    lse is ln 2^22 above its.

    65536 spans are joined one after the other in fp32: their sum, and the
    outputs', are off by 2^16 2^-24 of it each; a span's own 4096 positions and
    its weights (11 bits) add less than 2^-10, bf16 2^-8."""
    hk, dim, blocks = 1024, 64, 1 << 22
    c = Cache([64], hk, dim, seed=92, extra_pages=0, extra_width=0)
    q = c.q(1, hk)
    ref_out, ref_lse, weight, reach, _ = _ref(c, q, [1], 0.125)
    codes, scales, _, _ = c.device()
    i32 = dict(dtype=torch.int32, device=DEV)
    table, lens = torch.zeros((1, blocks), **i32), torch.tensor([64 * blocks], **i32)
    out = torch.full((1, 1, hk, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((1, 1, hk), 7.0, device=DEV)
    need = ds.kv8_decode_workspace_size(1, 1, hk, hk, dim, blocks)
    free, _ = torch.cuda.mem_get_info()
    if need + (1 << 30) > free:
        pytest.skip(f"needs {need >> 30} GiB of workspace")
    ds.kv8_decode(q.to(DEV)[None], codes, scales, table, lens, 0.125, out=out, lse=lse)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    o, l = out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
    assert (np.abs(o - ref_out) <= 2.0 ** -8 * np.abs(ref_out) +
            (2 * 2.0 ** -8 + 2.0 ** -10) * 1.01 * weight).all()
    want = ref_lse + math.log(blocks)
    assert (np.abs(l - want) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -20 * np.abs(want)).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [32768, 32769, 45000, 65537, 131072, 131073, 140000])
def test_decode_of_long_contexts(ds, length, dim):
    """Spans of 1024, 2048 and 4096 positions (32 and 64 pages, a lane looks up
    two of the latter), up to 32 and more of them; a page of the last span is
    outside the pool."""
    c = Cache([length, 300], 1, dim, seed=100, extra_width=0)
    c.table[0, -(-length // 64) - 2] = -1
    counts, heads, scale = [2, 2], 3, 1 / math.sqrt(dim)
    q = c.q(4, heads)
    codes, scales, table, lens = c.device()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = ds.kv8_decode(q.to(DEV).view(2, 2, heads, dim), codes, scales, table, lens, scale,
                             err_flag=err)
    _close(out.flatten(0, 1), lse.flatten(0, 1), _ref(c, q, counts, scale), dim, length)
    assert int(err) == ds.DEVERR_PAGE


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("exponent", [-12, -9, -7, -5])
def test_append_to_scales_that_are_no_powers_of_two(ds, exponent, few, dim):
    """Partly filled pages whose scale is 1.2345 2^exponent: kept where it covers
    the new tokens, grown (to a power of two) where it does not; a few tokens a
    request (a warp each) or many (a CTA a page)."""
    counts = [1, 5, 0, 12, 3] if few else [40, 100, 0, 64, 130]
    lens = [n + had for n, had in zip(counts, [7, 60, 30, 64 + 33, 1])]
    c = Cache([max(x, 0) for x in lens], 3, dim, seed=110 + exponent)
    c.scales[...] = np.float32(1.2345) * 2.0 ** exponent
    before = [x - n for x, n in zip(lens, counts)]
    for r, x in enumerate(before):
        for b in range(c.table.shape[1]):
            if c.table[r, b] >= 0 and 64 * b + 64 > x:
                at = c.codes[c.table[r, b], :, :, max(0, x - 64 * b):]
                at[...] = c.rng.integers(0, 256, at.shape)
    x = torch.as_tensor(c.rng.standard_normal((sum(counts), 2, 3, dim)).astype(np.float32))
    x = (x * torch.exp2(torch.as_tensor(c.rng.integers(-3, 4, (sum(counts), 2, 3, 1))).float())) \
        .to(torch.bfloat16)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    want = oracle.kv8_append(bits(x[:, 0]), bits(x[:, 1]), starts, lens, c.table, c.codes, c.scales)
    codes, scales, table, lens_d = c.device()
    kv = x.to(DEV)
    ds.kv8_append(kv[:, 0], kv[:, 1], torch.as_tensor(starts).to(DEV), table, lens_d, codes, scales)
    torch.cuda.synchronize()
    assert np.array_equal(scales.cpu().numpy(), want[1])
    got, ref = (oracle.e4m3_to_float64(a) for a in (codes.cpu().numpy(), want[0]))
    assert np.array_equal(got, ref, equal_nan=True)
    # (Both kinds are there, in one of the exponents at least.)
    firsts = [c.table[r, x // 64] for r, x in enumerate(before) if counts[r] and x % 64]
    grown = want[1][firsts] != c.scales[firsts]
    assert exponent > -12 or grown.all()
    assert exponent < -5 or not grown.all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("mid,top", [(11, 26), (11, 24), (9, 22), (8, 26), (11, 28), (0, 14)])
def test_a_reference_that_moves_far_keeps_the_weights_beside_it(ds, mid, top, first, dim):
    """One page of a tile 2^mid above the tile before, and one position of the
    other page 2^top above it, whose value is 0: the output is the page's, whose
    weights are 2^(mid - top) of the largest."""
    c = Cache([400], 1, dim, seed=120)
    c.scales[:] = 1.0
    for p in c.table[0][c.table[0] >= 0]:
        c.codes[p] = 0
    code = {0: 0, 8: 0x50, 9: 0x51, 11: 0x53, 14: 0x56, 22: 0x5B, 24: 0x5C, 26: 0x5D, 28: 0x5E}
    assert all(oracle.e4m3_to_float64(np.uint8(v)) == k for k, v in code.items())
    a, b = c.table[0, 2 + first], c.table[0, 3 - first]      # pages of the second tile
    c.codes[a, 0, 0, :, 0], c.codes[a, 1] = code[mid], 0x38
    c.codes[b, 0, 0, 17, 0] = code[top]
    q = torch.zeros((3, 2, dim), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    ref = _ref(c, q, [3], math.log(2))
    assert (ref[0] > 2.0 ** (mid - top)).all()
    for _, out, lse in _both(ds, c, q, [3], math.log(2)):
        _close(out, lse, ref, dim, 400)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests,kv_heads", [(24, 8), (64, 4), (200, 1), (1000, 2)])
@pytest.mark.parametrize("length,n", [(300, 1), (700, 3), (2000, 40), (129, 129)])
def test_prefill_of_one_request_among_many_without_tokens(ds, length, n, requests, kv_heads, dim):
    """A padded batch in which one request brings tokens, fewer tiles than there
    are CTAs: its bits are those of a call of its own."""
    c = Cache([length], kv_heads, dim, seed=140)
    codes, scales, one, _ = c.device()
    i32 = dict(dtype=torch.int32, device=DEV)
    q = c.q(n, 3 * kv_heads).to(DEV)
    alone = ds.kv8_prefill(q, torch.tensor([0, n], **i32), codes, scales, one,
                           torch.tensor([length], **i32), 0.1)
    err = torch.zeros(1, **i32)
    for at in (0, requests // 3, requests - 1):
        table = torch.full((requests, one.shape[1]), -1, **i32)
        table[at] = one[0]
        lens = torch.zeros(requests, **i32)
        lens[at] = length
        starts = torch.where(torch.arange(requests + 1, device=DEV) > at, n, 0).int()
        got = ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1, err_flag=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])


@pytest.mark.parametrize("dim", [64, 128])
def test_a_million_requests_most_without_tokens(ds, dim):
    """2^20 requests (the most there may be), few of them with positions and
    tokens: the same outputs as alone, in time that the empty ones do not fill."""
    n, hk = 1 << 20, 2
    c = Cache([300], hk, dim, seed=130)
    codes, scales, one, _ = c.device()
    i32 = dict(dtype=torch.int32, device=DEV)
    table = one.expand(n, -1).contiguous()
    err = torch.zeros(1, **i32)
    q = c.q(1, 6).to(DEV)
    want = ds.kv8_decode(q[None], codes, scales, one, torch.tensor([300], **i32), 0.1)
    alone = ds.kv8_prefill(q, torch.tensor([0, 1], **i32), codes, scales, one,
                           torch.tensor([300], **i32), 0.1)
    for where in ([0, n - 1], [n - 1], [0], [5, 77777, 77778, n // 2, n - 9]):
        full = torch.zeros(n, dtype=torch.bool, device=DEV)
        full[where] = True
        starts = torch.cat([torch.zeros(1, **i32), torch.cumsum(full, 0).int()])
        lens = torch.where(full, 300, 0).int()
        out, lse = ds.kv8_prefill(q.expand(len(where), -1, -1).contiguous(), starts, codes, scales,
                                  table, lens, 0.1, err_flag=err)
        assert (out == alone[0]).all() and (lse == alone[1]).all() and int(err) == 0
        out, lse = ds.kv8_decode(q.expand(n, -1, -1)[:, None].contiguous(), codes, scales, table,
                                 lens, 0.1, err_flag=err)
        assert (out[full] == want[0][0]).all() and (lse[full] == want[1][0]).all()
        assert (out[~full] == 0).all() and torch.isneginf(lse[~full]).all() and int(err) == 0
        del out, lse


def test_a_captured_serving_step(ds):
    """extend, append, decode and prefill of a step in one graph, replayed with
    new tokens: the states and outputs of the same steps run one by one."""
    hk, d, heads, rows, pages = 2, 128, 8, 5, 40
    i32 = dict(dtype=torch.int32, device=DEV)
    counts = torch.tensor([5, 0, 1, 17, 40], **i32)
    starts = torch.cat([torch.zeros(1, **i32), torch.cumsum(counts, 0).int()])
    which, t = torch.arange(rows, **i32), int(counts.sum())
    x = torch.empty((t, 2, hk, d), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((t, heads, d), dtype=torch.bfloat16, device=DEV)

    def state():
        return (torch.zeros(pages, **i32), torch.full((rows, 6), -1, **i32), torch.zeros(rows, **i32),
                torch.full((pages, 2, hk, 64, d), 0x7F, dtype=torch.uint8, device=DEV),
                torch.full((pages, 2, hk), float("nan"), device=DEV), torch.zeros(1, **i32))

    def step(refs, table, lens, codes, scales, err):
        ds.pages_extend(refs, table, lens, which, lens + counts, err_flag=err)
        ds.kv8_append(x[:, 0], x[:, 1], starts, table, lens, codes, scales, err_flag=err)
        out = ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.09, err_flag=err)
        return out + ds.kv8_decode(q[:rows, None], codes, scales, table, lens, 0.09, err_flag=err)

    fill = lambda k: [y.normal_(generator=torch.Generator(device=DEV).manual_seed(k))  # noqa: E731
                      for y in (x, q)]
    eager, kept = state(), state()
    fill(0)
    step(*state())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*kept)
    for k in range(7):
        fill(k)
        want = step(*eager)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for a, b in zip(kept[:3] + kept[5:], eager[:3] + eager[5:]):
            assert torch.equal(a, b)
        assert torch.equal(kept[3], eager[3]) and torch.equal(kept[4].nan_to_num(9),
                                                              eager[4].nan_to_num(9))
    assert int(kept[5]) == 0 and kept[2].tolist() == [35, 0, 7, 119, 280]

"""GPU tests of the block-scaled 8-bit cache: append (byte for byte) and the
decode and prefill attention against the float64 oracle.

Attention bounds come from oracle.kv8_bounds: fp32 scores and sums, softmax
weights rounded to 8 significant bits, the output rounded to bf16. Unused
slots hold NaN codes and unused pages NaN scales, so that anything read from
them shows.
"""

import math
import threading

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


# ----------------------------------------------------------------- append
def _values(codes):
    v = oracle.e4m3_to_float64(codes)
    return np.where(np.isnan(v), 1e9, v)


def _append_case(ds, lens, counts, kv_heads, dim, seed, mag=None, stride_pad=0, bad=()):
    """Earlier positions are in the cache; the last counts[r] are appended."""
    before = [x - n for x, n in zip(lens, counts)]
    c = Cache([max(x, 0) for x in lens], kv_heads, dim, seed)
    rng = c.rng
    for r, x in enumerate(before):   # what lies behind the earlier positions is garbage
        for b in range(c.table.shape[1]):
            p = c.table[r, b]
            if p >= 0 and 64 * b + 64 > x:
                lo = max(0, x - 64 * b)
                c.codes[p, :, :, lo:] = rng.integers(0, 256, c.codes[p, :, :, lo:].shape)
                if lo == 0:
                    c.scales[p] = np.nan
    for r, b, p in bad:
        c.table[r, b] = p
    t = sum(counts)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = rng.standard_normal((t, 2, kv_heads, dim)).astype(np.float32)
    x *= np.exp(rng.standard_normal((t, 2, kv_heads, 1)) * 2) if mag is None else mag
    x = torch.as_tensor(x).to(torch.bfloat16)
    buf = torch.zeros((t, 2 * kv_heads * dim + stride_pad), dtype=torch.bfloat16, device=DEV)
    buf[:, :2 * kv_heads * dim] = x.view(t, -1).to(DEV)
    kv = buf[:, :2 * kv_heads * dim].unflatten(1, (2, kv_heads, dim))
    codes, scales, table, _ = c.device()
    want = oracle.kv8_append(bits(x[:, 0]), bits(x[:, 1]), starts, lens, c.table, c.codes,
                             c.scales)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ds.kv8_append(kv[:, 0], kv[:, 1], torch.as_tensor(starts).to(DEV), table,
                  torch.as_tensor(lens, dtype=torch.int32).to(DEV), codes, scales, err_flag=err)
    torch.cuda.synchronize()
    assert np.array_equal(_values(codes.cpu().numpy()), _values(want[0]))
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    assert int(err) == (ds.DEVERR_LEN if want[2] else 0) | (ds.DEVERR_PAGE if want[3] else 0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,counts", [
    ([1], [1]),
    ([64, 65, 63], [64, 1, 2]),
    ([700, 5, 0, 130, 64], [699, 5, 0, 3, 0]),
    ([300, 257, 129, 1, 66, 500], [5, 5, 5, 1, 5, 5]),
])
def test_append_bytes(ds, lens, counts, dim):
    _append_case(ds, lens, counts, 3, dim, seed=len(lens) + dim)


def test_append_strided_and_many_heads(ds):
    _append_case(ds, [200, 90], [33, 90], 8, 64, seed=5, stride_pad=24)


@pytest.mark.parametrize("mag", [0.0, 1e-30, 2.0 ** -70, 1e35, 448.0])
def test_append_magnitudes(ds, mag):
    """All zeros (smallest scale), scales at their limits, and values whose
    growth pushes earlier codes below the normal range."""
    _append_case(ds, [100, 70], [40, 70], 2, 128, seed=6, mag=mag)


def test_append_specials(ds):
    """Infinities saturate (at the largest scale), NaN keeps to itself."""
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16)
    k[1, 0, 5] = float("nan")
    v = k.clone()
    v[2, 0, 7] = -float("inf")
    codes = torch.zeros((1, 2, 1, 64, 64), dtype=torch.uint8, device=DEV)
    scales = torch.ones((1, 2, 1), device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    ds.kv8_append(k.to(DEV), v.to(DEV), torch.tensor([0, 3], **i32), torch.zeros((1, 1), **i32),
                  torch.tensor([3], **i32), codes, scales)
    val = oracle.e4m3_to_float64(codes.cpu().numpy())[0] * scales.cpu().numpy()[0][..., None, None]
    assert np.isnan(val[0, 0, 1, 5]) and np.isnan(val[0, 0]).sum() == 1
    assert (val[0, 0, 0] == 1).all() and scales[0, 0, 0].item() == 2.0 ** -8
    assert scales[0, 1, 0].item() == 2.0 ** 120 and val[1, 0, 2, 7] == -448 * 2.0 ** 120


def test_append_flags_and_leaves(ds):
    """A request shorter than its tokens, pages outside the pool or the table."""
    _append_case(ds, [3, 70, 128], [5, 70, 10], 2, 64, seed=8, bad=[(1, 0, 10 ** 6), (2, 1, -1)])


def test_append_ignores_rows_behind_the_last_request(ds):
    i32 = dict(dtype=torch.int32, device=DEV)
    k = torch.randn((9, 2, 64), device=DEV).to(torch.bfloat16)
    codes = torch.full((4, 2, 2, 64, 64), 0x11, dtype=torch.uint8, device=DEV)
    scales = torch.full((4, 2, 2), 7.0, device=DEV)
    ds.kv8_append(k, k, torch.tensor([2, 2, 6], **i32), torch.tensor([[0], [3]], **i32),
                  torch.tensor([0, 4], **i32), codes, scales)
    torch.cuda.synchronize()
    assert (codes[:3] == 0x11).all() and (scales[:3] == 7).all()
    assert (codes[3, :, :, 4:] == 0x11).all() and (scales[3] != 7).all()


def test_append_round_by_round_then_decode(ds):
    """A request written in rounds of 1 to 40 tokens, read back by decode."""
    rng = np.random.default_rng(9)
    torch.manual_seed(9)
    hk, d, total = 2, 128, 200
    i32 = dict(dtype=torch.int32, device=DEV)
    codes = torch.full((6, 2, hk, 64, d), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((6, 2, hk), float("nan"), device=DEV)
    table = torch.tensor([[4, 1, 0, 5]], **i32)
    x = torch.randn((total, 2, hk, d), device=DEV).to(torch.bfloat16)
    done = 0
    while done < total:
        n = min(int(rng.integers(1, 41)), total - done)
        y = x[done:done + n]
        done += n
        ds.kv8_append(y[:, 0], y[:, 1], torch.tensor([0, n], **i32), table,
                      torch.tensor([done], **i32), codes, scales)
    q = torch.randn((1, 2, 8, d), device=DEV).to(torch.bfloat16)
    out, lse = ds.kv8_decode(q, codes, scales, table, torch.tensor([total], **i32), 0.09)
    rows = oracle.kv8_visible([total], [2], 4)
    ref = oracle.kv8_attention(bits(q[0]), rows, codes.cpu().numpy(), scales.cpu().numpy(),
                               table.cpu().numpy(), 0.09)
    _close(out[0], lse[0], ref, d, total)
    val = oracle.e4m3_to_float64(codes.cpu().numpy()) * scales.cpu().numpy()[..., None, None]
    got = val[[4, 1, 0, 5]].transpose(0, 3, 1, 2, 4).reshape(256, 2, hk, d)[:total]
    # A code in the normal range is off by 2^-4 of the value, once: dividing it
    # by a power of two is exact while it stays there. A subnormal code at scale
    # s is off by half a step, 2^-10 s, and by that of each smaller scale the
    # page had before: less than 2^-10 s (1 + 1/2 + 1/4 + ...) = 2^-9 s.
    step = np.repeat(scales.cpu().numpy()[[4, 1, 0, 5]], 64, 0)[:total, :, :, None]
    exact = x.double().cpu().numpy()
    assert (np.abs(got - exact) <= 2.0 ** -4 * np.abs(exact) + 2.0 ** -9 * step).all()


# -------------------------------------------------------------- attention
def _close(out, lse, ref, dim, length):
    ref_out, ref_lse, weight, reach, _ = ref
    tol, tol_lse = oracle.kv8_bounds(ref_out, ref_lse, weight, reach, dim, length)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = ~(np.abs(o - ref_out) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs off, worst "
                           f"{np.nanmax(np.abs(o - ref_out) / tol)} of the bound, first at "
                           f"{tuple(np.argwhere(bad)[0])}, {np.isnan(o).sum()} NaN")
    fin = np.isfinite(ref_lse)
    assert np.array_equal(np.isneginf(l), ~fin)
    assert (np.abs(l[fin] - ref_lse[fin]) <= tol_lse[fin]).all(), \
        np.max(np.abs(l[fin] - ref_lse[fin]) / tol_lse[fin])


def _decode(ds, c, next_n, heads, scale=None, gain=2.5, q=None, **kw):
    scale = 1 / math.sqrt(c.dim) if scale is None else scale
    q = c.q(len(c.lens) * next_n, heads, gain) if q is None else q
    codes, scales, table, lens = c.device()
    out, lse = ds.kv8_decode(q.to(DEV).view(len(c.lens), next_n, heads, c.dim), codes, scales,
                             table, lens, scale, **kw)
    rows = oracle.kv8_visible(c.lens, [next_n] * len(c.lens), c.table.shape[1])
    ref = oracle.kv8_attention(bits(q), rows, c.codes, c.scales, c.table, scale)
    torch.cuda.synchronize()
    _close(out.flatten(0, 1), lse.flatten(0, 1), ref, c.dim, max(c.lens + [1]))
    return out, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 8), (3, 7), (1, 16), (4, 3)])
def test_decode_heads(ds, dim, kv_heads, group):
    c = Cache([1, 63, 64, 65, 200, 0, 129], kv_heads, dim, seed=group)
    _decode(ds, c, 1, kv_heads * group)


@pytest.mark.parametrize("next_n,group", [(2, 1), (5, 8), (7, 3), (4, 16), (11, 12), (64, 2)])
def test_decode_several_tokens(ds, next_n, group):
    """Tokens before the context's start see nothing; causal within the step."""
    c = Cache([next_n, 3, 0, 200, 64, 129, -5], 2, 128, seed=next_n)
    _decode(ds, c, next_n, 2 * group)


@pytest.mark.parametrize("length", [127, 128, 511, 512, 513, 1023, 1025, 3000])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_lengths(ds, length, dim):
    _decode(ds, Cache([length, 17], 2, dim, seed=length), 1, 8)
    _decode(ds, Cache([length, 17], 1, dim, seed=length + 1), 5, 4)


def test_decode_uniform_and_peaked(ds):
    c = Cache([2500], 2, 128, seed=1)
    _decode(ds, c, 1, 4, gain=0.0)
    _decode(ds, c, 1, 4, gain=40.0)
    _decode(ds, c, 1, 4, scale=-0.05)


@pytest.mark.parametrize("nats", [4.0, 8.0, 12.0])
@pytest.mark.parametrize("where", [0, 1999])
def test_decode_one_position_far_above_a_long_tail(ds, nats, where):
    """An attention sink: one key stands `nats` above 2000 equal ones, whose
    small weights together still count. The tail is one value, so that errors
    of its weights do not average out."""
    c = Cache([2000], 1, 64, seed=2)
    one = 0x38                                       # code of 1.0
    for p in c.table[0][c.table[0] >= 0]:
        c.codes[p, 0], c.codes[p, 1] = 0, one
    c.scales[:] = 1.0
    p = c.table[0, where // 64]
    c.codes[p, 0, 0, where % 64, 0] = one
    c.codes[p, 1, 0, where % 64] = one | 0x80        # value -1
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([1.0, 0.5, 0.25, 2.0]) * nats
    _decode(ds, c, 1, 4, scale=1.0, q=q)


def test_decode_scales_of_any_size(ds):
    """Pages whose scales are hundreds of powers of two apart, all-zero pages
    at the smallest scale, scales that are no power of two."""
    c = Cache([700, 300], 2, 64, seed=3)
    used = ~np.isnan(c.scales[:, 1])
    c.scales[:, 1] = np.where(used, 2.0 ** c.rng.integers(-60, 30, c.scales[:, 1].shape), np.nan)
    c.scales[:, 0] *= 1.2345
    p = c.table[0, 3]
    c.codes[p] = 0
    c.scales[p] = 2.0 ** -60
    c.codes[c.table[1, :4]] &= 0x80
    c.scales[c.table[1, :4]] = 2.0 ** -60
    c.codes[c.table[1, 4], :, :, :44] = 0x01
    _decode(ds, c, 1, 8)


def test_decode_bad_pages_are_left_out_and_flagged(ds):
    c = Cache([300, 100, 64], 2, 128, seed=4)
    c.table[0, 1], c.table[1, 1], c.table[2, 0] = -1, c.pages, 2 ** 30
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _decode(ds, c, 2, 8, err_flag=err)
    assert int(err) == ds.DEVERR_PAGE


def test_decode_lengths_beyond_the_table_are_clamped(ds):
    c = Cache([128], 1, 64, seed=5, extra_width=0)
    c.lens = [1000]
    _decode(ds, c, 3, 4)


def test_decode_strided_queries_and_given_outputs(ds):
    c = Cache([200, 70], 2, 64, seed=6)
    buf = torch.randn((2, 3, 12 * 64), device=DEV).to(torch.bfloat16)
    q = buf[:, :, 64:64 + 8 * 64].unflatten(2, (8, 64))
    codes, scales, table, lens = c.device()
    want = ds.kv8_decode(q.contiguous(), codes, scales, table, lens, 0.1)
    out = torch.full((2, 3, 8, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, 3, 8), 9.0, device=DEV)
    ws = torch.full((ds.kv8_decode_workspace_size(2, 3, 8, 2, 64, table.shape[1]),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    got = ds.kv8_decode(q, codes, scales, table, lens, 0.1, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_decode_nonfinite_query_stays_in_its_head(ds):
    c = Cache([100], 1, 64, seed=7)
    q = c.q(1, 4)
    q[0, 2, 3] = float("inf")
    codes, scales, table, lens = c.device()
    out, lse = ds.kv8_decode(q.to(DEV)[None], codes, scales, table, lens, 0.1)
    assert torch.isnan(out[0, 0, 2]).all() and torch.isfinite(out[0, 0, [0, 1, 3]].float()).all()


def test_decode_rows_do_not_depend_on_the_batch(ds):
    c = Cache([1500, 77, 640, 0, 2049], 2, 128, seed=8)
    q = c.q(5 * 2, 16).to(DEV).view(5, 2, 16, 128)
    codes, scales, table, lens = c.device()
    out, lse = ds.kv8_decode(q, codes, scales, table, lens, 0.09)
    for r in range(5):
        o, l = ds.kv8_decode(q[r:r + 1].clone(), codes, scales, table[r:r + 1].contiguous(),
                             lens[r:r + 1].contiguous(), 0.09)
        assert torch.equal(o[0], out[r]) and torch.equal(l[0], lse[r])


def test_decode_captured_and_on_another_stream(ds):
    c = Cache([900, 130], 2, 128, seed=9)
    q = c.q(2, 8).to(DEV).view(2, 1, 8, 128)
    codes, scales, table, lens = c.device()
    want = ds.kv8_decode(q, codes, scales, table, lens, 0.09)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(ds.kv8_decode_workspace_size(2, 1, 8, 2, 128, table.shape[1]),
                     dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.kv8_decode(q, codes, scales, table, lens, 0.09, out=out, lse=lse, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    lens.copy_(torch.tensor([333, 64], dtype=torch.int32))      # the graph reads the new lengths
    g.replay()
    again = ds.kv8_decode(q, codes, scales, table, lens, 0.09)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = ds.kv8_decode(q, codes, scales, table, lens, 0.09, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(side[0], again[0])


def test_empty_calls(ds):
    c = Cache([10], 1, 64, seed=10)
    codes, scales, table, lens = c.device()
    i32 = dict(dtype=torch.int32, device=DEV)
    none = torch.empty((0, table.shape[1]), **i32)
    q = torch.empty((0, 2, 4, 64), dtype=torch.bfloat16, device=DEV)
    assert ds.kv8_decode(q, codes, scales, none, lens[:0], 0.1)[0].shape == (0, 2, 4, 64)
    assert ds.kv8_prefill(q[:, 0], torch.zeros(2, **i32), codes, scales, table, lens,
                          0.1)[0].shape == (0, 4, 64)
    ds.kv8_append(q[:, 0, :1], q[:, 0, :1], torch.zeros(2, **i32), table, lens, codes, scales)
    torch.cuda.synchronize()


def _prefill(ds, c, counts, heads, scale=None, gain=2.5, **kw):
    scale = 1 / math.sqrt(c.dim) if scale is None else scale
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = c.q(int(starts[-1]), heads, gain)
    codes, scales, table, lens = c.device()
    out, lse = ds.kv8_prefill(q.to(DEV), torch.as_tensor(starts).to(DEV), codes, scales, table,
                              lens, scale, **kw)
    rows = oracle.kv8_visible(c.lens, counts, c.table.shape[1])
    ref = oracle.kv8_attention(bits(q), rows, c.codes, c.scales, c.table, scale)
    torch.cuda.synchronize()
    _close(out, lse, ref, c.dim, max(c.lens + [1]))
    return out, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 8), (1, 7), (2, 5)])
def test_prefill_heads(ds, dim, kv_heads, group):
    c = Cache([70, 200, 1], kv_heads, dim, seed=20 + group)
    _prefill(ds, c, [70, 33, 1], kv_heads * group)


@pytest.mark.parametrize("lens,counts", [
    ([1], [1]), ([128], [128]), ([129, 127], [129, 127]), ([600, 40], [65, 0]),
    ([0, 5, 300, 64], [0, 5, 257, 64]), ([3, 1000], [5, 300]), ([0], [4]),
])
def test_prefill_lengths(ds, lens, counts):
    """Prompts, chunks of prompts, requests without tokens, and (3 of 5) tokens
    that see nothing."""
    _prefill(ds, Cache(lens, 2, 128, seed=30 + len(lens)), counts, 4)


def test_prefill_uniform_and_peaked(ds):
    c = Cache([500], 1, 64, seed=40)
    _prefill(ds, c, [200], 2, gain=0.0)
    _prefill(ds, c, [200], 2, gain=40.0)


def test_prefill_scales_of_any_size(ds):
    c = Cache([400], 2, 64, seed=41)
    used = ~np.isnan(c.scales[:, 1])
    c.scales[:, 1] = np.where(used, 2.0 ** c.rng.integers(-60, 30, c.scales[:, 1].shape), np.nan)
    c.codes[c.table[0, 2]] = 0
    c.scales[c.table[0, 2]] = 2.0 ** -60
    _prefill(ds, c, [300], 4)


def test_prefill_bad_pages_are_left_out_and_flagged(ds):
    c = Cache([300, 100], 2, 128, seed=42)
    c.table[0, 1], c.table[1, 1] = -7, c.pages
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _prefill(ds, c, [300, 64], 8, err_flag=err)
    assert int(err) == ds.DEVERR_PAGE


def test_prefill_leaves_rows_of_no_request(ds):
    c = Cache([40, 30], 1, 64, seed=43)
    q = c.q(100, 4).to(DEV)
    codes, scales, table, lens = c.device()
    starts = torch.tensor([3, 43, 73], dtype=torch.int32, device=DEV)
    out = torch.full((100, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((100, 4), 5.0, device=DEV)
    ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1, out=out, lse=lse)
    want = ds.kv8_prefill(q[3:73].contiguous(), starts - 3, codes, scales, table, lens, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(out[3:73], want[0]) and torch.equal(lse[3:73], want[1])
    for t in (out, lse):
        assert (t[:3] == 5).all() and (t[73:] == 5).all()


def test_prefill_tokens_do_not_depend_on_the_batch_or_the_chunking(ds):
    c = Cache([700, 200], 2, 128, seed=44)
    q = c.q(900, 8).to(DEV)
    codes, scales, table, lens = c.device()
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = ds.kv8_prefill(q, torch.tensor([0, 700, 900], **i32), codes, scales, table, lens,
                              0.09)
    for lo, hi in ((0, 300), (300, 301), (301, 700)):
        o, l = ds.kv8_prefill(q[lo:hi], torch.tensor([0, hi - lo], **i32), codes, scales,
                              table[:1].contiguous(), torch.tensor([hi], **i32), 0.09)
        assert torch.equal(o, out[lo:hi]) and torch.equal(l, lse[lo:hi])


def test_prefill_captured(ds):
    c = Cache([300, 90], 2, 64, seed=45)
    q = c.q(150, 4).to(DEV)
    codes, scales, table, lens = c.device()
    starts = torch.tensor([0, 100, 150], dtype=torch.int32, device=DEV)
    want = ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    need = ds.kv8_prefill_workspace_size(150, 2, 4, 2, 64)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1, out=out, lse=lse, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_prefill_strided_queries(ds):
    c = Cache([100], 2, 64, seed=46)
    buf = torch.randn((100, 20 * 64), device=DEV).to(torch.bfloat16)
    q = buf[:, 128:128 + 6 * 64].unflatten(1, (6, 64))
    codes, scales, table, lens = c.device()
    starts = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    a = ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1)
    b = ds.kv8_prefill(q.contiguous(), starts, codes, scales, table, lens, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_kept_workspaces_of_streams_and_graphs(ds):
    """Calls of several sizes in turn on two streams and in a captured graph,
    replayed between them: each with its own workspace."""
    cases = [Cache([900, 130], 2, 128, seed=50), Cache([2000, 700, 65, 1500], 4, 64, seed=51)]
    args, want = [], []
    for c in cases:
        q = c.q(len(c.lens), 16).to(DEV).view(len(c.lens), 1, 16, c.dim)
        args.append((q, *c.device(), 0.09))
        ws = torch.empty(ds.kv8_decode_workspace_size(len(c.lens), 1, 16, c.kv_heads, c.dim,
                                                      c.table.shape[1]),
                         dtype=torch.uint8, device=DEV)
        want.append(ds.kv8_decode(*args[-1], workspace=ws)[0].clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        inside = ds.kv8_decode(*args[1])[0]
    side = torch.cuda.Stream()
    got = []
    for _ in range(5):
        for i in (0, 1):
            got.append((i, ds.kv8_decode(*args[i])[0]))
            got.append((i, ds.kv8_decode(*args[i], stream=side)[0]))
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(inside, want[1])
    assert all(torch.equal(o, want[i]) for i, o in got)


def _poisoned(c, r, pos, side, head, dim_at):
    """The cache with a NaN code at one position, and with a 0 there."""
    p = c.table[r, pos // 64]
    out = []
    for code in (0x7F, 0x00):
        codes = c.codes.copy()
        codes[p, side, head, pos % 64, dim_at] = code
        out.append(torch.as_tensor(codes).to(DEV))
    return out


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [130, 1100])
def test_decode_nan_of_a_later_token_stays_with_those_that_see_it(ds, dim, length):
    """A NaN value at the third of five tokens: earlier tokens' bits are those
    of a cache without it, later ones are NaN in that dim alone; a NaN key
    makes later tokens' outputs NaN and leaves earlier ones."""
    c = Cache([length, 70], 2, dim, seed=60)
    q = c.q(10, 6).to(DEV).view(2, 5, 6, dim)
    _, scales, table, lens = c.device()
    for side in (1, 0):
        nan, zero = _poisoned(c, 0, length - 3, side, 1, 37)
        got = ds.kv8_decode(q, nan, scales, table, lens, 0.1)
        want = ds.kv8_decode(q, zero, scales, table, lens, 0.1)
        torch.cuda.synchronize()
        clean = torch.ones(2, 5, 6, dim, dtype=torch.bool, device=DEV)
        clean[0, 2:, 3:] = False
        if side == 1:
            clean[0, 2:, 3:] = torch.arange(dim, device=DEV) != 37
            assert torch.equal(got[1], want[1])
        assert torch.equal(got[0][clean], want[0][clean])
        assert torch.isnan(got[0][~clean]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_nan_of_a_later_token_stays_with_those_that_see_it(ds, dim):
    c = Cache([400, 90], 2, dim, seed=61)
    q = c.q(300, 6).to(DEV)
    _, scales, table, lens = c.device()
    starts = torch.tensor([0, 250, 300], dtype=torch.int32, device=DEV)
    for side in (1, 0):
        for pos in (399, 300, 151):                 # first seen by token pos - 150
            nan, zero = _poisoned(c, 0, pos, side, 1, 37)
            got = ds.kv8_prefill(q, starts, nan, scales, table, lens, 0.1)
            want = ds.kv8_prefill(q, starts, zero, scales, table, lens, 0.1)
            torch.cuda.synchronize()
            clean = torch.ones(300, 6, dim, dtype=torch.bool, device=DEV)
            clean[pos - 150:250, 3:] = False
            if side == 1:
                clean[pos - 150:250, 3:] = torch.arange(dim, device=DEV) != 37
                assert torch.equal(got[1], want[1])
            assert torch.equal(got[0][clean], want[0][clean])
            assert torch.isnan(got[0][~clean]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_runs_cut_inside_items(ds, dim):
    """Items of very different lengths, so that the CTAs' runs end inside them:
    the bits are those of calls of one request each."""
    lens = [3000, 40, 2900, 129, 1500, 2, 2222]
    counts = [700, 40, 1, 129, 300, 2, 60]
    c = Cache(lens, 3, dim, seed=62)
    q = c.q(sum(counts), 12).to(DEV)
    codes, scales, table, lens_d = c.device()
    i32 = dict(dtype=torch.int32, device=DEV)
    starts = np.concatenate([[0], np.cumsum(counts)])
    out, lse = ds.kv8_prefill(q, torch.as_tensor(starts, **i32), codes, scales, table, lens_d, 0.09)
    for r, n in enumerate(counts):
        lo, hi = int(starts[r]), int(starts[r + 1])
        o, l = ds.kv8_prefill(q[lo:hi], torch.tensor([0, n], **i32), codes, scales,
                              table[r:r + 1].contiguous(), lens_d[r:r + 1].contiguous(), 0.09)
        assert torch.equal(o, out[lo:hi]) and torch.equal(l, lse[lo:hi])
    for r in (2, 5):                                # and against the oracle
        lo, hi = int(starts[r]), int(starts[r + 1])
        rows = [(r, v) for _, v in oracle.kv8_visible([lens[r]], [counts[r]], c.table.shape[1])]
        ref = oracle.kv8_attention(bits(q[lo:hi]), rows, c.codes, c.scales, c.table, 0.09)
        _close(out[lo:hi], lse[lo:hi], ref, dim, lens[r])


def test_prefill_growing_scores_move_the_reference(ds):
    """Keys that grow along the context: the running reference has to move
    again and again, in either half of a tile."""
    c = Cache([900], 1, 64, seed=63, spread=1)
    for b in range(15):
        c.scales[c.table[0, b], 0] = 2.0 ** (b - 9)
    _prefill(ds, c, [400], 4)
    _decode(ds, c, 3, 4)


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_nan_query_leaves_its_neighbours(ds, dim):
    """A NaN in one head of one token: that row is NaN, the others' bits stay,
    also where references move."""
    c = Cache([900], 1, dim, seed=64, spread=1)
    for b in range(15):
        c.scales[c.table[0, b], 0] = 2.0 ** (b - 9)
    q = c.q(300, 3).to(DEV)
    codes, scales, table, lens = c.device()
    starts = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    out, lse = ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1)
    bad = q.clone()
    bad[17, 1, 5] = float("nan")
    bad[200, 2, 0] = float("inf")
    got, glse = ds.kv8_prefill(bad, starts, codes, scales, table, lens, 0.1)
    torch.cuda.synchronize()
    clean = torch.ones(300, 3, dtype=torch.bool, device=DEV)
    clean[17, 1] = clean[200, 2] = False
    assert torch.equal(got[clean], out[clean]) and torch.equal(glse[clean], lse[clean])
    assert torch.isnan(got[~clean]).all() and torch.isnan(glse[~clean]).all()


def _staircase(dim, length, seed):
    """Keys whose first dim climbs through the positive codes along the context
    (the others are 0), with several positions on each."""
    c = Cache([length], 1, dim, seed=seed, spread=1)
    codes = (np.arange(length) * 126 // length + 1).astype(np.uint8)
    for i in range(length):
        c.codes[c.table[0, i // 64], 0, 0, i % 64] = 0
        c.codes[c.table[0, i // 64], 0, 0, i % 64, 0] = codes[i]
    c.scales[c.table[0, :-(-length // 64)], 0] = 1.0
    return c, oracle.e4m3_to_float64(codes)


def _both(ds, c, q, n):
    """(out, lse) of the last n tokens by decode and by prefill."""
    codes, scales, table, lens = c.device()
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o, l = ds.kv8_decode(q[None], codes, scales, table, lens, 1.0)
    yield o[0], l[0]
    yield ds.kv8_prefill(q, starts, codes, scales, table, lens, 1.0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lift", [6, 10, 13])
def test_large_scores(ds, dim, lift):
    """Scores of up to 2^21.8: equal ones share, smaller ones get nothing.

    q . k is exact here (one dim, a power of two); times log2 e and less the
    reference it is rounded twice to 2^-24 of x = |score| log2 e at most, which
    moves a weight, and the sum that divides it, by a factor of 2^(2^-23 x) each
    (equal scores of the reference's own tile and of a later one are rounded
    apart, so that it shows). Steps differ by 2^-4 of a score.
    out: that, half a step of bf16 (2^-8) and of the f16 weights (2^-11), and
    2^-16 for weights too small for 11 bits; lse: fewer than 16 roundings of
    2^-24 of it."""
    n = 60
    c, keys = _staircase(dim, 700, seed=65)
    q = torch.zeros((n, 2, dim), dtype=torch.bfloat16)
    q[:, :, 0] = 2.0 ** lift
    rows = [(0, 700 - n + 1 + j) for j in range(n)]
    out, lse, weight = oracle.kv8_attention(bits(q), rows, c.codes, c.scales, c.table, 1.0)[:3]
    x = keys.max() * 2.0 ** lift * math.log2(math.e)
    tol = 2.0 ** -8 + 2.0 ** -10 + 2 * math.expm1(math.log(2) * 2.0 ** -23 * x)
    for o, l in _both(ds, c, q.to(DEV), n):
        o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
        assert (np.abs(o - out) <= tol * weight).all()
        assert (np.abs(l - lse) <= 2.0 ** -20 * (np.abs(lse) + 1)).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lift", [20, 40, 100, 125])
@pytest.mark.parametrize("length", [90, 400])
def test_scores_beyond_the_grain_of_a_float_are_nan(ds, length, lift, dim):
    """2^lift log2(e) times the largest visible key is far above 2^23 in the
    last tokens, in the first tile or a later one: they are NaN, and tokens
    whose largest is below 2^22 are not."""
    n = 60
    c, keys = _staircase(dim, length, seed=66)
    q = torch.zeros((n, 2, dim), dtype=torch.bfloat16)
    q[:, 0, 0] = 2.0 ** lift
    q[:, 1, 0] = 2.0 ** 4
    top = np.array([keys[:length - n + 1 + j].max() for j in range(n)]) * 2.0 ** lift
    over = torch.as_tensor(top * math.log2(math.e) >= 2.0 ** 24)
    under = torch.as_tensor(top < 2.0 ** 22)
    assert over.any()
    for o, l in _both(ds, c, q.to(DEV), n):
        o, l = o.cpu(), l.cpu()
        assert torch.isnan(l[over, 0]).all() and torch.isnan(o[over, 0]).all()
        assert torch.isfinite(l[under, 0]).all() and torch.isfinite(o[under, 0]).all()
        assert torch.isfinite(l[:, 1]).all() and torch.isfinite(o[:, 1]).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("exponent", [117, -60])
def test_value_scales_at_their_limits(ds, dim, exponent):
    c = Cache([700, 90], 1, dim, seed=67)
    c.scales[:, 1] *= np.float32(2.0 ** (exponent + 6))
    _decode(ds, c, 3, 4)
    _prefill(ds, c, [300, 70], 4)


def test_refusals_of_the_bindings(ds):
    """Shapes that no kernel serves are the library's errors, calls without
    requests or tokens do nothing."""
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, table = torch.tensor([5], **i32), torch.zeros((1, 1), **i32)
    starts = torch.tensor([0, 5], **i32)
    for dim, heads, what in ((32, 4, "head_dim"), (64, 3, "num_heads")):
        codes = torch.zeros((1, 2, 2, 64, dim), dtype=torch.uint8, device=DEV)
        scales = torch.ones((1, 2, 2), device=DEV)
        q = torch.zeros((5, heads, dim), dtype=torch.bfloat16, device=DEV)
        with pytest.raises(Exception, match=what):
            ds.kv8_prefill(q, starts, codes, scales, table, lens, 0.1)
        with pytest.raises(Exception, match=what):
            ds.kv8_decode(q[None], codes, scales, table, lens, 0.1)
    codes = torch.zeros((1, 2, 2, 64, 64), dtype=torch.uint8, device=DEV)
    q = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device=DEV)
    none = torch.zeros((0, 1), **i32), torch.zeros(0, **i32)
    out = torch.full_like(q, 7.0)
    ds.kv8_prefill(q, torch.zeros(1, **i32), codes, scales, *none, 0.1, out=out)
    assert (out == 7).all()                       # rows of no request stay
    assert ds.kv8_prefill(q[:0], starts * 0, codes, scales, table, lens, 0.1)[0].shape == (0, 2, 64)
    assert ds.kv8_decode(q[:0, None], codes, scales, *none, 0.1)[0].shape == (0, 1, 2, 64)
    ds.kv8_append(q[:0], q[:0], starts * 0, table, lens, codes, scales)
    torch.cuda.synchronize()
    assert (scales == 1).all()


def test_threads_have_workspaces_of_their_own(ds):
    """Two threads on one stream: the launches of their calls come in any order."""
    c = Cache([900, 1300], 2, 128, seed=68)
    codes, scales, table, lens = c.device()
    starts = torch.tensor([0, 200, 500], dtype=torch.int32, device=DEV)
    q = c.q(500, 4).to(DEV)
    want = [ds.kv8_prefill(q * s, starts, codes, scales, table, lens, 0.1)[0] for s in (1, -1)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        x = q * (1, -1)[i]
        for _ in range(50):
            o, _ = ds.kv8_prefill(x, starts, codes, scales, table, lens, 0.1)
            if not torch.equal(o, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


@pytest.mark.parametrize("dim", [64, 128])
def test_append_dozens_of_tokens_to_many_requests(ds, dim):
    """Up to 40 tokens a request, more than a lane holds in registers."""
    counts = [(37 * i) % 79 for i in range(66)]
    assert sum(counts) <= 40 * len(counts)
    _append_case(ds, [n + (53 * i) % 130 for i, n in enumerate(counts)], counts, 8, dim, seed=69)


def test_offsets_beyond_32_bits(ds):
    """The same request in a small cache and in the last pages of one of more
    than 4 GB: append, decode and prefill give the same bits."""
    hk, dim, length = 8, 128, 300
    pages = (9 << 29) // (2 * hk * 64 * dim)               # 4.8 GB
    i32 = dict(dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(70)
    kv = torch.randn((length, 2, hk, dim), device=DEV, generator=g).to(torch.bfloat16)
    q = torch.randn((40, 16, dim), device=DEV, generator=g).to(torch.bfloat16)
    starts, lens = torch.tensor([0, length], **i32), torch.tensor([length], **i32)
    qs = torch.tensor([0, 40], **i32)
    got = []
    for n in (8, pages):
        codes = torch.empty((n, 2, hk, 64, dim), dtype=torch.uint8, device=DEV)
        scales = torch.empty((n, 2, hk), device=DEV)
        ids = torch.arange(n - 1, n - 6, -1, device=DEV)
        table = ids.int()[None].contiguous()
        ds.kv8_append(kv[:, 0], kv[:, 1], starts, table, lens, codes, scales)
        got.append((ds.kv8_decode(q[None], codes, scales, table, lens, 0.09)[0][0],
                    ds.kv8_prefill(q, qs, codes, scales, table, lens, 0.09)[0],
                    codes[ids].clone()))
        ds.pages_copy([codes, scales], ids[:1].int(), torch.tensor([0], **i32))
        torch.cuda.synchronize()
        assert torch.equal(codes[0], codes[ids[0]]) and torch.equal(scales[0], scales[ids[0]])
        del codes
    a, b = got
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    held = torch.arange(320, device=DEV).view(5, 1, 1, 64, 1) < length
    assert torch.equal(torch.where(held, a[2], 0), torch.where(held, b[2], 0))


def test_prefill_on_two_streams_at_once(ds):
    c = Cache([2500, 1300, 3000], 2, 64, seed=71)
    codes, scales, table, lens = c.device()
    starts = torch.tensor([0, 700, 1500, 2300], dtype=torch.int32, device=DEV)
    q = c.q(2300, 8).to(DEV)
    qs = [q, -q]
    want = [ds.kv8_prefill(x, starts, codes, scales, table, lens, 0.1)[0] for x in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            got.append((i, ds.kv8_prefill(qs[i], starts, codes, scales, table, lens, 0.1,
                                          stream=s)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_of_one_long_request(ds, dim):
    """One token on a long context, and a group whose rows fill one row tile and
    a little of the next."""
    c = Cache([20000], 1, dim, seed=72)
    _prefill(ds, c, [1], 3)
    _prefill(ds, c, [43], 3)

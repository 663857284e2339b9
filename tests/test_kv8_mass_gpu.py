"""GPU tests of the attention mass against float64, and of a run of mass and
eviction as a server would use them."""

import numpy as np
import pytest
import torch

import oracle
from harness import ensure_built
from kv8_cases import Cache, bits

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


def _starts(counts, lead=0):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + lead


def _lse_of(q, starts, c, scale):
    """float32 lse of causal attention, as the attention calls give it."""
    counts = np.diff(starts)
    rows = oracle.kv8_visible(c.lens, counts, c.table.shape[1])
    lse = np.full(q.shape[:2], np.nan, np.float32)
    got = oracle.kv8_attention(bits(q)[starts[0]:starts[-1]], rows, c.codes, c.scales, c.table, scale)
    lse[starts[0]:starts[-1]] = got[1]
    return lse


def _check(got, want, old, reach, dim, steps, starts, lens, width):
    """A score is a dim-term fp32 sum, its exponent two more roundings of it and of
    the lse; a weight is off by that and by 2^-21 of the exponential, a sum of
    columns and steps by a half step each."""
    for r, raw in enumerate(lens):
        n, length = int(starts[r + 1] - starts[r]), min(max(raw, 0), 64 * width)
        for g in range(got.shape[1]):
            base = np.where(np.arange(got.shape[2]) < raw - n, old[r, g], 0.0)
            added = np.maximum(want[r, g] - base, 0.0)
            rel = np.expm1((dim + 16) * 2.0 ** -24 * reach[r, g]) + (80 + steps) * 2.0 ** -24 + 2.0 ** -20
            tol = rel * added + 2.0 ** -23 * np.abs(want[r, g]) + 1e-37
            bad = ~(np.abs(got[r, g] - want[r, g]) <= tol)
            bad &= ~(np.isnan(got[r, g]) & np.isnan(want[r, g]))
            assert not bad[:length].any(), (r, g, np.nonzero(bad)[0][:5])
            # nothing behind the last position, nothing of requests without tokens
            keep = slice(length if n else 0, None)
            assert np.array_equal(got[r, g, keep], old[r, g, keep], equal_nan=True)


def _case(ds, lens, counts, heads, hk, dim, seed, gain=2.5, lead=0, tail=0, pad=0, bad=(), extra=0,
          edit=None, spread=3, err_want=0):
    c = Cache(lens, hk, dim, seed, spread=spread)
    for r, b, p in bad:
        c.table[r, b] = p
    starts = _starts(counts, lead)
    t = int(starts[-1]) + tail
    q = c.q(t, heads + pad, gain)
    scale = dim ** -0.5
    if edit is not None:
        edit(q, c)
    lse = _lse_of(q[:, :heads], starts, c, scale)
    mass = np.abs(c.rng.standard_normal((len(lens), hk, 64 * c.table.shape[1] + extra))) \
        .astype(np.float32)
    codes, scales, table, lens_d = c.device()
    md = torch.as_tensor(mass).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = ds.kv8_mass(q.to(DEV)[:, :heads], torch.as_tensor(lse).to(DEV),
                      torch.as_tensor(starts).to(DEV), codes, scales, table, lens_d, scale, md,
                      err_flag=err)
    torch.cuda.synchronize()
    assert got is md and int(err) == err_want
    want, reach = oracle.kv8_mass(bits(q[:, :heads]), lse, starts, c.codes, c.scales, c.table,
                                  c.lens, scale, mass)
    _check(md.cpu().numpy(), want, mass, reach, dim, max(counts) * heads // hk // 128 + 1, starts,
           c.lens, c.table.shape[1])
    return md


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,hk", [(1, 1), (8, 1), (6, 2), (16, 2), (28, 4), (130, 1)])
def test_one_token(ds, heads, hk, dim):
    _case(ds, [1, 64, 65, 128, 129, 700, 0, 300], [1, 1, 1, 1, 1, 1, 1, 1], heads, hk, dim, seed=heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,counts,heads,hk", [
    ([1], [1], 3, 1), ([200], [200], 4, 2), ([500, 130, 64, 7], [3, 130, 0, 7], 14, 2),
    ([900, 257], [33, 256], 8, 1), ([128, 128, 129], [128, 127, 1], 2, 2), ([640], [129], 1, 1),
    ([300, 40, 0, -3, 77], [17, 1, 0, 0, 16], 40, 8)])
def test_ragged(ds, lens, counts, heads, hk, dim):
    _case(ds, lens, counts, heads, hk, dim, seed=len(lens) + dim, lead=3, tail=2, pad=heads % 3)


def test_many_items_per_cta(ds):
    """More items than the GPU has SMs, of several requests: rings wrap."""
    rng = np.random.default_rng(1)
    lens = rng.integers(100, 1500, 24)
    _case(ds, lens, rng.integers(0, 4, 24), 16, 8, 128, seed=1)
    _case(ds, lens, rng.integers(0, 30, 24), 16, 8, 64, seed=2)


def test_a_request_shorter_than_its_tokens(ds):
    _case(ds, [5, 100], [9, 130], 4, 2, 64, seed=3)


def test_pages_outside_the_pool(ds):
    _case(ds, [300, 200], [4, 70], 4, 2, 128, seed=4, bad=[(0, 1, -1), (0, 4, 10 ** 6), (1, 2, -7)],
          err_want=2)


def test_every_code_and_magnitude(ds):
    """All E4M3 codes (subnormal ones too) and q far from 1, exactly."""
    def edit(q, c):
        flat = c.codes[c.table[0, 0], 0, 0]
        flat[:] = np.arange(flat.size, dtype=np.int64).reshape(flat.shape) % 0x7F
        flat[1::2] |= 0x80
        q[:] = 0
        q[:, :, 0] = 1.0
        q[:, :, 7] = 2.0 ** -9
        q[:, 0, 9] = 3e-5
    _case(ds, [64], [3], 2, 1, 64, seed=5, edit=edit, spread=1)
    _case(ds, [64, 200], [3, 9], 2, 1, 128, seed=6, gain=1e-30)
    _case(ds, [64, 200], [3, 9], 2, 1, 128, seed=6, gain=40.0)


@pytest.mark.parametrize("counts", [[3, 2], [60, 30]])
def test_non_finite_inputs(ds, counts):
    """Few rows and many: a request's rows are multiplied in pieces or as they are."""
    c = Cache([200, 150], 2, 64, 7)
    scale, n0, n1 = 0.125, counts[0], counts[1]
    q = c.q(n0 + n1, 4)
    starts = _starts(counts)
    lse = _lse_of(q, starts, c, scale)
    codes, scales, table, lens = c.device()

    def run(q, lse, codes=codes):
        mass = torch.ones((2, 2, 64 * table.shape[1]), device=DEV)
        ds.kv8_mass(q.to(DEV), torch.as_tensor(lse).to(DEV), torch.as_tensor(starts).to(DEV), codes,
                    scales, table, lens, scale, mass)
        torch.cuda.synchronize()
        return mass.cpu()
    want = run(q, lse)
    # a NaN key: its position alone, in its head alone
    bad = codes.clone()
    bad[table[0, 1].item(), 0, 1, 5, 40] = 0xFF
    got = run(q, lse, bad)
    assert got[0, 1, 69].isnan() and got.isnan().sum() == 1
    got[0, 1, 69] = want[0, 1, 69]
    assert torch.equal(got, want)
    # a row whose lse is -inf adds nothing, one of +inf neither; NaN shows where it sees
    l2 = lse.copy()
    l2[0, 0], l2[-1, 3] = -np.inf, np.nan
    got = run(q, l2)
    # (token 0's weights sum to 1; one far below the sum it is added to is lost)
    assert not got[0].isnan().any() and (got[0, 0] <= want[0, 0] * (1 + 2.0 ** -20)).all()
    less = (want[0, 0].double() - got[0, 0].double()).sum().item()
    assert abs(less - 1.0) <= want[0, 0].sum().item() * 2.0 ** -20
    assert torch.equal(got[0, 1], want[0, 1])
    assert got[1, 1, :150].isnan().all() and not got[1, 0].isnan().any()
    q2 = q.clone()
    q2[1, 2, 3] = float("nan")     # token 1 of request 0 sees 200 - n0 + 2 positions
    got = run(q2, lse)
    sees = 200 - n0 + 2
    assert got[0, 1, :sees].isnan().all() and not got[0, 1, sees:].isnan().any()
    assert not got[0, 0].isnan().any() and torch.equal(got[1], want[1])
    # the next request's q and what lies behind the last token reach nobody else
    q2 = torch.cat([q, torch.full((9, 4, 64), float("nan"), dtype=torch.bfloat16)])
    q2[n0:n0 + n1] = float("inf")
    l2 = np.concatenate([lse, np.zeros((9, 4), np.float32)])
    got = run(q2, l2)
    assert torch.equal(got[0], want[0]) and got[1, :, :150].isnan().all()


@pytest.mark.parametrize("heads,hk", [(7, 1), (46, 2), (39, 1), (40, 1), (41, 1), (100, 1), (113, 1),
                                      (128, 1), (200, 1), (300, 1)])
def test_groups_that_fill_a_step_and_do_not(ds, heads, hk):
    """Steps of whole tokens with rows to spare, of one token, of parts of one."""
    _case(ds, [300, 129, 64], [1, 40, 23], heads, hk, 64, seed=heads, tail=1)
    _case(ds, [200, 66], [5, 2], heads, hk, 128, seed=heads)


def test_few_rows_and_many_in_one_call(ds):
    rng = np.random.default_rng(14)
    _case(ds, rng.integers(70, 900, 30), rng.choice([0, 1, 2, 5, 11, 60], 30), 8, 2, 128, seed=14)


def test_small_elements_of_q(ds):
    """Elements down to 2^-19 of a row's largest count exactly, smaller ones within
    2^-27 of it."""
    def edit(q, c):
        c.codes[:, 0, :, :, 0] = 0                    # the large element's keys
        q[:] = (q.float() * 2.0 ** -17).to(torch.bfloat16)
        q[:, :, 0] = 8.0
    c_scale = 64 ** -0.5
    assert c_scale == 0.125
    _case(ds, [150, 80], [2, 1], 4, 1, 64, seed=15, edit=edit)


def test_bits_do_not_depend_on_the_batch(ds):
    rng = np.random.default_rng(8)
    lens, counts = [1500, 300, 2000, 64, 900, 1100], [1, 40, 5, 64, 700, 0]
    c = Cache(lens, 4, 128, 8)
    starts, scale = _starts(counts), 128 ** -0.5
    q = c.q(int(starts[-1]), 12)
    lse = torch.as_tensor(rng.standard_normal((len(q), 12)).astype(np.float32) + 8).to(DEV)
    codes, scales, table, ln = c.device()
    qd, sd = q.to(DEV), torch.as_tensor(starts).to(DEV)
    whole = torch.zeros((6, 4, 64 * table.shape[1]), device=DEV)
    ds.kv8_mass(qd, lse, sd, codes, scales, table, ln, scale, whole)
    for r in range(6):
        a, b = starts[r], starts[r + 1]
        one = torch.zeros((1, 4, 64 * table.shape[1]), device=DEV)
        ds.kv8_mass(qd[a:b], lse[a:b], sd[r:r + 2] - int(a), codes, scales, table[r:r + 1].contiguous(),
                    ln[r:r + 1], scale, one)
        assert torch.equal(one[0], whole[r])


def test_weights_of_a_row_sum_to_one(ds):
    """With the lse of the cache's own attention the mass of a step is one per
    query row, and repeated calls add up."""
    lens = [3000, 128, 777]
    c = Cache(lens, 2, 128, 9)
    codes, scales, table, ln = c.device()
    q = c.q(3, 16).to(DEV)
    out, lse = ds.kv8_decode(q[:, None], codes, scales, table, ln, 0.09)
    starts = torch.arange(4, dtype=torch.int32, device=DEV)
    mass = torch.zeros((3, 2, 64 * table.shape[1]), device=DEV)
    for i in range(1, 4):
        ds.kv8_mass(q, lse[:, 0].contiguous(), starts, codes, scales, table, ln, 0.09, mass)
        # (the last position is the call's own: it is set, not added to)
        last = torch.stack([mass[r, :, n - 1] for r, n in enumerate(lens)])
        total = mass.double().sum(-1) - last
        rest = (total / i + last).cpu()
        # decode's scores are off by up to 2^-14 and more roundings
        assert (rest - 8).abs().max() <= 8 * 2.0 ** -13


@pytest.mark.parametrize("counts", [[1, 2], [5, 1], [3, 70], [90, 1]])
def test_long_runs_of_items(ds, counts):
    """Dozens of items for every CTA, few rows and many: the weights of a row sum to
    one (what lies behind the rows' own positions was 0)."""
    lens, hk, heads, d = [90000, 60000], 8, 32, 64
    c = Cache([64, 64], hk, d, 12)
    rng = np.random.default_rng(12)
    pages = 1400
    codes = torch.randint(0, 0x70, (pages, 2, hk, 64, d), dtype=torch.uint8, device=DEV)
    scales = torch.full((pages, 2, hk), 2.0 ** -7, device=DEV)
    table = torch.as_tensor(rng.integers(0, pages, (2, 1408)), dtype=torch.int32).to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    starts = torch.as_tensor(_starts(counts)).to(DEV)
    q = c.q(sum(counts), heads, gain=0.05).to(DEV)
    _, lse = ds.kv8_prefill(q, starts, codes, scales, table, ln, 0.125)
    mass = torch.zeros((2, hk, 64 * 1408), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ds.kv8_mass(q, lse, starts, codes, scales, table, ln, 0.125, mass, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    want = torch.tensor(counts, dtype=torch.float64)[:, None] * (heads // hk)
    assert ((mass.double().sum(-1).cpu() / want - 1).abs() <= 2.0 ** -13).all()
    assert all((mass[r, :, n:] == 0).all() and (mass[r, :, :n] > 0).all() for r, n in enumerate(lens))


def test_a_batch_of_mostly_empty_requests(ds):
    """2^20 requests, tokens in few of them, at the ends of the list above all."""
    reqs, n = 1 << 20, 50
    rng = np.random.default_rng(13)
    full = np.array([0, 1, 3, 40, 500_000, reqs - 1] + list(range(100, 700)))
    codes = torch.as_tensor(rng.integers(0, 0x70, (4, 2, 1, 64, 64)), dtype=torch.uint8).to(DEV)
    scales = torch.full((4, 2, 1), 2.0 ** -7, device=DEV)
    table = torch.as_tensor(rng.integers(0, 4, (reqs, 1)), dtype=torch.int32).to(DEV)
    lens = torch.full((reqs,), n, dtype=torch.int32, device=DEV)
    counts = np.zeros(reqs, np.int64)
    counts[full] = 1
    starts = torch.as_tensor(_starts(counts)).to(DEV)
    q = torch.as_tensor(rng.standard_normal((len(full), 2, 64))).to(torch.bfloat16).to(DEV)
    _, lse = ds.kv8_decode(q[:, None], codes, scales, table[np.sort(full)], lens[:len(full)], 0.125)
    mass = torch.full((reqs, 1, 64), 3.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ds.kv8_mass(q, lse[:, 0], starts, codes, scales, table, lens, 0.125, mass, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    got = mass[np.sort(full), 0].double().cpu()
    assert (got[:, n:] == 3).all() and (got[:, :n - 1] > 3).all()
    # Sums of the two heads' weights, on 3 but for the token's own position.
    assert ((got[:, :n].sum(-1) - 3 * (n - 1)) / 2 - 1).abs().max() <= n * 2.0 ** -23 + 2.0 ** -13
    mass[np.sort(full)] = 3.0
    assert (mass == 3).all()


def test_one_token_has_no_stride(ds):
    c = Cache([100], 2, 64, 14)
    codes, scales, table, ln = c.device()
    starts = torch.as_tensor(_starts([1])).to(DEV)
    q, lse = c.q(1, 4).to(DEV), torch.full((1, 4), 5.0, device=DEV)
    mass = torch.zeros((2, 1, 2, 64 * table.shape[1]), device=DEV)
    for stride, m in ((256, mass[0]), (1 << 60, mass[1])):
        status = ds.lib().ds_kv8_mass(
            q.data_ptr(), stride, lse.data_ptr(), 1, starts.data_ptr(), 1, codes.data_ptr(),
            scales.data_ptr(), codes.shape[0], table.data_ptr(), table.shape[1], ln.data_ptr(), 4, 2,
            64, 0.125, m.data_ptr(), m.shape[2], None, torch.cuda.current_stream().cuda_stream)
        assert status == 0
    torch.cuda.synchronize()
    assert mass[0].any() and torch.equal(mass[0], mass[1])


def test_capture_streams_and_two_at_once(ds):
    c = Cache([1500, 800], 2, 64, 10)
    codes, scales, table, ln = c.device()
    starts = torch.as_tensor(_starts([40, 8])).to(DEV)
    q, lse = c.q(48, 4).to(DEV), torch.full((48, 4), 6.0, device=DEV)
    z = torch.zeros((2, 2, 64 * table.shape[1]), device=DEV)

    def run(mass, **kw):
        return ds.kv8_mass(q, lse, starts, codes, scales, table, ln, 0.125, mass, **kw)
    want = run(z.clone())
    a, b, m = z.clone(), z.clone(), z.clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.zero_()
        b.zero_()
        torch.cuda.synchronize()
        run(a, stream=s1)
        run(b, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(m)
    for _ in range(2):
        m.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(m, want)


def test_refusals(ds):
    c = Cache([100], 2, 64, 11)
    codes, scales, table, ln = c.device()
    starts = torch.as_tensor(_starts([2])).to(DEV)
    q, lse = c.q(2, 4).to(DEV), torch.zeros((2, 4), device=DEV)
    mass = torch.zeros((1, 2, 64 * table.shape[1]), device=DEV)
    with pytest.raises(ValueError):
        ds.kv8_mass(q, lse[:1], starts, codes, scales, table, ln, 0.1, mass)
    with pytest.raises(ValueError):
        ds.kv8_mass(q, lse, starts[:1], codes, scales, table, ln, 0.1, mass)
    with pytest.raises(ValueError):
        ds.kv8_mass(q, lse, starts, codes, scales, table, ln, 0.1, mass[:, :1].contiguous())
    with pytest.raises(ds.DSError, match="mass_stride"):
        ds.kv8_mass(q, lse, starts, codes, scales, table, ln, 0.1, mass[..., :64].contiguous())
    with pytest.raises(TypeError):
        ds.kv8_mass(q, lse.double(), starts, codes, scales, table, ln, 0.1, mass)
    with pytest.raises(ds.DSError, match="num_heads=3"):
        ds.kv8_mass(q[:, :3].contiguous(), lse[:, :3].contiguous(), starts, codes, scales, table, ln,
                    0.1, mass)
    ds.kv8_mass(q[:0], lse[:0], starts * 0, codes, scales, table, ln, 0.1, mass)
    assert (mass == 0).all()


def _mass(ds, c, q, lse, starts, scale, codes=None):
    """The kernel's mass on top of ones, as a host tensor."""
    dev_codes, scales, table, lens = c.device()
    mass = torch.ones((len(c.lens), c.kv_heads, 64 * table.shape[1]), device=DEV)
    ds.kv8_mass(q.to(DEV), torch.as_tensor(lse).to(DEV), torch.as_tensor(starts).to(DEV),
                dev_codes if codes is None else codes.to(DEV), scales, table, lens, scale, mass)
    torch.cuda.synchronize()
    return mass.cpu()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,counts,heads,hk", [
    ([200, 150], [3, 2], 4, 2), ([300, 64], [1, 1], 16, 2), ([700, 500], [200, 250], 4, 2),
    ([600, 129], [40, 1], 14, 2), ([400, 300], [130, 128], 300, 1)])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38])
def test_a_row_of_lse_minus_infinity_is_left_out_whatever_its_q(ds, lens, counts, heads, hk, dim, fill):
    """Padding: q that holds anything, or scores that overflow, under an lse of -inf."""
    if heads > 100:
        counts = [x // 40 for x in counts]
    c = Cache(lens, hk, dim, 21)
    starts, scale = _starts(counts), dim ** -0.5
    q = c.q(int(starts[-1]), heads)
    lse = _lse_of(q, starts, c, scale)
    dead = c.rng.random(lse.shape) < 0.1
    for a, b in zip(starts, starts[1:]):
        dead[(a + b) // 2] = True              # a whole token, in the middle
        dead[b - 1, heads // 2] = True         # a head of the one that sees everything
        dead[a, 0] = True                      # a step's first row
    lse[dead] = -np.inf
    junk = q.clone()
    q[torch.as_tensor(dead)] = 0.0
    junk[torch.as_tensor(dead)] = fill
    want, got = _mass(ds, c, q, lse, starts, scale), _mass(ds, c, junk, lse, starts, scale)
    assert torch.isfinite(want).all() and torch.equal(got, want)
    # and those are the sums without these rows
    old = np.ones(tuple(want.shape), np.float32)
    ref, reach = oracle.kv8_mass(bits(q), lse, starts, c.codes, c.scales, c.table, c.lens, scale, old)
    _check(got.numpy(), ref, old, reach, dim, max(counts) * heads // hk // 128 + 1, starts, c.lens,
           c.table.shape[1])
    # no row at all: what lies before the call's tokens stays, their own positions are 0
    none = _mass(ds, c, torch.full_like(q, fill), np.full_like(lse, -np.inf), starts, scale)
    for r, (n, length) in enumerate(zip(counts, lens)):
        assert (none[r, :, :length - n] == 1).all() and (none[r, :, length - n:length] == 0).all()


@pytest.mark.parametrize("counts", [[3, 2], [60, 90]])
def test_lse_of_plus_infinity_adds_nothing(ds, counts):
    c = Cache([200, 300], 2, 64, 22)
    starts = _starts(counts)
    q = c.q(sum(counts), 4)
    lse = _lse_of(q, starts, c, 0.125)
    minus, plus = lse.copy(), lse.copy()
    minus[1, 0] = minus[-1, 3] = -np.inf
    plus[1, 0] = plus[-1, 3] = np.inf
    want = _mass(ds, c, q, minus, starts, 0.125)
    assert torch.equal(_mass(ds, c, q, plus, starts, 0.125), want) and torch.isfinite(want).all()


@pytest.mark.parametrize("lens,counts", [([200], [3]), ([400], [1]), ([300], [60]), ([700], [250])])
@pytest.mark.parametrize("at", [3, 60])
def test_a_nan_key_shows_where_a_row_of_weight_sees_it(ds, lens, counts, at):
    """Its dim in either half of the head; a position that only rows of lse -inf see
    gets nothing."""
    c = Cache(lens, 2, 64, 23)
    n, starts = counts[0], _starts(counts)
    q = c.q(n, 4)
    lse = _lse_of(q, starts, c, 0.125)
    codes, _, table, _ = c.device()

    def poisoned(pos):
        bad = codes.clone()
        bad[table[0, pos // 64].item(), 0, 1, pos % 64, at] = 0xFF
        return bad
    last = lens[0] - 1
    for pos in (0, lens[0] - n, last):
        want = _mass(ds, c, q, lse, starts, 0.125)
        got = _mass(ds, c, q, lse, starts, 0.125, poisoned(pos))
        assert got[0, 1, pos].isnan() and got.isnan().sum() == 1
        got[0, 1, pos] = want[0, 1, pos]
        assert torch.equal(got, want)
    # the last token's rows of kv head 1 have no weight: nobody else sees its position
    lse[-1, 2:] = -np.inf
    want = _mass(ds, c, q, lse, starts, 0.125)
    got = _mass(ds, c, q, lse, starts, 0.125, poisoned(last))
    assert got[0, 1, last] == 0 and torch.equal(got, want)
    # one of its two heads has: the position is NaN
    lse[-1, 3] = 5.0
    got = _mass(ds, c, q, lse, starts, 0.125, poisoned(last))
    assert got[0, 1, last].isnan() and got.isnan().sum() == 1


@pytest.mark.parametrize("counts,heads,hk", [([1, 3], 1024, 1024), ([40, 2], 512, 256), ([2, 1], 1024, 1)])
def test_many_heads(ds, counts, heads, hk):
    _case(ds, [130, 70], counts, heads, hk, 64, seed=31)

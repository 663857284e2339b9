"""GPU tests of the page operations against the list oracle, states and
payloads exact; and a run of them with the block-scaled cache as a server
would use them together."""

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


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


FLAGS = {"row": 4, "page": 2, "nopage": 16, "len": 32}


class State:
    """Random rows over a pool; some rows share their first pages."""

    def __init__(self, pages, width, lens, seed, share=()):
        rng = np.random.default_rng(seed)
        self.refs = [0] * pages
        self.table = [[-1] * width for _ in lens]
        self.lens = list(lens)
        perm = iter(rng.permutation(pages).tolist())
        for r, n in enumerate(lens):
            for j in range(oracle.pages.held(n, width)):
                self.table[r][j] = next(perm)
                self.refs[self.table[r][j]] = 1
        for a, b, n in share:   # row b's first n entries become row a's
            for j in range(n):
                self.refs[self.table[b][j]] -= 1
                self.table[b][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
        # payloads of several shapes, one whose pages allow only 4-byte words
        g = torch.Generator(device=DEV).manual_seed(seed)
        shapes = [(pages, 2, 1, 64, 64), (pages, 3), (pages, 40000 // 4), (pages, 4)]
        self.pools = [torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=g, device=DEV,
                                    dtype=torch.int32) for s in shapes]
        self.pools[0] = torch.randint(0, 256, shapes[0], generator=g, device=DEV,
                                      dtype=torch.uint8)

    def device(self):
        self.d = (_i32(self.refs), _i32(self.table), _i32(self.lens))
        return self.d

    def check(self, refs, table, lens, flags, err):
        torch.cuda.synchronize()
        assert self.d[0].tolist() == refs
        assert self.d[1].tolist() == table
        assert self.d[2].tolist() == lens
        assert int(err) == sum(FLAGS[f] for f in flags)


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows", [[0], [3, -1, 1], [2, 2, 0], [9, 1], list(range(5))])
def test_free(ds, rows):
    s = State(60, 12, [700, 64, 1, 0, 130], seed=1, share=[(0, 4, 2)])
    s.table[0][3] = 10 ** 6 if 9 in rows else s.table[0][3]
    refs, table, lens = s.device()
    err = _err()
    ds.pages_free(refs, table, lens, _i32(rows), err_flag=err)
    s.check(*oracle.pages_free(s.refs, s.table, s.lens, rows)[:4], err)


def test_free_flags_what_it_cannot_count(ds):
    s = State(10, 4, [200, 100], seed=2)
    s.table[0][1], s.refs[s.table[1][0]] = 77, 0
    refs, table, lens = s.device()
    err = _err()
    ds.pages_free(refs, table, lens, _i32([0, 1]), err_flag=err)
    want = oracle.pages_free(s.refs, s.table, s.lens, [0, 1])
    assert want[3] == {"page"}
    s.check(*want, err)


def _copied(pools, moves):
    want = [p.clone() for p in pools]
    for a, b in moves:
        for w, p in zip(want, pools):
            w[b] = p[a]
    return want


@pytest.mark.parametrize("pages,n", [(40, 1), (1500, 300), (5000, 37)])
def test_copy(ds, pages, n):
    s = State(pages, 1, [], seed=3)
    perm = np.random.default_rng(4).permutation(pages)
    src, dst = perm[:n].copy(), perm[n:2 * n].copy() if 2 * n <= pages else perm[-n:].copy()
    n = min(n, len(dst))
    src, dst = src[:n], dst[:n]
    moves = list(zip(src.tolist(), dst.tolist()))
    if n > 10:
        src[3], dst[4], src[5], dst[6] = -1, -2, pages, pages + 5
        moves = [m for i, m in enumerate(moves) if i not in (3, 4, 5, 6)]
    want = _copied(s.pools, moves)
    err = _err()
    ds.pages_copy(s.pools, _i32(src), _i32(dst), err_flag=err)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))
    assert int(err) == (2 if n > 10 else 0)


@pytest.mark.parametrize("parents,children", [
    ([0], [3]), ([0, 0, 1, 2], [3, 5, 6, 7]), ([0, -1, 1], [-1, 3, 5]),
    ([0, 0], [3, 3]), ([0, 1], [1, 5]), ([99, 0], [3, 99]), ([3, 0], [5, 3]),
])
def test_fork(ds, parents, children):
    s = State(1300, 14, [700, 64, 1, 0, 130, 0, 0, 0], seed=5)
    refs, table, lens = s.device()
    r, t, l, flags, moves = oracle.pages_fork(s.refs, s.table, s.lens, parents, children)
    want = _copied(s.pools, moves)
    err = _err()
    ds.pages_fork(s.pools, refs, table, lens, _i32(parents), _i32(children), err_flag=err)
    s.check(r, t, l, flags, err)
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))


def test_fork_without_pages_enough(ds):
    s = State(9, 4, [130, 70, 64, 0, 0, 0, 0], seed=6)     # 6 held, 3 free
    for children, parents in (([3, 4, 5, 6], [0, 1, 0, 2]), ([3, 4, 5, 6], [0, 0, 0, 1])):
        refs, table, lens = s.device()
        r, t, l, flags, moves = oracle.pages_fork(s.refs, s.table, s.lens, parents, children)
        pools = [p.clone() for p in s.pools]
        err = _err()
        ds.pages_fork(pools, refs, table, lens, _i32(parents), _i32(children), err_flag=err)
        s.check(r, t, l, flags, err)
        assert all(torch.equal(a, b) for a, b in zip(pools, _copied(s.pools, moves)))


def test_fork_without_pools(ds):
    s = State(50, 4, [100, 0], seed=7)
    refs, table, lens = s.device()
    err = _err()
    ds.pages_fork([], refs, table, lens, _i32([0]), _i32([1]), err_flag=err)
    s.check(*oracle.pages_fork(s.refs, s.table, s.lens, [0], [1])[:4], err)


@pytest.mark.parametrize("rows,new", [
    ([3], [1]), ([0, 1, 2, 3], [768, 65, 64, 500]), ([0, 0], [720, 740]),
    ([1, -1, 7, 2], [64, 5, 5, 0]), ([1, 3], [897, 896]),
])
def test_extend(ds, rows, new):
    s = State(2100, 14, [700, 64, 1, 0, 130], seed=8)
    refs, table, lens = s.device()
    err = _err()
    ds.pages_extend(refs, table, lens, _i32(rows), _i32(new), err_flag=err)
    s.check(*oracle.pages_extend(s.refs, s.table, s.lens, rows, new), err)


def test_extend_without_pages_enough(ds):
    s = State(12, 8, [64, 1, 0, 100], seed=9)              # 4 held, 8 free
    rows, new = [0, 2, 1, 3], [256, 512, 64, 128]
    refs, table, lens = s.device()
    err = _err()
    ds.pages_extend(refs, table, lens, _i32(rows), _i32(new), err_flag=err)
    want = oracle.pages_extend(s.refs, s.table, s.lens, rows, new)
    assert want[3] == {"nopage"}
    s.check(*want, err)


def test_lists_longer_than_a_block(ds):
    n = 700
    s = State(3500, 3, [65] * n + [0] * n, seed=10)
    parents, children = list(range(n)), list(range(n, 2 * n))
    refs, table, lens = s.device()
    r, t, l, flags, moves = oracle.pages_fork(s.refs, s.table, s.lens, parents, children)
    want = _copied(s.pools, moves)
    err = _err()
    ds.pages_fork(s.pools, refs, table, lens, _i32(parents), _i32(children), err_flag=err)
    s.check(r, t, l, flags, err)
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))
    r, t, l, f2 = oracle.pages_extend(r, t, l, children, [130] * n)
    ds.pages_extend(refs, table, lens, _i32(children), _i32([130] * n), err_flag=err)
    s.check(r, t, l, flags | f2, err)


@pytest.mark.parametrize("pages,lens,share", [
    (40, [700, 64, 1, 0, 130], [(0, 4, 2)]), (13, [64] * 13, []), (20, [0, 0], []),
    (3000, [640] * 100, [(0, 1, 5)]), (1, [5], []), (1025, [64 * 7] * 70, []),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(ds, pages, lens, share, in_place):
    s = State(pages, 12, lens, seed=pages, share=share)
    if pages == 40:
        s.table[0][9], s.table[1][0] = 10 ** 6, s.refs.index(0)
    refs, table, lens_d = s.device()
    r, t, flags, n, moves = oracle.pages_compact(s.refs, s.table, s.lens)
    want = _copied(s.pools, moves)
    err = _err()
    kw = dict(block_table_out=table, refcounts_out=refs) if in_place else {}
    t2, r2, n2 = ds.pages_compact(s.pools, refs, table, lens_d, err_flag=err, **kw)
    torch.cuda.synchronize()
    assert int(n2) == n and t2.tolist() == t and r2.tolist() == r
    assert int(err) == sum(FLAGS[f] for f in flags)
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))
    if not in_place:
        s.check(s.refs, s.table, s.lens, flags, err)


def test_captured_step_replays(ds):
    """free, fork, extend in one graph: the state of each replay follows from
    the state before it."""
    s = State(300, 10, [500, 130, 64, 0], seed=11)
    refs, table, lens = s.device()
    kids, parents, new = _i32([3, 2]), _i32([0, 1]), _i32([510, 200])
    ws = torch.empty(ds.pages_workspace_size(300, 2), dtype=torch.uint8, device=DEV)
    ds.pages_free(refs, table, lens, _i32([-1]))      # loads the kernel before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.pages_free(refs, table, lens, kids)
        ds.pages_fork(s.pools, refs, table, lens, parents, kids, workspace=ws)
        ds.pages_extend(refs, table, lens, kids, new, workspace=ws)
    r, t, l = s.refs, s.table, s.lens
    pools = [p.clone() for p in s.pools]
    for _ in range(3):
        g.replay()
        r, t, l, _f = oracle.pages_free(r, t, l, [3, 2])
        r, t, l, _f, moves = oracle.pages_fork(r, t, l, [0, 1], [3, 2])
        pools = _copied(pools, moves)
        r, t, l, _f = oracle.pages_extend(r, t, l, [3, 2], [510, 200])
        s.check(r, t, l, set(), _err())
        assert all(torch.equal(a, b) for a, b in zip(s.pools, pools))


def test_a_server_run(ds):
    """Prompts, decode steps, a fork, diverging tails, a free and a compaction:
    after each step the attention of every live row equals the oracle's on
    that row's own history of appended tokens."""
    hk, d, heads, pages, width, rows = 2, 64, 8, 40, 6, 4
    rng = np.random.default_rng(12)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    codes = torch.full((pages, 2, hk, 64, d), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages, 2, hk), float("nan"), device=DEV)
    pools = [codes, scales]
    host = [0] * rows
    err = _err()

    def grow(which, n):
        for r, m in zip(which, n):
            host[r] += m
        ds.pages_extend(refs, table, lens, _i32(which), _i32([host[r] for r in which]),
                        err_flag=err)
        counts = [n[which.index(r)] if r in which else 0 for r in range(rows)]
        starts = _i32(np.concatenate([[0], np.cumsum(counts)]))
        x = torch.as_tensor(rng.standard_normal((sum(counts), 2, hk, d)) *
                            np.exp(rng.standard_normal((sum(counts), 1, 1, 1)))) \
            .to(torch.bfloat16).to(DEV)
        ds.kv8_append(x[:, 0], x[:, 1], starts, table, lens, codes, scales, err_flag=err)

    def look():
        q = torch.randn((rows, 1, heads, d), device=DEV).to(torch.bfloat16)
        out, lse = ds.kv8_decode(q, codes, scales, table, lens, 0.125, err_flag=err)
        ref = oracle.kv8_attention(bits(q[:, 0]), oracle.kv8_visible(host, [1] * rows, width),
                                   codes.cpu().numpy(), scales.cpu().numpy(),
                                   table.cpu().numpy(), 0.125)
        tol, tol_lse = oracle.kv8_bounds(ref[0], ref[1], ref[2], ref[3], d, max(host))
        assert (np.abs(out[:, 0].double().cpu().numpy() - ref[0]) <= tol).all()
        live = np.array(host) > 0
        got = lse[:, 0].double().cpu().numpy()
        assert (np.abs(got[live] - ref[1][live]) <= tol_lse[live]).all()
        assert lens.tolist() == host and int(err) == 0
        return out, lse

    grow([0, 2], [150, 64])
    look()
    for _ in range(3):
        grow([2, 0], [1, 5])
    before = look()
    ds.pages_fork(pools, refs, table, lens, _i32([0, 2]), _i32([1, 3]), err_flag=err)
    host[1], host[3] = host[0], host[2]
    q = torch.randn((rows, 1, heads, d), device=DEV).to(torch.bfloat16)
    q[1], q[3] = q[0], q[2]
    out, _ = ds.kv8_decode(q, codes, scales, table, lens, 0.125)
    assert torch.equal(out[1], out[0]) and torch.equal(out[3], out[2])
    grow([0, 1, 2, 3], [3, 40, 1, 2])
    look()
    ds.pages_free(refs, table, lens, _i32([0]), err_flag=err)
    host[0] = 0
    kept = ds.kv8_decode(q, codes, scales, table, lens, 0.125)
    _, _, live = ds.pages_compact(pools, refs, table, lens, block_table_out=table,
                                  refcounts_out=refs, err_flag=err)
    after = ds.kv8_decode(q, codes, scales, table, lens, 0.125)
    assert torch.equal(kept[0], after[0]) and torch.equal(kept[1], after[1])
    held = {p for r in range(rows) for p in table[r, :-(-host[r] // 64)].tolist()}
    assert held == set(range(int(live)))
    grow([3, 0], [60, 10])
    look()
    assert before is not None


def test_refusals_of_pools(ds):
    i32 = dict(dtype=torch.int32, device=DEV)
    one = torch.zeros(1, **i32)
    with pytest.raises(ValueError, match="no pages"):
        ds.pages_copy([torch.zeros((0, 64), device=DEV)], one, one)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ds.pages_copy([None], one, one)
    with pytest.raises(ValueError, match="contiguous"):
        ds.pages_copy([torch.zeros((4, 64), device=DEV), torch.zeros((5, 64), device=DEV)], one, one)
    with pytest.raises(Exception, match="page_bytes"):
        ds.pages_copy([torch.zeros((4, 6), dtype=torch.uint8, device=DEV)], one, one)


@pytest.mark.parametrize("count", [16, 17, 128])
def test_many_pools_on_another_stream(ds, count):
    s = State(90, 12, [700, 64, 130, 0, 0], seed=12, share=[(0, 2, 2)])
    g = torch.Generator(device=DEV).manual_seed(13)
    s.pools = [torch.randint(-9, 9, (90, 4 * (i % 5 + 1)), generator=g, device=DEV,
                             dtype=torch.int32) for i in range(count)]
    refs, table, lens = s.device()
    parents, kids = _i32([0, 2]), _i32([3, 4])
    moves = [(50, 80), (3, 85)]
    want = _copied(s.pools, moves)
    r, t, l, flags, m = oracle.pages_fork(s.refs, s.table, s.lens, [0, 2], [3, 4])
    want = _copied(want, m)
    side, err = torch.cuda.Stream(), _err()
    src, dst = _i32([50, 3]), _i32([80, 85])
    torch.cuda.synchronize()
    ds.pages_copy(s.pools, src, dst, err_flag=err, stream=side)
    ds.pages_fork(s.pools, refs, table, lens, parents, kids, err_flag=err, stream=side)
    s.check(r, t, l, flags, err)
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))
    r2, t2, f2, n, m = oracle.pages_compact(r, t, l)
    want = _copied(want, m)
    out = ds.pages_compact(s.pools, refs, table, lens, err_flag=err, stream=side)
    torch.cuda.synchronize()
    assert int(out[2]) == n and out[0].tolist() == t2 and out[1].tolist() == r2
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_fork_takes_a_last_page_outside_the_pool_over(ds, bad):
    """No page is taken for it, the child's entry is the parent's, and both rows'
    attention leaves its positions out."""
    s = State(40, 14, [700, 130, 100, 0, 0, 0], seed=14)
    s.table[1][2] = bad
    parents, children = [0, 1, 2], [3, 4, 5]
    refs, table, lens = s.device()
    r, t, l, flags, moves = oracle.pages_fork(s.refs, s.table, s.lens, parents, children)
    assert flags == {"page"} and len(moves) == 2 and t[4][2] == bad
    want = _copied(s.pools, moves)
    err = _err()
    ds.pages_fork(s.pools, refs, table, lens, _i32(parents), _i32(children), err_flag=err)
    s.check(r, t, l, flags, err)
    assert all(torch.equal(a, b) for a, b in zip(s.pools, want))
    codes = torch.randint(0, 0x7F, (40, 2, 1, 64, 64), dtype=torch.uint8, device=DEV)
    q = torch.randn((1, 1, 2, 64), device=DEV).to(torch.bfloat16).expand(6, 1, 2, 64).contiguous()
    out, lse = ds.kv8_decode(q, codes, torch.full((40, 2, 1), 0.01, device=DEV), table, lens, 0.1)
    assert torch.equal(out[4], out[1]) and torch.equal(lse[4], lse[1])


def test_a_fork_leaves_its_parents_outputs(ds):
    """Attention of every row before a fork, after it, and after the children
    have appended: the parents' is unchanged, the children's starts as theirs."""
    hk, d, rows, pages = 2, 64, 4, 30
    g = torch.Generator(device=DEV).manual_seed(15)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    table = torch.full((rows, 4), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    codes = torch.full((pages, 2, hk, 64, d), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages, 2, hk), float("nan"), device=DEV)
    err = _err()

    def grow(which, counts, new_lens):
        ds.pages_extend(refs, table, lens, _i32(which), _i32(new_lens), err_flag=err)
        x = torch.randn((sum(counts), 2, hk, d), generator=g, device=DEV).to(torch.bfloat16)
        ds.kv8_append(x[:, 0], x[:, 1], _i32(np.concatenate([[0], np.cumsum(counts)])), table, lens,
                      codes, scales, err_flag=err)

    q = torch.randn((1, 1, 8, d), generator=g, device=DEV).to(torch.bfloat16)
    q = q.expand(rows, 1, 8, d).contiguous()
    look = lambda: ds.kv8_decode(q, codes, scales, table, lens, 0.125, err_flag=err)  # noqa: E731
    grow([0, 1], [150, 64, 0, 0], [150, 64])
    before = look()
    ds.pages_fork([codes, scales], refs, table, lens, _i32([0, 1]), _i32([2, 3]), err_flag=err)
    after = look()
    grow([2, 3], [0, 0, 30, 7], [180, 71])
    later = look()
    torch.cuda.synchronize()
    assert int(err) == 0
    for b, a, x in zip(before, after, later):
        assert torch.equal(a[:2], b[:2]) and torch.equal(a[2:], b[:2])
        assert torch.equal(x[:2], b[:2]) and not (x[2:] == b[:2]).flatten(1).all(1).any()

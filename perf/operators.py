"""What is measured of the block-scaled 8-bit KV cache and of the paged-cache maintenance.

Operators: the cache write (``kv8_append``), attention over that cache for
single or few tokens (``kv8_decode``) and for prompts (``kv8_prefill``), and
the page operations (``pages_copy``, ``pages_free``, ``pages_fork``,
``pages_extend``, ``pages_compact``).

The cache of one layer is ``kv_pages`` uint8 [pages, 2, kv_heads, 64, dim]
(E4M3 codes; index 0 of the second axis keys, 1 values) with ``kv_scales``
float32 [pages, 2, kv_heads]: a value is its code times the scale of its page,
side and head. Sizes are those of the repository's serving workloads (pages of
64, contexts of 1024, 4096-32768 and 8192-131072, 32 requests, 5 tokens under
multi-token prediction) or generic ones.
"""

import math

import torch

own = False

PAGE = 64
MIN_EXP, MAX_EXP = -60, 120   # exponents a scale may have
CODE_MAX = 448.0              # largest finite E4M3 magnitude


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of a batch writes its 5 speculative tokens per request.
        dict(name="append_mtp", op="append", reqs=128, lo=5, hi=5, ctx_lo=256, ctx_hi=4096,
             kv_heads=8, dim=128),
        # Prompts of odd lengths, some of them continuing a cached prefix.
        dict(name="append_prompts", op="append", reqs=8, lo=700, hi=4001, ctx_lo=4001,
             ctx_hi=8192, kv_heads=8, dim=128),
        # The smallest decode call, where latency is everything.
        dict(name="decode_small", op="decode", reqs=2, next_n=1, heads=16, kv_heads=2, dim=64,
             ctx_lo=1024, ctx_hi=1024),
        # A serving batch under multi-token prediction (1 target and 4 draft tokens).
        dict(name="decode_mtp", op="decode", reqs=32, next_n=5, heads=64, kv_heads=8, dim=128,
             ctx_lo=4096, ctx_hi=32768),
        # Long contexts, one token per request.
        dict(name="decode_long", op="decode", reqs=16, next_n=1, heads=128, kv_heads=8, dim=128,
             ctx_lo=8192, ctx_hi=131072),
        # A chunk of a long prompt: the last 2048 tokens of a 32768 context.
        dict(name="prefill_chunk", op="prefill", reqs=1, lo=2048, hi=2048, ctx_lo=32768,
             ctx_hi=32768, heads=64, kv_heads=8, dim=128),
        # A mixed batch: ragged prompts and prefixes, head groups of 7, dim 64.
        dict(name="prefill_ragged", op="prefill", reqs=12, lo=1, hi=1500, ctx_lo=1500,
             ctx_hi=5000, heads=28, kv_heads=4, dim=64),
        # Beam search / parallel sampling step: losers freed, winners forked and
        # extended by 5 tokens; few rows and layers.
        dict(name="beam_small", op="beam", rows=16, forks=4, ctx_lo=500, ctx_hi=4000, pages=2048,
             layers=4, kv_heads=2, dim=64),
        # The same on a large pool with many rows and layers.
        dict(name="beam_large", op="beam", rows=256, forks=96, ctx_lo=4096, ctx_hi=8192,
             pages=16384, layers=8, kv_heads=4, dim=128),
        # Compaction of a small fragmented pool.
        dict(name="compact_small", op="compact", rows=12, ctx_lo=100, ctx_hi=3000, pages=1500,
             layers=3, kv_heads=2, dim=64),
        # Compaction of a large one.
        dict(name="compact_large", op="compact", rows=128, ctx_lo=1000, ctx_hi=4000, pages=12000,
             layers=4, kv_heads=8, dim=128),
        # Pages copied by a list (a prefix duplicated for writing).
        dict(name="copy_pages", op="copy", pages=4096, copies=700, layers=4, kv_heads=4, dim=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "beam", "compact",
                     "copy"])
    kv_heads, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    if op == "append":
        hi = _log(rng, 1, 3000)
        ctx = hi + _log(rng, 1, 4000)
        reqs = _log(rng, 1, 8 if hi > 300 else 128)
        return dict(op=op, reqs=reqs, lo=rng.randint(0 if reqs > 5 else 1, hi), hi=hi, ctx_lo=hi,
                    ctx_hi=ctx, kv_heads=kv_heads, dim=dim)
    if op == "decode":
        ctx = _log(rng, 16, 100000)
        return dict(op=op, reqs=_log(rng, 1, max(1, min(64, 1000000 // ctx))),
                    next_n=rng.choice([1, 1, 2, 3, 4, 5, 7]),
                    heads=kv_heads * rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16]), kv_heads=kv_heads,
                    dim=dim, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    if op == "prefill":
        hi = _log(rng, 2, 2000)
        ctx = hi + _log(rng, 1, 12000)
        reqs = _log(rng, 1, max(1, min(12, 6000 // hi)))
        return dict(op=op, reqs=reqs, lo=rng.randint(0 if reqs > 5 else 1, hi), hi=hi, ctx_lo=hi,
                    ctx_hi=ctx,
                    heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv_heads=kv_heads, dim=dim)
    layers = rng.randint(1, 6)
    if op == "beam":
        rows = _log(rng, 4, 200)
        ctx = _log(rng, 64, 6000)
        return dict(op=op, rows=rows, forks=rng.randint(1, max(1, rows // 3)),
                    ctx_lo=rng.randint(1, ctx), ctx_hi=ctx,
                    pages=rows * (ctx // PAGE + 3) + rng.randint(0, 2000), layers=layers,
                    kv_heads=min(kv_heads, 4), dim=dim)
    if op == "compact":
        rows = _log(rng, 1, 100)
        ctx = _log(rng, 64, 4000)
        return dict(op=op, rows=rows, ctx_lo=rng.randint(1, ctx), ctx_hi=ctx,
                    pages=rows * (ctx // PAGE + 1) + rng.randint(1, 3000), layers=min(layers, 4),
                    kv_heads=min(kv_heads, 4), dim=dim)
    pages = _log(rng, 16, 4096)
    return dict(op=op, pages=pages, copies=rng.randint(1, pages // 2), layers=min(layers, 4),
                kv_heads=kv_heads, dim=dim)


# ----------------------------------------------------------------- inputs
def _host(case):
    """A generator for the case's lengths: they follow from the case alone, so
    every seed has the same amount of work."""
    return torch.Generator().manual_seed(20240 + sum(v for v in case.values()
                                                     if isinstance(v, int)))


def _between(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _pages_of(lens):
    return (lens + PAGE - 1) // PAGE


def _codes(shape, gen, dev):
    """Codes of N(0, 100) values: what a scale of about amax / 448 gives."""
    x = torch.empty(shape, dtype=torch.float16, device=dev).normal_(0.0, 100.0, generator=gen)
    return x.clamp_(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, gen, dev):
    """Powers of two around 1/128, another for every page, side and head."""
    return torch.exp2(torch.randint(-8, -5, shape, generator=gen, device=dev).float())


def _tables(lens, width, pages, gen, dev):
    """Random distinct pages for every row; -1 in entries that hold none."""
    held = _pages_of(lens)
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    j = torch.arange(width)[None, :]
    at = (first[:, None] + j).clamp(max=pages - 1).to(dev)
    return torch.where((j < held[:, None]).to(dev), perm[at], -1).to(torch.int32).contiguous()


def _lengths(case):
    """Context lengths and new-token counts of the requests (host tensors)."""
    g = _host(case)
    n, op = case["reqs"], case["op"]
    ctx = _between(g, case["ctx_lo"], case["ctx_hi"], n)
    if op == "decode":
        return ctx, torch.full((n,), case["next_n"])
    new = _between(g, case["lo"], case["hi"], n)
    return torch.maximum(ctx, new), new


def _beam_plan(case):
    g = _host(case)
    rows, forks = case["rows"], case["forks"]
    perm = torch.randperm(rows, generator=g)
    lens = _between(g, case["ctx_lo"], case["ctx_hi"], rows)
    return lens, perm[forks:][torch.randint(0, rows - forks, (forks,), generator=g)], perm[:forks]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    if op in ("append", "decode", "prefill"):
        lens, new = _lengths(case)
        hk, d = case["kv_heads"], case["dim"]
        width = max(1, int(_pages_of(lens).max()))
        pages = int(_pages_of(lens).sum()) + 3
        st = dict(op=op, lens=lens.to(dev, torch.int32),
                  block_table=_tables(lens, width, pages, gen, dev),
                  kv_pages=_codes((pages, 2, hk, PAGE, d), gen, dev),
                  kv_scales=_scales((pages, 2, hk), gen, dev))
        starts = torch.zeros(len(new) + 1, dtype=torch.int64)
        starts[1:] = torch.cumsum(new, 0)
        tokens = int(starts[-1])
        st["token_starts"] = starts.to(dev, torch.int32)
        if op == "append":
            # Keys and values as slices of one fused projection's output.
            kv = torch.randn((tokens, 2, hk, d), generator=gen, device=dev)
            kv *= torch.exp(0.5 * torch.randn((tokens, 1, hk, 1), generator=gen, device=dev))
            kv = kv.to(torch.bfloat16)
            st.update(k=kv[:, 0], v=kv[:, 1])
            return st
        st["scale"] = 1.0 / math.sqrt(d)
        q = 2.5 * torch.randn((tokens, case["heads"], d), generator=gen, device=dev)
        st["q"] = q.to(torch.bfloat16)
        st["max_new"] = int(new.max())
        if op == "decode":
            st["q"] = st["q"].view(case["reqs"], case["next_n"], case["heads"], d)
        # What the last pages hold behind the last position is whatever their
        # previous owners left, NaN codes among it.
        last = (lens - 1).clamp(min=0)
        page = st["block_table"].gather(1, (last // PAGE).to(dev)[:, None]).long()[:, 0].clamp(min=0)
        behind = torch.arange(PAGE)[None, :] > (last % PAGE)[:, None]
        tail = st["kv_pages"][page]
        tail.masked_fill_((behind.to(dev) & (st["lens"] > 0)[:, None])[:, None, None, :, None], 0x7F)
        st["kv_pages"][page] = tail
        return st
    pages, hk, d = case["pages"], case["kv_heads"], case["dim"]
    pools = []
    for _ in range(case["layers"]):
        pools.append(torch.randint(0, 256, (pages, 2, hk, PAGE, d), generator=gen, device=dev,
                                   dtype=torch.uint8))
        pools.append(_scales((pages, 2, hk), gen, dev))
    st = dict(op=op, pools=pools)
    if op == "copy":
        perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        st["src"] = perm[: case["copies"]].clone()
        st["dst"] = perm[pages - case["copies"]:].clone()
        return st
    if op == "beam":
        lens, parents, children = _beam_plan(case)
        st["parents"] = parents.to(dev, torch.int32)
        st["children"] = children.to(dev, torch.int32)
        st["new_lens"] = (lens[parents] + 5).to(dev, torch.int32)
        width = int(lens.max()) // PAGE + 2
    else:
        lens = _between(_host(case), case["ctx_lo"], case["ctx_hi"], case["rows"])
        width = int(_pages_of(lens).max())
    st["lens"] = lens.to(dev, torch.int32)
    st["block_table"] = _tables(lens, width, pages, gen, dev)
    held = st["block_table"].flatten().long()
    refs = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
    refs.index_add_(0, torch.where(held >= 0, held, pages), torch.ones_like(held, dtype=torch.int32))
    st["refcounts"] = refs[:pages].clone()
    if op == "compact":
        # Two rows share their first pages, as forked rows do.
        if case["rows"] > 1:
            n = int(min(lens[0], lens[1])) // PAGE // 2
            bt, r = st["block_table"], st["refcounts"]
            r[bt[1, :n].long()] -= 1
            bt[1, :n] = bt[0, :n]
            r[bt[0, :n].long()] += 1
    return st


# ------------------------------------------------------------ plain forms
def _need_scale(amax):
    """Smallest power of two s with amax <= 448 s, exponent limited; 0 for 0."""
    m, e = torch.frexp(amax / CODE_MAX)
    e = torch.where(m == 0.5, e - 1, e).clamp(MIN_EXP, MAX_EXP)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _append_plain(s):
    """The new codes are scattered; the page that a request's first new token
    goes to is gathered, rounded again where its scale grew, and put back."""
    k, v, starts, lens = s["k"], s["v"], s["token_starts"].long(), s["lens"].long()
    pool, scales, bt = s["kv_pages"], s["kv_scales"], s["block_table"].long()
    t = torch.arange(k.shape[0], device=k.device)
    req = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[req] - (starts[req + 1] - t)
    page, slot = bt[req, pos // PAGE], pos % PAGE
    x = torch.stack([k, v], 1).float()                             # [T, 2, H, D]
    need = _need_scale(torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax"))
    new = starts[1:] - starts[:-1]
    some = torch.nonzero(new)[:, 0]                                # requests with new tokens
    first = lens[some] - new[some]
    part, had = bt[some, first // PAGE], first % PAGE              # their first page
    old = torch.zeros_like(scales)
    old[part] = torch.where((had > 0)[:, None, None], scales[part], 0.0)
    grown = torch.maximum(old, need)
    grown = torch.where(grown > 0, grown, 2.0 ** MIN_EXP)
    codes = pool[part].view(torch.float8_e4m3fn).float()
    again = (codes * (old / grown)[part][..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    earlier = torch.arange(PAGE, device=k.device)[None, :] < had[:, None]
    change = earlier[:, None, None, :, None] & (old != grown)[part][..., None, None]
    pool[part] = torch.where(change, again, pool[part])
    y = (x / grown[page][..., None]).clamp(-CODE_MAX, CODE_MAX)
    pool[page, :, :, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    scales[page] = grown[page]


def _attention_plain(q, visible, s):
    """q [N, Q, H, D], visible [N, Q] positions each query sees."""
    n, nq, h, d = q.shape
    pool, bt = s["kv_pages"], s["block_table"].long().clamp(min=0)
    hk = pool.shape[2]
    length = bt.shape[1] * PAGE
    at = torch.arange(length, device=q.device)
    kv = pool[bt].view(torch.float8_e4m3fn).float() * s["kv_scales"][bt][..., None, None]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, n, hk, length, d)
    kv = torch.where((at < s["lens"][:, None])[None, :, None, :, None], kv, torch.zeros_like(kv))
    qg = q.float().view(n, nq, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    sc = torch.matmul(qg, kv[0].transpose(-1, -2)).mul_(s["scale"])
    seen = (at[None, None, :] < visible[:, :, None])[:, None, :, None, :]
    sc = sc.view(n, hk, nq, h // hk, length).masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hk, -1, length), kv[1]).view(n, hk, nq, h // hk, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + l.log())[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(n, nq, h, d).to(torch.bfloat16),
            lse.permute(0, 2, 1, 3).reshape(n, nq, h))


def _decode_plain(s):
    n, nq = s["q"].shape[:2]
    visible = s["lens"][:, None] - nq + 1 + torch.arange(nq, device=s["q"].device)
    return _attention_plain(s["q"], visible, s)


def _prefill_plain(s):
    q, starts = s["q"], s["token_starts"].long()
    i = torch.arange(s["max_new"], device=q.device)
    new = starts[1:] - starts[:-1]
    there = i < new[:, None]
    rows = torch.where(there, starts[:-1, None] + i, torch.zeros_like(there, dtype=torch.long))
    visible = torch.where(there, s["lens"][:, None] - new[:, None] + 1 + i, 0)
    o, lse = _attention_plain(q[rows], visible, s)
    t = torch.arange(q.shape[0], device=q.device)
    req = torch.searchsorted(starts, t, right=True) - 1
    return o[req, t - starts[req]], lse[req, t - starts[req]]


def _lowest_free(refs):
    return torch.argsort((refs != 0).to(torch.uint8), stable=True)


def _beam_plain(s):
    refs, bt, lens = s["refcounts"], s["block_table"], s["lens"]
    pages, width = refs.shape[0], bt.shape[1]
    par, ch = s["parents"].long(), s["children"].long()
    j = torch.arange(width, device=bt.device)[None, :]

    def count(entries, held, by):
        at = torch.where(held, entries.long(), pages).flatten()
        padded = torch.cat([refs, refs.new_zeros(1)])
        padded.index_add_(0, at, torch.full_like(at, by, dtype=torch.int32))
        refs.copy_(padded[:pages])

    # free the losers
    held = j < ((lens[ch] + PAGE - 1) // PAGE)[:, None]
    count(bt[ch], held, -1)
    bt[ch] = torch.where(held, torch.full_like(bt[ch], -1), bt[ch])
    lens[ch] = 0
    # fork the winners into their rows
    free = _lowest_free(refs).to(torch.int32)
    plen = lens[par]
    part = plen % PAGE != 0
    page = free[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    full = j < (plen // PAGE)[:, None]
    rows = torch.where(full, bt[par], bt[ch])
    rows = torch.where((j == (plen // PAGE)[:, None]) & part[:, None], page[:, None], rows)
    count(bt[par], full, 1)
    src = bt[par].gather(1, (plen // PAGE).long()[:, None].clamp(max=width - 1))[:, 0]
    src, dst = src[part].long(), page[part].long()
    refs[dst] = 1
    for pool in s["pools"]:
        pool[dst] = pool[src]
    # extend them
    have, want = (plen + PAGE - 1) // PAGE, (s["new_lens"] + PAGE - 1) // PAGE
    grow = want - have
    free = _lowest_free(refs).to(torch.int32)
    base = (torch.cumsum(grow, 0) - grow)[:, None]
    new = (j >= have[:, None]) & (j < want[:, None])
    got = free[(base + j - have[:, None]).clamp(0, pages - 1).long()]
    rows = torch.where(new, got, rows)
    count(rows, new, 1)
    bt[ch] = rows
    lens[ch] = s["new_lens"]


def _compact_plain(s):
    refs, bt, lens = s["refcounts"], s["block_table"], s["lens"]
    pages = refs.shape[0]
    live = refs > 0
    n = live.sum()
    at = torch.arange(pages, device=refs.device)
    src = torch.nonzero(live & (at >= n))[:, 0]
    dst = torch.nonzero(~live & (at < n))[:, 0]
    new_id = at.clone()
    new_id[src] = dst
    new_refs = refs.clone()
    new_refs[dst] = refs[src]
    new_refs[src] = 0
    held = torch.arange(bt.shape[1], device=bt.device) < ((lens + PAGE - 1) // PAGE)[:, None]
    new_bt = torch.where(held, new_id[bt.long().clamp(min=0)].to(torch.int32), bt)
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return new_bt, new_refs, n.to(torch.int32).view(1)


def run(s):
    op = s["op"]
    if own:
        import invariant_sparse_mla_gb300 as ds
    if op == "append":
        if own:
            ds.kv8_append(s["k"], s["v"], s["token_starts"], s["block_table"], s["lens"],
                          s["kv_pages"], s["kv_scales"])
        else:
            _append_plain(s)
        return s["kv_pages"].view(torch.float8_e4m3fn), s["kv_scales"]
    if op == "decode":
        if own:
            return ds.kv8_decode(s["q"], s["kv_pages"], s["kv_scales"], s["block_table"],
                                 s["lens"], s["scale"])
        return _decode_plain(s)
    if op == "prefill":
        if own:
            return ds.kv8_prefill(s["q"], s["token_starts"], s["kv_pages"], s["kv_scales"],
                                  s["block_table"], s["lens"], s["scale"])
        return _prefill_plain(s)
    if op == "copy":
        if own:
            ds.pages_copy(s["pools"], s["src"], s["dst"])
        else:
            for pool in s["pools"]:
                pool[s["dst"].long()] = pool[s["src"].long()]
        return s["pools"]
    if op == "beam":
        if own:
            ds.pages_free(s["refcounts"], s["block_table"], s["lens"], s["children"])
            ds.pages_fork(s["pools"], s["refcounts"], s["block_table"], s["lens"], s["parents"],
                          s["children"])
            ds.pages_extend(s["refcounts"], s["block_table"], s["lens"], s["children"],
                            s["new_lens"])
        else:
            _beam_plain(s)
        return s["block_table"], s["lens"], s["refcounts"], s["pools"]
    if own:
        got = ds.pages_compact(s["pools"], s["refcounts"], s["block_table"], s["lens"])
    else:
        got = _compact_plain(s)
    return got, s["pools"]


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    hk, d = case["kv_heads"], case["dim"]
    if op in ("append", "decode", "prefill"):
        lens, new = _lengths(case)
        tokens = int(new.sum())
        if op == "append":
            touched = (lens + PAGE - 1) // PAGE - (lens - new) // PAGE
            touched = int(torch.where(new > 0, touched, torch.zeros_like(touched)).sum())
            return {"bytes": max(1, tokens * 2 * hk * d * 3 + touched * 2 * hk * 4), "flops": 0}
        h = case["heads"]
        span = (lens - new + 1).clamp(min=0) + lens.clamp(min=0)
        seen = torch.where(lens >= new, span * new // 2, lens * (lens + 1) // 2)
        byt = int(lens.sum()) * 2 * hk * d + tokens * h * (4 * d + 4)
        return {"bytes": max(1, byt), "flops": 4 * h * d * int(seen.sum())}
    page = case["layers"] * (2 * hk * PAGE * d + 2 * hk * 4)
    if op == "copy":
        return {"bytes": 2 * page * case["copies"], "flops": 0}
    if op == "beam":
        lens, parents, _ = _beam_plan(case)
        held = lens[parents]
        entries = int(_pages_of(held).sum())
        return {"bytes": 2 * page * int((held % PAGE != 0).sum()) + entries * 4 * 5
                + case["pages"] * 4, "flops": 0}
    lens = _between(_host(case), case["ctx_lo"], case["ctx_hi"], case["rows"])
    held = int(_pages_of(lens).sum())
    if case["rows"] > 1:
        held -= int(min(lens[0], lens[1])) // PAGE // 2
    # Pages lie at random: the share of the live ones behind the first `held`.
    moved = held * (case["pages"] - held) // case["pages"]
    return {"bytes": 2 * page * moved + case["rows"] * int(_pages_of(lens).max()) * 8
            + case["pages"] * 8, "flops": 0}


# ------------------------------------------------------------------ exact
def _exact_append(s):
    """Page by page from the definition: scale by search over powers of two,
    codes by distance to the representable values."""
    grid = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    grid = grid[torch.isfinite(grid)].unique()                     # ascending, one zero

    def near(y):
        y = y.clamp(-CODE_MAX, CODE_MAX)
        i = torch.searchsorted(grid, y.contiguous()).clamp(1, grid.numel() - 1)
        lo, hi = grid[i - 1], grid[i]
        below = (y - lo) < (hi - y)
        tie = (y - lo) == (hi - y)
        step = hi - lo                                              # a tie goes to the even multiple
        even = torch.remainder(torch.div(lo, step), 2) == 0
        return torch.where(tie, torch.where(even, lo, hi), torch.where(below, lo, hi))

    pool = s["kv_pages"].view(torch.float8_e4m3fn).double()
    scales = s["kv_scales"].double()
    starts, lens, bt = s["token_starts"].tolist(), s["lens"].tolist(), s["block_table"].tolist()
    x = torch.stack([s["k"], s["v"]], 1).double()
    for r, length in enumerate(lens):
        n = starts[r + 1] - starts[r]
        first = length - n
        for b in range(first // PAGE, (length + PAGE - 1) // PAGE) if n else ():
            lo, hi = max(first, b * PAGE), min(length, (b + 1) * PAGE)
            new = x[starts[r] + lo - first: starts[r] + hi - first]      # [m, 2, H, D]
            p, had = bt[r][b], lo - b * PAGE
            amax = new.abs().amax((0, 3))
            want = torch.zeros_like(amax)
            # 448 * 2^e covers amax for the first e from below
            e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / CODE_MAX))
            e = torch.where(CODE_MAX * torch.exp2(e - 1) >= amax, e - 1, e)
            e = torch.where(CODE_MAX * torch.exp2(e) < amax, e + 1, e).clamp(MIN_EXP, MAX_EXP)
            want = torch.where(amax > 0, torch.exp2(e), want)
            old = scales[p] if had else torch.zeros_like(want)
            s_new = torch.maximum(old, want)
            s_new = torch.where(s_new > 0, s_new, torch.full_like(s_new, 2.0 ** MIN_EXP))
            if had:
                again = near(pool[p, :, :, :had] * (old / s_new)[..., None, None])
                keep = (old == s_new)[..., None, None]
                pool[p, :, :, :had] = torch.where(keep, pool[p, :, :, :had], again)
            pool[p, :, :, had:had + hi - lo] = near(new.permute(1, 2, 0, 3) / s_new[..., None, None])
            scales[p] = s_new
    return pool, scales


def _exact_attention(s, visible_of):
    q = s["q"].reshape(-1, *s["q"].shape[-2:])
    h, d = q.shape[1:]
    hk = s["kv_pages"].shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    starts, lens = s["token_starts"].tolist(), s["lens"].tolist()
    for r, length in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        if a == b or length <= 0:
            continue
        pg = s["block_table"][r, : (length + PAGE - 1) // PAGE].long()
        vis = visible_of(length, b - a).to(q.device)
        for g in range(hk):
            codes = s["kv_pages"][pg, :, g].view(torch.float8_e4m3fn).double()
            val = codes * s["kv_scales"][pg, :, g].double()[..., None, None]
            key, value = (val[:, i].reshape(-1, d)[:length] for i in (0, 1))
            for c in range(a, b, 256):
                e = min(b, c + 256)
                z = torch.einsum("qhd,kd->qhk", q[c:e, g * (h // hk):(g + 1) * (h // hk)].double(), key)
                z *= s["scale"]
                hide = torch.arange(length, device=q.device)[None, :] >= vis[c - a: e - a, None]
                z.masked_fill_(hide[:, None, :], -math.inf)
                ls = torch.logsumexp(z, -1)
                w = torch.exp(z - torch.where(ls > -math.inf, ls, torch.zeros_like(ls))[..., None])
                out[c:e, g * (h // hk):(g + 1) * (h // hk)] = torch.einsum("qhk,kd->qhd", w, value)
                lse[c:e, g * (h // hk):(g + 1) * (h // hk)] = ls
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def exact(case, seed):
    """The append and the attentions; what the page operations give is whole."""
    if case["op"] not in ("append", "decode", "prefill"):
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attention(s, lambda length, n: length - n + 1 + torch.arange(n))

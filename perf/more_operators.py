"""What is measured of the operators around the 8-bit cache of a serving step.

Operators: per-head norms of queries and keys with the position rotation
(``qk_norm_rope``), attention of a tree of drafted tokens over the cache
(``kv8_tree_decode``), the bookkeeping after drafts were verified
(``kv8_accept`` and ``pages_shrink``), the attention weight that positions have
received (``kv8_mass``) and eviction by it (``kv8_evict``).

The cache of one layer is ``kv_pages`` uint8 [pages, 2, kv_heads, 64, dim]
(E4M3 codes; index 0 of the second axis keys, 1 values) with ``kv_scales``
float32 [pages, 2, kv_heads]: a value is its code times the scale of its page,
side and head. Sizes are those of the repository's serving workloads (pages of
64, contexts of 1024 and 4096-32768, 32 requests, latent rows of 512 + 64 dims
under 128 heads) or generic ones.
"""

import math

import torch

own = False

PAGE = 64
CODE_MAX = 448.0              # largest finite E4M3 magnitude
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of two requests of a small model: latency is everything.
        dict(name="rope_step", op="rope", tokens=2, heads=16, kv_heads=2, dim=64, norm=64, rot=64,
             rot_start=0, pairs=False, q_norm=True, max_pos=4096),
        # Prompts of a batch: every head normed, the whole head rotated.
        dict(name="rope_prompt", op="rope", tokens=16384, heads=64, kv_heads=8, dim=128, norm=128,
             rot=128, rot_start=0, pairs=False, q_norm=True, max_pos=131072),
        # Latent rows: the 512 latent dims normed, the last 64 rotated by
        # neighbouring pairs; the queries are rotated only.
        dict(name="rope_latent", op="rope", tokens=4095, heads=128, kv_heads=1, dim=576, norm=512,
             rot=64, rot_start=512, pairs=True, q_norm=False, max_pos=65536),
        # The smallest draft tree, where latency counts.
        dict(name="tree_small", op="tree", reqs=2, nodes=8, heads=16, kv_heads=2, dim=64,
             ctx_lo=1024, ctx_hi=1024),
        # A serving batch that drafts trees of 24 tokens.
        dict(name="tree_batch", op="tree", reqs=16, nodes=24, heads=64, kv_heads=8, dim=128,
             ctx_lo=4096, ctx_hi=32768),
        # Room for the drafts, the accepted ones moved, the rest given back.
        dict(name="accept_small", op="accept", reqs=4, nodes=8, width=4, layers=2, kv_heads=2,
             dim=64, ctx_lo=200, ctx_hi=2000),
        # The same for a large batch of wide trees over several layers.
        dict(name="accept_large", op="accept", reqs=128, nodes=64, width=16, layers=6, kv_heads=8,
             dim=128, ctx_lo=500, ctx_hi=4000),
        # One decode step's weights over a serving batch.
        dict(name="mass_step", op="mass", reqs=32, lo=1, hi=1, heads=64, kv_heads=8, dim=128,
             ctx_lo=4096, ctx_hi=32768),
        # A chunk of a long prompt.
        dict(name="mass_chunk", op="mass", reqs=1, lo=2048, hi=2048, heads=64, kv_heads=8, dim=128,
             ctx_lo=32768, ctx_hi=32768),
        # Ragged prompts, head groups of 7.
        dict(name="mass_ragged", op="mass", reqs=12, lo=1, hi=1500, heads=28, kv_heads=4, dim=64,
             ctx_lo=1500, ctx_hi=5000),
        # A few short requests held to 512 positions.
        dict(name="evict_small", op="evict", reqs=4, kv_heads=2, dim=64, ctx_lo=400, ctx_hi=2000,
             budget=512, first=4, recent=64),
        # A serving batch held to 4096 positions.
        dict(name="evict_large", op="evict", reqs=32, kv_heads=8, dim=128, ctx_lo=4096,
             ctx_hi=32768, budget=4096, first=4, recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "accept", "mass", "mass", "evict"])
    kv_heads, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256, 576])
        norm = rng.choice([0, dim, dim, dim // 2])
        rot = rng.choice([r for r in (16, 32, 64, 128, 192, 256) if r <= dim])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
        most = max(2, 16384 * 72 * 128 // ((heads + kv_heads) * dim))
        return dict(op=op, tokens=_log(rng, 1, min(16384, most)), heads=heads, kv_heads=kv_heads,
                    dim=dim, norm=norm, rot=rot, rot_start=rng.choice([0, dim - rot]),
                    pairs=rng.random() < 0.5, q_norm=rng.random() < 0.8,
                    max_pos=_log(rng, 100, 1000000))
    if op == "tree":
        ctx = _log(rng, 64, 60000)
        nodes = rng.choice([1, 2, 5, 8, 13, 16, 24, 33, 48, 64])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 7, 8])
        most = max(1, min(32, 16 * 24 * 64 * 16000 // (nodes * heads * ctx)))
        return dict(op=op, reqs=_log(rng, 1, most), nodes=nodes, heads=heads, kv_heads=kv_heads,
                    dim=dim, ctx_lo=rng.randint(nodes // 2, ctx), ctx_hi=ctx)
    if op == "accept":
        nodes, ctx = rng.choice([2, 5, 8, 16, 31, 64]), _log(rng, 64, 4000)
        return dict(op=op, reqs=_log(rng, 1, 128), nodes=nodes, width=rng.randint(1, min(nodes, 16)),
                    layers=rng.randint(1, 6), kv_heads=kv_heads, dim=dim, ctx_lo=rng.randint(0, ctx),
                    ctx_hi=ctx)
    if op == "mass":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
        if rng.random() < 0.4:
            ctx, hi = _log(rng, 16, 60000), rng.choice([1, 1, 2, 5, 16])
            reqs = _log(rng, 1, max(1, min(64, 600000 // ctx)))
        else:
            hi = _log(rng, 2, 2000)
            ctx = hi + _log(rng, 1, 12000)
            reqs = _log(rng, 1, max(1, min(12, 6000 // hi)))
        return dict(op=op, reqs=reqs, lo=rng.randint(0 if reqs > 5 else 1, hi), hi=hi, heads=heads,
                    kv_heads=kv_heads, dim=dim, ctx_lo=min(hi, ctx), ctx_hi=max(hi, ctx))
    budget = _log(rng, 16, 6000)
    ctx = _log(rng, budget + 1, 30000)
    first = rng.choice([0, 0, 1, 4, 8])
    return dict(op=op, reqs=_log(rng, 1, max(1, min(64, 4000000 // (kv_heads * ctx)))),
                kv_heads=kv_heads, dim=dim, ctx_lo=rng.randint(budget // 2, ctx), ctx_hi=ctx,
                budget=budget, first=first, recent=rng.randint(0, budget - first))


# ----------------------------------------------------------------- inputs
def _host(case):
    """A generator for the case's lengths: they follow from the case alone, so
    every seed has the same amount of work."""
    return torch.Generator().manual_seed(4711 + sum(v for v in case.values()
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
    if op == "tree":
        return ctx, torch.full((n,), case["nodes"])
    if op == "mass":
        new = _between(g, case["lo"], case["hi"], n)
        return torch.maximum(ctx, new), new
    return ctx, torch.zeros(n, dtype=torch.int64)


def _parents(case):
    """The draft trees: node 0 is the root, every other node has an earlier
    parent."""
    g = _host(case)
    n, m = case["reqs"], case["nodes"]
    u = torch.rand((n, m), generator=g)
    return (u * torch.arange(m)).long().clamp(max=m - 1)


def _masks(parents):
    """Bit i of mask j: node j is node i or one of its descendants."""
    n, m = parents.shape
    sees = torch.zeros((n, m, m), dtype=torch.bool)
    rows = torch.arange(n)
    for j in range(m):
        if j > 0:
            sees[:, j] = sees[rows, parents[:, j]]
        sees[:, j, j] = True
    return sees


def _accept_plan(case):
    """Lengths before the drafts and the accepted nodes of every request (-1
    behind them): the way from the root to a random node, cut to `width`."""
    g = _host(case)
    n, m, w = case["reqs"], case["nodes"], case["width"]
    lens = _between(g, case["ctx_lo"], case["ctx_hi"], n)
    sees = _masks(_parents(case))
    node = torch.randint(0, m, (n,), generator=g)
    path = sees[torch.arange(n), node]                              # [n, m]
    at = torch.where(path, torch.arange(m)[None, :], m)
    at = torch.sort(at, 1).values[:, :w]
    return lens, torch.where(at < m, at, -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, d, hk = case["op"], case["dim"], case["kv_heads"]
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        # Queries and keys as slices of one fused projection's output.
        x = torch.randn((t, (h + 2 * hk) * d), generator=gen, device=dev)
        x *= torch.exp(0.5 * torch.randn((t, 1), generator=gen, device=dev))
        x = x.to(torch.bfloat16)
        st = dict(op=op, q=x[:, : h * d].unflatten(1, (h, d)),
                  k=x[:, h * d: (h + hk) * d].unflatten(1, (hk, d)),
                  positions=torch.randint(0, case["max_pos"], (t,), generator=gen, device=dev,
                                          dtype=torch.int32),
                  inv_freq=(1e6 ** (-torch.arange(0, case["rot"], 2, device=dev).double()
                                    / case["rot"])).float(),
                  norm=case["norm"], rot_start=case["rot_start"], pairs=case["pairs"])
        for name, there in (("q_weight", case["q_norm"]), ("k_weight", True)):
            w = 1.0 + 0.2 * torch.randn(case["norm"], generator=gen, device=dev)
            st[name] = w.to(torch.bfloat16) if there and case["norm"] else None
        return st
    if op == "accept":
        lens, accepted = _accept_plan(case)
        full = lens + case["nodes"]
        width, pages = int(_pages_of(full).max()), int(_pages_of(full).sum()) + 5
        st = dict(op=op, nodes=case["nodes"], lens=lens.to(dev, torch.int32),
                  rows=torch.arange(case["reqs"], device=dev, dtype=torch.int32),
                  full=full.to(dev, torch.int32), accepted=accepted.to(dev, torch.int32),
                  block_table=_tables(lens, width, pages, gen, dev))
        st["layers"] = [(_codes((pages, 2, hk, PAGE, d), gen, dev), _scales((pages, 2, hk), gen, dev))
                        for _ in range(case["layers"])]
        held = st["block_table"].flatten().long()
        refs = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
        refs.index_add_(0, torch.where(held >= 0, held, pages), torch.ones_like(held, dtype=torch.int32))
        st["refcounts"] = refs[:pages].clone()
        return st
    lens, new = _lengths(case)
    width, pages = max(1, int(_pages_of(lens).max())), int(_pages_of(lens).sum()) + 3
    st = dict(op=op, lens=lens.to(dev, torch.int32),
              block_table=_tables(lens, width, pages, gen, dev),
              kv_pages=_codes((pages, 2, hk, PAGE, d), gen, dev),
              kv_scales=_scales((pages, 2, hk), gen, dev))
    if op in ("mass", "evict"):
        # What earlier steps gave: a few positions got most of it, about as much in
        # all as this call adds.
        m = torch.exp(2.0 * torch.randn((case["reqs"], hk, width * PAGE), generator=gen, device=dev))
        if op == "mass":
            m *= 0.15 * case["heads"] / hk * case["hi"] / case["ctx_hi"]
        st["mass"] = m
    if op == "evict":
        st.update(budget=case["budget"], first=case["first"], recent=case["recent"])
        return st
    st["scale"] = 1.0 / math.sqrt(d)
    starts = torch.zeros(len(new) + 1, dtype=torch.int64)
    starts[1:] = torch.cumsum(new, 0)
    st["token_starts"] = starts.to(dev, torch.int32)
    q = 2.5 * torch.randn((int(starts[-1]), case["heads"], d), generator=gen, device=dev)
    st["q"] = q.to(torch.bfloat16)
    st["max_new"] = int(new.max())
    if op == "tree":
        st["q"] = st["q"].view(case["reqs"], case["nodes"], case["heads"], d)
        bits = torch.ones(1, dtype=torch.int64) << torch.arange(case["nodes"])
        st["masks"] = (_masks(_parents(case)) * bits).sum(-1).to(dev)
    # What the last pages hold behind the last position is whatever their
    # previous owners left, NaN codes among it.
    last = (lens - 1).clamp(min=0)
    page = st["block_table"].gather(1, (last // PAGE).to(dev)[:, None]).long()[:, 0].clamp(min=0)
    behind = torch.arange(PAGE)[None, :] > (last % PAGE)[:, None]
    tail = st["kv_pages"][page]
    tail.masked_fill_((behind.to(dev) & (st["lens"] > 0)[:, None])[:, None, None, :, None], 0x7F)
    st["kv_pages"][page] = tail
    if op == "mass":
        st["lse"] = _by_token(_weights_plain(st)[1], st)            # as attention gave it
    return st


# ------------------------------------------------------------ plain forms
def _rope_plain(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    got = []
    for name in ("q", "k"):
        x, w, n, a = s[name].float(), s[name + "_weight"], s["norm"], s["rot_start"]
        if w is not None:
            r = torch.rsqrt(x[..., :n].square().mean(-1, keepdim=True) + EPS)
            x = torch.cat([x[..., :n] * r * w.float(), x[..., n:]], -1)
        half = cos.shape[-1]
        rot = x[..., a: a + 2 * half]
        u, v = (rot[..., 0::2], rot[..., 1::2]) if s["pairs"] else (rot[..., :half], rot[..., half:])
        y = [u * cos - v * sin, v * cos + u * sin]
        y = torch.stack(y, -1).flatten(-2) if s["pairs"] else torch.cat(y, -1)
        got.append(torch.cat([x[..., :a], y, x[..., a + 2 * half:]], -1).to(torch.bfloat16))
    return got


def _cache_plain(s, sides):
    """Keys (and values) of every request [sides, N, Hk, L, D]; 0 behind its end."""
    pool, bt = s["kv_pages"][:, :sides], s["block_table"].long().clamp(min=0)
    hk, d, length = pool.shape[2], pool.shape[4], bt.shape[1] * PAGE
    kv = pool[bt].view(torch.float8_e4m3fn).float() * s["kv_scales"][:, :sides][bt][..., None, None]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(sides, bt.shape[0], hk, length, d)
    there = torch.arange(length, device=bt.device) < s["lens"][:, None]
    return torch.where(there[None, :, None, :, None], kv, torch.zeros_like(kv))


def _scores_plain(q, key, seen, scale):
    """q [N, Q, H, D], seen [N, Q, L] to scores [N, Hk, Q, G, L], -inf unseen."""
    n, nq, h, d = q.shape
    hk, length = key.shape[1], key.shape[2]
    qg = q.float().view(n, nq, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    sc = torch.matmul(qg, key.transpose(-1, -2)).mul_(scale)
    return sc.view(n, hk, nq, h // hk, length).masked_fill_(~seen[:, None, :, None, :], -math.inf)


def _tree_plain(s):
    q = s["q"]
    n, nq, h, d = q.shape
    key, value = _cache_plain(s, 2)
    at = torch.arange(key.shape[2], device=q.device)
    node = at[None, :] - (s["lens"][:, None] - nq)                  # [N, L] < 0: before the drafts
    bit = torch.bitwise_right_shift(s["masks"][:, :, None], node.clamp(0, 63)[:, None, :]) & 1
    seen = (node < 0)[:, None, :] | ((node < nq)[:, None, :] & (bit != 0))
    sc = _scores_plain(q, key, seen & (at < s["lens"][:, None])[:, None, :], s["scale"])
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    hk = key.shape[1]
    o = torch.matmul(p.view(n, hk, -1, key.shape[2]), value).view(n, hk, nq, h // hk, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + l.log())[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(n, nq, h, d).to(torch.bfloat16),
            lse.permute(0, 2, 1, 3).reshape(n, nq, h))


def _token_rows(s):
    """(which padded [N, Q] entries are tokens, their row of q)."""
    starts = s["token_starts"].long()
    i = torch.arange(s["max_new"], device=starts.device)
    new = starts[1:] - starts[:-1]
    there = i < new[:, None]
    return there, torch.where(there, starts[:-1, None] + i, torch.zeros_like(there, dtype=torch.long))


def _by_token(x, s):
    """[N, Q, ...] padded to [T, ...]."""
    starts = s["token_starts"].long()
    t = torch.arange(s["q"].shape[0], device=x.device)
    req = torch.searchsorted(starts, t, right=True) - 1
    return x[req, t - starts[req]].contiguous()


def _weights_plain(s):
    """Scores [N, Hk, Q, G, L] of the new tokens, and their lse [N, Q, H]."""
    there, rows = _token_rows(s)
    key, = _cache_plain(s, 1)
    new = there.sum(1, keepdim=True)
    i = torch.arange(s["max_new"], device=rows.device)
    visible = torch.where(there, s["lens"].long()[:, None] - new + 1 + i, 0)
    seen = torch.arange(key.shape[2], device=rows.device)[None, None, :] < visible[:, :, None]
    sc = _scores_plain(s["q"][rows], key, seen, s["scale"])
    lse = torch.logsumexp(sc, -1)
    return sc, lse.permute(0, 2, 1, 3).reshape(rows.shape[0], rows.shape[1], -1)


def _mass_plain(s):
    there, rows = _token_rows(s)
    key, = _cache_plain(s, 1)
    n, nq = rows.shape
    new = there.sum(1, keepdim=True)
    lens = s["lens"].long()[:, None]
    i = torch.arange(s["max_new"], device=rows.device)
    at = torch.arange(key.shape[2], device=rows.device)
    visible = torch.where(there, lens - new + 1 + i, 0)
    sc = _scores_plain(s["q"][rows], key, at[None, None, :] < visible[:, :, None], s["scale"])
    lse = s["lse"][rows].view(n, nq, key.shape[1], -1).permute(0, 2, 1, 3)
    got = sc.sub_(lse[..., None]).exp_().sum((2, 3))                 # [N, Hk, L]
    fresh = (at >= lens - new) & (at < lens)
    s["mass"].copy_(torch.where(fresh[:, None, :], got, s["mass"] + got))
    return s["mass"]


def _requantise(codes, ratio):
    """Codes [..., D] under a scale `1 / ratio` times their own."""
    y = (codes.view(torch.float8_e4m3fn).float() * ratio[..., None]).clamp(-CODE_MAX, CODE_MAX)
    y = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where((ratio == 1.0)[..., None], codes, y)


def _evict_plain(s):
    lens, bt, mass = s["lens"].long(), s["block_table"].long(), s["mass"]
    budget, first, recent = s["budget"], s["first"], s["recent"]
    pool, scales = s["kv_pages"], s["kv_scales"]
    hk = mass.shape[1]
    act = torch.nonzero(lens > budget)[:, 0]
    new_lens = lens.clamp(max=budget).to(torch.int32)
    at = torch.arange(mass.shape[2], device=lens.device)
    may = (at >= first) & (at < lens[act, None] - recent)
    ranked = torch.where(may[:, None, :], mass[act], -math.inf)
    ranked = torch.sort(ranked, dim=-1, descending=True, stable=True).indices
    top = torch.sort(ranked[..., : budget - first - recent], dim=-1).values
    ends = torch.arange(first, device=lens.device).expand(len(act), hk, first)
    late = (lens[act, None, None] - recent + torch.arange(recent, device=lens.device))
    kept = torch.cat([ends, top, late.expand(-1, hk, -1)], -1)       # [A, Hk, budget] ascending
    head = torch.arange(hk, device=lens.device)[None, :, None]
    row = act[:, None, None]
    page, slot = bt[row, kept // PAGE], kept % PAGE
    dst = torch.arange(budget, device=lens.device)
    to = bt[row, (dst // PAGE)[None, None, :].expand_as(kept)]
    codes = pool[page, :, head, slot]                                # [A, Hk, budget, 2, D]
    old = scales[page, :, head]                                      # [A, Hk, budget, 2]
    blocks = (budget + PAGE - 1) // PAGE
    by_page = old.new_zeros((len(act), hk, blocks * PAGE, 2))
    by_page[:, :, :budget] = old
    grown = by_page.view(len(act), hk, blocks, PAGE, 2).amax(3)
    codes = _requantise(codes, old / grown[:, :, dst // PAGE])
    moved = mass[act].gather(-1, kept)
    pool[to, :, head, (dst % PAGE)[None, None, :]] = codes
    scales[to, :, head] = grown[:, :, dst // PAGE]
    mass[act, :, :budget] = moved
    return new_lens


def _refs_add(refs, entries, held, by):
    at = torch.where(held, entries.long(), refs.shape[0]).flatten()
    padded = torch.cat([refs, refs.new_zeros(1)])
    padded.index_add_(0, at, torch.full_like(at, by, dtype=torch.int32))
    refs.copy_(padded[:-1])


def _accept_plain(s):
    refs, bt, lens, full, acc = (s[x] for x in ("refcounts", "block_table", "lens", "full", "accepted"))
    j = torch.arange(bt.shape[1], device=bt.device)[None, :]
    # room for the drafts
    have, want = _pages_of(lens)[:, None], _pages_of(full)[:, None]
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True).to(torch.int32)
    grow = want - have
    rank = torch.cumsum(grow, 0) - grow + j - have
    new = (j >= have) & (j < want)
    bt.copy_(torch.where(new, free[rank.clamp(0, refs.shape[0] - 1).long()], bt))
    _refs_add(refs, bt, new, 1)
    # the accepted ones move to the front: both pages that the drafts lie in
    base, count = full.long() - s["nodes"], (acc >= 0).sum(1)
    off = (base % PAGE)[:, None]
    two = (base // PAGE)[:, None] + torch.arange(2, device=bt.device)
    there = two < want
    page = bt.gather(1, two.clamp(max=bt.shape[1] - 1)).long()
    page = torch.where(there, page, page[:, :1])                      # [R, 2]
    at = torch.arange(2 * PAGE, device=bt.device)[None, :]
    nth = (at - off).clamp(0, acc.shape[1] - 1)
    src = torch.where(at < off, at, off + acc.long().gather(1, nth).clamp(min=0))
    held = at < off + count[:, None]                                  # [R, 128]
    row = torch.arange(len(base), device=bt.device)[:, None]
    from_page, to_page = page[row, src // PAGE], page[row, at.expand_as(src) // PAGE]
    put = torch.nonzero(held)
    r, l = put[:, 0], put[:, 1]
    for pool, scales in s["layers"]:
        old = scales[from_page]                                       # [R, 128, 2, H]
        grown = torch.where(held[..., None, None], old, 0.0).unflatten(1, (2, PAGE)).amax(2)
        codes = _requantise(pool[from_page, :, :, src % PAGE], old / grown.repeat_interleave(PAGE, 1))
        pool[to_page[r, l], :, :, l % PAGE] = codes[r, l]
        scales[to_page[r, l]] = grown[r, l // PAGE]
    # what the drafts no longer need goes back
    lens.copy_(base + count)
    gone = (j >= _pages_of(lens)[:, None]) & (j < want)
    _refs_add(refs, bt, gone, -1)
    bt.masked_fill_(gone, -1)


def run(s):
    op = s["op"]
    if own:
        import invariant_sparse_mla_gb300 as ds
    if op == "rope":
        if own:
            return ds.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"],
                                   s["k_weight"], eps=EPS, norm_dim=s["norm"],
                                   rot_start=s["rot_start"], interleaved=s["pairs"])
        return _rope_plain(s)
    if op == "accept":
        if own:
            ds.pages_extend(s["refcounts"], s["block_table"], s["lens"], s["rows"], s["full"])
            left = ds.kv8_accept(s["layers"], s["block_table"], s["lens"], s["nodes"], s["accepted"])
            ds.pages_shrink(s["refcounts"], s["block_table"], s["lens"], s["rows"], left)
        else:
            _accept_plain(s)
        return (s["block_table"], s["lens"], s["refcounts"],
                [(pool.view(torch.float8_e4m3fn), scales) for pool, scales in s["layers"]])
    if op == "tree":
        if own:
            return ds.kv8_tree_decode(s["q"], s["masks"], s["kv_pages"], s["kv_scales"],
                                      s["block_table"], s["lens"], s["scale"])
        return _tree_plain(s)
    if op == "mass":
        if own:
            return ds.kv8_mass(s["q"], s["lse"], s["token_starts"], s["kv_pages"], s["kv_scales"],
                               s["block_table"], s["lens"], s["scale"], s["mass"])
        return _mass_plain(s)
    if own:
        left = ds.kv8_evict(s["mass"], s["budget"], s["first"], s["recent"], s["kv_pages"],
                            s["kv_scales"], s["block_table"], s["lens"])
    else:
        left = _evict_plain(s)
    return left, s["mass"], s["kv_pages"].view(torch.float8_e4m3fn), s["kv_scales"]


# ------------------------------------------------------------------- work
def work(case):
    op, d, hk = case["op"], case["dim"], case["kv_heads"]
    if op == "rope":
        n = case["tokens"] * (case["heads"] + hk)
        return {"bytes": n * d * 4 + case["tokens"] * 4, "flops": n * (4 * case["norm"]
                                                                      + 3 * case["rot"])}
    if op == "accept":
        lens, acc = _accept_plan(case)
        moved = int(((acc >= 0) & (acc != torch.arange(acc.shape[1]))).sum())
        pages = _pages_of(lens + case["nodes"])
        return {"bytes": max(1, case["layers"] * moved * 2 * hk * d * 2 + acc.numel() * 4
                             + int(pages.sum()) * 4), "flops": 0}
    lens, new = _lengths(case)
    if op == "evict":
        act = lens[lens > case["budget"]]
        kept = len(act) * case["budget"] * 2 * hk * d
        return {"bytes": max(4 * len(lens), 2 * kept + int(act.sum()) * hk * 4
                             + len(act) * case["budget"] * hk * 4), "flops": 0}
    h = case["heads"]
    if op == "tree":
        seen = int((lens - new).clamp(min=0).sum()) * case["nodes"]
        seen += int(_masks(_parents(case)).sum())
        rows = case["reqs"] * case["nodes"]
        return {"bytes": int(lens.sum()) * 2 * hk * d + rows * (h * (4 * d + 4) + 8),
                "flops": 4 * h * d * seen}
    span = (lens - new + 1) + lens
    seen = int((span * new // 2).sum())
    return {"bytes": max(1, int(torch.where(new > 0, lens, 0).sum()) * hk * (d + 8)
                         + int(new.sum()) * h * (2 * d + 4)), "flops": 2 * h * d * seen}


# ------------------------------------------------------------------ exact
def _exact_rope(s):
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    n, a, half = s["norm"], s["rot_start"], s["inv_freq"].numel()
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double().clone()
        if w is not None:
            ms = (y[..., :n] ** 2).sum(-1, keepdim=True) / n
            y[..., :n] = y[..., :n] / torch.sqrt(ms + EPS) * w.double()
        part = y[..., a: a + 2 * half].clone()
        i = torch.arange(half, device=y.device)
        lo, hi = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + half)
        z = torch.complex(part[..., lo], part[..., hi]) * torch.polar(torch.ones_like(angle), angle)
        part[..., lo], part[..., hi] = z.real, z.imag
        y[..., a: a + 2 * half] = part
        got.append(y)
    return got


def _request_kv(s, r, length, g, sides):
    """Keys (and values) of head g of request r in 64 bits, [length, D] each."""
    pg = s["block_table"][r, : (length + PAGE - 1) // PAGE].long()
    codes = s["kv_pages"][pg, :sides, g].view(torch.float8_e4m3fn).double()
    val = codes * s["kv_scales"][pg, :sides, g].double()[..., None, None]
    return [val[:, i].reshape(-1, val.shape[-1])[:length] for i in range(sides)]


def _exact_tree(s):
    q, masks, lens = s["q"], s["masks"].tolist(), s["lens"].tolist()
    n, m, h, d = q.shape
    hk = s["kv_pages"].shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    for r, length in enumerate(lens):
        if length <= 0:
            continue
        sees = [[p < length - m or bool(masks[r][j] >> (p - length + m) & 1)
                 for p in range(max(0, length - m), length)] for j in range(m)]
        hide = ~torch.tensor(sees, device=q.device)
        for g in range(hk):
            key, value = _request_kv(s, r, length, g, 2)
            z = torch.einsum("qhd,kd->qhk", q[r, :, g * (h // hk):(g + 1) * (h // hk)].double(), key)
            z *= s["scale"]
            z[..., length - hide.shape[1]:].masked_fill_(hide[:, None, :], -math.inf)
            ls = torch.logsumexp(z, -1)
            w = torch.exp(z - torch.where(ls > -math.inf, ls, torch.zeros_like(ls))[..., None])
            out[r, :, g * (h // hk):(g + 1) * (h // hk)] = torch.einsum("qhk,kd->qhd", w, value)
            lse[r, :, g * (h // hk):(g + 1) * (h // hk)] = ls
    return out, lse


def _exact_mass(s):
    q, mass = s["q"], s["mass"].double()
    starts, lens = s["token_starts"].tolist(), s["lens"].tolist()
    hk, group = mass.shape[1], q.shape[1] // mass.shape[1]
    for r, length in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        if a == b or length <= 0:
            continue
        mass[r, :, max(0, length - (b - a)): length] = 0.0
        for g in range(hk):
            key, = _request_kv(s, r, length, g, 1)
            for c in range(a, b, 256):
                e = min(b, c + 256)
                z = torch.einsum("qhd,kd->qhk", q[c:e, g * group:(g + 1) * group].double(), key)
                z = z * s["scale"] - s["lse"][c:e, g * group:(g + 1) * group].double()[..., None]
                seen = length - (b - a) + 1 + torch.arange(c - a, e - a, device=q.device)
                hide = torch.arange(length, device=q.device)[None, :] >= seen[:, None]
                mass[r, g, :length] += z.masked_fill_(hide[:, None, :], -math.inf).exp_().sum((0, 1))
    return mass


def _nearest(y):
    """The E4M3 value next to y (64 bits), by distance; a tie goes to the even
    multiple of the step."""
    grid = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    grid = grid[torch.isfinite(grid)].unique()
    y = y.clamp(-CODE_MAX, CODE_MAX).contiguous()
    i = torch.searchsorted(grid, y).clamp(1, grid.numel() - 1)
    lo, hi = grid[i - 1], grid[i]
    even = torch.remainder(torch.div(lo, hi - lo), 2) == 0
    below = ((y - lo) < (hi - y)) | (((y - lo) == (hi - y)) & even)
    return torch.where(below, lo, hi)


def _move_exact(pool, scales, table, heads, kept):
    """Positions `kept` (ascending) to the front, for the given heads of one
    request: pool and scales in 64 bits."""
    src = [(table[p // PAGE], p % PAGE) for p in kept]
    pages = torch.tensor([p for p, _ in src], device=pool.device)
    slots = torch.tensor([t for _, t in src], device=pool.device)
    hs = torch.tensor(heads, device=pool.device)
    codes = pool[pages[:, None], :, hs[None, :], slots[:, None]]             # [n, H, 2, D]
    own_scale = scales[pages[:, None], :, hs[None, :]]                       # [n, H, 2]
    for b in range((len(kept) + PAGE - 1) // PAGE):
        lo, hi = b * PAGE, min(len(kept), (b + 1) * PAGE)
        if all(kept[i] == i for i in range(lo, hi)):
            continue
        top = own_scale[lo:hi].amax(0)
        page = table[b]
        value = _nearest(codes[lo:hi] * (own_scale[lo:hi] / top)[..., None])
        at = torch.arange(hi - lo, device=pool.device)
        pool[page][:, hs[None, :], at[:, None]] = value.permute(2, 0, 1, 3)
        scales[page][:, hs] = top.T


def _exact_evict(s):
    pool, scales = s["kv_pages"].view(torch.float8_e4m3fn).double(), s["kv_scales"].double()
    mass, budget = s["mass"].double(), s["budget"]
    table = s["block_table"].tolist()
    for r, length in enumerate(s["lens"].tolist()):
        if length <= budget:
            continue
        for g in range(mass.shape[1]):
            m = s["mass"][r, g].cpu()
            middle = range(s["first"], length - s["recent"])
            order = torch.sort(-m[s["first"]: length - s["recent"]], stable=True).indices.tolist()
            best = sorted(middle[i] for i in order[: budget - s["first"] - s["recent"]])
            kept = [*range(s["first"]), *best, *range(length - s["recent"], length)]
            _move_exact(pool, scales, table[r], [g], kept)
            mass[r, g, :budget] = m.double()[kept].to(mass.device)
    return None, mass, pool, scales


def _exact_accept(case, seed):
    """The caches after the call; the tables hold whole numbers. The drafts'
    pages are the lowest free ones, in the rows' order."""
    s = prepare(case, seed)
    lens, table = s["lens"].tolist(), s["block_table"].tolist()
    free = [p for p, c in enumerate(s["refcounts"].tolist()) if c == 0]
    layers = [(a.view(torch.float8_e4m3fn).double(), b.double()) for a, b in s["layers"]]
    heads = list(range(case["kv_heads"]))
    for r, length in enumerate(lens):
        for b in range((length + PAGE - 1) // PAGE, (length + case["nodes"] + PAGE - 1) // PAGE):
            table[r][b] = free.pop(0)
        kept = [length + a for a in s["accepted"][r].tolist() if a >= 0]
        first = length // PAGE * PAGE                     # the page that the drafts begin in
        local = [p - first for p in [*range(first, length), *kept]]
        for pool, scales in layers:
            _move_exact(pool, scales, table[r][first // PAGE:], heads, local)
    return None, None, None, layers


def exact(case, seed):
    op = case["op"]
    if op == "accept":
        return _exact_accept(case, seed)
    s = prepare(case, seed)
    if op == "rope":
        return _exact_rope(s)
    if op == "tree":
        return _exact_tree(s)
    return _exact_mass(s) if op == "mass" else _exact_evict(s)

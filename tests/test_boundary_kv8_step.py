"""Refusals of the norm with rotation, the draft tree, accepted drafts, mass,
eviction and shrinking, on the host: bad arguments are rejected, with a message
that names the parameter, before anything reaches the CUDA runtime."""

import ctypes

import pytest
import torch

from harness import ensure_built
from test_boundary import (A, DS_ERR_ALIGN, DS_ERR_NULL, DS_ERR_SHAPE, DS_ERR_UNSUPPORTED,
                           DS_ERR_WORKSPACE, DS_OK, host_only)
from test_boundary_kv8 import DECODE, PREFILL, STATE, _call, _msg


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


@pytest.fixture(scope="module")
def L(ds):
    return ds.lib()


class Layer(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


def _layers(*pairs):
    return ctypes.cast((Layer * len(pairs))(*[Layer(a, b) for a, b in pairs]), ctypes.c_void_p)


CACHE = dict(pages=16, bt=A, bts=4, lens=A, N=2, hk=2, d=128)
TREE = {"q": A, "qs": 1024, "masks": A, **{k: v for k, v in DECODE.items() if k not in ("q", "qs")}}
MASS = dict(q=A, qs=1024, lse=A, T=10, starts=A, N=2, kv=A, sc=A, pages=16, bt=A, bts=4, lens=A, h=8,
            hk=2, d=128, scale=0.1, mass=A, ms=256, err=None)
ACCEPT = dict(layers=_layers((A, A)), nl=1, pages=16, bt=A, bts=4, lens=A, N=2, hk=2, d=128, nn=8,
              acc=A, width=4, new=A + 64, err=None)
EVICT = dict(mass=A, ms=256, budget=100, first=4, recent=10, kv=A, sc=A, pages=16, refs=None, bt=A,
             bts=4, lens=A, N=2, hk=2, d=128, new=A + 64, ws=A, wsb=1 << 40, err=None)
ROPE = dict(q=A, qs=1024, h=8, qw=A, k=A, ks=256, hk=2, kw=A, T=10, d=128, nd=128, eps=1e-6, pos=A,
            freq=A, rs=0, rd=64, inter=0, qo=A, qos=1024, ko=A, kos=256)


def _bad(L, name, base):
    def bad(status, word, **kw):
        assert _call(L, name, base, **kw) == status and word in _msg(L), (kw, _msg(L))
    return bad


@host_only
@pytest.mark.parametrize("name,base", [("ds_kv8_tree_decode", TREE), ("ds_kv8_mass", MASS),
                                       ("ds_kv8_accept", ACCEPT), ("ds_kv8_evict", EVICT)])
def test_cache_arguments(L, name, base):
    bad = _bad(L, name, base)
    bad(DS_ERR_UNSUPPORTED, "head_dim=96", d=96)
    bad(DS_ERR_UNSUPPORTED, "num_kv_heads=0", hk=0)
    bad(DS_ERR_SHAPE, "num_pages=0", pages=0)
    bad(DS_ERR_SHAPE, "bt_stride=0", bts=0)
    bad(DS_ERR_UNSUPPORTED, "bt_stride", bts=1 << 26)
    bad(DS_ERR_SHAPE, "num_requests=-1", N=-1)
    bad(DS_ERR_ALIGN, "err_flag", err=A + 2)
    for p in ("bt", "lens"):
        bad(DS_ERR_NULL, "is NULL", **{p: None})
    assert _call(L, name, base, N=0) == DS_OK


@host_only
def test_tree(L):
    bad = _bad(L, "ds_kv8_tree_decode", TREE)
    bad(DS_ERR_NULL, "masks", masks=None)
    bad(DS_ERR_ALIGN, "masks", masks=A + 4)
    bad(DS_ERR_UNSUPPORTED, "next_n=65", nn=65)
    bad(DS_ERR_UNSUPPORTED, "next_n=0", nn=0)
    bad(DS_ERR_WORKSPACE, "workspace_bytes=8", wsb=8)
    assert PREFILL["scale"] == TREE["scale"]


@host_only
def test_mass(L):
    bad = _bad(L, "ds_kv8_mass", MASS)
    bad(DS_ERR_SHAPE, "mass_stride=255", ms=255)
    bad(DS_ERR_UNSUPPORTED, "bt_stride", bts=(1 << 20) + 1, ms=1 << 40)
    bad(DS_ERR_SHAPE, "num_tokens=-1", T=-1)
    bad(DS_ERR_UNSUPPORTED, "num_tokens", T=1 << 24, h=1024, qs=131072)
    bad(DS_ERR_SHAPE, "q_stride=1020", qs=1020)
    bad(DS_ERR_SHAPE, "scale", scale=float("nan"))
    bad(DS_ERR_UNSUPPORTED, "num_heads=7", h=7)
    for p, word in (("q", "q"), ("lse", "lse"), ("mass", "mass"), ("starts", "token_starts"),
                    ("kv", "kv_pages"), ("sc", "kv_scales")):
        bad(DS_ERR_NULL, word, **{p: None})
    bad(DS_ERR_ALIGN, "mass", mass=A + 2)
    assert _call(L, "ds_kv8_mass", MASS, T=0, q=None) == DS_OK


@host_only
def test_accept(L):
    bad = _bad(L, "ds_kv8_accept", ACCEPT)
    bad(DS_ERR_UNSUPPORTED, "num_layers=0", nl=0)
    bad(DS_ERR_UNSUPPORTED, "num_layers=129", nl=129)
    bad(DS_ERR_UNSUPPORTED, "next_n=65", nn=65)
    bad(DS_ERR_SHAPE, "width=9", width=9)
    bad(DS_ERR_SHAPE, "width=0", width=0)
    bad(DS_ERR_NULL, "layers is NULL", layers=None)
    bad(DS_ERR_NULL, "layers[0].kv_pages", layers=_layers((None, A)))
    bad(DS_ERR_NULL, "layers[1].kv_scales", layers=_layers((A, A), (A + 64, None)), nl=2)
    bad(DS_ERR_ALIGN, "layers[0]", layers=_layers((A + 8, A)))
    bad(DS_ERR_SHAPE, "same cache", layers=_layers((A, A), (A, A + 64)), nl=2)
    bad(DS_ERR_SHAPE, "same cache", layers=_layers((A, A), (A + 64, A)), nl=2)
    bad(DS_ERR_SHAPE, "new_lens", new=A)
    bad(DS_ERR_NULL, "accepted", acc=None)
    bad(DS_ERR_UNSUPPORTED, "num_requests", N=1 << 20, hk=1024)


@host_only
def test_evict(L):
    bad = _bad(L, "ds_kv8_evict", EVICT)
    bad(DS_ERR_SHAPE, "mass_stride=0", ms=0)
    bad(DS_ERR_SHAPE, "mass_stride=258", ms=258)
    bad(DS_ERR_SHAPE, "budget=0", budget=0, first=0, recent=0)
    bad(DS_ERR_SHAPE, "recent=97", recent=97)
    bad(DS_ERR_SHAPE, "first=-1", first=-1)
    bad(DS_ERR_UNSUPPORTED, "16385", budget=16385, first=0, recent=0)
    bad(DS_ERR_SHAPE, "new_lens", new=A)
    bad(DS_ERR_ALIGN, "mass", mass=A + 4)
    bad(DS_ERR_ALIGN, "refcounts", refs=A + 2)
    bad(DS_ERR_NULL, "workspace", ws=None)
    bad(DS_ERR_UNSUPPORTED, "num_requests=1048576", N=1 << 20, hk=128)
    need = L.ds_kv8_evict_workspace_size(2, 2, 256, 100, 4, 10)
    bad(DS_ERR_WORKSPACE, str(need), wsb=need - 1)
    assert need > 0
    for args in ((2, 2, 258, 100, 4, 10), (2, 0, 256, 100, 4, 10), (2, 2, 256, 100, 60, 50)):
        assert L.ds_kv8_evict_workspace_size(*args) == 0 and _msg(L)


@host_only
def test_norm_rope(L):
    bad = _bad(L, "ds_qk_norm_rope", ROPE)
    for d in (0, 8, 72, 1040):
        bad(DS_ERR_UNSUPPORTED, f"head_dim={d}", d=d)
    bad(DS_ERR_UNSUPPORTED, "num_q_heads=0", h=0)
    bad(DS_ERR_UNSUPPORTED, "num_k_heads=-1", hk=-1)
    bad(DS_ERR_SHAPE, "num_tokens=-1", T=-1)
    bad(DS_ERR_SHAPE, "norm_dim=136", nd=136)
    bad(DS_ERR_SHAPE, "norm_dim=4", nd=4)
    bad(DS_ERR_SHAPE, "norm_dim=0", nd=0)
    bad(DS_ERR_SHAPE, "rot_dim=24", rd=24)
    bad(DS_ERR_SHAPE, "rot_start=72", rs=72)
    bad(DS_ERR_SHAPE, "rot_start=4", rs=4)
    bad(DS_ERR_SHAPE, "rot_dim=144", rd=144)
    bad(DS_ERR_SHAPE, "eps", eps=-1.0)
    bad(DS_ERR_SHAPE, "eps", eps=float("nan"))
    for p in ("qs", "ks", "qos", "kos"):
        bad(DS_ERR_SHAPE, "_stride=12", **{p: 12})
    for p in ("q", "k", "pos", "freq", "qo", "ko"):
        bad(DS_ERR_NULL, "is NULL", **{p: None})
    for p in ("q", "k", "qw", "kw", "qo", "ko"):
        bad(DS_ERR_ALIGN, "16-byte", **{p: A + 8})
    assert _call(L, "ds_qk_norm_rope", ROPE, T=0, q=None) == DS_OK


@host_only
def test_shrink(L):
    form = {**STATE, "list": A, "new": A, "n": 3, "err": None}
    bad = _bad(L, "ds_pages_shrink", form)
    bad(DS_ERR_SHAPE, "num_pages=0", pages=0)
    bad(DS_ERR_SHAPE, "n=-1", n=-1)
    bad(DS_ERR_UNSUPPORTED, "65535", n=65536)
    bad(DS_ERR_NULL, "rows", list=None)
    bad(DS_ERR_NULL, "new_lens", new=None)
    bad(DS_ERR_ALIGN, "err_flag", err=A + 1)
    assert _call(L, "ds_pages_shrink", form, n=0) == DS_OK


def test_bindings_reject_cpu_tensors(ds):
    z = torch.zeros
    pages, scales = z(2, 2, 1, 64, 64, dtype=torch.uint8), z(2, 2, 1)
    i = z(1, dtype=torch.int32)
    q = z(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ds.qk_norm_rope(q, None, i, z(32))
    with pytest.raises(ValueError):
        ds.kv8_tree_decode(q[None], z(1, 1, dtype=torch.int64), pages, scales, i.view(1, 1), i, 0.1)
    with pytest.raises(ValueError):
        ds.kv8_mass(q, z(1, 4), z(2, dtype=torch.int32), pages, scales, i.view(1, 1), i, 0.1,
                    z(1, 1, 64))
    with pytest.raises(ValueError):
        ds.kv8_accept([(pages, scales)], i.view(1, 1), i, 1, i.view(1, 1))
    with pytest.raises(ValueError):
        ds.kv8_evict(z(1, 1, 64), 32, 0, 0, pages, scales, i.view(1, 1), i)
    with pytest.raises(ValueError):
        ds.pages_shrink(i, i.view(1, 1), i, i, i)


@host_only
def test_tree_workspace(L):
    """Its size changes with the form (rows of a kv head), and the call asks for it."""
    size = L.ds_kv8_tree_decode_workspace_size
    few, many = (2, 20, 8, 2, 128, 64), (2, 21, 8, 2, 128, 64)
    assert size(*few) == L.ds_kv8_decode_workspace_size(*few)
    # 4 spans at most (4096 positions) of 84 rows, for 2 requests x 2 kv heads
    assert size(*many) >= 2 * 2 * 4 * 84 * (128 * 4 + 8)
    for nn, need in ((20, size(*few)), (21, size(*many))):
        _bad(L, "ds_kv8_tree_decode", TREE)(DS_ERR_WORKSPACE, f"the {need} bytes needed", nn=nn, bts=64,
                                            wsb=need - 1)
    for i, (value, word) in enumerate([(-1, "num_requests"), (65, "next_n"), (9, "num_heads"),
                                       (0, "num_kv_heads"), (96, "head_dim"), (0, "bt_stride")]):
        args = list(many)
        args[i] = value
        assert size(*args) == 0 and word in _msg(L), (args, _msg(L))

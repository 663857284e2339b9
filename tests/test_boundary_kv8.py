"""Refusals of the block-scaled cache and page calls, on the host: bad
arguments are rejected, with a message that names the parameter, before
anything reaches the CUDA runtime."""

import ctypes

import pytest
import torch

from harness import ensure_built
from test_boundary import (A, DS_ERR_ALIGN, DS_ERR_NULL, DS_ERR_SHAPE, DS_ERR_UNSUPPORTED,
                           DS_ERR_WORKSPACE, DS_OK, host_only)


@pytest.fixture(scope="module")
def ds():
    return ensure_built()


@pytest.fixture(scope="module")
def L(ds):
    return ds.lib()


def _msg(L):
    return L.ds_last_error().decode()


def _call(L, name, defaults, **kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(L, name)(*a.values(), None)


APPEND = dict(k=A, v=A, ks=256, vs=256, T=10, starts=A, N=2, bt=A, bts=4, lens=A, hk=2, d=128,
              kv=A, sc=A, pages=16, err=None)
DECODE = dict(q=A, qs=1024, kv=A, sc=A, pages=16, bt=A, bts=4, lens=A, N=2, nn=1, h=8, hk=2, d=128,
              scale=0.1, out=A, lse=A, ws=A, wsb=1 << 40, err=None)
PREFILL = dict(q=A, qs=1024, T=10, starts=A, N=2, kv=A, sc=A, pages=16, bt=A, bts=4, lens=A, h=8,
               hk=2, d=128, scale=0.1, out=A, lse=A, ws=A, wsb=1 << 40, err=None)


@host_only
@pytest.mark.parametrize("name,base", [("ds_kv8_append", APPEND), ("ds_kv8_decode", DECODE),
                                       ("ds_kv8_prefill", PREFILL)])
def test_cache_calls_reject_bad_arguments(L, name, base):
    def bad(status, word, **kw):
        assert _call(L, name, base, **kw) == status and word in _msg(L), (kw, _msg(L))
    bad(DS_ERR_UNSUPPORTED, "head_dim=96", d=96)
    bad(DS_ERR_UNSUPPORTED, "num_kv_heads=0", hk=0)
    bad(DS_ERR_SHAPE, "num_pages=0", pages=0)
    bad(DS_ERR_UNSUPPORTED, "num_pages", pages=1 << 25)
    bad(DS_ERR_SHAPE, "bt_stride=0", bts=0)
    bad(DS_ERR_UNSUPPORTED, "bt_stride", bts=1 << 26)
    bad(DS_ERR_SHAPE, "num_requests=-1", N=-1)
    for p in ("kv", "sc", "bt", "lens"):
        bad(DS_ERR_NULL, "is NULL", **{p: None})
    bad(DS_ERR_ALIGN, "kv_pages", kv=A + 8)
    bad(DS_ERR_ALIGN, "err_flag", err=A + 2)
    if name == "ds_kv8_append":
        bad(DS_ERR_SHAPE, "k_stride=255", ks=255)
        bad(DS_ERR_SHAPE, "v_stride=128", vs=128)
        bad(DS_ERR_SHAPE, "num_tokens=-3", T=-3)
        bad(DS_ERR_NULL, "token_starts", starts=None)
        bad(DS_ERR_UNSUPPORTED, "num_tokens", T=1 << 24, N=1 << 20, hk=1024, ks=131072, vs=131072)
        bad(DS_ERR_ALIGN, "k must be 16-byte", k=A + 4)
        assert _call(L, name, base, T=0, k=None, v=None) == DS_OK
        return
    bad(DS_ERR_UNSUPPORTED, "num_heads=7", h=7)
    bad(DS_ERR_SHAPE, "q_stride=1020", qs=1020)
    bad(DS_ERR_SHAPE, "q_stride=512", qs=512)
    bad(DS_ERR_SHAPE, "scale", scale=float("inf"))
    bad(DS_ERR_NULL, "out is NULL", out=None)
    bad(DS_ERR_ALIGN, "out", out=A + 8)
    bad(DS_ERR_ALIGN, "workspace", ws=A + 64)
    if name == "ds_kv8_decode":
        bad(DS_ERR_UNSUPPORTED, "next_n=0", nn=0)
        bad(DS_ERR_UNSUPPORTED, "next_n=65", nn=65)
        bad(DS_ERR_UNSUPPORTED, "num_requests=1048576", N=1 << 20, nn=64, h=64, qs=8192)
        need = L.ds_kv8_decode_workspace_size(2, 1, 8, 2, 128, 4)
        bad(DS_ERR_WORKSPACE, str(need), wsb=need - 1)
        assert _call(L, name, base, N=0, q=None) == DS_OK
    else:
        bad(DS_ERR_SHAPE, "num_tokens=-1", T=-1)
        bad(DS_ERR_UNSUPPORTED, "num_tokens", T=1 << 24, h=1024, qs=131072)
        bad(DS_ERR_UNSUPPORTED, "bt_stride", bts=(1 << 20) + 1)
        bad(DS_ERR_NULL, "token_starts", starts=None)
        assert _call(L, name, base, T=0, q=None) == DS_OK


def test_cache_workspace_sizes_refuse(L):
    assert L.ds_kv8_decode_workspace_size(4, 1, 8, 2, 128, 100) > 0
    for args in ((4, 1, 8, 3, 128, 100), (4, 1, 8, 2, 32, 100), (4, 65, 8, 2, 128, 100),
                 (-1, 1, 8, 2, 128, 100), (4, 1, 8, 2, 128, 0)):
        assert L.ds_kv8_decode_workspace_size(*args) == 0 and _msg(L)


class Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("bytes", ctypes.c_int64)]


def _pool_array(*pools):
    arr = (Pool * len(pools))(*[Pool(p, b) for p, b in pools])
    return ctypes.cast(arr, ctypes.c_void_p)


STATE = dict(refs=A, pages=100, bt=A, bts=4, lens=A, rows=8)


def _pages(L, name, **kw):
    pools = dict(pools=kw.pop("pools", _pool_array((A, 64))), np=1)
    ws = dict(ws=A, wsb=1 << 30)
    form = {
        "ds_pages_copy": {**pools, "pages": 100, "src": A, "dst": A, "n": 3, "err": None},
        "ds_pages_free": {**STATE, "list": A, "n": 3, "err": None},
        "ds_pages_fork": {**pools, **STATE, "a": A, "list": A, "n": 3, **ws, "err": None},
        "ds_pages_extend": {**STATE, "list": A, "new": A, "n": 3, **ws, "err": None},
        "ds_pages_compact": {**pools, **STATE, "ro": A, "to": A, "nl": A, **ws, "err": None},
    }[name]
    return _call(L, name, form, **kw)


@host_only
def test_page_calls_reject_bad_arguments(L):
    for name in ("ds_pages_copy", "ds_pages_free", "ds_pages_fork", "ds_pages_extend",
                 "ds_pages_compact"):
        assert _pages(L, name, pages=0) == DS_ERR_SHAPE and "num_pages=0" in _msg(L)
        assert _pages(L, name, pages=(1 << 22) + 1) == DS_ERR_UNSUPPORTED and "2^22" in _msg(L)
        assert _pages(L, name, err=A + 1) == DS_ERR_ALIGN
        if name != "ds_pages_compact":
            assert _pages(L, name, n=-1) == DS_ERR_SHAPE and "n=-1" in _msg(L)
            assert _pages(L, name, n=65536) == DS_ERR_UNSUPPORTED and "65535" in _msg(L)
            assert _pages(L, name, n=0) == DS_OK
        if name != "ds_pages_copy":
            assert _pages(L, name, refs=None) == DS_ERR_NULL and "refcounts" in _msg(L)
            assert _pages(L, name, bts=0) == DS_ERR_SHAPE and "bt_stride" in _msg(L)
            assert _pages(L, name, rows=0) == DS_ERR_SHAPE and "num_rows" in _msg(L)
        if name in ("ds_pages_copy", "ds_pages_fork", "ds_pages_compact"):
            for pool, word in (((None, 64), "data is NULL"), ((A + 2, 64), "4-byte"),
                               ((A, 6), "page_bytes=6"), ((A, 0), "page_bytes=0")):
                assert _pages(L, name, pools=_pool_array(pool)) != DS_OK and word in _msg(L)
            assert _pages(L, name, np=129) == DS_ERR_UNSUPPORTED and "num_pools" in _msg(L)
        if name in ("ds_pages_fork", "ds_pages_extend", "ds_pages_compact"):
            assert _pages(L, name, ws=None) == DS_ERR_NULL and "workspace" in _msg(L)
            assert _pages(L, name, wsb=10) == DS_ERR_WORKSPACE
    assert _pages(L, "ds_pages_free", list=None) == DS_ERR_NULL and "rows" in _msg(L)
    assert _pages(L, "ds_pages_copy", src=None) == DS_ERR_NULL and "src" in _msg(L)


def test_bindings_reject_wrong_tensors(ds):
    z = torch.zeros
    pages, scales = z(2, 2, 1, 64, 64, dtype=torch.uint8), z(2, 2, 1)
    i = z(1, dtype=torch.int32)
    q = z(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):            # CPU tensors
        ds.kv8_decode(q, pages, scales, i.view(1, 1), i, 0.1)
    with pytest.raises(TypeError):             # codes are uint8
        ds.kv8_decode(q, pages.float(), scales, i.view(1, 1), i, 0.1)
    with pytest.raises(ValueError):
        ds.pages_free(i, i.view(1, 1), i, i)
    with pytest.raises(TypeError):
        ds.pages_copy([pages], i.long(), i)

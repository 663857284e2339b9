"""Pages of a paged cache: copy, free, fork, extend, compact.

Argument marshalling for the ds_pages_* calls (see include/ds_sparse_mla.h).
The state is ``refcounts`` int32 [num_pages], ``block_table`` int32
[rows, bt_stride] and ``lens`` int32 [rows] on the device; ``pools`` is a list
of the tensors that the pages index, each [num_pages, ...] and contiguous.
"""

import ctypes

import torch

from ._native import _need, lib
from .kv8 import _launch, _p


def pages_workspace_size(num_pages, n):
    return int(lib().ds_pages_workspace_size(num_pages, n))


def _pools(pools, num_pages, dev):
    """The pools as the C array {pointer, bytes of a page}."""
    words = []
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"pools[{i}] must be a torch.Tensor")
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"pools[{i}] must be on {dev}, got {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"pools[{i}] must be contiguous")
        if t.dim() < 1 or t.shape[0] != num_pages:
            raise ValueError(f"pools[{i}] must have {num_pages} pages as its first dim")
        words += (t.data_ptr(), t.numel() // num_pages * t.element_size())
    return (ctypes.c_int64 * max(1, len(words)))(*words)


def _state(refcounts, block_table, lens, err_flag):
    _need(refcounts, "refcounts", torch.int32, None, 1)
    dev = refcounts.device
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(lens, "lens", torch.int32, dev, 1)
    if lens.numel() != block_table.shape[0]:
        raise ValueError("lens must have one entry per block_table row")
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32, dev)
        if err_flag.numel() < 1:
            raise ValueError("err_flag must have an element")
    return dev


def _list(t, name, dev, n=None):
    _need(t, name, torch.int32, dev, 1)
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} entries")
    return t.numel()


def _workspace(workspace, num_pages, n, dev):
    if workspace is None:
        need = pages_workspace_size(num_pages, n)
        return torch.empty(need or 256, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    return workspace


def pages_copy(pools, src, dst, err_flag=None, stream=None):
    """Copy page ``src[i]`` to page ``dst[i]`` in every pool."""
    _need(src, "src", torch.int32, None, 1)
    dev = src.device
    n = _list(dst, "dst", dev, src.numel())
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32, dev)
    if not pools:
        return
    num_pages = pools[0].shape[0]
    _launch(dev, lib().ds_pages_copy, _pools(pools, num_pages, dev), len(pools), num_pages,
            _p(src), _p(dst), n, _p(err_flag), stream)


def pages_free(refcounts, block_table, lens, rows, err_flag=None, stream=None):
    """Give up everything the listed rows hold (in place)."""
    dev = _state(refcounts, block_table, lens, err_flag)
    n = _list(rows, "rows", dev)
    _launch(dev, lib().ds_pages_free, _p(refcounts), refcounts.numel(), _p(block_table),
            block_table.shape[1], _p(lens), block_table.shape[0], _p(rows), n, _p(err_flag),
            stream)


def pages_fork(pools, refcounts, block_table, lens, parents, children, workspace=None,
               err_flag=None, stream=None):
    """Make row ``children[i]`` (empty) a copy of row ``parents[i]``: full pages
    shared, a partly filled last page copied in every pool (in place)."""
    dev = _state(refcounts, block_table, lens, err_flag)
    n = _list(children, "children", dev, _list(parents, "parents", dev))
    num_pages = refcounts.numel()
    workspace = _workspace(workspace, num_pages, n, dev)
    _launch(dev, lib().ds_pages_fork, _pools(pools, num_pages, dev), len(pools), _p(refcounts),
            num_pages, _p(block_table), block_table.shape[1], _p(lens), block_table.shape[0],
            _p(parents), _p(children), n, _p(workspace), workspace.numel(), _p(err_flag), stream)


def pages_extend(refcounts, block_table, lens, rows, new_lens, workspace=None, err_flag=None,
                 stream=None):
    """Grow row ``rows[i]`` to ``new_lens[i]`` positions with free pages, lowest
    first (in place)."""
    dev = _state(refcounts, block_table, lens, err_flag)
    n = _list(new_lens, "new_lens", dev, _list(rows, "rows", dev))
    num_pages = refcounts.numel()
    workspace = _workspace(workspace, num_pages, n, dev)
    _launch(dev, lib().ds_pages_extend, _p(refcounts), num_pages, _p(block_table),
            block_table.shape[1], _p(lens), block_table.shape[0], _p(rows), _p(new_lens), n,
            _p(workspace), workspace.numel(), _p(err_flag), stream)


def pages_compact(pools, refcounts, block_table, lens, block_table_out=None, refcounts_out=None,
                  num_live=None, workspace=None, err_flag=None, stream=None):
    """Move the live pages to the front of every pool (pools in place; the
    outputs may be the inputs). Returns (block_table, refcounts, num_live)."""
    dev = _state(refcounts, block_table, lens, err_flag)
    num_pages = refcounts.numel()
    if block_table_out is None:
        block_table_out = torch.empty_like(block_table)
    if refcounts_out is None:
        refcounts_out = torch.empty_like(refcounts)
    if num_live is None:
        num_live = torch.empty(1, dtype=torch.int32, device=dev)
    _need(block_table_out, "block_table_out", torch.int32, dev, 2)
    _list(refcounts_out, "refcounts_out", dev, num_pages)
    _list(num_live, "num_live", dev, 1)
    if block_table_out.shape != block_table.shape:
        raise ValueError(f"block_table_out must be {tuple(block_table.shape)}")
    workspace = _workspace(workspace, num_pages, 0, dev)
    _launch(dev, lib().ds_pages_compact, _pools(pools, num_pages, dev), len(pools), _p(refcounts),
            num_pages, _p(block_table), block_table.shape[1], _p(lens), block_table.shape[0],
            _p(refcounts_out), _p(block_table_out), _p(num_live), _p(workspace),
            workspace.numel(), _p(err_flag), stream)
    return block_table_out, refcounts_out, num_live

"""Pages of a paged cache: copy, free, fork, extend, shrink, compact.

Argument marshalling for the ds_pages_* calls (see include/ds_sparse_mla.h).
The state is ``refcounts`` int32 [num_pages], ``block_table`` int32
[rows, bt_stride] and ``lens`` int32 [rows] on the device; ``pools`` is a list
of the tensors that the pages index, each [num_pages, ...] and contiguous. A
``stream`` argument runs the call, and what it allocates, on that stream instead
of the current one.
"""

import struct

import torch

from ._native import lib
from .kv8 import _arg, _device, _flag, _run, _scratch


def pages_workspace_size(num_pages, n):
    return int(lib().ds_pages_workspace_size(num_pages, n))


def _pools(pools, num_pages, dev):
    """The pools as the C array {pointer, bytes of a page}, packed."""
    if num_pages < 1:
        raise ValueError("the pools have no pages")
    words = []
    index = dev.index
    for t in pools:
        if (not isinstance(t, torch.Tensor) or t.get_device() != index or not t.is_contiguous()
                or t.dim() < 1 or t.shape[0] != num_pages):
            raise ValueError(f"every pool must be a contiguous tensor on {dev} with {num_pages} "
                             "pages as its first dim")
        words.append(t.data_ptr())
        words.append(t.nbytes // num_pages)
    return struct.pack(f"{len(words)}q", *words)


def _state(refcounts, block_table, lens):
    """(device, the state's arguments of the C calls)."""
    dev = _device(refcounts, "refcounts", torch.int32)
    _arg(refcounts, "refcounts", torch.int32, dev, 1)
    _arg(block_table, "block_table", torch.int32, dev, 2)
    _arg(lens, "lens", torch.int32, dev, 1)
    rows, width = block_table.shape
    if lens.shape[0] != rows:
        raise ValueError("lens must have one entry per block_table row")
    return dev, (refcounts.data_ptr(), refcounts.shape[0], block_table.data_ptr(), width,
                 lens.data_ptr(), rows)


def _list(t, name, dev, n=None):
    _arg(t, name, torch.int32, dev, 1)
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries")
    return t.shape[0]


def _workspace(workspace, refcounts, n):
    if workspace is None:
        need = lib().ds_pages_workspace_size(refcounts.shape[0], n)
        dev = refcounts.device
        workspace = _scratch(need or 256, dev, torch._C._cuda_getCurrentRawStream(dev.index))
        return workspace, workspace.data_ptr(), workspace.numel()
    _arg(workspace, "workspace", torch.uint8, refcounts.device)
    return workspace, workspace.data_ptr(), workspace.numel()


def pages_copy(pools, src, dst, err_flag=None, stream=None):
    """Copy page ``src[i]`` to page ``dst[i]`` in every pool."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return pages_copy(pools, src, dst, err_flag)
    dev = _device(src, "src", torch.int32)
    n = _list(dst, "dst", dev, _list(src, "src", dev))
    flag = _flag(err_flag, dev)
    if not pools:
        return
    first = pools[0]
    if not isinstance(first, torch.Tensor) or first.dim() < 1:
        raise TypeError("every pool must be a torch.Tensor of pages")
    num_pages = first.shape[0]
    _run(dev, lib().ds_pages_copy, _pools(pools, num_pages, dev), len(pools), num_pages,
         src.data_ptr(), dst.data_ptr(), n, flag)


def pages_free(refcounts, block_table, lens, rows, err_flag=None, stream=None):
    """Give up everything the listed rows hold (in place)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return pages_free(refcounts, block_table, lens, rows, err_flag)
    dev, state = _state(refcounts, block_table, lens)
    n = _list(rows, "rows", dev)
    _run(dev, lib().ds_pages_free, *state, rows.data_ptr(), n, _flag(err_flag, dev))


def pages_fork(pools, refcounts, block_table, lens, parents, children, workspace=None,
               err_flag=None, stream=None):
    """Make row ``children[i]`` (empty) a copy of row ``parents[i]``: full pages
    shared, a partly filled last page copied in every pool (in place)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return pages_fork(pools, refcounts, block_table, lens, parents, children, workspace,
                              err_flag)
    dev, state = _state(refcounts, block_table, lens)
    n = _list(children, "children", dev, _list(parents, "parents", dev))
    workspace, ws, ws_bytes = _workspace(workspace, refcounts, n)
    _run(dev, lib().ds_pages_fork, _pools(pools, refcounts.shape[0], dev), len(pools), *state,
         parents.data_ptr(), children.data_ptr(), n, ws, ws_bytes, _flag(err_flag, dev))


def pages_extend(refcounts, block_table, lens, rows, new_lens, workspace=None, err_flag=None,
                 stream=None):
    """Grow row ``rows[i]`` to ``new_lens[i]`` positions with free pages, lowest
    first (in place)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return pages_extend(refcounts, block_table, lens, rows, new_lens, workspace, err_flag)
    dev, state = _state(refcounts, block_table, lens)
    n = _list(new_lens, "new_lens", dev, _list(rows, "rows", dev))
    workspace, ws, ws_bytes = _workspace(workspace, refcounts, n)
    _run(dev, lib().ds_pages_extend, *state, rows.data_ptr(), new_lens.data_ptr(), n, ws, ws_bytes,
         _flag(err_flag, dev))


def pages_shrink(refcounts, block_table, lens, rows, new_lens, err_flag=None, stream=None):
    """Lower row ``rows[i]`` to ``new_lens[i]`` positions and give back the pages
    behind them (in place)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return pages_shrink(refcounts, block_table, lens, rows, new_lens, err_flag)
    dev, state = _state(refcounts, block_table, lens)
    n = _list(new_lens, "new_lens", dev, _list(rows, "rows", dev))
    _run(dev, lib().ds_pages_shrink, *state, rows.data_ptr(), new_lens.data_ptr(), n,
         _flag(err_flag, dev))


def pages_compact(pools, refcounts, block_table, lens, block_table_out=None, refcounts_out=None,
                  num_live=None, workspace=None, err_flag=None, stream=None):
    """Move the live pages to the front of every pool (pools in place; the
    outputs may be the inputs). Returns (block_table, refcounts, num_live)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return pages_compact(pools, refcounts, block_table, lens, block_table_out,
                                 refcounts_out, num_live, workspace, err_flag)
    dev, state = _state(refcounts, block_table, lens)
    num_pages = refcounts.shape[0]
    if block_table_out is None:
        block_table_out = torch.empty_like(block_table)
    else:
        _arg(block_table_out, "block_table_out", torch.int32, dev, 2)
        if block_table_out.shape != block_table.shape:
            raise ValueError(f"block_table_out must be {tuple(block_table.shape)}")
    if refcounts_out is None:
        refcounts_out = torch.empty_like(refcounts)
    else:
        _list(refcounts_out, "refcounts_out", dev, num_pages)
    if num_live is None:
        num_live = torch.empty(1, dtype=torch.int32, device=dev)
    else:
        _list(num_live, "num_live", dev, 1)
    workspace, ws, ws_bytes = _workspace(workspace, refcounts, 0)
    _run(dev, lib().ds_pages_compact, _pools(pools, num_pages, dev), len(pools), *state,
         refcounts_out.data_ptr(), block_table_out.data_ptr(), num_live.data_ptr(), ws, ws_bytes,
         _flag(err_flag, dev))
    return block_table_out, refcounts_out, num_live

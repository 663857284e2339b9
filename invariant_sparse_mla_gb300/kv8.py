"""The block-scaled 8-bit KV cache: append, decode and prefill attention.

Argument marshalling for ds_kv8_append / ds_kv8_decode / ds_kv8_prefill (see
include/ds_sparse_mla.h). The cache of one layer is ``kv_pages`` uint8
[num_pages, 2, kv_heads, 64, dim] (E4M3 codes, keys then values) with
``kv_scales`` float32 [num_pages, 2, kv_heads]; block tables are those of the
latent cache. A ``stream`` argument runs the call, and what it allocates, on
that stream instead of the current one.
"""

import threading

import torch

from ._native import _check, _need, lib


# Workspaces kept for the streams they were allocated on, by (device, raw
# stream): calls of one thread on one stream run in order, so they share one.
# (Each thread has its own: the launches of two calls could come in turn. An
# allocation between launches costs about 4 us on the host, half of a small
# call.) Larger ones than this, and those of calls that are being captured into
# a graph, are allocated anew.
_KEEP_BYTES = 64 << 20


class _Kept(threading.local):
    def __init__(self):
        self.by_stream = {}


_kept = _Kept()


def _scratch(need, dev, raw):
    """A workspace of at least ``need`` bytes for a call on ``raw``, the current
    stream."""
    if (need > _KEEP_BYTES or torch.cuda.current_device() != dev.index
            or torch.cuda.is_current_stream_capturing()):
        return torch.empty(need, dtype=torch.uint8, device=dev)
    key = (dev.index, raw)
    by_stream = _kept.by_stream
    kept = by_stream.get(key)
    if kept is None or kept.numel() < need:
        # (Dropping the smaller one is safe: its memory goes back to this stream.)
        kept = by_stream[key] = torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=dev)
    return kept


def _run(dev, fn, *args):
    """Calls fn(*args, the device's current stream) with ``dev`` current (the
    runtime launches only into streams of the current device)."""
    raw = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status:
        _check(status)


def _arg(t, name, dtype, dev, ndim=None):
    """``_need`` for the usual case in one expression: these calls take a few
    microseconds on the GPU, and the checks of their arguments should not take
    more."""
    if (type(t) is not torch.Tensor or t.dtype is not dtype or t.device != dev
            or not t.is_contiguous() or (ndim is not None and t.dim() != ndim)):
        _need(t, name, dtype, dev, ndim)


def _tokens(t, name, dtype, dev, lead):
    """A [*lead, heads, dim] tensor whose tokens are evenly strided and whose
    [heads, dim] part is contiguous; returns the stride between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dim() != lead + 2:
        raise ValueError(f"{name} must have {lead + 2} dims, got {t.dim()}")
    if t.is_contiguous():
        return t.shape[-1] * t.shape[-2]
    shape, stride = t.shape, t.stride()
    if (shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1]):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row = shape[-2] * shape[-1]
    if lead == 2:
        if shape[0] > 1 and shape[1] > 1 and stride[0] != shape[1] * stride[1]:
            raise ValueError(f"{name}: tokens must be evenly strided")
        return stride[1] if shape[1] > 1 else (stride[0] if shape[0] > 1 else row)
    return stride[0] if shape[0] > 1 else row


def _device(t, name, dtype):
    """The device of the tensor that the others have to share it with."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda:
        _need(t, name, dtype)
    return t.device


def _cache(kv_pages, kv_scales, dev):
    _arg(kv_pages, "kv_pages", torch.uint8, dev, 5)
    _arg(kv_scales, "kv_scales", torch.float32, dev, 3)
    pages, two, hk, page, d = kv_pages.shape
    if two != 2 or page != 64:
        raise ValueError("kv_pages must be [num_pages, 2, kv_heads, 64, dim] codes, got "
                         f"{tuple(kv_pages.shape)}")
    if kv_scales.shape != (pages, 2, hk):
        raise ValueError(f"kv_scales must be [{pages}, 2, {hk}], got {tuple(kv_scales.shape)}")
    return pages, hk, d


def _flag(err_flag, dev):
    if err_flag is None:
        return None
    _arg(err_flag, "err_flag", torch.int32, dev)
    if err_flag.numel() < 1:
        raise ValueError("err_flag must have an element")
    return err_flag.data_ptr()


def _requests(block_table, lens, dev, err_flag):
    _arg(block_table, "block_table", torch.int32, dev, 2)
    _arg(lens, "lens", torch.int32, dev, 1)
    n, width = block_table.shape
    if lens.shape[0] != n:
        raise ValueError("lens must have one entry per block_table row")
    return n, width, _flag(err_flag, dev)


def _starts(token_starts, n, dev):
    _arg(token_starts, "token_starts", torch.int32, dev, 1)
    if token_starts.shape[0] != n + 1:
        raise ValueError("token_starts must have one entry more than block_table has rows")


def kv8_append(k, v, token_starts, block_table, lens, kv_pages, kv_scales, err_flag=None,
               stream=None):
    """Write new tokens' keys and values (bf16 [T, kv_heads, dim], tokens may
    be strided) at the ends of their requests, quantised in place; request r
    owns tokens ``token_starts[r]:token_starts[r + 1]`` and ``lens`` includes
    them. Returns ``kv_pages``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv8_append(k, v, token_starts, block_table, lens, kv_pages, kv_scales, err_flag)
    dev = _device(kv_pages, "kv_pages", torch.uint8)
    pages, hk, d = _cache(kv_pages, kv_scales, dev)
    ks = _tokens(k, "k", torch.bfloat16, dev, 1)
    vs = _tokens(v, "v", torch.bfloat16, dev, 1)
    if k.shape[1:] != (hk, d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [tokens, {hk}, {d}]")
    n, width, flag = _requests(block_table, lens, dev, err_flag)
    _starts(token_starts, n, dev)
    _run(dev, lib().ds_kv8_append, k.data_ptr(), v.data_ptr(), ks, vs, k.shape[0],
         token_starts.data_ptr(), n, block_table.data_ptr(), width, lens.data_ptr(), hk, d,
         kv_pages.data_ptr(), kv_scales.data_ptr(), pages, flag)
    return kv_pages


def kv8_decode_workspace_size(num_requests, next_n, num_heads, num_kv_heads, head_dim, bt_stride):
    return int(lib().ds_kv8_decode_workspace_size(num_requests, next_n, num_heads, num_kv_heads,
                                                  head_dim, bt_stride))


def kv8_prefill_workspace_size(num_tokens, num_requests, num_heads, num_kv_heads, head_dim):
    return int(lib().ds_kv8_prefill_workspace_size(num_tokens, num_requests, num_heads,
                                                   num_kv_heads, head_dim))


def _outputs(q, d, dev, out, lse):
    if q.shape[-1] != d:
        raise ValueError(f"q must have head dim {d}, got {q.shape[-1]}")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _arg(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}")
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    else:
        _arg(lse, "lse", torch.float32, dev)
        if lse.shape != q.shape[:-1]:
            raise ValueError(f"lse must be {tuple(q.shape[:-1])}")
    return out, lse


def kv8_decode(q, kv_pages, kv_scales, block_table, lens, scale, out=None, lse=None,
               workspace=None, err_flag=None, stream=None):
    """Attention of the last ``next_n`` tokens of every request over the
    block-scaled cache: q bf16 [R, next_n, H, dim] (tokens may be evenly
    strided); returns (out bf16 like q, lse fp32 [R, next_n, H])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv8_decode(q, kv_pages, kv_scales, block_table, lens, scale, out, lse,
                              workspace, err_flag)
    dev = _device(kv_pages, "kv_pages", torch.uint8)
    pages, hk, d = _cache(kv_pages, kv_scales, dev)
    qs = _tokens(q, "q", torch.bfloat16, dev, 2)
    n, width, flag = _requests(block_table, lens, dev, err_flag)
    r, nn, h, _ = q.shape
    if r != n:
        raise ValueError("q must have one row per block_table row")
    out, lse = _outputs(q, d, dev, out, lse)
    L = lib()
    if workspace is None:
        need = r and L.ds_kv8_decode_workspace_size(r, nn, h, hk, d, width)
        workspace = _scratch(need or 256, dev, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        _arg(workspace, "workspace", torch.uint8, dev)
    _run(dev, L.ds_kv8_decode, q.data_ptr(), qs, kv_pages.data_ptr(), kv_scales.data_ptr(), pages,
         block_table.data_ptr(), width, lens.data_ptr(), r, nn, h, hk, d, float(scale),
         out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(), flag)
    return out, lse


def kv8_prefill(q, token_starts, kv_pages, kv_scales, block_table, lens, scale, out=None, lse=None,
                workspace=None, err_flag=None, stream=None):
    """Causal attention of ragged prompts over the block-scaled cache: q bf16
    [T, H, dim] (tokens may be strided), request r owning tokens
    ``token_starts[r]:token_starts[r + 1]``, the last of its ``lens[r]``
    positions; returns (out bf16 [T, H, dim], lse fp32 [T, H]). Rows of no
    request are left as they are (unset in outputs allocated here)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv8_prefill(q, token_starts, kv_pages, kv_scales, block_table, lens, scale, out,
                               lse, workspace, err_flag)
    dev = _device(kv_pages, "kv_pages", torch.uint8)
    pages, hk, d = _cache(kv_pages, kv_scales, dev)
    qs = _tokens(q, "q", torch.bfloat16, dev, 1)
    n, width, flag = _requests(block_table, lens, dev, err_flag)
    _starts(token_starts, n, dev)
    t, h, _ = q.shape
    out, lse = _outputs(q, d, dev, out, lse)
    L = lib()
    if workspace is None:
        need = t and L.ds_kv8_prefill_workspace_size(t, n, h, hk, d)
        workspace = _scratch(need or 256, dev, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        _arg(workspace, "workspace", torch.uint8, dev)
    _run(dev, L.ds_kv8_prefill, q.data_ptr(), qs, t, token_starts.data_ptr(), n,
         kv_pages.data_ptr(), kv_scales.data_ptr(), pages, block_table.data_ptr(), width,
         lens.data_ptr(), h, hk, d, float(scale), out.data_ptr(), lse.data_ptr(),
         workspace.data_ptr(), workspace.numel(), flag)
    return out, lse

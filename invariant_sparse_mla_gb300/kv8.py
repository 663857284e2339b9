"""The block-scaled 8-bit KV cache: append, decode and prefill attention.

Argument marshalling for ds_kv8_append / ds_kv8_decode / ds_kv8_prefill (see
include/ds_sparse_mla.h). The cache of one layer is ``kv_pages`` uint8
[num_pages, 2, kv_heads, 64, dim] (E4M3 codes, keys then values) with
``kv_scales`` float32 [num_pages, 2, kv_heads]; block tables are those of the
latent cache.
"""

import torch

from ._native import _check, _need, lib


def _launch(dev, fn, *args):
    """Calls fn(*args, stream) with ``dev`` current (the runtime launches only
    into streams of the current device)."""
    stream = args[-1]
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    args = args[:-1] + (stream.cuda_stream,)
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args))


def _p(t):
    return None if t is None else t.data_ptr()


def _tokens(t, name, dtype, dev, lead):
    """A [*lead, heads, dim] tensor whose tokens are evenly strided and whose
    [heads, dim] part is contiguous; returns the stride between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dim() != lead + 2:
        raise ValueError(f"{name} must have {lead + 2} dims, got {t.dim()}")
    shape, stride = t.shape, t.stride()
    if (shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1]):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row = shape[-2] * shape[-1]
    if lead == 2:
        if shape[0] > 1 and shape[1] > 1 and stride[0] != shape[1] * stride[1]:
            raise ValueError(f"{name}: tokens must be evenly strided")
        return stride[1] if shape[1] > 1 else (stride[0] if shape[0] > 1 else row)
    return stride[0] if shape[0] > 1 else row


def _cache(kv_pages, kv_scales, dev):
    _need(kv_pages, "kv_pages", torch.uint8, dev, 5)
    _need(kv_scales, "kv_scales", torch.float32, dev, 3)
    pages, two, hk, page, d = kv_pages.shape
    if two != 2 or page != 64:
        raise ValueError("kv_pages must be [num_pages, 2, kv_heads, 64, dim] codes, got "
                         f"{tuple(kv_pages.shape)}")
    if tuple(kv_scales.shape) != (pages, 2, hk):
        raise ValueError(f"kv_scales must be [{pages}, 2, {hk}], got {tuple(kv_scales.shape)}")
    return pages, hk, d


def _requests(block_table, lens, dev, err_flag):
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(lens, "lens", torch.int32, dev, 1)
    if err_flag is not None:
        _need(err_flag, "err_flag", torch.int32, dev)
        if err_flag.numel() < 1:
            raise ValueError("err_flag must have an element")
    n, width = block_table.shape
    if lens.numel() != n:
        raise ValueError("lens must have one entry per block_table row")
    return n, width


def _starts(token_starts, n, dev):
    _need(token_starts, "token_starts", torch.int32, dev, 1)
    if token_starts.numel() != n + 1:
        raise ValueError("token_starts must have one entry more than block_table has rows")


def kv8_append(k, v, token_starts, block_table, lens, kv_pages, kv_scales, err_flag=None,
               stream=None):
    """Write new tokens' keys and values (bf16 [T, kv_heads, dim], tokens may
    be strided) at the ends of their requests, quantised in place; request r
    owns tokens ``token_starts[r]:token_starts[r + 1]`` and ``lens`` includes
    them. Returns ``kv_pages``."""
    dev = kv_pages.device
    pages, hk, d = _cache(kv_pages, kv_scales, dev)
    ks = _tokens(k, "k", torch.bfloat16, dev, 1)
    vs = _tokens(v, "v", torch.bfloat16, dev, 1)
    if tuple(k.shape[1:]) != (hk, d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [tokens, {hk}, {d}]")
    n, width = _requests(block_table, lens, dev, err_flag)
    _starts(token_starts, n, dev)
    _launch(dev, lib().ds_kv8_append, _p(k), _p(v), ks, vs, k.shape[0], _p(token_starts), n,
            _p(block_table), width, _p(lens), hk, d, _p(kv_pages), _p(kv_scales), pages,
            _p(err_flag), stream)
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
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}")
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", torch.float32, dev)
        if lse.shape != q.shape[:-1]:
            raise ValueError(f"lse must be {tuple(q.shape[:-1])}")
    return out, lse


def kv8_decode(q, kv_pages, kv_scales, block_table, lens, scale, out=None, lse=None,
               workspace=None, err_flag=None, stream=None):
    """Attention of the last ``next_n`` tokens of every request over the
    block-scaled cache: q bf16 [R, next_n, H, dim] (tokens may be evenly
    strided); returns (out bf16 like q, lse fp32 [R, next_n, H])."""
    dev = kv_pages.device
    pages, hk, d = _cache(kv_pages, kv_scales, dev)
    qs = _tokens(q, "q", torch.bfloat16, dev, 2)
    n, width = _requests(block_table, lens, dev, err_flag)
    r, nn, h, _ = q.shape
    if r != n:
        raise ValueError("q must have one row per block_table row")
    out, lse = _outputs(q, d, dev, out, lse)
    L = lib()
    if workspace is None and r > 0:
        need = L.ds_kv8_decode_workspace_size(r, nn, h, hk, d, width)
        workspace = torch.empty(need or 256, dtype=torch.uint8, device=dev)
    elif workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    _launch(dev, L.ds_kv8_decode, _p(q), qs, _p(kv_pages), _p(kv_scales), pages, _p(block_table),
            width, _p(lens), r, nn, h, hk, d, float(scale), _p(out), _p(lse), _p(workspace),
            0 if workspace is None else workspace.numel(), _p(err_flag), stream)
    return out, lse


def kv8_prefill(q, token_starts, kv_pages, kv_scales, block_table, lens, scale, out=None, lse=None,
                workspace=None, err_flag=None, stream=None):
    """Causal attention of ragged prompts over the block-scaled cache: q bf16
    [T, H, dim] (tokens may be strided), request r owning tokens
    ``token_starts[r]:token_starts[r + 1]``, the last of its ``lens[r]``
    positions; returns (out bf16 [T, H, dim], lse fp32 [T, H]). Rows of no
    request are left as they are (unset in outputs allocated here)."""
    dev = kv_pages.device
    pages, hk, d = _cache(kv_pages, kv_scales, dev)
    qs = _tokens(q, "q", torch.bfloat16, dev, 1)
    n, width = _requests(block_table, lens, dev, err_flag)
    _starts(token_starts, n, dev)
    t, h, _ = q.shape
    out, lse = _outputs(q, d, dev, out, lse)
    L = lib()
    if workspace is None and t > 0:
        need = L.ds_kv8_prefill_workspace_size(t, n, h, hk, d)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    elif workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    _launch(dev, L.ds_kv8_prefill, _p(q), qs, t, _p(token_starts), n, _p(kv_pages),
            _p(kv_scales), pages, _p(block_table), width, _p(lens), h, hk, d, float(scale),
            _p(out), _p(lse), _p(workspace), 0 if workspace is None else workspace.numel(),
            _p(err_flag), stream)
    return out, lse

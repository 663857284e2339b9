"""Norms of queries and keys per head with the position rotation.

Argument marshalling for ds_qk_norm_rope (see include/ds_sparse_mla.h).
"""

import torch

from ._native import lib
from .kv8 import _arg, _device, _run, _tokens


def _out(x, out, name, dev):
    """The output of a side and its stride between tokens."""
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        return out, x.shape[1] * x.shape[2]
    stride = _tokens(out, name, torch.bfloat16, dev, 1)
    if out.shape != x.shape:
        raise ValueError(f"{name} must be {tuple(x.shape)}")
    return out, stride


def _weight(w, name, norm_dim, dev):
    if w is None:
        return None
    _arg(w, name, torch.bfloat16, dev, 1)
    if w.shape[0] != norm_dim:
        raise ValueError(f"{name} must have norm_dim = {norm_dim} entries")
    return w.data_ptr()


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, norm_dim=None,
                 rot_start=0, interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of every head's first ``norm_dim`` dims (all of them by default)
    times its weights (bf16; a side without weights is not normed), then the
    rotation of ``2 * len(inv_freq)`` dims from ``rot_start`` on by
    ``positions`` (int32 [T]): q bf16 [T, H, dim] and k [T, Hk, dim] (tokens may
    be strided, k may be None). Returns (q_out, k_out), new tensors unless given;
    q and k themselves may be given."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, norm_dim,
                                rot_start, interleaved, q_out, k_out)
    dev = _device(q, "q", torch.bfloat16)
    qs = _tokens(q, "q", torch.bfloat16, dev, 1)
    t, h, d = q.shape
    q_out, qos = _out(q, q_out, "q_out", dev)
    hk, ks, kos, kp, kop = 0, 0, 0, None, None
    if k is not None:
        ks = _tokens(k, "k", torch.bfloat16, dev, 1)
        if k.shape[0] != t or k.shape[2] != d:
            raise ValueError(f"k must be [{t}, kv_heads, {d}], got {tuple(k.shape)}")
        hk = k.shape[1]
        k_out, kos = _out(k, k_out, "k_out", dev)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    _arg(positions, "positions", torch.int32, dev, 1)
    if positions.shape[0] != t:
        raise ValueError(f"positions must have {t} entries")
    _arg(inv_freq, "inv_freq", torch.float32, dev, 1)
    if norm_dim is None:
        norm_dim = d if q_weight is not None or k_weight is not None else 0
    qw = _weight(q_weight, "q_weight", norm_dim, dev)
    kw = _weight(k_weight, "k_weight", norm_dim, dev)
    _run(dev, lib().ds_qk_norm_rope, q.data_ptr(), qs, h, qw, kp, ks, hk, kw, t, d, norm_dim,
         float(eps), positions.data_ptr(), inv_freq.data_ptr(), rot_start, 2 * inv_freq.shape[0],
         int(bool(interleaved)), q_out.data_ptr(), qos, kop, kos)
    return q_out, k_out

"""Seeded inputs of the block-scaled 8-bit cache tests (no method arithmetic)."""

import numpy as np
import torch

DEV = "cuda:0"


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


class Cache:
    """A cache of E4M3 codes with random tables: NaN codes in every slot that
    no position owns, -1 in every table entry that no row holds."""

    def __init__(self, lens, kv_heads, dim, seed, extra_pages=3, extra_width=1, spread=3):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.lens = [int(x) for x in lens]
        self.kv_heads, self.dim = kv_heads, dim
        held = [max(0, -(-x // 64)) for x in self.lens]
        self.pages = sum(held) + extra_pages
        width = max(held + [1]) + extra_width
        perm = rng.permutation(self.pages)
        self.table = np.full((len(lens), width), -1, np.int32)
        codes = rng.standard_normal((self.pages, 2, kv_heads, 64, dim)) * 100
        codes = torch.as_tensor(np.clip(codes, -448, 448)).to(torch.float8_e4m3fn)
        codes = codes.view(torch.uint8).numpy().copy()
        own = np.zeros((self.pages, 64), bool)
        at = 0
        for r, n in enumerate(held):
            self.table[r, :n] = perm[at:at + n]
            for b in range(n):
                own[perm[at + b], :max(0, min(64, self.lens[r] - 64 * b))] = True
            at += n
        codes[~np.broadcast_to(own[:, None, None, :], codes.shape[:4])] = 0x7F
        self.codes = codes
        # Scales of unused pages are NaN.
        self.scales = (2.0 ** rng.integers(-8, -8 + spread, (self.pages, 2, kv_heads))) \
            .astype(np.float32)
        self.scales[~own.any(1)] = np.nan

    def device(self, dev=DEV):
        return (torch.as_tensor(self.codes).to(dev), torch.as_tensor(self.scales).to(dev),
                torch.as_tensor(self.table).to(dev),
                torch.as_tensor(self.lens, dtype=torch.int32).to(dev))

    def q(self, tokens, heads, gain=2.5):
        x = self.rng.standard_normal((tokens, heads, self.dim)).astype(np.float32) * gain
        return torch.as_tensor(x).to(torch.bfloat16)

"""Test infrastructure for the ragged append and single-token attention: a pool
with sequences of any lengths in shuffled pages, filled from host tensors."""
from __future__ import annotations

import numpy as np
import torch

import paged_kv_chunk_query_b200 as pk

DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy(rng.normal(size=shape) * std).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


class Pages:
    """A device pool whose every unwritten K/V value is NaN (what stands behind a
    sequence's end must not matter)."""

    def __init__(self, num_pages, P, Hkv, d, grad=False, seed=11, fill=float("nan")):
        self.P, self.Hkv, self.d = P, Hkv, d
        self.pool = pk.pool_create(num_pages, P, Hkv, d, pk.LOC_DEVICE, grad, seed, 0)
        self.kv, self.grad, self.mean = pk.pool_views(self.pool)
        self.kv.fill_(fill)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        torch.cuda.synchronize()
        pk.pool_destroy(self.pool)

    def take(self, tokens):
        return [pk.pool_alloc_page(self.pool) for _ in range(-(-tokens // self.P))]

    def put(self, ids, k, v):
        """Host K, V [tokens][Hkv][d] into the pages `ids` (test set-up, no library call)."""
        n, P = k.shape[0], self.P
        for i, page in enumerate(ids):
            m = min(P, n - i * P)
            if m > 0:
                kv = torch.stack([k[i * P:i * P + m], v[i * P:i * P + m]])  # [2][m][Hkv][d]
                self.kv[page, :, :, :m] = kv.permute(2, 0, 1, 3).to(DEV)

    def rows(self, ids, n, which, buf=None):
        """Rows 0..n-1 of the pages in order [n][Hkv][d], 0 = K, 1 = V."""
        src = self.kv if buf is None else buf
        x = src[torch.tensor(ids, dtype=torch.long, device=DEV), :, which]
        return x.permute(0, 2, 1, 3).reshape(-1, self.Hkv, self.d)[:n]

    def status(self):
        return pk.get_device_status(self.pool)


def tables(lists, width=None, pad=0x3FFFFFFF):
    """Page tables [len(lists)][width]; places behind a list hold an id that is no page."""
    width = width or max([1, *(len(x) for x in lists)])
    return i32([list(x) + [pad] * (width - len(x)) for x in lists])


def starts_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()

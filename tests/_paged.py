"""A paged cache for the tests, and plain fp64 forms of what the library does with it.

Nothing here calls the library: rows are placed and read back by their position, attention
is a masked softmax, and 8-bit codes are the nearest of the oracle's e4m3 values."""
from __future__ import annotations

import numpy as np
import torch

import oracle

F8 = torch.float8_e4m3fn


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def e4m3_values(codes: torch.Tensor) -> np.ndarray:
    """fp64 values of uint8 e4m3 codes."""
    return codes.cpu().view(F8).to(torch.float64).numpy()


def encode(y: np.ndarray) -> np.ndarray:
    """e4m3 codes (uint8) of finite fp64 values: the nearest of the format's values, ties to the
    even code, magnitudes past 448 to 448."""
    table = oracle.e4m3_decode_table()[:127]            # 0 .. 448, ascending
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(table, a), 1, 126)
    lo = hi - 1
    up, down = table[hi] - a, a - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """(codes uint8, scale fp32) of fp64 rows [..., d] that hold bf16 values."""
    x32 = x.astype(np.float32)
    amax = np.abs(x32).max(-1)
    amax = np.where((amax > 0) & (amax < np.float32(2.0) ** -100), np.float32(2.0) ** -100, amax)
    amax = amax.astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(amax > 0, np.float32(448.0) / amax, np.float32(0.0)).astype(np.float32)
    y = (x32 * inv[..., None]).astype(np.float32)
    return encode(y.astype(np.float64)), (amax / np.float32(448.0)).astype(np.float32)


class Cache:
    """A pool with a random assignment of pages to sequences of the given capacities.
    fill: what every row holds before anything is written ("normal" or "nan")."""

    def __init__(self, caps, Hkv, d, ps, kv, seed, fill="normal", spare=3, max_pages=None):
        self.Hkv, self.d, self.ps, self.kv = Hkv, d, ps, kv
        gen = torch.Generator().manual_seed(seed)
        counts = [-(-c // ps) for c in caps]
        self.n_pages = sum(counts) + spare
        self.max_pages = max_pages or max(1, max(counts))
        order = torch.randperm(self.n_pages, generator=gen).tolist()
        self.table = torch.full((len(caps), self.max_pages), -1, dtype=torch.int32)
        for b, c in enumerate(counts):
            self.table[b, :c] = torch.tensor([order.pop() for _ in range(c)], dtype=torch.int32)
        shape = (self.n_pages, Hkv, ps, d)
        rows = [torch.randn(shape, generator=gen).to(torch.bfloat16) for _ in range(2)]
        self.scales = None
        if kv == "e4m3":
            both = [quantise(f64(r)) for r in rows]
            self.k, self.v = (torch.from_numpy(c).view(F8) for c, _ in both)
            self.scales = torch.stack([torch.from_numpy(s) for _, s in both], 2).contiguous()
        else:
            self.k, self.v = rows
        if fill == "nan":
            for t in (self.k, self.v):
                if kv == "e4m3":
                    t.view(torch.uint8).fill_(0x7F)
                else:
                    t.fill_(float("nan"))
            if self.scales is not None:
                self.scales.fill_(float("nan"))

    def cuda(self):
        """(k_pages, v_pages, table, scales) on the device."""
        return (self.k.cuda(), self.v.cuda(), self.table.cuda(),
                None if self.scales is None else self.scales.cuda())

    def set_row(self, which, b, pos, row, scale=None):
        """row: [Hkv, d], bf16 or uint8 codes with scale [Hkv]."""
        page, r = int(self.table[b, pos // self.ps]), pos % self.ps
        pages = (self.k, self.v)[which]
        if self.kv == "e4m3":
            pages.view(torch.uint8)[page, :, r] = row
            self.scales[page, :, which, r] = scale
        else:
            pages[page, :, r] = row

    def rows(self, which, b, n, first=0):
        """fp64 [Hkv, n, d]: positions first .. first + n - 1 of sequence b."""
        page, r = self._at(b, first, n)
        x = f64((self.k, self.v)[which])[page, :, r]                   # [n, Hkv, d]
        if self.scales is not None:
            x = x * f64(self.scales)[page, :, which, r][:, :, None]
        return x.transpose(1, 0, 2)

    def scale_rows(self, which, b, n):
        page, r = self._at(b, 0, n)
        return f64(self.scales)[page, :, which, r].T

    def _at(self, b, first, n):
        pos = first + np.arange(n)
        return self.table[b].numpy()[pos // self.ps], pos % self.ps


def attend(q, k, v, n, causal, scale):
    """One sequence: q [H, Nq, d], k, v [Hkv, n, d] in fp64.  Returns (o, lse, weight): weight
    [H, Nq, n] are the softmax probabilities."""
    H, Nq, d = q.shape
    G = H // k.shape[0]
    o, lse, w = np.zeros((H, Nq, d)), np.full((H, Nq), -np.inf), np.zeros((H, Nq, n))
    for h in range(H):
        for i in range(Nq):
            seen = min(n, max(0, n - Nq + 1 + i)) if causal else n
            if seen == 0:
                continue
            x = scale * (k[h // G, :seen] @ q[h, i])
            m = x.max()
            e = np.exp(x - m)
            lse[h, i] = m + np.log(e.sum())
            w[h, i, :seen] = e / e.sum()
            o[h, i] = w[h, i, :seen] @ v[h // G, :seen]
    return o, lse, w

"""Plain float64 statements of the paged-cache operators (norm, rotation, quantised pages, causal attention) on the
CPU, and a small driver that holds a batch on both sides."""

from __future__ import annotations

import numpy as np
import torch

from hybrid_linear_attention_03_gb300 import kda

F64 = torch.float64


def norm_rotate(x, w, pos, inv_freq, interleaved, eps):
    """x [rows, heads, d] -> float64, per-head RMSNorm (w None: none) and rotation of the first 2 len(inv_freq) channels."""
    x = x.to(F64).clone()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = torch.tensor([float(p) * f for p in pos], dtype=F64)[:, None]
        xa, xb = x[..., a].clone(), x[..., b].clone()
        x[..., a] = xa * ang.cos() - xb * ang.sin()
        x[..., b] = xa * ang.sin() + xb * ang.cos()
    return x


def e4m3_grid() -> np.ndarray:
    """The finite non-negative e4m3 values."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    nor = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(sub + nor[:-1])  # the last pattern is NaN


def quantise(x):
    """float64 vectors -> (values on the e4m3 grid, biased exponent), round to nearest even, non-finite -> NaN."""
    x = np.asarray(x, np.float64)
    grid = e4m3_grid()
    fin = np.isfinite(x)
    amax = np.max(np.where(fin, np.abs(x), 0.0), -1)
    e = np.zeros(amax.shape, np.int64)
    nz = amax > 0
    e[nz] = np.clip(np.ceil(np.log2(amax[nz] / 448.0)), -126, 127) + 127
    y = np.where(fin, np.abs(x), 0.0) * 2.0 ** (127.0 - np.where(nz, e, 127))[..., None]
    hi = np.clip(np.searchsorted(grid, y), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - grid[lo], grid[hi] - y
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    q = np.copysign(grid[pick], x)
    return np.where(fin, q, np.nan), e


def attend(q, k, v, ctx, scale, group):
    """q [T, Hq, d]; k, v [L, Hkv, d] float64 with NaN-free visible keys handled key by key: masked keys take no part.
    Returns (out, sum p |v|, max |score|) in float64."""
    T, hq, d = q.shape
    out = torch.zeros(T, hq, v.shape[2], dtype=F64)
    mag = torch.zeros_like(out)
    for t in range(T):
        for h in range(hq):
            kk, vv = k[:ctx + t + 1, h // group], v[:ctx + t + 1, h // group]
            s = (kk @ q[t, h]) * scale
            p = torch.softmax(s, 0)
            out[t, h] = p @ vv
            mag[t, h] = p @ vv.abs()
    return out, mag


class Batch:
    """A cache and a batch's tables, with the pages in a shuffled order.  new / total: tokens of the call and cache
    length per sequence."""

    def __init__(self, new, total, hq, hkv, d, page, act, fmt, seed=0, spare=3, fill=None, extra_rows=0, num_pages=None):
        self.new, self.total, self.hq, self.hkv, self.d, self.page = list(new), list(total), hq, hkv, d, page
        self.act, self.fmt, self.group = act, fmt, hq // hkv
        g = torch.Generator().manual_seed(seed)
        per = [-(-t // page) for t in total]
        n_pages = sum(per) + spare
        num_pages = num_pages or n_pages
        order = (torch.randperm(num_pages, generator=g)[:n_pages]).to(torch.int32)
        width = max(per + [1])
        table = torch.full((len(new), width), -1, dtype=torch.int32)
        at = 0
        for i, c in enumerate(per):
            table[i, :c] = order[at:at + c]
            at += c
        self.table = table
        self.rows = sum(new)
        self.max_rows = self.rows + extra_rows
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.kv = kda.PagedKV(num_pages, page, hq, hkv, d, act, kv_format=fmt)
        if fill is not None:
            for t in (self.kv.k, self.kv.v):
                if fmt == "e4m3":
                    t.view(torch.uint8).fill_(0x7F)  # NaN
                else:
                    t.fill_(fill)
            if fmt == "e4m3":
                self.kv.k_scale.fill_(254)
                self.kv.v_scale.fill_(254)
        self.dev = (self.cu.cuda(), torch.tensor(total, dtype=torch.int32).cuda(), table.cuda())
        self.batch = kda.make_kv_batch(*self.dev, max_rows=max(self.max_rows, 1), max_new=max(list(new) + [1]))
        self.gen = g

    def positions(self):
        return [L - T + t for T, L in zip(self.new, self.total) for t in range(T)]

    def whole(self):
        """The same cache seen as a batch whose tokens are all of every sequence's."""
        b = Batch.__new__(Batch)
        b.__dict__.update(self.__dict__)
        b.new = list(self.total)
        b.rows = b.max_rows = sum(b.new)
        b.cu = torch.tensor(np.concatenate([[0], np.cumsum(b.new)]), dtype=torch.int32)
        b.dev = (b.cu.cuda(), self.dev[1], self.dev[2])
        b.batch = kda.make_kv_batch(*b.dev, max_rows=max(b.rows, 1), max_new=max(b.new + [1]))
        return b

    def randn(self, rows, heads):
        return torch.randn(rows, heads, self.d, generator=self.gen, dtype=torch.float32).to(self.act)

    def workspace(self, fill=0xA5):
        n = kda.kda_kv_attend_workspace_bytes(self.kv, self.batch)
        return torch.full((n,), fill, dtype=torch.uint8, device="cuda")

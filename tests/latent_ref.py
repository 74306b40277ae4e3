"""Plain float64 statements of the latent-attention operators (norm, rotation, quantised pages, both attention forms) on the
CPU, and small drivers that hold a batch on both sides."""

from __future__ import annotations

import numpy as np
import torch

from hybrid_linear_attention_03_gb300 import kda

from kv_ref import F64, norm_rotate, quantise

BF = torch.bfloat16


def rotate(x, pos, freq, inter):
    """x [rows, heads, d] -> float64, the first 2 len(freq) channels turned."""
    return norm_rotate(x, None, pos, freq, inter, 0.0)


def norm(x, w, eps):
    x = x.to(F64)
    return x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)


def attend(score, value, ctx, gone=()):
    """score [T, H, L] and value [L, H or 1, D] in float64, row t sees keys up to ctx + t but those in `gone`.  Returns
    (out, sum p |v|); a row without keys, or whose scores are all -inf, gives zeros.  Hidden keys take no part."""
    T, H, L = score.shape
    j = torch.arange(L)
    hidden = j[None] > ctx + torch.arange(T)[:, None]
    if len(gone):
        hidden[:, list(gone)] = True
    s = score.masked_fill(hidden[:, None], -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -torch.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out, mag = torch.zeros(T, H, value.shape[2], dtype=F64), torch.zeros(T, H, value.shape[2], dtype=F64)
    seen = ~hidden
    for t in range(T):
        v = value[seen[t]]
        w = p[t][:, seen[t]]
        if v.shape[1] == 1:
            out[t], mag[t] = w @ v[:, 0], w @ v[:, 0].abs()
        else:
            out[t], mag[t] = torch.einsum("hj,jhd->hd", w, v), torch.einsum("hj,jhd->hd", w, v.abs())
    return out, mag


def half_step(t):
    return torch.finfo(t).eps / 2


def check(got, ref, mag, qk, channels, act, what=""):
    """Rows [T, H, D] against their float64 values.  A score sums `channels` products (channels + 4 units of 2^-24 of at most
    qk = scale |q| |k|); its weight is off by that relatively, twice over for the sum, and by 2^-20 for the power of two and the
    sums; bf16 calls may round each weight to bf16 (2^-8) before it meets its value; the output is rounded once."""
    got = got.double().cpu()
    rel = (channels + 4) * 2.0 ** -24 * qk[..., None] * 2 + 2.0 ** -20
    tol = mag * (rel + (2 * half_step(BF) if act == BF else 0)) + ref.abs() * (half_step(BF) if act == BF else 0) + 1e-30
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    off = torch.nan_to_num((got - ref).abs() / tol)
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: worst error {worst:.2f} of the tolerance"


class Batch:
    """A latent cache and a batch's tables, with the pages in a shuffled order.  new / total: tokens of the call and cache
    length per sequence."""

    def __init__(self, new, total, heads, latent, rope, page, act, fmt, seed=0, spare=3, fill=None, extra_rows=0, num_pages=None):
        self.new, self.total, self.heads, self.latent, self.rope, self.page = list(new), list(total), heads, latent, rope, page
        self.act, self.fmt = act, fmt
        self.gen = torch.Generator().manual_seed(seed)
        per = [-(-t // page) for t in total]
        n_pages = sum(per) + spare
        num_pages = num_pages or n_pages
        order = torch.randperm(num_pages, generator=self.gen)[:n_pages].to(torch.int32)
        self.table = torch.full((len(new), max(per + [1])), -1, dtype=torch.int32)
        at = 0
        for i, c in enumerate(per):
            self.table[i, :c] = order[at:at + c]
            at += c
        self.rows = sum(new)
        self.max_rows = self.rows + extra_rows
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.kv = kda.PagedLatent(num_pages, page, heads, latent, rope, act, kv_format=fmt)
        if fill is not None:
            self.kv.kr.fill_(fill)
            if fmt == "e4m3":
                self.kv.c.view(torch.uint8).fill_(0x7F)  # NaN
                self.kv.c_scale.fill_(254)
            else:
                self.kv.c.fill_(fill)
        self.dev = (self.cu.cuda(), torch.tensor(total, dtype=torch.int32).cuda(), self.table.cuda())
        self.batch = kda.make_kv_batch(*self.dev, max_rows=max(self.max_rows, 1), max_new=max(list(new) + [1]))

    def set(self, new, total):
        """Other tokens and lengths over the same pages."""
        self.new, self.total, self.rows = list(new), list(total), sum(new)
        self.max_rows = self.rows
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.dev = (self.cu.cuda(), torch.tensor(total, dtype=torch.int32).cuda(), self.dev[2])
        self.batch = kda.make_kv_batch(*self.dev, max_rows=max(self.rows, 1), max_new=max(self.new + [1]))

    def whole(self):
        """The same cache seen as a batch whose tokens are all of every sequence's."""
        b = Batch.__new__(Batch)
        b.__dict__.update(self.__dict__)
        b.set(self.total, self.total)
        return b

    def positions(self):
        return [L - T + t for T, L in zip(self.new, self.total) for t in range(T)]

    def lines(self):
        """Page and line of every row of the batch."""
        seq = torch.tensor([i for i, T in enumerate(self.new) for _ in range(T)], dtype=torch.long)
        pos = torch.tensor(self.positions(), dtype=torch.long)
        return self.table[seq, pos // self.page].long(), pos % self.page

    def randn(self, *shape, gain=1.0):
        return (torch.randn(*shape, generator=self.gen, dtype=torch.float32) * gain).to(self.act)

    def queries(self, rows=None, gain=1.0):
        rows = self.max_rows if rows is None else rows
        return self.randn(rows, self.heads, self.latent, gain=gain).cuda(), self.randn(rows, self.heads, self.rope, gain=gain).cuda()

    def workspace(self, fill=0xA5):
        return torch.full((kda.kda_latent_attend_workspace_bytes(self.kv, self.batch),), fill, dtype=torch.uint8, device="cuda")

    def fill_cache(self, gain=1.0):
        """Random latents and key parts for every token, appended through the library; what the cache then holds."""
        w = self.whole()
        c, kr = w.randn(w.rows, self.latent, gain=gain), w.randn(w.rows, self.rope, gain=gain)
        kda.kda_latent_append(self.kv, None, kda.make_latent_io(c.cuda(), kr.cuda(), None, None), w.batch)
        return self.held()

    def held(self):
        """Per sequence (c, kr) in float64, read back through the library."""
        w = self.whole()
        c = torch.zeros(max(w.rows, 1), self.latent, dtype=self.act, device="cuda")
        kr = torch.zeros(max(w.rows, 1), self.rope, dtype=self.act, device="cuda")
        kda.kda_latent_read(self.kv, w.batch, c, kr)
        c, kr = c.double().cpu(), kr.double().cpu()
        cu = [int(x) for x in w.cu]
        return [(c[a:z], kr[a:z]) for a, z in zip(cu[:-1], cu[1:])]

    def no_error(self):
        st, flags = kda.kda_latent_poll_device_error(self.kv)
        assert st == kda.KDA_OK, hex(flags)

    def check_attend(self, q, out, held, scale, gone=None):
        """Every row of the batch against the absorbed form over what the cache holds."""
        qc, qr = q[0].double().cpu(), q[1].double().cpu()
        for i, (T, L) in enumerate(zip(self.new, self.total)):
            if T == 0:
                continue
            a = int(self.cu[i])
            c, kr = held[i]
            s = (torch.einsum("thl,jl->thj", qc[a:a + T], c) + torch.einsum("thr,jr->thj", qr[a:a + T], kr)) * scale
            ref, mag = attend(s, c[:, None], L - T, gone[i] if gone else ())
            top = torch.cat((c, kr), -1).nan_to_num(0.0, 0.0, 0.0).norm(dim=-1).max()
            qk = torch.cat((qc[a:a + T], qr[a:a + T]), -1).norm(dim=-1) * float(top) * scale
            check(out[a:a + T], ref, mag, qk, self.latent + self.rope, self.act, f"sequence {i}")


class Rows:
    """Keys and values in rows, and the queries, of an expanded call; total: key rows per sequence.  The tensors are slices
    of wider projections."""

    def __init__(self, new, total, heads, nope, rope, value, act, seed=0, extra_rows=0, extra_keys=0, fill=9.0, gain=1.0):
        self.new, self.total, self.heads, self.act = list(new), list(total), heads, act
        self.nope, self.rope, self.value = nope, rope, value
        self.gen = torch.Generator().manual_seed(seed)
        self.rows, self.keys = sum(new), sum(total)
        self.max_rows, self.max_keys = max(self.rows + extra_rows, 1), max(self.keys + extra_keys, 1)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.cu_kv = torch.tensor(np.concatenate([[0], np.cumsum(total)]), dtype=torch.int32)

        def randn(*shape):
            return torch.randn(*shape, generator=self.gen, dtype=torch.float32).to(act).cuda()

        q, kv = randn(self.max_rows, heads, nope + rope) * gain, randn(self.max_keys, heads, nope + value)
        if extra_keys:
            kv[self.keys:] = float("nan")  # behind the last sequence's keys
        self.qn, self.qr, self.k, self.v = q[..., :nope], q[..., nope:], kv[..., :nope], kv[..., nope:]
        self.kr = randn(self.max_keys, rope + 8)[:, :rope]
        self.wide = torch.full((self.max_rows, heads * value + 8), fill, dtype=act, device="cuda")
        self.out = self.wide[:, :heads * value].unflatten(1, (heads, value))
        self.cache = kda.PagedLatent(1, 16, heads, 128, rope, act)
        self.dev = (self.cu.cuda(), self.cu_kv.cuda())
        self.batch = kda.make_latent_prefill_batch(*self.dev, max_rows=self.max_rows, max_kv_rows=self.max_keys,
                                                   max_new=max(self.new + [1]))
        self.scale = (nope + rope) ** -0.5
        self.io = kda.make_latent_prefill_io(self.qn, self.qr, self.k, self.kr, self.v, self.out)

    def workspace(self, fill=0xA5):
        return torch.full((kda.kda_latent_prefill_workspace_bytes(self.cache, self.io, self.batch),), fill, dtype=torch.uint8,
                          device="cuda")

    def call(self, ws=None, stream=None):
        kda.kda_latent_prefill(self.cache, self.io, self.batch, self.workspace() if ws is None else ws, stream=stream)

    def no_error(self):
        st, flags = kda.kda_latent_poll_device_error(self.cache)
        assert st == kda.KDA_OK, hex(flags)

    def check(self, scale=None, only=None):
        scale = self.scale if scale is None else scale
        qn, qr, k, kr, v = (t.double().cpu() for t in (self.qn, self.qr, self.k, self.kr, self.v))
        for i, (T, L) in enumerate(zip(self.new, self.total)):
            if T == 0 or (only is not None and i not in only):
                continue
            a, b = int(self.cu[i]), int(self.cu_kv[i])
            kk, kkr, vv = k[b:b + L], kr[b:b + L], v[b:b + L]
            s = (torch.einsum("thn,jhn->thj", qn[a:a + T], kk) + torch.einsum("thr,jr->thj", qr[a:a + T], kkr)) * scale
            ref, mag = attend(s, vv, L - T)
            top = (kk.nan_to_num(0.0, 0.0, 0.0).square().sum(-1) + kkr.nan_to_num(0.0, 0.0, 0.0).square().sum(-1)[:, None]).sqrt().max()
            qk = torch.cat((qn[a:a + T], qr[a:a + T]), -1).norm(dim=-1) * float(top) * scale
            check(self.out[a:a + T], ref, mag, qk, self.nope + self.rope, self.act, f"sequence {i}")
        assert (self.wide[:, self.heads * self.value:] == 9.0).all() and (self.out[self.rows:] == 9.0).all()

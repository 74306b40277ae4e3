"""Latent attention on a GPU held to the precision that include/kda.h states, element by element, norm against norm, and weight by
weight where channels show them apart (see latent_precision.py)."""

from __future__ import annotations

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import latent_precision as P
import latent_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ACTS = pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
FMTS = pytest.mark.parametrize("fmt", ["act", "e4m3"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()


def attend(b, q, scale):
    out = torch.full_like(q[0], 9.0)
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, scale), b.batch, b.workspace())
    b.no_error()
    return out


def rel_of(channels, qk):
    """latent_ref.check's: a score of `channels` products in 32 bits, twice over for the sum, and 2^-20."""
    return (channels + 4) * 2.0 ** -24 * qk[..., None] * 2 + 2.0 ** -20


def scored(b, i, q, held, scale):
    """Sequence i's scores [T, H, L] in float64, and what 32-bit arithmetic may move a weight by, [T, H, 1]; over e4m3 pages with
    that of q_c's second terms: elements below 2^-10 of their row's largest are off by 2^-18 of that."""
    a, T = int(b.cu[i]), b.new[i]
    (c, kr), qc, qr = held[i], q[0][a:a + T].double().cpu(), q[1][a:a + T].double().cpu()
    s = (torch.einsum("thl,jl->thj", qc, c) + torch.einsum("thr,jr->thj", qr, kr)) * scale
    qk = torch.cat((qc, qr), -1).norm(dim=-1) * float(torch.cat((c, kr), -1).norm(dim=-1).max()) * scale
    rel = rel_of(b.latent + b.rope, qk)
    if b.fmt == "e4m3" and b.act == BF:
        top = qc.abs().amax(-1, keepdim=True)
        small = (qc.abs() < top * 2.0 ** -10).double()
        rel = rel + 2 * scale * 2.0 ** -18 * top * torch.einsum("thl,jl->thj", small, c.abs()).amax(-1, keepdim=True)
    return s, rel


def unit_term(b, i, p, held):
    """Over e4m3 pages: a weight times its key's scale is off by 2^-22 of the largest weight times the largest scale, times the
    key's code; [T, H, latent]."""
    if b.fmt != "e4m3" or b.act != BF:
        return 0.0
    w = b.whole()
    pg, line = w.lines()
    at = int(w.cu[i])
    unit = 2.0 ** (b.kv.c_scale.cpu()[pg, line][at:at + b.total[i]].double() - 127)
    code = held[i][0].abs() / unit[:, None]
    return 2.0 ** -22 * float(unit.max()) * p.amax(-1, keepdim=True) * code.sum(0)


@FMTS
@ACTS
@pytest.mark.parametrize("n", [2, 3, 4])
@pytest.mark.parametrize("heads,latent", [(64, 512), (5, 256)])
def test_weights_of_few_keys(act, fmt, n, heads, latent):
    """Each key has channels of its own, so that outputs show the weights one by one."""
    b = R.Batch([1] * 6, [n] * 6, heads, latent, 64, 16, act, fmt, seed=n + heads)
    w = b.whole()
    c = torch.cat([P.disjoint(n, latent, b.gen) for _ in range(6)]).to(act)
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(c.cuda(), w.randn(w.rows, 64).cuda(), None, None), w.batch)
    held, q = b.held(), b.queries()
    out = attend(b, q, 0.07)
    for i in range(6):
        s, rel = scored(b, i, q, held, 0.07)
        p = torch.softmax(s, -1)
        bad = P.weights_within(out[i:i + 1], held[i][0], p, rel[..., 0], act, fmt)
        assert bad == 0, f"{bad} weights out of {p.numel()}"


@FMTS
@ACTS
@pytest.mark.parametrize("new,total,heads,latent", [([1, 1, 1], [2, 17, 300], 64, 512), ([1], [5000], 16, 512), ([9, 40], [200, 333], 5, 256),
                                                    ([8, 8], [8, 150], 16, 128)])
def test_absorbed_within_the_contract(act, fmt, new, total, heads, latent):
    b = R.Batch(new, total, heads, latent, 64, 64, act, fmt, seed=sum(total))
    held, q = b.fill_cache(), b.queries()
    out = attend(b, q, 0.05)
    for i, (T, L) in enumerate(zip(new, total)):
        a = int(b.cu[i])
        s, rel = scored(b, i, q, held, 0.05)
        ref, mag = R.attend(s, held[i][0][:, None], L - T)
        hidden = torch.arange(L) > L - T + torch.arange(T)[:, None, None]
        p = torch.softmax(s.masked_fill(hidden, -torch.inf), -1)
        P.within_contract(out[a:a + T], ref, mag, rel, act, unit_term(b, i, p, held), f"sequence {i}")
        if L - T >= 150:
            P.flat_rows(out[a:a + T], ref, act, fmt, f"sequence {i}")


@ACTS
@pytest.mark.parametrize("new,total,heads,nope,value", [([1, 3, 100], [2, 4, 300], 8, 128, 128), ([300], [2500], 2, 128, 128),
                                                        ([128, 129], [700, 130], 3, 64, 64), ([20], [6000], 2, 128, 64)])
def test_expanded_within_the_contract(act, new, total, heads, nope, value):
    r = R.Rows(new, total, heads, nope, 64, value, act, seed=sum(total))
    r.call()
    r.no_error()
    qn, qr, k, kr, v = (t.double().cpu() for t in (r.qn, r.qr, r.k, r.kr, r.v))
    for i, (T, L) in enumerate(zip(new, total)):
        a, z = int(r.cu[i]), int(r.cu_kv[i])
        kk, kkr = k[z:z + L], kr[z:z + L]
        s = (torch.einsum("thn,jhn->thj", qn[a:a + T], kk) + torch.einsum("thr,jr->thj", qr[a:a + T], kkr)) * r.scale
        ref, mag = R.attend(s, v[z:z + L], L - T)
        top = (kk.square().sum(-1) + kkr.square().sum(-1)[:, None]).sqrt().max()
        qk = torch.cat((qn[a:a + T], qr[a:a + T]), -1).norm(dim=-1) * float(top) * r.scale
        P.within_contract(r.out[a:a + T], ref, mag, rel_of(nope + 64, qk), act, what=f"sequence {i}")
        if L - T >= 150:
            P.flat_rows(r.out[a:a + T], ref, act, what=f"sequence {i}")

"""Latent attention at its corners on a GPU, against the plain float64 statements of latent_ref.py: values that are not finite
under weights too small for 32 bits, values next to the end of the type's range, many short items in a CTA, and heads
that do not fill their groups."""

from __future__ import annotations

import itertools
import math

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import latent_precision as P
import latent_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
ACTS = pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()


@ACTS
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("new,ctx", [(100, 200), (300, 200), (1, 400), (60, 0)])
def test_values_under_weights_too_small_for_32_bits(act, bad, new, ctx):
    """A key that scores 200 below all others (2^-288 of their weight) with a value that is not finite: no row that sees it has a
    finite output in that channel, wherever the key lies; rows before it and other channels do not change."""
    total = new + ctx
    far = float(torch.tensor(-200.0 * (128 + 64) ** 0.5).to(act))
    for at in sorted({0, 5, 64, total // 2, total - new, total - 1}):
        if at >= total:
            continue
        r = R.Rows([new, 3], [total, 50], 2, 128, 64, 128, act, seed=at + new)
        r.qn[..., 0], r.k[..., 0] = 1.0, 0.0
        r.k[at, :, 1:] = 0.0
        r.kr[at] = 0.0
        r.k[at, :, 0] = far
        r.call()
        r.check()
        kept = r.out.clone()
        r.v[at, :, 1] = bad
        r.call()
        r.no_error()
        got, first = r.out, max(at - ctx, 0)  # the first row that sees the key
        assert not torch.isfinite(got[first:new, :, 1]).any(), at
        others = [c for c in range(128) if c != 1]
        assert torch.equal(got[:first], kept[:first]) and torch.equal(got[new:], kept[new:]), at
        a, b = got[first:new][..., others].double(), kept[first:new][..., others].double()
        # in a tile that some row does not see in full the value's other channels join in another order: total units of 2^-24
        # of sum p |v| <= max |v|, and then a rounding to the neighbour
        step = b.abs() * (2 * R.half_step(BF) if act == BF else 2.0 ** -23)
        top = float(r.v[:total].float().nan_to_num(0.0, 0.0, 0.0).abs().max())
        assert ((a - b).abs() <= step + total * 2.0 ** -24 * top).all(), at


@ACTS
@pytest.mark.parametrize("new", [30, 200])
def test_rows_without_weights_beside_values_that_are_not_finite(act, new):
    """All scores -inf: zeros, but in the channel that holds an infinity, which may be NaN."""
    r = R.Rows([new], [new + 100], 2, 128, 64, 64, act, seed=new)
    r.kr[:, 0] = -INF
    r.qr[..., 0] = 1.0
    r.v[new + 50, :, 3] = INF
    r.call()
    r.no_error()
    first = max(new - 50, 0)  # the first row that sees it
    assert (r.out[..., :3] == 0).all() and (r.out[..., 4:] == 0).all() and (r.out[:first, :, 3] == 0).all()
    seen = r.out[first:, :, 3]
    assert (torch.isnan(seen) | (seen == 0)).all()


@ACTS
@pytest.mark.parametrize("new", [4, 300])
def test_large_values_under_rising_scores(act, new):
    """The first 64 keys score 2^9 below the others, which together stay below where the reference would move: 64 values of
    2^105 (up to 2^107) weigh 2^15 there, 8 times over, and their weighted mean is as finite as they are."""
    total, gain = 500, 2.0 ** 105
    r = R.Rows([new], [total], 2, 128, 64, 128, act, seed=new)
    for t in (r.qn, r.qr, r.k, r.kr):
        t.zero_()
    r.qn[..., 0] = 1.0
    r.k[64:, :, 0] = 9 * math.log(2.0) / r.scale
    r.v.mul_(gain)
    assert float(r.v.float().abs().max()) * 2.0 ** 16 * -(-total // 64) < 2.0 ** 127
    r.call()
    r.no_error()
    s = (torch.einsum("thn,jhn->thj", r.qn.double().cpu(), r.k.double().cpu())) * r.scale
    ref, mag = R.attend(s, r.v.double().cpu() / gain, total - new)
    P.within_contract(r.out.double().cpu() / gain, ref, mag, 2.0 ** -14, act)


@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act"), (F32, "e4m3")])
@pytest.mark.parametrize("new,heads", [(1, 16), (40, 3)])
def test_large_latents_under_rising_scores(act, fmt, new, heads):
    """As above for the absorbed form, whose reference moves when a score leads it by 8."""
    total, gain, scale = 300, 2.0 ** 105, 0.05
    b = R.Batch([new], [total], heads, 512, 64, 64, act, fmt, seed=new)
    w = b.whole()
    kr = torch.zeros(total, 64)
    kr[64:, 0] = 7.5 * math.log(2.0) / scale
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(w.randn(total, 512, gain=gain).cuda(), kr.to(act).cuda(), None, None), w.batch)
    c, kr = b.held()[0]
    assert float(c.abs().max()) * 2.0 ** 8 * total < 2.0 ** 127
    q = b.queries()
    q[0].mul_(2.0 ** -105 / 64), q[1].zero_()
    q[1][..., 0] = 1.0
    out = torch.empty_like(q[0])
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, scale), b.batch, b.workspace())
    b.no_error()
    s = (torch.einsum("thl,jl->thj", q[0].double().cpu(), c) + torch.einsum("thr,jr->thj", q[1].double().cpu(), kr)) * scale
    ref, mag = R.attend(s, c[:, None] / gain, total - new)
    # scores of at most 6: 576 products and 4 more, in 32 bits; over e4m3 pages q_c's small elements and the smallest weights
    extra = 2.0 ** -22 * total * float(c.abs().max()) / gain if fmt == "e4m3" and act == BF else 0.0
    P.within_contract(out.double().cpu() / gain, ref, mag, 2.0 ** -10 if fmt == "e4m3" and act == BF else 2.0 ** -11, act, extra)


ORDERS = [k for t in itertools.product(range(1, 5), repeat=3) for k in t]  # every order of three items of one to four tiles


@ACTS
@pytest.mark.parametrize("n,heads,news,max_new", [
    (100, 64, [1, 2], 2),              # sides by keys, a sequence's heads in a row
    (1500, 1, [1, 3, 2], 3),           # by keys, other numbers of tiles from item to item
    (1500, 1, [1, 130, 7, 2], 200),    # by rows: the second side sits most items out
    (600, 2, [130, 1, 129, 128, 5], 130),
])
def test_short_items_in_every_order(act, n, heads, news, max_new):
    """A CTA's items of one to four tiles of 128 keys one after the other: what one leaves in rings, barriers and tensor memory is
    the next one's beginning."""
    total = [128 * ORDERS[i % len(ORDERS)] - (37 * i) % 128 for i in range(n)]
    new = [min(news[i % len(news)], t) for i, t in enumerate(total)]
    if act == F32:
        n = n // 4
        total, new = total[:n], new[:n]
    gen = torch.Generator(device="cuda").manual_seed(n + heads)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(act)

    rows, keys, N, Rr, V = sum(new), sum(total), 64, 64, 64
    qn, qr, k, kr, v = randn(rows, heads, N), randn(rows, heads, Rr), randn(keys, heads, N), randn(keys, Rr), randn(keys, heads, V)
    out = torch.full((rows + 1, heads, V), 9.0, dtype=act, device="cuda")
    cache = kda.PagedLatent(1, 16, heads, 128, Rr, act)
    cu, cu_kv = (torch.tensor([0, *itertools.accumulate(x)], dtype=torch.int32, device="cuda") for x in (new, total))
    batch = kda.make_latent_prefill_batch(cu, cu_kv, rows, keys, max_new)
    io = kda.make_latent_prefill_io(qn, qr, k, kr, v, out)
    ws = torch.empty(kda.kda_latent_prefill_workspace_bytes(cache, io, batch), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        kda.kda_latent_prefill(cache, io, batch, ws)
    assert kda.kda_latent_poll_device_error(cache) == (kda.KDA_OK, 0)
    assert (out[rows:] == 9.0).all()
    scale = (N + Rr) ** -0.5
    j = torch.arange(512, device="cuda")
    for a in range(0, n, 50):  # 50 sequences at a time, padded, in float64 on the device
        ids = torch.arange(a, min(a + 50, n), device="cuda")
        T, L = (cu[ids + 1] - cu[ids]).long(), (cu_kv[ids + 1] - cu_kv[ids]).long()
        t = torch.arange(int(T.max()), device="cuda")
        row, key = (cu[ids].long()[:, None] + t).clamp(max=rows - 1), (cu_kv[ids].long()[:, None] + j).clamp(max=keys - 1)
        s = torch.einsum("nthc,njhc->nthj", qn[row].double(), k[key].double())
        s = (s + torch.einsum("nthc,njc->nthj", qr[row].double(), kr[key].double())) * scale
        seen = j <= (L - T)[:, None, None] + t[:, None]
        p = torch.softmax(s.masked_fill(~seen[:, :, None], -torch.inf), -1)
        ref, mag = (torch.einsum("nthj,njhc->nthc", p, x) for x in (v[key].double(), v[key].double().abs()))
        real = t < T[:, None]
        top = torch.cat((k[key].double(), kr[key].double()[:, :, None].expand(-1, -1, heads, -1)), -1).norm(dim=-1).max()
        qk = torch.cat((qn[row], qr[row]), -1).double().norm(dim=-1) * top * scale
        rel = (N + Rr + 4) * 2.0 ** -24 * qk[..., None] * 2 + 2.0 ** -20
        P.within_contract(out[row][real], ref[real].cpu(), mag[real].cpu(), rel[real].cpu(), act, what=f"sequences from {a}")


@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act"), (F32, "e4m3")])
@pytest.mark.parametrize("heads,new,total,latent", [
    (65, [1, 1], [300, 64], 512), (67, [1] * 40, [1 + 29 * i % 400 for i in range(40)], 512), (71, [2, 1], [2000, 65], 256),
    (127, [1, 3], [129, 700], 128), (129, [1], [900], 512), (131, [5, 0, 1], [5, 9, 190], 128), (33, [1, 2], [300, 80], 512),
    (37, [7, 1], [90, 1500], 256), (193, [1], [333], 128)])
def test_heads_that_do_not_fill_their_groups(act, fmt, heads, new, total, latent):
    """Rows past the last head are nobody's: what stands behind and between the heads of out stays, whole items and parts."""
    b = R.Batch(new, total, heads, latent, 64, 64, act, fmt, seed=heads, fill=NAN, extra_rows=1)
    held, q = b.fill_cache(), b.queries()
    guard = torch.full((b.max_rows, heads + 3, latent + 8), 9.0, dtype=act, device="cuda")
    out = guard[:, 1:1 + heads, 8:]
    # queries whose next rows hold NaN, so that one read for a head that is not there would show
    wide = [torch.full((b.max_rows, heads + 2, t.shape[2]), NAN, dtype=act, device="cuda") for t in q]
    for w, t in zip(wide, q):
        w[:, :heads] = t
    io = kda.make_latent_attn_io(*(w[:, :heads] for w in wide), out, 0.07)
    kda.kda_latent_attend(b.kv, io, b.batch, b.workspace())
    b.no_error()
    b.check_attend(q, out, held, 0.07)
    assert (out[b.rows:] == 9.0).all() and (guard[:, 0] == 9.0).all() and (guard[:, heads + 1:] == 9.0).all() and (guard[..., :8] == 9.0).all()


@ACTS
def test_time_follows_the_groups_of_heads(act):
    """A head or three past a full group cost another pass over the pages, not one a head (67 times where that was so)."""
    us = {}
    per = 64 if act == BF else 32
    for heads in (per, per + 3, 2 * per):
        b = R.Batch([1] * 8, [4000 + 300 * i for i in range(8)], heads, 512, 64, 64, act, "act", seed=1)
        q = b.queries()
        io, ws = kda.make_latent_attn_io(*q, torch.empty_like(q[0]), 0.05), b.workspace()
        for _ in range(3):
            kda.kda_latent_attend(b.kv, io, b.batch, ws)
        torch.cuda.synchronize()
        kda.kda_profile_start(64)
        for _ in range(10):
            kda.kda_latent_attend(b.kv, io, b.batch, ws)
        torch.cuda.synchronize()
        us[heads] = kda.kda_profile_stop()["latent_attend"][1]
    assert us[per + 3] < 4 * us[per] and us[2 * per] < 4 * us[per], us

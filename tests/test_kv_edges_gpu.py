"""Paged-cache operators at the edges of their contract, on a GPU: tables that contradict themselves, values that are not
finite, and what the plain tests of test_kv_gpu.py leave out.  Tolerances are those of that file's docstring."""

from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import kv_ref as R
from test_kv_gpu import check_attend, fill_cache, held, stored

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()


# ---- tables that contradict themselves -----------------------------------------------------------------------------------

DECREASING = [[0, 10, 3, 8], [0, 12, 14, 15, 1, 1, 30], [0, 8, 0, 2, 8]]


def with_cu(cu, length, act, fmt, hq=4, hkv=2, d=64, page=16):
    """A cache of `length` tokens per sequence and a batch with these cu_seqlens; (batch driver, its consistent sequences
    as (index, first row, tokens))."""
    n, rows = len(cu) - 1, max(cu)
    b = R.Batch([0] * n, [length] * n, hq, hkv, d, page, act, fmt, seed=7, extra_rows=rows)
    b.dev[0].copy_(torch.tensor(cu, dtype=torch.int32))
    b.batch = kda.make_kv_batch(*b.dev, max_rows=rows, max_new=rows)
    good = [(i, a, e - a) for i, (a, e) in enumerate(zip(cu[:-1], cu[1:])) if 0 <= a <= e <= rows and e - a <= length]
    return b, rows, good


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cu", DECREASING)
def test_decreasing_cu_seqlens_touch_no_other_line(cu, act, fmt):
    """Only rows and lines of the consistent sequences change, and the error word says that something is wrong."""
    length, page = 64, 16
    b, rows, good = with_cu(cu, length, act, fmt, page=page)
    lines = torch.zeros(b.kv.num_pages, page, dtype=torch.bool)
    owned = torch.zeros(rows, dtype=torch.bool)
    for i, a, T in good:
        owned[a:a + T] = True
        for p in range(length - T, length):
            lines[int(b.table[i, p // page]), p % page] = True
    pools = [t for t in (b.kv.k.view(torch.uint8), b.kv.v.view(torch.uint8), b.kv.k_scale, b.kv.v_scale) if t is not None]
    before = [t.clone() for t in pools]
    q, k, v = (b.randn(rows, n).cuda() for n in (4, 2, 2))
    q_out = torch.full_like(q, 7.0)
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(q, k, v, q_out), b.batch)
    assert kda.kda_kv_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_META)
    for old, new in zip(before, pools):
        same = (old == new).flatten(3).all(3) if old.dim() > 3 else old == new  # [page, head, line]
        assert same.all(1).cpu()[~lines].all()
    assert (q_out.cpu()[~owned] == 7.0).all()
    ko, vo = (torch.full((rows, 2, 64), 5.0, dtype=act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, b.batch, ko, vo)
    assert kda.kda_kv_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_META)
    assert (ko.cpu()[~owned] == 5.0).all() and (vo.cpu()[~owned] == 5.0).all()
    out = torch.full_like(q, 9.0)
    ws = torch.empty(kda.kda_kv_attend_workspace_bytes(b.kv, b.batch), dtype=torch.uint8, device="cuda")
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, ws)
    assert kda.kda_kv_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_META)
    assert (out.cpu()[~owned] == 9.0).all()


@pytest.mark.parametrize("which", ["first", "middle", "last"])
@pytest.mark.parametrize("length", [-1, -2 ** 31, 65, 2 ** 31 - 1])
def test_empty_sequences_with_bad_lengths_are_reported(length, which):
    """A sequence without rows in the call is as inconsistent as another: all three calls say so and serve the others."""
    at = {"first": 0, "middle": 20, "last": 39}[which]
    new = [1] * 40
    new[at] = 0
    b = R.Batch(new, [64] * 40, 2, 1, 32, 16, BF, "act", seed=3)
    b.dev[1][at] = length
    q, k, v = (b.randn(b.rows, n).cuda() for n in (2, 1, 1))
    q_out, out = torch.full_like(q, 7.0), torch.full_like(q, 9.0)
    bad = (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_META)
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(q, k, v, q_out), b.batch)
    assert kda.kda_kv_poll_device_error(b.kv) == bad
    ko, vo = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
    kda.kda_kv_read(b.kv, b.batch, ko, vo)
    assert kda.kda_kv_poll_device_error(b.kv) == bad
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    assert kda.kda_kv_poll_device_error(b.kv) == bad
    assert torch.equal(q_out, q) and torch.equal(ko, k) and torch.equal(vo, v) and not (out == 9.0).any()


# ---- the last positions --------------------------------------------------------------------------------------------------

def exact_angle(p, f):
    """p * f in (-pi, pi], the product and its reduction exact (pi to 50 digits)."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937511")
    x = Fraction(float(f)) * p
    x -= 2 * pi * round(x / (2 * pi))
    return float(x)


@pytest.mark.parametrize("base", [10000.0, 500000.0, None])
def test_angles_of_the_last_positions(base):
    """Angles are good to the cosine's 7e-8 up to the last position there is: a frequency in turns as a 53-bit number would
    be off by up to 5e-7 there."""
    page, d = 128, 128
    last = 2 ** 31 - 1024
    freq = ([base ** (-2.0 * i / d) for i in range(d // 2)] if base else
            [-1.0, -0.3, 0.75, 1e-9, 37.5, 1000.0, -2500.125, 123456.789] * 8)
    b = R.Batch([4], [4], 1, 1, d, page, F32, "act", seed=5)
    table = torch.zeros(1, -(-last // page), dtype=torch.int32, device="cuda")
    batch = kda.make_kv_batch(b.dev[0], torch.tensor([last], dtype=torch.int32, device="cuda"), table, max_rows=4, max_new=4)
    q = torch.zeros(4, 1, d, device="cuda")
    q[..., :d // 2] = 1.0
    q_out, kv = torch.empty_like(q), torch.zeros_like(q)
    kda.kda_kv_append(b.kv, kda.make_qk_params(None, None, 1e-5, freq), kda.make_kv_io(q, kv, kv, q_out), batch)
    assert kda.kda_kv_poll_device_error(b.kv)[0] == kda.KDA_OK
    ang = torch.tensor([[exact_angle(last - 4 + t, f) for f in freq] for t in range(4)], dtype=torch.float64)
    got = q_out[:, 0].double().cpu()
    worst = max(float((got[:, :d // 2] - ang.cos()).abs().max()), float((got[:, d // 2:] - ang.sin()).abs().max()))
    assert worst <= 7.2e-8, worst


# ---- values that are not finite ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", [False, True], ids=["", "norm"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(128, 64), (128, 96), (64, 24), (32, 24), (16, 8)])
def test_non_finite_values_stay_in_their_pair(d, rot, inter, norm, act, fmt):
    """An infinity or NaN reaches the other channel of its pair and, with the norm, the row; channels that do not turn are
    those that came."""
    b = R.Batch([6], [40], 2, 1, d, 16, act, fmt, seed=d + rot)
    q, k, v = (b.randn(6, n) for n in (2, 1, 1))
    for x in (q, k):
        x[0, :, 1] = float("inf")           # turns
        x[1, :, rot - 1] = float("-inf")    # turns
        x[2, :, 0] = float("nan")           # turns
        x[3, :, rot] = float("inf")         # does not turn
        x[4, :, d - 1] = float("nan")       # does not turn
    w = (1 + 0.1 * torch.randn(2, d, generator=b.gen)).to(act) if norm else (None, None)
    freq = [1000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    params = kda.make_qk_params(*(None if x is None else x.cuda() for x in w), 1e-5, freq, inter)
    q_out = torch.full_like(q, 7.0, device="cuda")
    kda.kda_kv_append(b.kv, params, kda.make_kv_io(q.cuda(), k.cuda(), v.cuda(), q_out), b.batch)
    ko, vo = (torch.full((6, 1, d), 5.0, dtype=act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, b.batch, ko, vo)
    assert kda.kda_kv_poll_device_error(b.kv)[0] == kda.KDA_OK
    for got, x, wx, e4m3 in ((q_out, q, w[0], False), (ko, k, w[1], fmt == "e4m3")):
        got, ref = got.double().cpu(), R.norm_rotate(x, wx, b.positions(), freq, inter, 1e-5)
        if e4m3:  # stored as NaN
            ref = torch.where(torch.isfinite(ref), ref, torch.nan)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        fin = torch.isfinite(ref)
        assert torch.equal(got[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
        top = torch.where(fin, ref, 0.0).abs().amax(-1, keepdim=True)
        tol = ref.abs() * (2.0 ** -8 if act == BF else 0.0) + 2.0 ** -18 * top
        if e4m3:  # half a step of e4m3, at the small end half of 2^-9 of a unit that is at most max / 224
            tol = tol + ref.abs() * 2.0 ** -4 + top * (2.0 ** -10 / 224)
        assert ((got - ref).abs() <= tol)[fin].all()
        if not norm and not e4m3:
            assert torch.equal(got[..., rot:].nan_to_num(), x[..., rot:].double().nan_to_num())


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,hq,hkv,d", [(1, 2, 1, 128), (9, 2, 1, 128), (40, 8, 2, 128), (150, 4, 2, 64), (3, 2, 1, 32)])
@pytest.mark.parametrize("scale", [1e-9, 1e-30, 2e-45])
def test_rows_of_zeros_and_small_scales(scale, new, hq, hkv, d, act, fmt):
    """A query of zeros weighs its keys alike, whatever the scale; so does any query at a scale this small."""
    b = R.Batch([new], [new + 60], hq, hkv, d, 16, act, fmt, seed=89)
    v = b.whole().randn(new + 60, hkv)
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, v.cuda(), v.cuda(), None), b.whole().batch)
    ko, vo = (torch.empty(new + 60, hkv, d, dtype=act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, b.whole().batch, ko, vo)
    q = b.randn(new, hq)
    q[::2] = 0.0
    out = torch.full_like(q, 9.0, device="cuda")
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q.cuda(), out, scale), b.batch, b.workspace())
    assert kda.kda_kv_poll_device_error(b.kv)[0] == kda.KDA_OK
    vo = vo.double().cpu()
    for t in range(new):  # scores below 1e-6: weights alike to 1e-6
        ref = vo[:61 + t].mean(0).repeat_interleave(hq // hkv, 0)
        mag = vo[:61 + t].abs().mean(0).repeat_interleave(hq // hkv, 0)
        tol = mag * (4e-6 + (2 * 2.0 ** -8 if act == BF else 0.0)) + (ref.abs() * 2.0 ** -8 if act == BF else 0.0)
        assert ((out[t].double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
def test_quantised_largest_and_smallest_values(act):
    """The type's largest values (what rounds to 2^128 reads back as infinity), and vectors below every e4m3 step of the
    smallest scale (in bf16 multiples of 2^-133 read back)."""
    d, top = 16, torch.finfo(act).max
    rows = torch.zeros(8, 1, d, dtype=torch.float64)
    rows[0, 0, 0], rows[0, 0, 1] = top, -top / 3
    rows[1, 0, 0] = -top
    rows[2, 0, 0], rows[2, 0, 1] = 1.921875 * 2.0 ** 127, 1.0  # below the border at 1.9375 * 2^127
    rows[3, 0, 0] = 1.75 * 2.0 ** 127
    rows[4, 0] = torch.arange(d) * 2.0 ** -133
    rows[5, 0, 0] = 2.0 ** -133
    rows[6, 0, 0], rows[6, 0, 1] = 2.0 ** -126, -3 * 2.0 ** -133
    rows[7, 0, 0], rows[7, 0, 1] = top, float("inf")
    x = rows.to(act)
    b = R.Batch([8], [8], 1, 1, d, 16, act, "e4m3")
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, x.cuda(), x.cuda(), None), b.batch)
    qv, qe = R.quantise(x.double().numpy())
    for vals, e in stored(b):
        assert np.array_equal(e.numpy(), qe) and np.array_equal(vals.numpy(), qv, equal_nan=True)
    ko, vo = (torch.empty(8, 1, d, dtype=act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, b.batch, ko, vo)
    want = torch.from_numpy(qv * 2.0 ** (qe - 127.0)[..., None]).to(torch.float32).to(act)
    assert torch.isinf(want[0, 0, 0]) and torch.isinf(want[1, 0, 0]) and torch.isfinite(want[2:7]).all()
    for got in (ko, vo):
        assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,hq,hkv,d", [(1, 16, 2, 128), (9, 4, 2, 128), (150, 4, 2, 64), (40, 2, 1, 32), (1, 2, 1, 16)])
def test_non_finite_queries_stay_in_their_row(new, hq, hkv, d, act, fmt):
    """A query with a NaN or an infinity gives NaN (an infinity of keys of both signs is one of +inf scores) and leaves the
    other heads and tokens alone."""
    b = R.Batch([new, 1], [new + 90, 200], hq, hkv, d, 32, act, fmt, seed=101)
    cache = fill_cache(b)
    q = b.randn(b.rows, hq)
    hit = [(0, 0, float("nan")), (new // 2, hq - 1, float("inf")), (new, 1, float("-inf"))]
    clean = q.clone()
    for t, h, x in hit:
        q[t, h, d // 2] = x
    out, want = (torch.empty_like(q, device="cuda") for _ in range(2))
    for x, o in ((q, out), (clean, want)):
        kda.kda_kv_attend(b.kv, kda.make_attn_io(x.cuda(), o), b.batch, b.workspace())
        assert kda.kda_kv_poll_device_error(b.kv)[0] == kda.KDA_OK
    check_attend(b, clean, want, cache, d ** -0.5)
    for t, h, _ in hit:
        assert torch.isnan(out[t, h]).all()
        out[t, h] = want[t, h]
    check_attend(b, clean, out, cache, d ** -0.5)


# ---- tighter looks at attention ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,total,hq,hkv,d", [([1, 6], [300, 200], 4, 2, 64), ([1, 1], [900, 50], 16, 2, 128),
                                                ([40, 7], [333, 7], 4, 2, 128), ([200], [390], 2, 1, 64),
                                                ([3, 20], [100, 260], 2, 1, 32), ([1], [70], 3, 1, 16)])
def test_far_apart_scores_pick_their_value(new, total, hq, hkv, d, act, fmt):
    """Scores thousands apart: every row whose best key leads by more than the scores' error gives that key's value."""
    b = R.Batch(new, total, hq, hkv, d, 16, act, fmt, seed=97)
    cache = fill_cache(b, gain=100.0)
    q = (b.randn(b.rows, hq) * 50).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out, 1.0), b.batch, b.workspace())
    assert kda.kda_kv_poll_device_error(b.kv)[0] == kda.KDA_OK
    got, q = out.double().cpu(), q.double().cpu()
    sure, at = 0, 0
    for (T, L), (k, v) in zip(zip(new, total), cache):
        for t in range(T):
            for h in range(hq):
                kk, vv, qq = k[:L - T + t + 1, h // b.group], v[:L - T + t + 1, h // b.group], q[at + t, h]
                s, order = torch.sort(kk @ qq, descending=True)
                # products and sums in 32 bits; with e4m3 keys q is good to 2^-18 of its largest channel
                err = (d + 4) * 2.0 ** -24 * float(qq.norm() * kk.norm(dim=-1).max())
                err += 2.0 ** -18 * float(qq.abs().max() * kk.abs().sum(-1).max())
                if len(s) > 1 and float(s[0] - s[1]) < 40 + 2 * err:
                    continue
                sure += 1
                ref = vv[order[0]]
                # the others weigh e^-40 at most; bf16: rn(rn(w) v / w), two roundings by 2^-8 of what they round
                tol = ref.abs() * (2 * 2.0 ** -8 + 2.0 ** -15 if act == BF else 2.0 ** -22) + 1e-12
                assert ((got[at + t, h] - ref).abs() <= tol).all()
        at += T
    assert sure >= 0.8 * b.rows * hq


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,hq,hkv,d", [(4, 4, 2, 128), (100, 4, 2, 128), (300, 2, 1, 64), (20, 3, 1, 32)])
def test_masked_values_may_be_anything_in_32_bits(bad, new, hq, hkv, d, fmt):
    """The masked-value checks with the bound that 32-bit calls have, over all rows."""
    total = new + 70
    b = R.Batch([new], [total], hq, hkv, d, 32, F32, fmt, seed=11)
    fill_cache(b)
    at = total - new // 2
    page, line = int(b.table[0, at // 32]), at % 32
    last = int(b.table[0, (total - 1) // 32]), (total - 1) % 32
    if fmt == "e4m3":
        b.kv.v.view(torch.uint8)[page, :, line, 1] = 0xFF
        b.kv.k.view(torch.uint8)[last[0], :, last[1], 0] = 0x7F
    else:
        b.kv.v[page, :, line, 1] = bad
        b.kv.k[last[0], :, last[1], 0] = float("nan")
    q = b.randn(b.rows, hq).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    check_attend(b, q, out, held(b), d ** -0.5)
    t_bad = at - (total - new)
    assert torch.isfinite(out[:t_bad]).all() and not torch.isfinite(out[t_bad:, :, 1]).any()
    assert torch.isfinite(out[t_bad:-1, :, 2:]).all() and torch.isnan(out[-1]).all()

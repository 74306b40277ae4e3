"""Paged-cache operators on a GPU against plain float64 statements: kda_kv_append, kda_kv_read, kda_kv_attend and runs
of them together.

Tolerances.  A rounding to type t is off by at most eps(t) / 2 of the value (bf16 2^-8, e4m3 2^-4 and, below its normal
range, 2^-10 of the scale's unit).  Arithmetic is in 32 bits (unit 2^-24):
  append  the sum of squares is a tree of depth at most 12, then a root, a division, two products, and two products and
          a sum with a cosine and a sine good to 2 units and an angle good to pi units: under 32 units, of a value whose
          partner may be the row's largest: 2^-18 max|row| covers both terms of the rotation.
  attend  a score sums d products (d + 4 units of sum |q k| scale at most); its weight is off by that much relatively,
          and by 2^-20 for the power of two and the sums.  bf16 inputs may have their weights rounded to bf16 before
          they meet the values (2^-8 of each weight in the numerator, and in the sum).  All of it times sum p |v|."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import kv_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()


def half_step(t):
    return torch.finfo(t).eps / 2


def no_device_error(kv):
    st, flags = kda.kda_kv_poll_device_error(kv)
    assert st == kda.KDA_OK, hex(flags)


def run_append(b, rot=0, inter=False, norm=True, strided=False, seed=1, in_place=False, base=10000.0):
    """Appends b's rows; returns (inputs, float64 q and k after norm and rotation, q_out)."""
    q, k, v = b.randn(b.max_rows, b.hq), b.randn(b.max_rows, b.hkv), b.randn(b.max_rows, b.hkv)
    wq = (1 + 0.1 * torch.randn(b.d, generator=b.gen)).to(b.act) if norm else None
    wk = (1 + 0.1 * torch.randn(b.d, generator=b.gen)).to(b.act) if norm else None
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if strided:
        pad = 16
        fused = torch.zeros(b.max_rows, (b.hq + 2 * b.hkv) * b.d + pad, dtype=b.act, device="cuda")
        dq = fused[:, :b.hq * b.d].unflatten(1, (b.hq, b.d))
        dk = fused[:, b.hq * b.d:(b.hq + b.hkv) * b.d].unflatten(1, (b.hkv, b.d))
        dv = fused[:, (b.hq + b.hkv) * b.d:-pad].unflatten(1, (b.hkv, b.d))
        dq.copy_(q), dk.copy_(k), dv.copy_(v)
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    q_out = dq if in_place else torch.full_like(q, 7.0, device="cuda")
    params = kda.make_qk_params(None if wq is None else wq.cuda(), None if wk is None else wk.cuda(), 1e-5, freq, inter)
    kda.kda_kv_append(b.kv, params, kda.make_kv_io(dq, dk, dv, q_out), b.batch)
    pos = b.positions()
    rq = R.norm_rotate(q[:b.rows], wq, pos, freq, inter, 1e-5)
    rk = R.norm_rotate(k[:b.rows], wk, pos, freq, inter, 1e-5)
    return (q, k, v), rq, rk, q_out


def check_rows(got, ref, act):
    got = got.double().cpu()
    tol = ref.abs() * (half_step(act) if act == BF else 0) + 2.0 ** -18 * ref.abs().amax(-1, keepdim=True)
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} values off, worst {float(((got - ref).abs() / tol.clamp(min=1e-300)).max()):.2f} tolerances"


def stored(b):
    """The batch rows' lines from the raw pages: values [rows, hkv, d] and biased exponents [rows, hkv] (or None)."""
    out = []
    pages = [(b.kv.k, b.kv.k_scale), (b.kv.v, b.kv.v_scale)]
    seq = [i for i, T in enumerate(b.new) for _ in range(T)]
    pos = b.positions()
    page = torch.tensor([int(b.table[s, p // b.page]) for s, p in zip(seq, pos)], dtype=torch.long)
    line = torch.tensor([p % b.page for p in pos], dtype=torch.long)
    for t, e in pages:
        x = t.float().cpu()[page, :, line].double()
        out.append((x, None if e is None else e.cpu()[page, :, line].long()))
    return out


APPEND = [
    # new, total, hq, hkv, d, page, rot, inter, norm
    ([1], [1], 8, 1, 128, 16, 128, False, True),
    ([1], [100001], 64, 8, 128, 64, 128, False, True),
    ([5, 0, 1, 17], [5, 0, 33, 130], 6, 2, 64, 16, 64, True, True),
    ([3, 2], [3, 70], 7, 1, 16, 32, 8, False, True),
    ([33, 40], [33, 41], 4, 4, 32, 128, 24, False, False),
    ([70, 9], [71, 90], 12, 4, 64, 64, 40, True, True),
    ([1] * 40, list(range(1, 41)), 14, 2, 128, 32, 0, False, True),
    ([300], [1000], 3, 3, 128, 64, 96, False, True),
]


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_and_read(case, act, fmt):
    new, total, hq, hkv, d, page, rot, inter, norm = APPEND[case]
    b = R.Batch(new, total, hq, hkv, d, page, act, fmt, seed=case, extra_rows=2)
    before = (b.kv.k.view(torch.uint8).clone(), b.kv.v.view(torch.uint8).clone())
    (q, k, v), rq, rk, q_out = run_append(b, rot, inter, norm, strided=case % 2 == 1)
    no_device_error(b.kv)
    check_rows(q_out[:b.rows], rq, act)
    assert (q_out[b.rows:] == 7.0).all()  # rows behind the last sequence
    (ks, ke), (vs, ve) = stored(b)
    rv = v[:b.rows].double()
    if fmt == "act":
        check_rows(ks, rk, act)
        assert torch.equal(vs, rv)
    else:
        qv, qe = R.quantise(rv.numpy())
        assert np.array_equal(ve.numpy(), qe) and np.array_equal(vs.numpy(), qv)
        unit = 2.0 ** (ke.double() - 127)[..., None]
        amax = rk.abs().amax(-1)
        slack = 2.0 ** -18 * amax
        assert (unit[..., 0] * 448 >= amax - slack).all() and (unit[..., 0] * 224 <= amax + slack).all()
        err = (ks * unit - rk).abs()
        assert (err <= rk.abs() * 2.0 ** -4 + unit * 2.0 ** -10 + slack[..., None]).all()
    # only the batch's lines changed
    touched = torch.zeros(b.kv.num_pages, page, dtype=torch.bool)
    for i, (T, L) in enumerate(zip(new, total)):
        for p in range(L - T, L):
            touched[int(b.table[i, p // page]), p % page] = True
    keep = ~touched[:, None, :, None].expand(-1, hkv, -1, d)
    for old, t in zip(before, (b.kv.k, b.kv.v)):
        old = old.view(t.dtype).float().cpu()
        assert torch.equal(old[keep], t.float().cpu()[keep])
    # and read back
    ko, vo = (torch.full((b.max_rows, hkv, d), 5.0, dtype=act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, b.batch, ko, vo)
    no_device_error(b.kv)
    for o, (x, e) in ((ko, (ks, ke)), (vo, (vs, ve))):
        ref = x if e is None else x * 2.0 ** (e.double() - 127)[..., None]
        assert torch.equal(o[:b.rows].double().cpu(), ref)
        assert (o[b.rows:] == 5.0).all()


def test_append_in_place_and_keys_only():
    b = R.Batch([20, 3], [20, 50], 8, 2, 64, 16, BF, "act", seed=3)
    _, rq, _, q_out = run_append(b, 64, False, True, in_place=True)
    check_rows(q_out, rq, BF)
    k, v = b.randn(b.rows, 2).cuda(), b.randn(b.rows, 2).cuda()
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, k, v, None), b.batch)
    (ks, _), (vs, _) = stored(b)
    assert torch.equal(ks, k.double().cpu()) and torch.equal(vs, v.double().cpu())


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act,hq,hkv,d", [(BF, 2, 1, 64), (F32, 3, 1, 16), (BF, 5, 5, 128)])
def test_append_and_read_many_rows(act, hq, hkv, d, fmt):
    """Tens of thousands of rows: every line is in its place in the raw pages, and comes back."""
    b = R.Batch([9001, 0, 11000, 1], [9001, 5, 11033, 70], hq, hkv, d, 64, act, fmt, seed=83, extra_rows=7)
    q, k, v = b.randn(b.max_rows, hq), b.randn(b.max_rows, hkv), b.randn(b.max_rows, hkv)
    q_out = torch.full_like(q, 7.0, device="cuda")
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(q.cuda(), k.cuda(), v.cuda(), q_out), b.batch)
    no_device_error(b.kv)
    assert torch.equal(q_out[:b.rows].cpu(), q[:b.rows]) and (q_out[b.rows:] == 7.0).all()
    seq = torch.tensor([i for i, T in enumerate(b.new) for _ in range(T)])
    pos = torch.tensor(b.positions())
    page, line = b.table[seq, pos // 64].long(), pos % 64
    ko, vo = (torch.full((b.max_rows, hkv, d), 5.0, dtype=act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, b.batch, ko, vo)
    no_device_error(b.kv)
    for x, pages, exps, back in ((k, b.kv.k, b.kv.k_scale, ko), (v, b.kv.v, b.kv.v_scale, vo)):
        raw = pages.float().cpu()[page, :, line].double()
        if fmt == "act":
            ref = x[:b.rows].double()
            assert torch.equal(raw, ref)
        else:
            val, e = R.quantise(x[:b.rows].double().numpy())
            assert np.array_equal(raw.numpy(), val) and np.array_equal(exps.cpu()[page, :, line].numpy(), e)
            ref = torch.from_numpy(val * 2.0 ** (e - 127.0)[..., None])
        assert torch.equal(back[:b.rows].double().cpu(), ref) and (back[b.rows:] == 5.0).all()


def test_far_positions_keep_their_angle():
    """A position of tens of millions: an angle formed in 32 bits would be off by whole radians."""
    far = 50_000_003
    b = R.Batch([2], [2], 2, 1, 64, 128, F32, "act", seed=5)
    width = far // 128 + 2
    b.table = torch.zeros(1, width, dtype=torch.int32)
    b.total = [far + 1]
    dev = (b.dev[0], torch.tensor([far + 1], dtype=torch.int32).cuda(), b.table.cuda())
    b.batch = kda.make_kv_batch(*dev, max_rows=2, max_new=2)
    _, rq, _, q_out = run_append(b, 64, False, False)
    # the frequencies are rounded to 2^-64 turns on a 53-bit product: 2^-53 of an angle of at most 8e6 turns
    got = q_out.double().cpu()
    assert (got - rq).abs().max() <= 2.0 ** -18 * rq.abs().max()


@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
def test_quantising_edge_values(act):
    """Zero vectors, borders of the scale, subnormals, the type's largest values, infinities and NaN."""
    d = 16
    rows = torch.zeros(10, 1, d, dtype=F32)
    rows[1, 0, 3] = 448.0
    rows[2, 0, 3] = 450.0
    rows[3, 0] = torch.arange(d) * 2.0 ** -12
    rows[4, 0, 0], rows[4, 0, 1] = 1e30, -3e29
    rows[5, 0, 0], rows[5, 0, 1] = float("inf"), 2.0
    rows[6, 0, 0], rows[6, 0, 1] = float("nan"), -3.0
    rows[7, 0] = -0.0
    rows[8, 0] = float("-inf")
    rows[9, 0, 0] = 2.0 ** -120
    rows = rows.to(act)
    b = R.Batch([10], [10], 1, 1, d, 16, act, "e4m3")
    x = rows.cuda()
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, x, x, None), b.batch)
    qv, qe = R.quantise(rows.double().numpy())
    for vals, e in stored(b):
        assert np.array_equal(e.numpy(), qe)
        assert np.array_equal(np.isnan(vals.numpy()), np.isnan(qv))
        assert np.array_equal(np.nan_to_num(vals.numpy()), np.nan_to_num(qv))


# ---- attention -------------------------------------------------------------------------------------------------------

def fill_cache(b, gain=1.0):
    """Random keys and values for every token of every sequence, appended through the library; returns them as the
    cache holds them, per sequence."""
    w = b.whole()
    k, v = w.randn(w.rows, b.hkv) * gain, w.randn(w.rows, b.hkv)
    kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, k.cuda(), v.cuda(), None), w.batch)
    return held(b)


def held(b):
    w = b.whole()
    ko, vo = (torch.zeros(max(w.rows, 1), b.hkv, b.d, dtype=b.act, device="cuda") for _ in range(2))
    kda.kda_kv_read(b.kv, w.batch, ko, vo)
    ko, vo = ko.double().cpu(), vo.double().cpu()
    cu = [int(x) for x in w.cu]
    return [(ko[a:z], vo[a:z]) for a, z in zip(cu[:-1], cu[1:])]


def check_attend(b, q, out, cache, scale):
    """Every row within the bound of the module's docstring."""
    got = out.double().cpu()
    worst = 0.0
    for i, (T, L) in enumerate(zip(b.new, b.total)):
        a = int(b.cu[i])
        if T == 0:
            continue
        k, v = cache[i]
        qq = q[a:a + T].double().cpu()
        ref, mag = R.attend(qq, k, v, L - T, scale, b.group)
        qk = (qq.abs().amax(-1) * 0 + qq.norm(dim=-1)) * float(torch.nan_to_num(k).norm(dim=-1).max()) * abs(scale)
        rel = (b.d + 4) * 2.0 ** -24 * qk[..., None] * 2 + 2.0 ** -20
        if b.act == BF:
            rel = rel + 2 * half_step(BF)
        tol = mag * rel + ref.abs() * (half_step(BF) if b.act == BF else 0) + 1e-30
        g = got[a:a + T]
        assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"sequence {i}: NaN in other places"
        off = torch.nan_to_num((g - ref).abs() / tol)
        worst = max(worst, float(off.max()))
    assert worst <= 1.0, f"worst error {worst:.2f} of the tolerance"


ATTEND = [
    # new, total, hq, hkv, d, page
    ([1], [1], 8, 1, 128, 16),
    ([1] * 9, [1, 2, 15, 16, 17, 63, 64, 65, 300], 8, 2, 128, 16),
    ([1, 1], [129, 1000], 16, 1, 64, 64),
    ([1, 1, 1], [7, 40, 222], 3, 3, 32, 32),
    ([1, 1], [31, 500], 7, 1, 16, 128),
    ([1], [700], 64, 1, 128, 64),
    ([2, 4, 0, 3], [2, 100, 0, 77], 4, 2, 128, 32),
    ([8, 8], [8, 150], 16, 2, 64, 16),
    ([5, 1], [64, 127], 21, 3, 128, 64),
    ([64], [64], 4, 1, 128, 64),
    ([130, 1, 33], [130, 200, 129], 6, 2, 64, 32),
    ([100, 65], [356, 65], 8, 8, 128, 16),
    ([129], [257], 5, 1, 32, 128),
    ([40, 90], [200, 90], 2, 2, 16, 16),
    ([3], [131], 64, 1, 64, 64),
    ([257, 300], [300, 300], 2, 1, 128, 64),
]


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(case, act, fmt):
    """Pages start as NaN, so a line behind a sequence's end that took part would show."""
    new, total, hq, hkv, d, page = ATTEND[case]
    b = R.Batch(new, total, hq, hkv, d, page, act, fmt, seed=100 + case, fill=float("nan"), extra_rows=1)
    cache = fill_cache(b)
    q = b.randn(b.max_rows, hq).cuda()
    wide = torch.full((b.max_rows, hq * d + 16), 9.0, dtype=act, device="cuda")
    out = wide[:, :hq * d].unflatten(1, (hq, d))
    scale = d ** -0.5
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out, scale), b.batch, b.workspace())
    no_device_error(b.kv)
    check_attend(b, q, out, cache, scale)
    assert (out[b.rows:] == 9.0).all() and (wide[:, hq * d:] == 9.0).all()


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,total,hq,hkv,d", [([1], [5000], 4, 1, 128), ([1, 1], [3000, 17], 8, 2, 64),
                                                ([20], [3000], 2, 1, 128)])
def test_attend_long_cut_into_parts(act, fmt, new, total, hq, hkv, d):
    """One cache head over many CTAs: parts joined, and sharp scores whose maximum sits in one part."""
    b = R.Batch(new, total, hq, hkv, d, 64, act, fmt, seed=7)
    cache = fill_cache(b, gain=3.0)
    q = b.randn(b.rows, hq).cuda()
    out = torch.empty_like(q)
    io = kda.make_attn_io(q, out)
    kda.kda_kv_attend(b.kv, io, b.batch, b.workspace(0xFF))
    check_attend(b, q, out, cache, d ** -0.5)
    again = out.clone()
    kda.kda_kv_attend(b.kv, io, b.batch, b.workspace(0))
    assert torch.equal(again.view(torch.uint8), out.view(torch.uint8))  # the workspace's contents do not matter


@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,hq,hkv,d", [(4, 4, 2, 128), (100, 4, 2, 128), (300, 2, 1, 64), (20, 3, 1, 32)])
def test_masked_values_may_be_anything(act, bad, new, hq, hkv, d):
    """A token's non-finite key or value reaches its own and later rows only."""
    total = new + 70
    b = R.Batch([new], [total], hq, hkv, d, 32, act, "act", seed=11)
    fill_cache(b)
    at = total - new // 2  # a position inside the chunk
    page, line = int(b.table[0, at // 32]), at % 32
    b.kv.v[page, :, line, 1] = bad
    b.kv.k[int(b.table[0, (total - 1) // 32]), :, (total - 1) % 32, 0] = float("nan")  # the last token's key
    q = b.randn(b.rows, hq).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    got = out.double().cpu()
    t_bad = at - (total - new)
    assert torch.isfinite(got[:t_bad]).all()
    assert not torch.isfinite(got[t_bad:-1, :, 1]).any()
    assert torch.isfinite(got[t_bad:-1, :, 2:]).all() and torch.isfinite(got[t_bad:-1, :, 0]).all()
    assert torch.isnan(got[-1]).all()
    # the untouched rows have their values
    k, v = held(b)[0]
    ref, mag = R.attend(q[:t_bad].double().cpu(), k, v, total - new, d ** -0.5, hq // hkv)
    assert ((got[:t_bad] - ref).abs() <= 3 * half_step(BF) * mag + 1e-12).all()


def test_extreme_scores():
    """Scores of thousands apart, and a row whose every score is -inf."""
    d = 64
    b = R.Batch([1, 6], [300, 200], 4, 2, d, 16, BF, "act", seed=13)
    cache = fill_cache(b, gain=100.0)
    q = (b.randn(b.rows, 4) * 50).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out, 1.0), b.batch, b.workspace())
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    a = 0
    for (T, L), (k, v) in zip(zip(b.new, b.total), cache):
        ref, _ = R.attend(q[a:a + T].double().cpu(), k, v, L - T, 1.0, 2)
        # one key holds all the weight unless two scores are within a few units of each other
        assert (got[a:a + T] - ref).abs().median() <= half_step(BF) * ref.abs().max()
        a += T
    b.kv.k[..., 0] = float("-inf")
    q[:, :, 0] = 1.0
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out, 1.0), b.batch, b.workspace())
    assert (out == 0).all()


def test_bad_pages_and_tables_on_the_device():
    """A page outside the cache: its tokens are absent; inconsistent tables: the sequence's rows are left alone."""
    d = 64
    for new, total in (([1, 1], [100, 90]), ([40, 50], [100, 90])):
        b = R.Batch(new, total, 4, 2, d, 16, BF, "act", seed=17)
        cache = fill_cache(b)
        q = b.randn(b.rows, 4).cuda()
        out = torch.full_like(q, 9.0)
        io, ws = kda.make_attn_io(q, out), b.workspace()
        cu, lens, table = b.dev
        table[0, 1] = b.kv.num_pages  # positions 16..31 of sequence 0
        table[1, 2] = -5              # positions 32..47 of sequence 1
        kda.kda_kv_attend(b.kv, io, b.batch, ws)
        st, flags = kda.kda_kv_poll_device_error(b.kv)
        assert st == kda.KDA_ERR_DEVICE and flags == kda.KDA_DEVERR_PAGE_RANGE
        got = out.double().cpu()
        a = 0
        for i, (T, L) in enumerate(zip(new, total)):
            k, v = cache[i]
            gone = range(16, 32) if i == 0 else range(32, 48)
            for t in range(T):
                keys = [j for j in range(L - T + t + 1) if j not in gone]
                for h in range(4):
                    p = torch.softmax(k[keys, h // 2] @ q[a + t, h].double().cpu() * d ** -0.5, 0)
                    ref, mag = p @ v[keys, h // 2], p @ v[keys, h // 2].abs()
                    assert ((got[a + t, h] - ref).abs() <= 4 * half_step(BF) * mag).all()
            a += T
        ko, vo = (torch.full((b.rows, 2, d), 5.0, dtype=BF, device="cuda") for _ in range(2))
        kda.kda_kv_read(b.kv, b.batch, ko, vo)
        kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, ko, vo, None), b.batch)
        kda.kda_kv_poll_device_error(b.kv)
        # inconsistent: the second sequence claims fewer cached tokens than it brings
        lens[1] = new[1] - 1
        out.fill_(9.0)
        kda.kda_kv_attend(b.kv, io, b.batch, ws)
        st, flags = kda.kda_kv_poll_device_error(b.kv)
        assert st == kda.KDA_ERR_DEVICE and flags & kda.KDA_DEVERR_META
        assert (out[new[0]:] == 9.0).all() and not (out[:new[0]] == 9.0).any()
        # longer than its row of the page table
        lens[1] = table.shape[1] * 16 + 1
        kda.kda_kv_attend(b.kv, io, b.batch, ws)
        k2 = torch.full((b.rows, 2, d), 5.0, dtype=BF, device="cuda")
        kda.kda_kv_read(b.kv, b.batch, k2, k2.clone())
        st, flags = kda.kda_kv_poll_device_error(b.kv)
        assert flags & kda.KDA_DEVERR_META
        assert (out[new[0]:] == 9.0).all() and (k2[new[0]:] == 5.0).all()


def test_all_pages_of_a_sequence_absent_gives_zeros():
    for new in ([1, 1], [30, 30]):
        b = R.Batch(new, [60, 60], 4, 2, 128, 16, BF, "act", seed=19)
        fill_cache(b)
        b.dev[2][0] = -1
        q = b.randn(b.rows, 4).cuda()
        out = torch.full_like(q, 9.0)
        kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
        assert (out[:new[0]] == 0).all() and not (out[new[0]:] == 0).all()
        assert kda.kda_kv_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_PAGE_RANGE


def test_offsets_past_32_bits():
    """A cache of more than 2^31 values, its sequences on the far pages."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 31) // (page * hkv * d) + 200
    b = R.Batch([1, 3, 70], [200, 130, 70], 16, hkv, d, page, BF, "act", seed=23, num_pages=n_pages)
    per = [-(-t // page) for t in b.total]
    at = n_pages - sum(per)
    for i, c in enumerate(per):
        b.table[i, :c] = torch.arange(at, at + c, dtype=torch.int32)
        at += c
    b.dev[2].copy_(b.table)
    cache = fill_cache(b)
    q = b.randn(b.rows, 16).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    no_device_error(b.kv)
    check_attend(b, q, out, cache, d ** -0.5)
    assert b.kv.k[:100].abs().max() == 0


def test_no_sequences_and_no_rows_are_no_ops():
    b = R.Batch([1], [5], 2, 1, 32, 16, BF, "act")
    x = torch.zeros(1, 1, 32, dtype=BF, device="cuda")
    q = torch.full((1, 2, 32), 3.0, dtype=BF, device="cuda")
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for batch in (kda.make_kv_batch(one, empty, empty.view(0, 4), 0, 1),
                  kda.make_kv_batch(b.dev[0], b.dev[1], b.dev[2], 0, 1)):
        assert kda.kda_kv_attend_workspace_bytes(b.kv, batch) == 0
        kda.kda_kv_append(b.kv, None, kda.make_kv_io(None, x, x, None), batch)
        kda.kda_kv_read(b.kv, batch, x, x)
        kda.kda_kv_attend(b.kv, kda.make_attn_io(q, q.clone()), batch, None)
    none = R.Batch([0, 0], [0, 7], 2, 1, 32, 16, BF, "act")
    out = torch.full((1, 2, 32), 9.0, dtype=BF, device="cuda")
    kda.kda_kv_attend(none.kv, kda.make_attn_io(q, out), none.batch, none.workspace())
    no_device_error(none.kv)
    assert (out == 9.0).all()


MANY = [
    # lengths from one token up, sequences by the hundred: items of one tile, and pieces that hold many items
    ([1] * 300, [1 + 37 * i % 160 for i in range(300)], 8, 1, 128, 16),
    ([1] * 180, [1 + 211 * i % 1500 for i in range(180)], 16, 2, 128, 64),
    ([3] * 200, [3 + 53 * i % 400 for i in range(200)], 8, 1, 128, 32),
    ([5] * 170, [5 + i % 123 for i in range(170)], 4, 2, 64, 128),
    ([1 + 7 * i % 40 for i in range(60)], [40 + 97 * i % 700 for i in range(60)], 8, 1, 128, 128),
    ([128 * (i % 3) for i in range(30)], [256 + 64 * (i % 5) for i in range(30)], 2, 1, 128, 64),
]


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attend_many_sequences(case, fmt):
    new, total, hq, hkv, d, page = MANY[case]
    b = R.Batch(new, total, hq, hkv, d, page, BF, fmt, seed=200 + case, fill=float("nan"))
    cache = fill_cache(b)
    q = b.randn(b.rows, hq).cuda()
    out = torch.full_like(q, 9.0)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    no_device_error(b.kv)
    check_attend(b, q, out, cache, d ** -0.5)


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new,group,d", [(1, 16, 128), (1, 17, 128), (2, 8, 128), (16, 1, 128), (17, 1, 128), (8, 16, 128),
                                         (43, 3, 128), (1, 1, 64), (64, 2, 64), (129, 1, 64)])
def test_attend_rows_of_a_tile(new, group, d, page, fmt):
    """One row to a little over a tile, over caches that end at a tile's border and one token to either side of it."""
    tops = [max(t, new) for t in (127, 128, 129, 256, 384)]
    b = R.Batch([new] * 5, tops, group, 1, d, page, BF, fmt, seed=300 + new, fill=float("nan"))
    cache = fill_cache(b)
    q = b.randn(b.rows, group).cuda()
    out = torch.full_like(q, 9.0)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    no_device_error(b.kv)
    check_attend(b, q, out, cache, d ** -0.5)


@pytest.mark.parametrize("new,group,d,act", [(1, 2, 128, BF), (4, 8, 128, BF), (40, 8, 64, BF), (1, 2, 64, BF), (1, 3, 32, F32),
                                             (5, 2, 16, BF)])
def test_attend_few_items_of_any_length(new, group, d, act):
    """Fewer items than CTAs, of lengths that put the cuts between CTAs at every place of a key step."""
    rng = np.random.default_rng(73)
    for trial in range(25):
        total = [new + int(x) for x in rng.integers(0, int(rng.choice([300, 1500, 4000])), int(rng.integers(1, 7)))]
        b = R.Batch([new] * len(total), total, group, 1, d, 64, act, "act", seed=400 + trial)
        cache = fill_cache(b)
        q = b.randn(b.rows, group).cuda()
        out = torch.full_like(q, 9.0)
        kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
        no_device_error(b.kv)
        check_attend(b, q, out, cache, d ** -0.5)


@pytest.mark.parametrize("new,hq,hkv,d", [(4, 4, 2, 128), (100, 4, 2, 128), (300, 2, 1, 64), (20, 3, 1, 32)])
def test_masked_e4m3_lines_may_be_anything(new, hq, hkv, d):
    """A quantised line that holds NaN, or a scale past bf16's range, reaches its own and later rows only."""
    total = new + 70
    for act in (BF, F32):
        b = R.Batch([new], [total], hq, hkv, d, 32, act, "e4m3", seed=43)
        cache = fill_cache(b)
        at = total - new // 2
        page, line = int(b.table[0, at // 32]), at % 32
        b.kv.v.view(torch.uint8)[page, :, line, 1] = 0xFF
        page, line = int(b.table[0, (total - 1) // 32]), (total - 1) % 32
        b.kv.v_scale[page, :, line] = 255
        b.kv.k.view(torch.uint8)[page, :, line, 0] = 0x7F
        q = b.randn(b.rows, hq).cuda()
        out = torch.empty_like(q)
        kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
        got = out.double().cpu()
        t_bad = at - (total - new)
        assert torch.isfinite(got[:t_bad]).all()
        assert torch.isnan(got[t_bad:-1, :, 1]).all()
        assert torch.isfinite(got[t_bad:-1, :, 2:]).all() and torch.isfinite(got[t_bad:-1, :, 0]).all()
        assert torch.isnan(got[-1]).all()
        k, v = cache[0]
        ref, mag = R.attend(q[:t_bad].double().cpu(), k, v, total - new, d ** -0.5, hq // hkv)
        assert ((got[:t_bad] - ref).abs() <= 3 * half_step(BF) * mag + 1e-12).all()


@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act"), (F32, "e4m3")])
@pytest.mark.parametrize("new,hq,d", [(2, 4, 128), (30, 2, 128), (150, 2, 64), (3, 64, 32)])
def test_far_positions_and_absent_pages(new, hq, d, act, fmt):
    """A context of tens of millions of tokens of which only the last pages are there (a window)."""
    page, far = 128, 40_000_000
    b = R.Batch([new], [new + 200], hq, 1, d, page, act, fmt, seed=47)
    cache = fill_cache(b)
    skip = far // page
    table = torch.full((1, skip + b.table.shape[1]), -1, dtype=torch.int32)
    table[0, skip:] = b.table[0]
    lens = torch.tensor([skip * page + new + 200], dtype=torch.int32).cuda()
    batch = kda.make_kv_batch(b.dev[0], lens, table.cuda(), max_rows=b.rows, max_new=new)
    q = b.randn(b.rows, hq).cuda()
    out = torch.full_like(q, 9.0)
    ws = torch.empty(kda.kda_kv_attend_workspace_bytes(b.kv, batch), dtype=torch.uint8, device="cuda")
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), batch, ws)
    assert kda.kda_kv_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_PAGE_RANGE)
    check_attend(b, q, out, cache, d ** -0.5)


def test_longest_positions_are_refused():
    """Past 2^31 - 1024 tokens a tile's last positions would not be 32-bit numbers: the sequence is left alone."""
    page = 128
    b = R.Batch([1, 1], [100, 50], 2, 1, 64, page, BF, "act", seed=53)
    cache = fill_cache(b)
    width = (1 << 31) // page
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[:, :1] = b.dev[2]
    b.dev[1][0] = (1 << 31) - 1
    batch = kda.make_kv_batch(b.dev[0], b.dev[1], table, max_rows=2, max_new=1)
    q = b.randn(2, 2).cuda()
    out = torch.full_like(q, 9.0)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), batch, b.workspace())
    assert kda.kda_kv_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_META)
    assert (out[0] == 9.0).all()
    ref, mag = R.attend(q[1:].double().cpu(), *cache[1], 49, 64 ** -0.5, 2)
    assert ((out[1:].double().cpu() - ref).abs() <= 4 * half_step(BF) * mag).all()


@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act")])
@pytest.mark.parametrize("new,hq,hkv,d", [(1, 8, 2, 128), (9, 8, 2, 128), (150, 4, 2, 64), (40, 4, 2, 16)])
def test_rows_16_bytes_apart_and_loose_bounds(new, hq, hkv, d, act, fmt):
    """Rows that start at 16-byte but not 32-byte places, and host bounds larger than what the tables hold."""
    b = R.Batch([new, 0, 1], [new + 150, 20, 33], hq, hkv, d, 32, act, fmt, seed=59, extra_rows=5)
    cache = fill_cache(b)
    pad = 8 if act == BF else 4
    q_wide = torch.zeros(b.max_rows, hq * d + pad, dtype=act, device="cuda")
    q = q_wide[:, pad:].unflatten(1, (hq, d))
    q.copy_(b.randn(b.max_rows, hq))
    wide = torch.full((b.max_rows, hq * d + pad), 9.0, dtype=act, device="cuda")
    out = wide[:, pad:].unflatten(1, (hq, d))
    for max_new in (new, new + 1, 70, 1000):
        if max_new < new:
            continue
        wide.fill_(9.0)
        batch = kda.make_kv_batch(*b.dev, max_rows=b.max_rows, max_new=max_new)
        ws = torch.empty(kda.kda_kv_attend_workspace_bytes(b.kv, batch), dtype=torch.uint8, device="cuda")
        kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), batch, ws)
        no_device_error(b.kv)
        check_attend(b, q, out, cache, d ** -0.5)
        assert (out[b.rows:] == 9.0).all() and (wide[:, :pad] == 9.0).all()


@pytest.mark.parametrize("fmt", ["act", "e4m3"])
def test_two_calls_at_once(fmt):
    """Two streams, each with its own workspace, over one cache and at the same time: what each gives alone."""
    streams, work = [torch.cuda.Stream() for _ in range(2)], []
    b = R.Batch([1] * 20, [900 + 31 * i for i in range(20)], 8, 2, 128, 64, BF, fmt, seed=61)
    fill_cache(b)
    c = R.Batch.__new__(R.Batch)
    c.__dict__.update(b.__dict__)
    c.new, c.rows = [30] * 20, 600
    c.cu = torch.arange(21, dtype=torch.int32) * 30
    c.dev = (c.cu.cuda(), b.dev[1], b.dev[2])
    c.batch = kda.make_kv_batch(*c.dev, max_rows=600, max_new=30)
    for x in (b, c):
        q = x.randn(x.rows, 8).cuda()
        io, ws = kda.make_attn_io(q, torch.empty_like(q)), x.workspace()
        kda.kda_kv_attend(x.kv, io, x.batch, ws)
        work.append((x, io, ws, io._tensors[1], io._tensors[1].clone()))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (x, io, ws, out, _) in zip(streams, work):
            kda.kda_kv_attend(x.kv, io, x.batch, ws, stream=st)
    torch.cuda.synchronize()
    no_device_error(b.kv)
    for _, _, _, out, alone in work:
        assert torch.equal(out, alone)


@pytest.mark.parametrize("act,fmt,new", [(BF, "e4m3", 1), (BF, "e4m3", 8), (BF, "act", 40), (F32, "act", 2)])
def test_replayed_with_other_lengths(act, fmt, new):
    """Captured once, replayed with tables that move work between CTAs, sequences that drop out and new pages."""
    hq, hkv, d, page = 8, 2, 128, 16
    b = R.Batch([new] * 3, [700, 600, 500], hq, hkv, d, page, act, fmt, seed=67)
    fill_cache(b)
    q = b.randn(b.rows, hq).cuda()
    out = torch.empty_like(q)
    ws, st = b.workspace(), torch.cuda.Stream()
    io = kda.make_attn_io(q, out)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        kda.kda_kv_attend(b.kv, io, b.batch, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            kda.kda_kv_attend(b.kv, io, b.batch, ws)
    torch.cuda.synchronize()
    for news, lens in (([new] * 3, [700, 600, 500]), ([new, 0, new], [new, 600, 333]), ([0, new, 0], [9, 17 + new, 9]),
                       ([1, 1, 1], [1, 2, 3]), ([new] * 3, [128, 640, 127 + new])):
        b.new, b.total, b.rows = news, lens, sum(news)
        b.cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32)
        b.dev[0].copy_(b.cu), b.dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        b.dev[2].copy_(b.table.flip(1)[:, :b.table.shape[1]].clamp(min=0))
        out.fill_(9.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        no_device_error(b.kv)
        check_attend(b, q, out, held(b), d ** -0.5)
        assert (out[b.rows:] == 9.0).all()


def test_a_page_twice_in_a_sequence():
    """A table may name a page more than once: its tokens then stand at several positions."""
    b = R.Batch([1, 20], [300, 310], 4, 2, 128, 32, BF, "act", seed=71)
    fill_cache(b)
    b.dev[2][:, 1:5] = b.dev[2][0, 0]
    q = b.randn(b.rows, 4).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    no_device_error(b.kv)
    check_attend(b, q, out, held(b), 128 ** -0.5)


# ---- together ----------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act")], ids=["bf16", "bf16-e4m3", "f32"])
def test_prompt_then_decode_then_verify(act, fmt):
    """A layer as it is served: a prompt in two chunks, single tokens, then drafts, each call appending before it attends;
    every output against attention over what the cache holds."""
    hq, hkv, d, page = 8, 2, 64, 16
    plan = [[50, 70], [40, 1], [1, 1], [1, 1], [4, 4], [1, 1]]
    totals = np.cumsum(plan, 0)
    last = totals[-1].tolist()
    b = R.Batch([1, 1], last, hq, hkv, d, page, act, fmt, seed=29)
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    w = (1 + 0.1 * torch.randn(2, d, generator=b.gen)).to(act)
    params = kda.make_qk_params(w[0].cuda(), w[1].cuda(), 1e-5, freq)
    lens = b.dev[1]
    for new, total in zip(plan, totals.tolist()):
        b.new, b.total = new, total
        b.rows = b.max_rows = sum(new)
        b.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        b.dev = (b.cu.cuda(), torch.tensor(total, dtype=torch.int32).cuda(), b.dev[2])
        b.batch = kda.make_kv_batch(*b.dev, max_rows=b.rows, max_new=max(new))
        q, k, v = (b.randn(b.rows, n) for n in (hq, hkv, hkv))
        q_out, out = (torch.empty(b.rows, hq, d, dtype=act, device="cuda") for _ in range(2))
        kda.kda_kv_append(b.kv, params, kda.make_kv_io(q.cuda(), k.cuda(), v.cuda(), q_out), b.batch)
        kda.kda_kv_attend(b.kv, kda.make_attn_io(q_out, out), b.batch, b.workspace())
        no_device_error(b.kv)
        check_rows(q_out, R.norm_rotate(q, w[0], b.positions(), freq, False, 1e-5), act)
        check_attend(b, q_out, out, held(b), d ** -0.5)
    assert lens.tolist() == last


def test_graph_replay_reads_new_tables():
    """append + attend captured once and replayed with other tables and inputs, on a stream of its own; two graphs that
    share a workspace, replayed in order."""
    hq, hkv, d, page = 8, 1, 128, 64
    b = R.Batch([1, 1], [400, 200], hq, hkv, d, page, BF, "act", seed=31)
    fill_cache(b)
    q, k, v = b.randn(2, hq).cuda(), b.randn(2, hkv).cuda(), b.randn(2, hkv).cuda()
    qs, outs = [torch.empty_like(q) for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    ws = b.workspace()
    params = kda.make_qk_params(None, None, 1e-5, [1.0 / (10.0 + i) for i in range(d // 2)])
    io = kda.make_kv_io(q, k, v, qs[0])
    st = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(st):
        kda.kda_kv_append(b.kv, params, io, b.batch)
        kda.kda_kv_attend(b.kv, kda.make_attn_io(qs[0], outs[0]), b.batch, ws)
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                kda.kda_kv_append(b.kv, params, kda.make_kv_io(q, k, v, qs[i]), b.batch)
                kda.kda_kv_attend(b.kv, kda.make_attn_io(qs[i], outs[i], 0.05 * (i + 1)), b.batch, ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for lens in ([400, 200], [399, 1], [65, 130]):
        b.dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(b.randn(2, hq))
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        b.total = lens
        for i in range(2):
            check_attend(b, qs[i], outs[i], held(b), 0.05 * (i + 1))


def test_calls_on_another_stream_and_profile():
    b = R.Batch([9, 1], [190, 70], 4, 2, 64, 32, BF, "e4m3", seed=37)
    cache = fill_cache(b)
    q = b.randn(b.rows, 4).cuda()
    out = torch.empty_like(q)
    st = torch.cuda.Stream()
    ws = b.workspace()
    torch.cuda.synchronize()
    kda.kda_profile_start(16)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, ws, stream=st)
    prof = kda.kda_profile_stop()
    st.synchronize()
    assert prof["kv_attend"][0] == 1 and prof["kv_combine"][0] == 1
    check_attend(b, q, out, cache, 64 ** -0.5)


@pytest.mark.parametrize("act,fmt,d,group,new", [(BF, "act", 128, 8, 1), (BF, "e4m3", 128, 4, 4), (BF, "act", 64, 8, 100),
                                                 (BF, "e4m3", 32, 8, 3), (F32, "act", 64, 1, 1), (F32, "e4m3", 128, 2, 30)])
def test_one_key_step_is_one_launch(act, fmt, d, group, new):
    """A page table of one key step: no item is cut, so there is nothing to join."""
    page = 32 if act == F32 and new == 1 else 64
    b = R.Batch([new] * 3, [page - 1 if new < 30 else page, page, new] if new <= page else [new] * 3, group, 1, d,
                page if new <= page else 128, act, fmt, seed=79)
    cache = fill_cache(b)
    q = b.randn(b.rows, group).cuda()
    out = torch.full_like(q, 9.0)
    ws = b.workspace(0xFF)
    torch.cuda.synchronize()
    kda.kda_profile_start(16)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, ws)
    prof = kda.kda_profile_stop()
    torch.cuda.synchronize()
    assert prof["kv_attend"][0] == 1 and prof["kv_combine"][0] == 0
    no_device_error(b.kv)
    check_attend(b, q, out, cache, d ** -0.5)


def test_shared_pages():
    """Two sequences over the same prefix pages give what each gives alone."""
    b = R.Batch([1, 1], [130, 128], 4, 2, 128, 32, BF, "act", seed=41)
    fill_cache(b)
    b.dev[2][1, :4] = b.dev[2][0, :4]
    b.table[1, :4] = b.table[0, :4]
    q = b.randn(2, 4).cuda()
    out = torch.empty_like(q)
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, out), b.batch, b.workspace())
    check_attend(b, q, out, held(b), 128 ** -0.5)

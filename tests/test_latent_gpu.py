"""Latent-attention operators on a GPU against plain float64 statements: kda_latent_append, kda_latent_read, kda_latent_attend,
kda_latent_prefill and runs of them together.

Tolerances.  A rounding to type t is off by at most eps(t) / 2 of the value (bf16 2^-8, e4m3 2^-4 and, below its normal
range, 2^-10 of the scale's unit).  Arithmetic is in 32 bits (unit 2^-24):
  append  the sum of squares is a tree of depth at most 25 (16 or 4 in a lane, then 5 of shuffles and 4 of pieces), then a quotient, a root, a
          division and two products, or two products and a sum with a cosine and a sine good to 2 units and an angle good to pi units:
          under 64 units, of a value whose partner may be the row's largest: 2^-18 max|row| covers both.
  attend  see latent_ref.check."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import latent_ref as R
from kv_ref import quantise

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()


half_step = R.half_step
ACTS = pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
FMTS = pytest.mark.parametrize("fmt", ["act", "e4m3"])


def check_rows(got, ref, act):
    got = got.double().cpu()
    tol = ref.abs() * (half_step(act) if act == BF else 0) + 2.0 ** -18 * ref.abs().amax(-1, keepdim=True)
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} values off, worst {float(((got - ref).abs() / tol.clamp(min=1e-300)).max()):.2f} tolerances"


# ---- append and read ---------------------------------------------------------------------------------------------------

def run_append(b, rot, inter, with_norm, strided=False, in_place=False, base=10000.0):
    """Appends b's rows; returns (c, kr, q in float64 after norm and rotation, q_out)."""
    H, L, Rr = b.heads, b.latent, b.rope
    if strided:  # c and kr slices of one projection, q of another, q_out head-major
        row = b.randn(b.max_rows, L + Rr + 8).cuda()
        c, kr = row[:, 8:8 + L], row[:, 8 + L:]
        q = b.randn(b.max_rows, H, Rr + 16).cuda()[..., 16:]
        q_out = torch.full((H, b.max_rows, Rr), 7.0, dtype=b.act, device="cuda").transpose(0, 1)
    else:
        c, kr, q = b.randn(b.max_rows, L).cuda(), b.randn(b.max_rows, Rr).cuda(), b.randn(b.max_rows, H, Rr).cuda()
        q_out = torch.full_like(q, 7.0)
    q0 = q.clone()
    if in_place:
        q_out = q
    w = (1 + 0.1 * torch.randn(L, generator=b.gen)).to(b.act) if with_norm else None
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    params = kda.make_latent_params(None if w is None else w.cuda(), 1e-5, freq, inter)
    kda.kda_latent_append(b.kv, params, kda.make_latent_io(c, kr, q, q_out), b.batch)
    pos, n = b.positions(), b.rows
    return (R.norm(c[:n].cpu(), w, 1e-5), R.rotate(kr[:n, None].cpu(), pos, freq, inter)[:, 0],
            R.rotate(q0[:n].cpu(), pos, freq, inter), q_out)


APPEND = [
    # new, total, heads, latent, rope, page, rot, inter, norm
    ([1], [1], 64, 512, 64, 64, 64, False, True),
    ([1], [100001], 16, 512, 64, 128, 64, True, True),
    ([5, 0, 1, 17], [5, 0, 33, 130], 6, 256, 32, 16, 32, True, True),
    ([3, 2], [3, 70], 7, 128, 16, 32, 8, False, True),
    ([33, 40], [33, 41], 4, 512, 64, 128, 24, False, False),
    ([70, 9], [71, 90], 12, 128, 64, 64, 40, True, True),
    ([1] * 40, list(range(1, 41)), 3, 256, 16, 32, 0, False, True),
    ([300], [1000], 1, 512, 32, 64, 16, False, True),
    ([2000, 700], [2000, 801], 5, 512, 64, 64, 64, False, True),
]


@FMTS
@ACTS
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_and_read(case, act, fmt):
    new, total, heads, latent, rope, page, rot, inter, with_norm = APPEND[case]
    b = R.Batch(new, total, heads, latent, rope, page, act, fmt, seed=case, extra_rows=2)
    before = b.kv.c.view(torch.uint8).clone(), b.kv.kr.clone()
    rc, rkr, rq, q_out = run_append(b, rot, inter, with_norm, strided=case % 2 == 1)
    b.no_error()
    check_rows(q_out[:b.rows], rq, act)
    assert (q_out[b.rows:] == 7.0).all()  # rows behind the last sequence
    pg, line = b.lines()
    got_kr = b.kv.kr.cpu()[pg, line].double()
    check_rows(got_kr, rkr, act)
    got_c = b.kv.c.float().cpu()[pg, line].double()
    if fmt == "act":
        check_rows(got_c, rc, act)
    else:
        e = b.kv.c_scale.cpu()[pg, line].double()
        unit, amax = 2.0 ** (e - 127)[:, None], rc.abs().amax(-1)
        slack = 2.0 ** -18 * amax
        assert (unit[:, 0] * 448 >= amax - slack).all() and (unit[:, 0] * 224 <= amax + slack).all()
        assert ((got_c * unit - rc).abs() <= rc.abs() * 2.0 ** -4 + unit * 2.0 ** -10 + slack[:, None]).all()
        got_c = got_c * unit
    # only the batch's lines changed
    touched = torch.zeros(b.kv.num_pages, page, dtype=torch.bool)
    touched[pg, line] = True
    for old, t in zip(before, (b.kv.c.view(torch.uint8), b.kv.kr)):
        assert torch.equal(old.cpu()[~touched], t.cpu()[~touched])
    # and read back, into slices of wider rows
    wide = torch.full((b.max_rows, latent + rope + 16), 5.0, dtype=act, device="cuda")
    co, ko = wide[:, 8:8 + latent], wide[:, 8 + latent:8 + latent + rope]
    kda.kda_latent_read(b.kv, b.batch, co, ko)
    b.no_error()
    assert torch.equal(co[:b.rows].double().cpu(), got_c) and torch.equal(ko[:b.rows].double().cpu(), got_kr)
    assert (wide[b.rows:] == 5.0).all() and (wide[:, :8] == 5.0).all() and (wide[:, -8:] == 5.0).all()


def test_append_in_place_and_cache_only():
    b = R.Batch([20, 3], [20, 50], 8, 256, 64, 16, BF, "act", seed=3)
    _, _, rq, q_out = run_append(b, 64, False, True, in_place=True)
    check_rows(q_out, rq, BF)
    c, kr = b.randn(b.rows, 256).cuda(), b.randn(b.rows, 64).cuda()
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(c, kr, None, None), b.batch)
    pg, line = b.lines()
    assert torch.equal(b.kv.c.cpu()[pg, line], c.cpu()) and torch.equal(b.kv.kr.cpu()[pg, line], kr.cpu())


@FMTS
@ACTS
def test_append_and_read_many_rows(act, fmt):
    """Tens of thousands of rows: every line is in its place in the raw pages, and comes back."""
    b = R.Batch([9001, 0, 11000, 1], [9001, 5, 11033, 70], 2, 128, 16, 64, act, fmt, seed=83, extra_rows=7)
    c, kr, q = b.randn(b.max_rows, 128), b.randn(b.max_rows, 16), b.randn(b.max_rows, 2, 16)
    q_out = torch.full_like(q, 7.0, device="cuda")
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(c.cuda(), kr.cuda(), q.cuda(), q_out), b.batch)
    b.no_error()
    assert torch.equal(q_out[:b.rows].cpu(), q[:b.rows]) and (q_out[b.rows:] == 7.0).all()
    pg, line = b.lines()
    co, ko = torch.full((b.max_rows, 128), 5.0, dtype=act, device="cuda"), torch.full((b.max_rows, 16), 5.0, dtype=act, device="cuda")
    kda.kda_latent_read(b.kv, b.batch, co, ko)
    b.no_error()
    assert torch.equal(b.kv.kr.cpu()[pg, line], kr[:b.rows]) and torch.equal(ko[:b.rows].cpu(), kr[:b.rows])
    raw, want = b.kv.c.float().cpu()[pg, line].double(), c[:b.rows].double()
    if fmt == "e4m3":
        val, e = quantise(want.numpy())
        assert np.array_equal(raw.numpy(), val) and np.array_equal(b.kv.c_scale.cpu()[pg, line].numpy(), e)
        want = torch.from_numpy(val * 2.0 ** (e - 127.0)[..., None])
    else:
        assert torch.equal(raw, want)
    assert torch.equal(co[:b.rows].double().cpu(), want) and (co[b.rows:] == 5.0).all() and (ko[b.rows:] == 5.0).all()


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions_keep_their_angle(inter):
    far = 50_000_003
    b = R.Batch([2], [2], 2, 128, 64, 128, F32, "act", seed=5)
    table = torch.zeros(1, far // 128 + 2, dtype=torch.int32)
    b.total = [far + 1]
    b.dev = (b.dev[0], torch.tensor([far + 1], dtype=torch.int32).cuda(), table.cuda())
    b.batch = kda.make_kv_batch(*b.dev, max_rows=2, max_new=2)
    _, _, rq, q_out = run_append(b, 64, inter, False)
    assert (q_out.double().cpu() - rq).abs().max() <= 2.0 ** -18 * rq.abs().max()


@ACTS
def test_quantising_edge_values(act):
    """Zero vectors, borders of the scale, subnormals, the type's largest values, infinities and NaN."""
    d = 128
    rows = torch.zeros(10, d, dtype=F32)
    rows[1, 3] = 448.0
    rows[2, 3] = 450.0
    rows[3, :16] = torch.arange(16) * 2.0 ** -12
    rows[4, 0], rows[4, 1] = 1e30, -3e29
    rows[5, 0], rows[5, 1] = INF, 2.0
    rows[6, 0], rows[6, 1] = NAN, -3.0
    rows[7] = -0.0
    rows[8] = -INF
    rows[9, 127] = 2.0 ** -120
    x = rows.to(act)
    b = R.Batch([10], [10], 1, d, 16, 16, act, "e4m3")
    kr = torch.zeros(10, 16, dtype=act, device="cuda")
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(x.cuda(), kr, None, None), b.batch)
    qv, qe = quantise(x.double().numpy())
    pg, line = b.lines()
    vals, e = b.kv.c.float().cpu()[pg, line].double().numpy(), b.kv.c_scale.cpu()[pg, line].numpy()
    assert np.array_equal(e, qe) and np.array_equal(np.isnan(vals), np.isnan(qv))
    assert np.array_equal(np.nan_to_num(vals), np.nan_to_num(qv))


@FMTS
@ACTS
@pytest.mark.parametrize("rope,rot,inter", [(64, 32, False), (64, 24, False), (32, 16, True), (16, 8, False)])
def test_non_finite_values_stay_in_their_pair(rope, rot, inter, act, fmt):
    """An infinity or NaN reaches its pair; channels that do not turn are those that came, bit for bit."""
    b = R.Batch([4], [40], 2, 128, rope, 16, act, fmt, seed=rope + rot)
    kr, q = b.randn(4, rope), b.randn(4, 2, rope)
    for x in (kr[:, None], q):
        x[1, :, 1], x[2, :, rot], x[3, :, rope - 1] = NAN, INF, -INF
    q_out = torch.zeros_like(q, device="cuda")
    freq = [0.1 * (i + 1) for i in range(rot // 2)]
    kda.kda_latent_append(b.kv, kda.make_latent_params(None, 1e-5, freq, inter),
                          kda.make_latent_io(b.randn(4, 128).cuda(), kr.cuda(), q.cuda(), q_out), b.batch)
    pg, line = b.lines()
    for x, got in ((kr[:, None], b.kv.kr[pg, line][:, None]), (q, q_out)):
        got, ref = got.double().cpu(), R.rotate(x, b.positions(), freq, inter)
        assert torch.equal(got[..., rot:].nan_to_num(1.5), x[..., rot:].double().nan_to_num(1.5))
        fin = torch.isfinite(ref)
        assert torch.equal(torch.isfinite(got), fin)
        top = torch.where(fin, ref, torch.zeros_like(ref)).abs().amax(-1, keepdim=True)
        assert ((got - ref).abs()[fin] <= (ref.abs() * half_step(BF) + 2.0 ** -18 * top)[fin]).all()


@FMTS
def test_bad_tables_touch_no_other_line(fmt):
    """Pages outside the cache and inconsistent sequences: what is consistent is written, nothing else is."""
    b = R.Batch([3, 2, 4], [20, 17, 30], 2, 128, 32, 16, BF, fmt, seed=9)
    b.dev[2][0, 1] = b.kv.num_pages  # positions 16..19 of sequence 0: all of its rows
    b.dev[1][1] = 1                  # sequence 1 brings more than it has
    before = b.kv.c.view(torch.uint8).clone(), b.kv.kr.clone()
    c, kr, q = b.randn(9, 128).cuda(), b.randn(9, 32).cuda(), b.randn(9, 2, 32).cuda()
    q_out = torch.full_like(q, 7.0)
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(c, kr, q, q_out), b.batch)
    assert kda.kda_latent_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_META | kda.KDA_DEVERR_PAGE_RANGE)
    assert torch.equal(q_out[:3], q[:3]) and (q_out[3:5] == 7.0).all() and torch.equal(q_out[5:], q[5:])
    pg, line = b.lines()
    touched = torch.zeros(b.kv.num_pages, 16, dtype=torch.bool)
    touched[pg[5:], line[5:]] = True
    for old, t in zip(before, (b.kv.c.view(torch.uint8), b.kv.kr)):
        assert torch.equal(old.cpu()[~touched], t.cpu()[~touched])
    assert torch.equal(b.kv.kr.cpu()[pg[5:], line[5:]], kr[5:].cpu())
    co, ko = torch.full((9, 128), 5.0, dtype=BF, device="cuda"), torch.full((9, 32), 5.0, dtype=BF, device="cuda")
    kda.kda_latent_read(b.kv, b.batch, co, ko)
    assert kda.kda_latent_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_META | kda.KDA_DEVERR_PAGE_RANGE
    assert (co[:3] == 0).all() and (ko[:3] == 0).all() and (co[3:5] == 5.0).all() and (ko[3:5] == 5.0).all()
    assert torch.equal(ko[5:], kr[5:])


# ---- absorbed form ------------------------------------------------------------------------------------------------------

ATTEND = [
    # new, total, heads, latent, rope, page
    ([1], [1], 64, 512, 64, 16),
    ([1] * 9, [1, 2, 15, 16, 17, 63, 64, 65, 300], 16, 512, 64, 16),
    ([1, 1], [129, 1000], 64, 512, 64, 64),
    ([1, 1, 1], [7, 40, 222], 3, 256, 32, 32),
    ([1, 1], [31, 500], 128, 128, 16, 128),
    ([1], [700], 67, 512, 64, 64),
    ([2, 4, 0, 3], [2, 100, 0, 77], 4, 512, 64, 32),
    ([8, 8], [8, 150], 64, 256, 64, 16),
    ([5, 1], [64, 127], 21, 128, 64, 64),
    ([64], [64], 1, 512, 32, 64),
    ([70, 1, 33], [70, 200, 129], 5, 128, 32, 32),
    ([40, 65], [196, 65], 8, 512, 64, 128),
    ([3], [131], 48, 512, 64, 128),
    ([6, 7], [300, 300], 12, 512, 64, 64),
]


@FMTS
@ACTS
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(case, act, fmt):
    """Pages start as NaN, so a line behind a sequence's end that took part would show; rows and heads in slices."""
    new, total, heads, latent, rope, page = ATTEND[case]
    b = R.Batch(new, total, heads, latent, rope, page, act, fmt, seed=100 + case, fill=NAN, extra_rows=1)
    held = b.fill_cache()
    q = b.queries()
    if case % 3 == 1:  # one tensor [rows, heads, latent + rope]
        joint = torch.cat(q, -1)
        q = joint[..., :latent], joint[..., latent:]
    elif case % 3 == 2:  # head-major
        q = tuple(t.transpose(0, 1).contiguous().transpose(0, 1) for t in q)
    wide = torch.full((b.max_rows, heads, latent + 8), 9.0, dtype=act, device="cuda")
    out = wide[..., 8:]
    scale = (128 + rope) ** -0.5
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, scale), b.batch, b.workspace())
    b.no_error()
    b.check_attend(q, out, held, scale)
    assert (out[b.rows:] == 9.0).all() and (wide[..., :8] == 9.0).all()


@FMTS
@ACTS
@pytest.mark.parametrize("new,total,heads,latent", [([1], [5000], 16, 512), ([1, 1], [3000, 17], 64, 256), ([9], [3000], 7, 128),
                                                    ([1], [20000], 4, 512)])
def test_attend_long_cut_into_parts(act, fmt, new, total, heads, latent):
    """One sequence over many CTAs: parts joined, and sharp scores whose maximum sits in one part."""
    b = R.Batch(new, total, heads, latent, 64, 64, act, fmt, seed=7)
    held = b.fill_cache(gain=2.0)
    q = b.queries()
    out = torch.empty_like(q[0])
    io = kda.make_latent_attn_io(*q, out, 0.1)
    kda.kda_latent_attend(b.kv, io, b.batch, b.workspace(0xFF))
    b.check_attend(q, out, held, 0.1)
    again = out.clone()
    kda.kda_latent_attend(b.kv, io, b.batch, b.workspace(0))
    assert torch.equal(again.view(torch.uint8), out.view(torch.uint8))  # the workspace's contents do not matter


MANY = [
    # lengths from one token up, sequences by the hundred: items of one tile, and pieces that hold many items
    ([1] * 300, [1 + 37 * i % 160 for i in range(300)], 8, 512, 16),
    ([1] * 180, [1 + 211 * i % 1500 for i in range(180)], 64, 512, 64),
    ([3] * 200, [3 + 53 * i % 400 for i in range(200)], 16, 256, 32),
    ([1 + 7 * i % 40 for i in range(60)], [40 + 97 * i % 700 for i in range(60)], 4, 512, 128),
    ([32 * (i % 3) for i in range(30)], [256 + 64 * (i % 5) for i in range(30)], 2, 128, 64),
]


@FMTS
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attend_many_sequences(case, fmt):
    new, total, heads, latent, page = MANY[case]
    b = R.Batch(new, total, heads, latent, 64, page, BF, fmt, seed=200 + case, fill=NAN)
    held = b.fill_cache()
    q = b.queries()
    out = torch.full_like(q[0], 9.0)
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    b.no_error()
    b.check_attend(q, out, held, 0.07)


@FMTS
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new,heads", [(1, 15), (1, 16), (1, 17), (1, 33), (1, 64), (1, 65), (2, 32), (3, 32), (64, 1), (65, 1), (5, 13)])
def test_attend_rows_of_a_tile(new, heads, page, fmt):
    """One row to a little over a tile, over caches that end at a tile's border and one token to either side of it."""
    b = R.Batch([new] * 6, [max(t, new) for t in (63, 64, 65, 127, 128, 193)], heads, 512, 64, page, BF, fmt, seed=300 + new, fill=NAN)
    held = b.fill_cache()
    q = b.queries()
    out = torch.full_like(q[0], 9.0)
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    b.no_error()
    b.check_attend(q, out, held, 0.07)


@pytest.mark.parametrize("new,heads,latent,act", [(1, 16, 512, BF), (4, 16, 256, BF), (9, 8, 128, BF), (1, 3, 128, F32)])
def test_attend_few_items_of_any_length(new, heads, latent, act):
    """Fewer items than CTAs, of lengths that put the cuts between CTAs at every place of a key step."""
    rng = np.random.default_rng(73)
    for trial in range(15):
        total = [new + int(x) for x in rng.integers(0, int(rng.choice([300, 1500, 4000])), int(rng.integers(1, 7)))]
        b = R.Batch([new] * len(total), total, heads, latent, 64, 64, act, "act", seed=400 + trial)
        held = b.fill_cache()
        q = b.queries()
        out = torch.full_like(q[0], 9.0)
        kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
        b.no_error()
        b.check_attend(q, out, held, 0.07)


@FMTS
@ACTS
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("new,heads,latent", [(4, 4, 512), (40, 2, 256), (100, 3, 128)])
def test_masked_latents_may_be_anything(act, bad, new, heads, latent, fmt):
    """A token's non-finite latent or key part reaches its own and later rows only."""
    total = new + 70
    b = R.Batch([new], [total], heads, latent, 64, 32, act, fmt, seed=11)
    held = b.fill_cache()
    at = total - new // 2  # a position inside the chunk
    page, line = int(b.table[0, at // 32]), at % 32
    if fmt == "e4m3":
        b.kv.c.view(torch.uint8)[page, line, 1] = 0x7F
    else:
        b.kv.c[page, line, 1] = bad
    b.kv.kr[int(b.table[0, (total - 1) // 32]), (total - 1) % 32, 0] = NAN  # the last token's key part
    q = b.queries()
    q[0][:] = q[0].abs() + 0.1  # so that an infinity scores +inf
    out = torch.empty_like(q[0])
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    got, t_bad = out.double().cpu(), at - (total - new)
    assert torch.isfinite(got[:t_bad]).all() and torch.isnan(got[t_bad:]).all()
    b.set([t_bad], [at])  # the rows before it, as they would be without it
    b.check_attend(tuple(t[:t_bad] for t in q), out[:t_bad], [(held[0][0][:at], held[0][1][:at])], 0.07)


@FMTS
@ACTS
@pytest.mark.parametrize("new,heads", [([1, 6], 4), ([1, 2], 40)])
def test_extreme_scores(act, fmt, new, heads):
    """Scores thousands apart (a row whose best key leads by more than the scores' error gives its latent), rows whose scores
    are all -inf, and queries that are not finite."""
    b = R.Batch(new, [300, 200], heads, 512, 64, 16, act, fmt, seed=13)
    held = b.fill_cache(gain=30.0)
    q = b.queries(gain=20.0)
    out = torch.empty_like(q[0])
    io = kda.make_latent_attn_io(*q, out, 1.0)
    kda.kda_latent_attend(b.kv, io, b.batch, b.workspace())
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    a, told = 0, 0
    for (T, L), (c, kr) in zip(zip(b.new, b.total), held):
        for t in range(T):
            n = L - T + t + 1
            s = q[0][a + t].double().cpu() @ c[:n].T + q[1][a + t].double().cpu() @ kr[:n].T
            best = s.topk(2, -1)
            qk = torch.cat((q[0][a + t], q[1][a + t]), -1).double().cpu().norm(dim=-1) * torch.cat((c, kr), -1).norm(dim=-1).max()
            clear = best.values[:, 0] - best.values[:, 1] > 60 + 4 * 580 * 2.0 ** -24 * qk
            want = c[best.indices[:, 0]]
            told += int(clear.sum())
            assert ((got[a + t] - want).abs()[clear] <= 2.0 ** -20 * c.abs().max() + want.abs()[clear] * 3 * half_step(BF)).all()
        a += T
    assert told > heads
    b.kv.kr[..., 0] = -INF
    q[1][:, :, 0] = 1.0
    kda.kda_latent_attend(b.kv, io, b.batch, b.workspace())
    assert (out == 0).all()
    held = b.fill_cache()
    q = b.queries()
    q[0][0, 1, 5], q[1][1, 0, 3] = NAN, INF
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[1, 0]).all()
    out[0, 1] = out[1, 0] = 0
    assert torch.isfinite(out).all()


@FMTS
@pytest.mark.parametrize("scale", [1e-30, 2.0 ** -149])
def test_small_scales_and_zero_queries(scale, fmt):
    """Such rows weigh their keys alike."""
    b = R.Batch([2], [70], 9, 512, 64, 16, BF, fmt, seed=89)
    held = b.fill_cache()
    q = b.queries()
    q[0][0], q[1][0] = 0, 0
    out = torch.empty_like(q[0])
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, scale), b.batch, b.workspace())
    b.check_attend(q, out, held, scale)


@FMTS
@pytest.mark.parametrize("power", [-117, -100, 100])
def test_latents_of_extreme_sizes(power, fmt):
    """Scales next to the ends of their range.  (In units of the latents, so that the tolerance's floor of 1e-30 means nothing;
    weights times scales are off by 2^-22 of the largest, of scales as of 2^-122 at least: with 70 keys and codes of up to 448
    less than 70 * 448 * 2^-144, where a 2^-7 of sum p |v| is above 2^-126.)"""
    b = R.Batch([2], [70], 9, 512, 64, 16, BF, fmt, seed=97)
    w = b.whole()
    c, kr = w.randn(w.rows, 512, gain=2.0 ** power), w.randn(w.rows, 64)
    kda.kda_latent_append(b.kv, None, kda.make_latent_io(c.cuda(), kr.cuda(), None, None), w.batch)
    held, kr = b.held()[0]
    q = b.queries()
    q[0].mul_(2.0 ** -power if power < 0 and power > -110 else 2.0 ** -100 if power > 0 else 1.0)
    out = torch.empty_like(q[0])
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.05), b.batch, b.workspace())
    b.no_error()
    qc, qr = q[0].double().cpu(), q[1].double().cpu()
    s = (torch.einsum("thl,jl->thj", qc, held) + torch.einsum("thr,jr->thj", qr, kr)) * 0.05
    ref, mag = R.attend(s, held[:, None] * 2.0 ** -power, 68)
    qk = (qc.norm(dim=-1) * held.norm(dim=-1).max() + qr.norm(dim=-1) * kr.norm(dim=-1).max()) * 0.05
    R.check(out.double().cpu() * 2.0 ** -power, ref, mag, qk, 576, BF)


def test_bad_pages_and_tables_on_the_device():
    """A page outside the cache: its tokens are absent; inconsistent tables: the sequence's rows are left alone."""
    for act, new, total, heads in ((BF, [1, 1], [100, 90], 16), (BF, [20, 30], [100, 90], 4), (F32, [2, 3], [100, 90], 4)):
        b = R.Batch(new, total, heads, 512, 64, 16, act, "act", seed=17)
        held = b.fill_cache()
        q = b.queries()
        out = torch.full_like(q[0], 9.0)
        io, ws = kda.make_latent_attn_io(*q, out, 0.07), b.workspace()
        b.dev[2][0, 1] = b.kv.num_pages  # positions 16..31 of sequence 0
        b.dev[2][1, 2] = -5              # positions 32..47 of sequence 1
        kda.kda_latent_attend(b.kv, io, b.batch, ws)
        assert kda.kda_latent_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_PAGE_RANGE)
        b.check_attend(q, out, held, 0.07, gone=[range(16, 32), range(32, 48)])
        b.dev[1][1] = new[1] - 1  # fewer cached tokens than it brings
        out.fill_(9.0)
        kda.kda_latent_attend(b.kv, io, b.batch, ws)
        assert kda.kda_latent_poll_device_error(b.kv)[1] & kda.KDA_DEVERR_META
        assert (out[new[0]:] == 9.0).all() and not (out[:new[0]] == 9.0).any()
        b.dev[1][1] = b.dev[2].shape[1] * 16 + 1  # longer than its row of the page table
        kda.kda_latent_attend(b.kv, io, b.batch, ws)
        assert kda.kda_latent_poll_device_error(b.kv)[1] & kda.KDA_DEVERR_META
        assert (out[new[0]:] == 9.0).all()
        b.dev[1][1] = total[1]
        b.dev[2][0] = -1  # all of a sequence's pages
        kda.kda_latent_attend(b.kv, io, b.batch, ws)
        assert kda.kda_latent_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_PAGE_RANGE
        assert (out[:new[0]] == 0).all() and not (out[new[0]:] == 0).all()


@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act")])
def test_far_positions_and_absent_pages(act, fmt):
    """A context of tens of millions of tokens of which only the last pages are there (a window)."""
    page, far, new = 128, 20_000_000, 2
    b = R.Batch([new], [new + 200], 4, 512, 64, page, act, fmt, seed=47)
    held = b.fill_cache()
    skip = far // page
    table = torch.full((1, skip + b.table.shape[1]), -1, dtype=torch.int32)
    table[0, skip:] = b.table[0]
    lens = torch.tensor([skip * page + new + 200], dtype=torch.int32).cuda()
    b.batch = kda.make_kv_batch(b.dev[0], lens, table.cuda(), max_rows=b.rows, max_new=new)
    q = b.queries()
    out = torch.full_like(q[0], 9.0)
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    assert kda.kda_latent_poll_device_error(b.kv) == (kda.KDA_ERR_DEVICE, kda.KDA_DEVERR_PAGE_RANGE)
    b.check_attend(q, out, held, 0.07)


@FMTS
def test_offsets_past_32_bits(fmt):
    """A cache of more than 2^31 values, its sequences on the far pages."""
    page, latent = 64, 512
    n_pages = (1 << 31) // (page * latent) + 200
    b = R.Batch([1, 3, 70], [200, 130, 70], 16, latent, 64, page, BF, fmt, seed=23, num_pages=n_pages)
    per = [-(-t // page) for t in b.total]
    at = n_pages - sum(per)
    for i, c in enumerate(per):
        b.table[i, :c] = torch.arange(at, at + c, dtype=torch.int32)
        at += c
    b.dev[2].copy_(b.table)
    held = b.fill_cache()
    q = b.queries()
    out = torch.empty_like(q[0])
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    b.no_error()
    b.check_attend(q, out, held, 0.07)
    assert b.kv.kr[:100].abs().max() == 0


def test_no_sequences_and_no_rows_are_no_ops():
    b = R.Batch([1], [5], 2, 128, 16, 16, BF, "act")
    x, y = torch.zeros(1, 128, dtype=BF, device="cuda"), torch.zeros(1, 16, dtype=BF, device="cuda")
    q = torch.full((1, 2, 128), 3.0, dtype=BF, device="cuda"), torch.full((1, 2, 16), 3.0, dtype=BF, device="cuda")
    empty, one = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for batch in (kda.make_kv_batch(one, empty, empty.view(0, 4), 0, 1), kda.make_kv_batch(*b.dev, 0, 1)):
        assert kda.kda_latent_attend_workspace_bytes(b.kv, batch) == 0
        kda.kda_latent_append(b.kv, None, kda.make_latent_io(x, y, None, None), batch)
        kda.kda_latent_read(b.kv, batch, x, y)
        kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, q[0].clone(), 1.0), batch, None)
    none = R.Batch([0, 0], [0, 7], 2, 128, 16, 16, BF, "act")
    out = torch.full((1, 2, 128), 9.0, dtype=BF, device="cuda")
    kda.kda_latent_attend(none.kv, kda.make_latent_attn_io(*q, out, 1.0), none.batch, none.workspace())
    none.no_error()
    assert (out == 9.0).all()


@pytest.mark.parametrize("act,fmt,new", [(BF, "act", 1), (BF, "e4m3", 1), (BF, "act", 5), (F32, "act", 2)])
def test_replayed_with_other_lengths(act, fmt, new):
    """Captured once, replayed with tables that move work between CTAs, sequences that drop out and new pages."""
    b = R.Batch([new] * 3, [700, 600, 500], 16, 512, 64, 16, act, fmt, seed=67)
    b.fill_cache()
    q = b.queries()
    out = torch.empty_like(q[0])
    ws, st, batch = b.workspace(), torch.cuda.Stream(), b.batch
    io, dev = kda.make_latent_attn_io(*q, out, 0.07), b.dev
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        kda.kda_latent_attend(b.kv, io, batch, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            kda.kda_latent_attend(b.kv, io, batch, ws)
    torch.cuda.synchronize()
    for news, lens in (([new] * 3, [700, 600, 500]), ([new, 0, new], [new, 600, 333]), ([0, new, 0], [9, 17 + new, 9]),
                       ([1, 1, 1], [1, 2, 3]), ([new] * 3, [128, 640, 127 + new])):
        b.table = b.table.flip(1)[:, :b.table.shape[1]].clamp(min=0)
        dev[2].copy_(b.table)
        b.set(news, lens)
        b.dev = (b.dev[0], b.dev[1], dev[2])
        dev[0].copy_(b.cu), dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(9.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        b.no_error()
        b.check_attend(q, out, b.held(), 0.07)
        assert (out[b.rows:] == 9.0).all()


@FMTS
def test_two_calls_at_once(fmt):
    """Two streams, each with its own workspace, over one cache and at the same time: what each gives alone."""
    streams, work = [torch.cuda.Stream() for _ in range(2)], []
    b = R.Batch([1] * 20, [900 + 31 * i for i in range(20)], 16, 512, 64, 64, BF, fmt, seed=61)
    b.fill_cache()
    for new in (1, 9):
        b.set([new] * 20, b.total)
        q = b.queries()
        out = torch.empty_like(q[0])
        io, ws, batch = kda.make_latent_attn_io(*q, out, 0.07), b.workspace(), b.batch
        kda.kda_latent_attend(b.kv, io, batch, ws)
        work.append((io, ws, batch, out, out.clone()))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (io, ws, batch, _, _) in zip(streams, work):
            kda.kda_latent_attend(b.kv, io, batch, ws, stream=st)
    torch.cuda.synchronize()
    b.no_error()
    for _, _, _, out, alone in work:
        assert torch.equal(out, alone)


@FMTS
def test_loose_bounds(fmt):
    """Host bounds larger than what the tables hold."""
    b = R.Batch([2, 0, 1], [152, 20, 33], 16, 512, 64, 32, BF, fmt, seed=59, extra_rows=5)
    held = b.fill_cache()
    q = b.queries()
    out = torch.empty_like(q[0])
    for max_new in (2, 3, 70, 1000):
        out.fill_(9.0)
        batch = kda.make_kv_batch(*b.dev, max_rows=b.max_rows, max_new=max_new)
        ws = torch.empty(kda.kda_latent_attend_workspace_bytes(b.kv, batch), dtype=torch.uint8, device="cuda")
        kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), batch, ws)
        b.no_error()
        b.check_attend(q, out, held, 0.07)
        assert (out[b.rows:] == 9.0).all()


def test_a_page_twice_in_a_sequence():
    b = R.Batch([1, 4], [300, 310], 16, 512, 64, 32, BF, "act", seed=71)
    b.fill_cache()
    b.dev[2][:, 1:5] = b.dev[2][0, 0]
    q = b.queries()
    out = torch.empty_like(q[0])
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, b.workspace())
    b.no_error()
    b.check_attend(q, out, b.held(), 0.07)


def test_calls_on_another_stream_and_profile():
    b = R.Batch([2, 1], [190, 70], 16, 512, 64, 32, BF, "e4m3", seed=37)
    held = b.fill_cache()
    q = b.queries()
    out = torch.empty_like(q[0])
    st, ws = torch.cuda.Stream(), b.workspace()
    torch.cuda.synchronize()
    kda.kda_profile_start(16)
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, out, 0.07), b.batch, ws, stream=st)
    prof = kda.kda_profile_stop()
    st.synchronize()
    assert prof["latent_attend"][0] == 1 and prof["latent_combine"][0] == 1
    b.check_attend(q, out, held, 0.07)


# ---- expanded form ------------------------------------------------------------------------------------------------------

PREFILL = [
    # new, total, heads, nope, rope, value
    ([1], [1], 2, 128, 64, 128),
    ([130, 1, 33], [130, 200, 129], 3, 128, 64, 128),
    ([5, 0, 64, 65], [64, 7, 64, 65], 5, 64, 32, 64),
    ([300], [300], 2, 128, 64, 64),
    ([257, 255], [257, 700], 2, 64, 64, 128),
    ([100, 17], [356, 530], 4, 128, 16, 128),
    ([1] * 7, [1, 63, 64, 65, 127, 128, 500], 64, 128, 64, 128),
    ([20, 30], [1500, 90], 1, 128, 32, 128),
]


@ACTS
@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill(case, act):
    """Key and value rows behind the last sequence hold NaN."""
    new, total, heads, nope, rope, value = PREFILL[case]
    r = R.Rows(new, total, heads, nope, rope, value, act, seed=500 + case, extra_rows=2, extra_keys=3)
    r.call()
    r.no_error()
    r.check()


@ACTS
@pytest.mark.parametrize("new,heads", [(127, 3), (128, 3), (129, 3), (255, 1), (256, 1), (257, 1), (513, 2)])
def test_prefill_rows_of_a_tile(new, heads, act):
    r = R.Rows([new, new], [new, new + 61], heads, 128, 64, 128, act, seed=new)
    r.call()
    r.no_error()
    r.check()


@ACTS
@pytest.mark.parametrize("new,total", [([20], [6000]), ([1, 3], [4000, 17]), ([300], [2500])])
def test_prefill_long_cut_into_parts(act, new, total):
    r = R.Rows(new, total, 2, 128, 64, 128, act, seed=7, gain=3.0)
    r.call(r.workspace(0xFF))
    r.no_error()
    r.check()
    first = r.out.clone()
    r.call(r.workspace(0))
    assert torch.equal(first.view(torch.uint8), r.out.contiguous().view(torch.uint8))


@ACTS
def test_prefill_many_sequences(act):
    new = [1 + 37 * i % 90 for i in range(90)]
    total = [n + 53 * i % 300 for i, n in enumerate(new)]
    r = R.Rows(new, total, 3, 64, 32, 64, act, seed=77)
    r.call()
    r.no_error()
    r.check()


@ACTS
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("new,value", [(4, 128), (100, 64), (300, 128), (600, 64)])
def test_masked_values_and_keys_may_be_anything(act, bad, new, value):
    """A token's non-finite value or key reaches its own and later rows only; the channel of a bad value alone."""
    total = new + 70
    r = R.Rows([new, 3], [total, 50], 2, 128, 64, value, act, seed=11)
    at, t_bad = total - new // 2, new - new // 2
    r.v[at, :, 1] = bad
    r.k[total - 1, :, 0] = NAN
    r.call()
    got = r.out.double().cpu()
    assert torch.isfinite(got[:t_bad]).all()
    assert not torch.isfinite(got[t_bad:new - 1, :, 1]).any()
    assert torch.isfinite(got[t_bad:new - 1, :, 2:]).all() and torch.isfinite(got[t_bad:new - 1, :, 0]).all()
    assert torch.isnan(got[new - 1]).all() and torch.isfinite(got[new:]).all()
    r.check(only=[1])
    r.v[at, :, 1], r.k[total - 1, :, 0] = 0, 0
    kept = r.out.clone()
    r.call()
    assert torch.equal(kept[:t_bad], r.out[:t_bad])
    # a sum of `total` terms in another order is off by at most total units of 2^-24 of sum p |v| <= max |v|, and may then
    # round to the neighbouring bf16 (a whole step)
    a, b = (x[t_bad:new - 1, :, 2:].double() for x in (kept, r.out))
    step = b.abs() * (2 * half_step(BF) if act == BF else 2.0 ** -23)
    assert ((a - b).abs() <= step + total * 2.0 ** -24 * float(r.v[:total].abs().max())).all()


@ACTS
def test_prefill_extreme_scores(act):
    r = R.Rows([60, 200], [90, 300], 2, 128, 64, 128, act, seed=13)
    r.io.scale = 100.0
    r.call()
    assert torch.isfinite(r.out).all()
    r.kr[:, 0] = -INF
    r.qr[..., 0] = 1.0
    r.call()
    assert (r.out == 0).all()
    r.kr[:, 0] = 1.0
    r.qn[3, 1, 0], r.qr[70, 0, 5] = NAN, INF
    r.io.scale = 0.07
    r.call()
    assert torch.isnan(r.out[3, 1]).all() and not torch.isfinite(r.out[70, 0]).any()
    r.out[3, 1] = r.out[70, 0] = 0
    assert torch.isfinite(r.out).all()
    r.qn[:], r.qr[:] = 0, 0
    r.io.scale = 2.0 ** -149
    r.call()
    r.check(scale=2.0 ** -149)


def test_prefill_bad_tables():
    """An inconsistent sequence's rows are left alone, the others served."""
    for act in (BF, F32):
        r = R.Rows([40, 50, 10], [60, 90, 10], 2, 128, 64, 128, act, seed=17)
        cu, cu_kv = r.dev
        for change in ("short", "past", "decreasing", "long"):
            cu.copy_(r.cu), cu_kv.copy_(r.cu_kv)
            r.batch.max_new = 50
            bad = 1
            if change == "short":
                cu_kv[1] = int(cu_kv[2]) - 49  # fewer keys than tokens (and sequence 0 has more keys than its own)
            elif change == "past":
                cu_kv[3], bad = r.max_keys + 1, 2
            elif change == "decreasing":
                cu_kv[2], bad = int(cu_kv[1]) - 1, 1
            else:
                r.batch.max_new = 49
            r.out.fill_(9.0)
            r.call()
            st, flags = kda.kda_latent_poll_device_error(r.cache)
            assert st == kda.KDA_ERR_DEVICE and flags == kda.KDA_DEVERR_META, change
            a, z = int(r.cu[bad]), int(r.cu[bad + 1])
            assert (r.out[a:z] == 9.0).all() and not (r.out[:a] == 9.0).any(), change
        cu.copy_(r.cu), cu_kv.copy_(r.cu_kv)
        r.batch.max_new = 50
        r.call()
        r.no_error()
        r.check()


@ACTS
def test_prefill_replayed_with_other_lengths(act):
    """Captured once, replayed with tables that move work between CTAs, sequences that drop out and one past the bound."""
    r = R.Rows([300, 129, 40], [700, 400, 333], 3, 128, 64, 128, act, seed=83)
    ws, st = r.workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        r.call(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            r.call(ws)
    torch.cuda.synchronize()
    for new, total in (([300, 129, 40], [700, 400, 333]), ([1, 0, 256], [1433, 0, 256]), ([0, 128, 0], [5, 1400, 9]),
                       ([7, 8, 9], [7, 8, 9]), ([255, 1, 128], [255, 1000, 129])):
        r.new, r.total, r.rows, r.keys = new, total, sum(new), sum(total)
        for host, dev, n in ((r.cu, r.dev[0], new), (r.cu_kv, r.dev[1], total)):
            host.copy_(torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32))
            dev.copy_(host)
        r.out.fill_(9.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        good = [i for i in range(3) if sum(total[:i + 1]) <= r.max_keys]
        if len(good) == 3:
            r.no_error()
        else:  # the last sequence's keys go past the bound: its rows are left alone
            assert kda.kda_latent_poll_device_error(r.cache)[1] == kda.KDA_DEVERR_META
            assert (r.out[int(r.cu[2]):] == 9.0).all()
        r.check(only=good)


def test_two_prefills_at_once():
    """Two streams, each with its own workspace, at the same time: what each gives alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [R.Rows([n] * 3, [n + 300, n, n + 77], 4, 128, 64, 128, BF, seed=n) for n in (90, 300)]
    work = [(r, r.workspace()) for r in work]
    for r, ws in work:
        r.call(ws)
    torch.cuda.synchronize()
    alone = [r.out.clone() for r, _ in work]
    for _ in range(20):
        for st, (r, ws) in zip(streams, work):
            r.call(ws, stream=st)
    torch.cuda.synchronize()
    for (r, _), out in zip(work, alone):
        r.no_error()
        assert torch.equal(r.out, out)
        r.check()


@ACTS
def test_prefill_layouts(act):
    """Head-major tensors, rows 16 bytes apart from any wider border, loose bounds, and replay from a graph."""
    new, total, heads = [70, 9], [130, 9], 3
    r = R.Rows(new, total, heads, 128, 32, 64, act, seed=31)
    pad = 8 if act == BF else 4
    for name in ("qn", "qr", "k", "v"):
        t = getattr(r, name)
        wide = torch.zeros(heads, t.shape[0], t.shape[2] + pad, dtype=act, device="cuda")
        wide[..., pad:] = t.transpose(0, 1)
        setattr(r, name, wide[..., pad:].transpose(0, 1))
    r.io = kda.make_latent_prefill_io(r.qn, r.qr, r.k, r.kr, r.v, r.out)
    r.batch = kda.make_latent_prefill_batch(*r.dev, max_rows=r.max_rows, max_kv_rows=r.max_keys, max_new=1000)
    ws, st = r.workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        r.call(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            r.call(ws)
    torch.cuda.synchronize()
    r.check()
    for new, total in (([9, 70], [9, 130]), ([0, 79], [60, 79]), ([1, 1], [2, 137])):
        r.new, r.total, r.rows = new, total, sum(new)
        r.cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32)
        r.cu_kv = torch.tensor([0, total[0], sum(total)], dtype=torch.int32)
        r.dev[0].copy_(r.cu), r.dev[1].copy_(r.cu_kv)
        r.out.fill_(9.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        r.no_error()
        r.check()


def test_prefill_no_rows_are_no_ops():
    r = R.Rows([3], [5], 2, 64, 16, 64, BF)
    for kw in (dict(max_rows=0), dict(max_rows=0, max_kv_rows=0)):
        batch = kda.make_latent_prefill_batch(*r.dev, **{**dict(max_rows=3, max_kv_rows=5, max_new=3), **kw})
        assert kda.kda_latent_prefill_workspace_bytes(r.cache, r.io, batch) == 0
        kda.kda_latent_prefill(r.cache, r.io, batch, None)
    r = R.Rows([0, 0], [0, 7], 2, 64, 16, 64, BF)
    r.call()
    r.no_error()
    assert (r.out == 9.0).all()


# ---- together ------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("act,fmt", [(BF, "act"), (BF, "e4m3"), (F32, "act")], ids=["bf16", "bf16-e4m3", "f32"])
def test_prompt_expanded_then_decode_absorbed(act, fmt):
    """A layer as it is served: a prompt in two chunks in the expanded form (latents appended, read back and multiplied out),
    then single tokens and drafts in the absorbed form; every call against float64 attention over what the cache holds, with
    the same up-projections."""
    H, L, Rr, N, V, page = 16, 128, 32, 64, 64, 16
    plan = [("expanded", [50, 70]), ("expanded", [40, 1]), ("absorbed", [1, 1]), ("absorbed", [4, 4]), ("absorbed", [1, 0])]
    last = np.sum([p[1] for p in plan], 0).tolist()
    b = R.Batch([1, 1], last, H, L, Rr, page, act, fmt, seed=29)
    uk, uv = b.randn(H, N, L, gain=L ** -0.5).cuda(), b.randn(H, V, L, gain=L ** -0.5).cuda()
    freq = [10000.0 ** (-2.0 * i / Rr) for i in range(Rr // 2)]
    w = (1 + 0.1 * torch.randn(L, generator=b.gen)).to(act)
    params = kda.make_latent_params(w.cuda(), 1e-5, freq)
    scale, total = (N + Rr) ** -0.5, np.zeros(2, dtype=int)
    for form, new in plan:
        total = total + new
        b.set(new, total.tolist())
        c, kr = b.randn(b.rows, L).cuda(), b.randn(b.rows, Rr).cuda()
        q = b.randn(b.rows, H, N + Rr).cuda()
        kda.kda_latent_append(b.kv, params, kda.make_latent_io(c, kr, q[..., N:], q[..., N:]), b.batch)
        if form == "absorbed":
            qc = torch.einsum("thn,hnl->thl", q[..., :N], uk)
            out = torch.empty(b.rows, H, L, dtype=act, device="cuda")
            kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(qc, q[..., N:], out, scale), b.batch, b.workspace())
            b.no_error()
            b.check_attend((qc, q[..., N:]), out, b.held(), scale)
            got = torch.einsum("thl,hvl->thv", out, uv)
        else:
            whole = b.whole()
            lat, key = torch.empty(whole.rows, L, dtype=act, device="cuda"), torch.empty(whole.rows, Rr, dtype=act, device="cuda")
            kda.kda_latent_read(b.kv, whole.batch, lat, key)
            k, v = torch.einsum("jl,hnl->jhn", lat, uk).contiguous(), torch.einsum("jl,hvl->jhv", lat, uv).contiguous()
            got = torch.empty(b.rows, H, V, dtype=act, device="cuda")
            batch = kda.make_latent_prefill_batch(b.dev[0], whole.dev[0], b.rows, whole.rows, max(new))
            io = kda.make_latent_prefill_io(q[..., :N], q[..., N:], k, key, v, got)
            ws = torch.empty(kda.kda_latent_prefill_workspace_bytes(b.kv, io, batch), dtype=torch.uint8, device="cuda")
            kda.kda_latent_prefill(b.kv, io, batch, ws)
            b.no_error()
        # both forms are the same function: float64 over the cache, roundings of the products around the calls included
        # (bf16: q U and U c are rounded to 2^-8 each, which moves a score by up to 2^-7 |q| |k| scale; then o U and out)
        for i, (T, n) in enumerate(zip(b.new, b.total)):
            if T == 0:
                continue
            a = int(b.cu[i])
            lat, key = b.held()[i]
            kk, vv = torch.einsum("jl,hnl->jhn", lat, uk.double().cpu()), torch.einsum("jl,hvl->jhv", lat, uv.double().cpu())
            qq = q[a:a + T].double().cpu()
            s = (torch.einsum("thn,jhn->thj", qq[..., :N], kk) + torch.einsum("thr,jr->thj", qq[..., N:], key)) * scale
            ref, mag = R.attend(s, vv, n - T)
            lat_mag = R.attend(s, lat[:, None], n - T)[1]
            up = torch.einsum("thl,hvl->thv", lat_mag, uv.double().cpu().abs())
            if act == BF:
                mags = torch.einsum("thn,hnl->thl", qq[..., :N].abs(), uk.double().cpu().abs()) @ lat.abs().T
                move = 2 * half_step(BF) * scale * mags.amax(-1, keepdim=True)
                tol = (2 * move + 6 * half_step(BF)) * up + 2 * half_step(BF) * ref.abs()
            else:
                tol = 2.0 ** -14 * up
            assert ((got[a:a + T].double().cpu() - ref).abs() <= tol).all(), form


def test_decode_step_from_a_graph():
    """append + absorbed attention captured once and replayed with other tables and inputs; two graphs share a workspace."""
    b = R.Batch([1, 1], [400, 200], 64, 512, 64, 64, BF, "act", seed=31)
    b.fill_cache()
    c, kr, q = b.randn(2, 512).cuda(), b.randn(2, 64).cuda(), b.randn(2, 64, 64).cuda()
    qc = b.queries()[0]
    qs, outs = [torch.empty_like(q) for _ in range(2)], [torch.empty_like(qc) for _ in range(2)]
    params = kda.make_latent_params(torch.ones(512, dtype=BF, device="cuda"), 1e-5, [1.0 / (10.0 + i) for i in range(32)])
    ws, st, graphs, batch, dev = b.workspace(), torch.cuda.Stream(), [], b.batch, b.dev

    def step(i):
        kda.kda_latent_append(b.kv, params, kda.make_latent_io(c, kr, q, qs[i]), batch)
        kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(qc, qs[i], outs[i], 0.05 * (i + 1)), batch, ws)

    with torch.cuda.stream(st):
        step(0)
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                step(i)
            graphs.append(g)
    torch.cuda.synchronize()
    for lens in ([400, 200], [399, 1], [65, 130]):
        dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(b.randn(2, 64, 64))
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        b.set([1, 1], lens)
        for i in range(2):
            b.check_attend((qc, qs[i]), outs[i], b.held(), 0.05 * (i + 1))

"""kda_latent_append in each of its forms (a row to a CTA, two rows, a row to a warp: by the number of rows and of the device's
SMs) with norm, rotation and many heads, against float64.  Tolerances: those of test_latent_gpu.py."""

from __future__ import annotations

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import latent_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()


# sizes well inside each form and next to where it ends, and so many more rows that a moved border leaves none out
FORMS = {"cta": lambda n: 2 * n - 1, "cta_most": lambda n: 6 * n, "half": lambda n: 6 * n + 3, "half_most": lambda n: 12 * n,
         "warp": lambda n: 12 * n + 3, "warp_many": lambda n: 32 * n + 5}


def rows_of(form):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return FORMS[form](sms)


def near(got, ref, act, slack=0.0):
    # half a step of the type, and 2^-18 of the row's largest (arithmetic in 32 bits)
    tol = ref.abs() * (R.half_step(BF) if act == BF else 0.0) + 2.0 ** -18 * ref.abs().amax(-1, keepdim=True) + slack
    assert ((got.double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("act,fmt,heads,latent,rope,rot,inter,in_place", [
    (BF, "e4m3", 64, 512, 64, 64, False, False),
    (BF, "act", 64, 512, 64, 64, True, True),
    (BF, "act", 17, 256, 64, 24, False, True),  # places of four channels
    (BF, "e4m3", 17, 512, 64, 40, True, False),
    (BF, "act", 33, 128, 16, 16, False, False),
    (BF, "e4m3", 17, 512, 64, 32, False, True),  # half of the channels turn
    (F32, "act", 17, 512, 64, 64, False, False),
    (F32, "e4m3", 17, 128, 32, 24, True, True),
])
def test_append_forms(form, act, fmt, heads, latent, rope, rot, inter, in_place):
    rows = rows_of(form)
    new = [rows // 3, 0, rows - rows // 3 - 1, 1]  # ragged, behind prefixes that put the sequences' ends inside pages
    total = [new[0] + 37, 9, new[2] + 1000, 70]
    b = R.Batch(new, total, heads, latent, rope, 64, act, fmt, seed=rows + heads, extra_rows=3)
    c, kr, q = (b.randn(b.max_rows, *s).cuda() for s in ((latent,), (rope,), (heads, rope)))
    q0, q_out = q.clone(), q if in_place else torch.full_like(q, 7.0)
    w = (1 + 0.1 * torch.randn(latent, generator=b.gen)).to(act)
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    kda.kda_latent_append(b.kv, kda.make_latent_params(w.cuda(), 1e-5, freq, inter), kda.make_latent_io(c, kr, q, q_out), b.batch)
    b.no_error()
    pos, (pg, line) = b.positions(), b.lines()
    assert torch.equal(q_out[b.rows:], q0[b.rows:] if in_place else torch.full_like(q0[b.rows:], 7.0))
    for a in range(0, b.rows, 1000):  # in pieces: the float64 queries of all rows are large
        z = min(b.rows, a + 1000)
        near(q_out[a:z], R.rotate(q0[a:z].cpu(), pos[a:z], freq, inter), act)
    near(b.kv.kr.cpu()[pg, line], R.rotate(kr[:b.rows, None].cpu(), pos, freq, inter)[:, 0], act)
    ref, got = R.norm(c[:b.rows].cpu(), w, 1e-5), b.kv.c.float().cpu()[pg, line].double()
    if fmt == "act":
        near(got, ref, act)
    else:
        unit, top = 2.0 ** (b.kv.c_scale.cpu()[pg, line].double() - 127)[:, None], ref.abs().amax(-1, keepdim=True)
        slack = 2.0 ** -18 * top
        assert (unit * 448 >= top - slack).all() and (unit * 224 <= top + slack).all()
        assert ((got * unit - ref).abs() <= ref.abs() * 2.0 ** -4 + unit * 2.0 ** -10 + slack).all()
    touched = torch.zeros(b.kv.num_pages, 64, dtype=torch.bool)
    touched[pg, line] = True
    assert not b.kv.kr.cpu()[~touched].any() and not b.kv.c.view(torch.uint8).cpu()[~touched].any()  # nothing else was written

"""Paged-cache operators at the edges of their contract, on a GPU: tables that contradict themselves, values that are not
finite, and what the plain tests of test_kv_gpu.py leave out.  Tolerances are those of that file's docstring."""

from __future__ import annotations

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

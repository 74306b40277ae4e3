"""Latent attention at its corners on a GPU, against the plain float64 statements of latent_ref.py: values that are not finite
under weights too small for 32 bits."""

from __future__ import annotations

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

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

"""What include/kda.h promises of latent attention's precision, as checks in float64.

half(t) is the most that a rounding to t is off by, relatively.  A call on bf16 rows may round each weight by half(bf16) = 2^-8 of
it, and rounds its output by as much; 32-bit calls round neither.  Over e4m3 pages the kernel means each weight as three e5m2
terms: 2^-11 for the f16 that they are split from and (1/9)^3 for the terms, together below 2^-9."""

from __future__ import annotations

import torch

import latent_ref as R

BF = torch.bfloat16
HALF = R.half_step(BF)


def weight_bound(act, fmt="act"):
    return 0.0 if act != BF else HALF / 2 if fmt == "e4m3" else HALF


def within_contract(got, ref, mag, rel, act, extra=0.0, what=""):
    """Element by element: rel is the 32-bit arithmetic's share of a weight (latent_ref.check), extra an absolute one."""
    half = HALF if act == BF else 0.0
    got = got.double().cpu()
    tol = mag * (rel + half) + ref.abs() * half + extra + 1e-30
    worst = float(((got - ref).abs() / tol).max())
    assert worst <= 1.0, f"{what}: {worst:.3f} of what the contract allows"


def flat_rows(got, ref, act, fmt="act", what=""):
    """Of many weights that are alike, norm against norm: a rounding that is off by at most h is off by h / sqrt(3) in the root of
    its mean square (less, as h belongs to the smallest significand), and those of weights and outputs are independent."""
    bound = ((weight_bound(act, fmt) ** 2 + HALF ** 2) / 3) ** 0.5 if act == BF else 2.0 ** -20
    e = float((got.double().cpu() - ref).norm() / ref.norm())
    assert e <= bound, f"{what}: {e:.3e} of the outputs' norm, at most {bound:.3e}"


def weights_within(got, latents, p, rel, act, fmt="act"):
    """got [..., D] holds in channels where only key j is not zero its weight times the key: [..., j] of p.  Each channel says
    between which bounds its weight lies before the output's rounding; all of a key's have to agree on one within the bound.
    Returns the weights out of it."""
    bad = 0
    bound = weight_bound(act, fmt) + 2.0 ** -20
    for j in range(latents.shape[0]):
        on = latents[j] != 0
        assert not (latents[:j, on].any() or latents[j + 1:, on].any())
        g, c = got[..., on].double().cpu().abs(), latents[j, on].abs()
        # half a step of the output: of 8 significant bits, or of 24
        half = torch.exp2(torch.floor(torch.log2(g.clamp(min=1e-300))) - (8 if act == BF else 24))
        low, high = ((g - half) / c).amax(-1), ((g + half) / c).amin(-1)
        b = bound + rel
        bad += int(((low > p[..., j] * (1 + b)) | (high < p[..., j] * (1 - b))).sum())
    return bad


def disjoint(n, channels, gen):
    """n latents of which each has a part of the channels to itself."""
    c = torch.zeros(n, channels)
    per = channels // n
    for j in range(n):
        c[j, j * per:(j + 1) * per] = torch.randn(per, generator=gen)
    return c

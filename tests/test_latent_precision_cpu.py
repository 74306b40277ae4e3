"""The precision checks themselves (no GPU): they pass what the contract allows, and fail for weights that lose a term."""

import pytest
import torch

from kv_ref import quantise

import latent_precision as P
import latent_ref as R

BF, F32 = torch.bfloat16, torch.float32


def split(w, terms):
    """Weights as f16, then the sum of that many e5m2 terms, each what those before leave."""
    rest, out = w.to(torch.float16), torch.zeros_like(w)
    for _ in range(terms):
        t = rest.to(torch.float8_e5m2)
        out, rest = out + t.double(), rest - t.to(torch.float16)
    return out


def weighed(p, how):
    return {"exact": lambda: p, "bf16": lambda: p.to(BF).double(), "one": lambda: split(p * 128, 1) / 128,
            "two": lambda: split(p * 128, 2) / 128, "three": lambda: split(p * 128, 3) / 128}[how]()


def latents(n, fmt, gen, full=False):
    c = torch.randn(n, 512, generator=gen) if full else P.disjoint(n, 512, gen)
    if fmt == "act":
        return c.to(BF).double()
    val, e = quantise(c.double().numpy())
    return torch.from_numpy(val * 2.0 ** (e - 127.0)[..., None])


@pytest.mark.parametrize("fmt,how,good", [("act", "exact", True), ("act", "bf16", True), ("act", "one", False),
                                          ("e4m3", "exact", True), ("e4m3", "three", True), ("e4m3", "two", False),
                                          ("e4m3", "bf16", False)])
@pytest.mark.parametrize("n", [2, 3, 4])
def test_few_keys_show_a_lost_term(n, fmt, how, good):
    gen = torch.Generator().manual_seed(n)
    c = latents(n, fmt, gen)
    s = torch.randn(64, n, generator=gen, dtype=torch.float64)
    w = torch.exp(s - s.amax(-1, keepdim=True))
    total = w.sum(-1, keepdim=True)
    out = (weighed(w, how) @ c / total).to(BF)
    bad = P.weights_within(out, c, w / total, 0.0, BF, fmt)
    assert (bad == 0) == good, bad


@pytest.mark.parametrize("fmt,how,good", [("act", "bf16", True), ("act", "one", False), ("e4m3", "three", True), ("e4m3", "two", False)])
def test_flat_rows_show_a_lost_term(fmt, how, good):
    gen = torch.Generator().manual_seed(5)
    c = latents(300, fmt, gen, full=True)
    s = torch.randn(64, 300, generator=gen, dtype=torch.float64)
    w = torch.exp(s - s.amax(-1, keepdim=True))
    total = w.sum(-1, keepdim=True)
    got, ref = (weighed(w, how) @ c / total).to(BF), w @ c / total
    if good:
        P.flat_rows(got, ref, BF, fmt)
        P.within_contract(got, ref, w @ c.abs() / total, 0.0, BF)
    else:
        with pytest.raises(AssertionError):
            P.flat_rows(got, ref, BF, fmt)


def test_weights_of_32_bits():
    gen = torch.Generator().manual_seed(7)
    c = P.disjoint(3, 128, gen).double()
    p = torch.softmax(torch.randn(8, 3, generator=gen, dtype=torch.float64), -1)
    assert P.weights_within((p @ c).float(), c, p, 0.0, F32) == 0
    assert P.weights_within((p * (1 + 2.0 ** -18) @ c).float(), c, p, 0.0, F32) > 0

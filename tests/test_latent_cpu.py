"""Host-side refusals of the latent-attention entry points and binding (no GPU), and the reference's pins."""

import ctypes

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import latent_ref as R


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.lib()


A = 0x10000  # an aligned address that no host check dereferences
ref = ctypes.byref
BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


def made(cls, base, kw):
    return cls(**{**base, **kw})


def cache(**kw):
    return made(kda.kda_latent_cache, dict(c=A, c_scale=None, kr=A, err=A, num_pages=4, page_size=16, num_heads=8, latent_dim=128,
                                           rope_dim=32, act=kda.KDA_BF16, format=kda.KDA_KV_ACT), kw)


def batch(**kw):
    return made(kda.kda_kv_batch, dict(cu_seqlens=A, kv_lens=A, page_table=A, n_seqs=2, table_stride=4, max_rows=2, max_new=1), kw)


def io(**kw):
    return made(kda.kda_latent_io, dict(c=A, kr=A, q=A, q_out=2 * A, c_stride=160, kr_stride=160, q_stride=512, q_head_stride=64,
                                        q_out_stride=256, q_out_head_stride=32), kw)


def attn_io(**kw):
    return made(kda.kda_latent_attn_io, dict(q_c=A, q_r=2 * A, out=3 * A, q_c_stride=1024, q_c_head_stride=128, q_r_stride=256,
                                             q_r_head_stride=32, out_stride=1024, out_head_stride=128, scale=0.1), kw)


def rows_io(**kw):
    return made(kda.kda_latent_prefill_io, dict(q_n=A, q_r=2 * A, k=3 * A, kr=4 * A, v=5 * A, out=6 * A, q_n_stride=512,
                                                q_n_head_stride=64, q_r_stride=256, q_r_head_stride=32, k_stride=512,
                                                k_head_stride=64, kr_stride=32, v_stride=1024, v_head_stride=128, out_stride=1024,
                                                out_head_stride=128, nope_dim=64, value_dim=128, scale=0.1), kw)


def rows_batch(**kw):
    return made(kda.kda_latent_prefill_batch, dict(cu_seqlens=A, cu_kv=A, n_seqs=2, max_rows=2, max_kv_rows=9, max_new=1), kw)


CACHES = [(dict(c=None), BAD), (dict(c=A + 8), BAD), (dict(kr=None), BAD), (dict(err=None), BAD), (dict(err=A + 2), BAD),
          (dict(num_pages=0), BAD), (dict(num_heads=0), BAD), (dict(act=2), BAD), (dict(format=2), BAD),
          (dict(format=kda.KDA_KV_E4M3), BAD), (dict(format=kda.KDA_KV_E4M3, c_scale=A + 8), BAD), (dict(latent_dim=0), BAD),
          (dict(rope_dim=0), BAD), (dict(page_size=48), UNSUP), (dict(page_size=256), UNSUP), (dict(latent_dim=64), UNSUP),
          (dict(latent_dim=384), UNSUP), (dict(rope_dim=48), UNSUP), (dict(rope_dim=128), UNSUP)]
BATCHES = [dict(n_seqs=-1), dict(max_rows=-1), dict(max_new=0), dict(max_new=-1), dict(cu_seqlens=None),
           dict(kv_lens=None), dict(page_table=None), dict(table_stride=0), dict(kv_lens=A + 2)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_bad_caches(lib, kw, status):
    c, b = cache(**kw), batch()
    assert lib.kda_latent_append(ref(c), None, ref(io()), ref(b), None) == status
    assert lib.kda_latent_read(ref(c), ref(b), A, 128, A, 32, None) == status
    assert lib.kda_latent_attend(ref(c), ref(attn_io()), ref(b), A, 1 << 40, None) == status
    assert lib.kda_latent_attend_workspace_bytes(ref(c), ref(b)) == 0


@pytest.mark.parametrize("kw", BATCHES)
def test_bad_batches(lib, kw):
    c, b = cache(), batch(**kw)
    assert lib.kda_latent_append(ref(c), None, ref(io()), ref(b), None) == BAD
    assert lib.kda_latent_read(ref(c), ref(b), A, 128, A, 32, None) == BAD
    assert lib.kda_latent_attend(ref(c), ref(attn_io()), ref(b), A, 1 << 40, None) == BAD
    assert lib.kda_latent_attend_workspace_bytes(ref(c), ref(b)) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(q_out=None), dict(c=None), dict(kr=A + 4), dict(c_stride=120),
                                dict(kr_stride=36), dict(kr_stride=24), dict(q_stride=24), dict(q_head_stride=36),
                                dict(q_out_head_stride=-32), dict(q_out=A), dict(c_stride=1 << 37)])
def test_bad_append_rows(lib, kw):
    assert lib.kda_latent_append(ref(cache()), None, ref(io(**kw)), ref(batch()), None) == BAD


def test_bad_norm_and_rotation(lib):
    freq = (ctypes.c_double * 16)(*[0.5] * 16)
    inf = (ctypes.c_double * 16)(*[float("inf")] * 16)
    for kw, status in ((dict(c_norm_w=A + 2), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(rot_dim=40), BAD),
                       (dict(rot_dim=-8), BAD), (dict(rot_dim=16, inv_freq=None), BAD), (dict(rot_dim=16, inv_freq=inf), BAD),
                       (dict(interleaved=2), BAD), (dict(rot_dim=12), UNSUP)):
        p = made(kda.kda_latent_params, dict(c_norm_w=A, eps=1e-5, rot_dim=32, interleaved=0, inv_freq=freq), kw)
        assert lib.kda_latent_append(ref(cache()), ref(p), ref(io()), ref(batch()), None) == status, kw


@pytest.mark.parametrize("args", [(None, 128, A, 32), (A, 128, None, 32), (A + 8, 128, A, 32), (A, 120, A, 32), (A, 129, A, 32),
                                  (A, 128, A, 24)])
def test_bad_read_rows(lib, args):
    assert lib.kda_latent_read(ref(cache()), ref(batch()), *args, None) == BAD


def test_bad_attend_arguments(lib):
    c, b = cache(), batch()
    for kw in (dict(q_c=None), dict(q_r=None), dict(out=A), dict(out=2 * A), dict(out=3 * A + 2), dict(q_c_stride=120),
               dict(q_c_head_stride=132), dict(q_r_stride=0), dict(out_head_stride=64), dict(out_stride=1 << 37),
               dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan"))):
        assert lib.kda_latent_attend(ref(c), ref(attn_io(**kw)), ref(b), A, 1 << 40, None) == BAD, kw
    need = lib.kda_latent_attend_workspace_bytes(ref(c), ref(b))
    assert need > 0
    for ws, n in ((None, need), (A, need - 1), (A + 64, need)):
        assert lib.kda_latent_attend(ref(c), ref(attn_io()), ref(b), ws, n, None) == kda.KDA_ERR_WORKSPACE
    assert lib.kda_latent_poll_device_error(None, None, None) == BAD
    for nothing in (batch(n_seqs=0), batch(max_rows=0)):
        assert lib.kda_latent_attend(ref(c), ref(attn_io()), ref(nothing), None, 0, None) == kda.KDA_OK
        assert lib.kda_latent_read(ref(c), ref(nothing), None, 0, None, 0, None) == kda.KDA_OK
        assert lib.kda_latent_append(ref(c), None, ref(io()), ref(nothing), None) == kda.KDA_OK


def test_bad_prefill_arguments(lib):
    c, b = cache(c=None, kr=None, num_pages=0), rows_batch()  # the pages are not this form's
    need = lib.kda_latent_prefill_workspace_bytes(ref(c), ref(rows_io()), ref(b))
    assert need > 0
    for kw, status in ((dict(q_n=None), BAD), (dict(q_r=None), BAD), (dict(k=None), BAD), (dict(kr=A + 8), BAD), (dict(v=None), BAD),
                       (dict(out=3 * A), BAD), (dict(out=5 * A), BAD), (dict(k_stride=56), BAD), (dict(k_head_stride=68), BAD),
                       (dict(v_head_stride=64), BAD), (dict(kr_stride=16), BAD), (dict(out_stride=0), BAD),
                       (dict(scale=float("nan")), BAD), (dict(scale=0.0), BAD), (dict(nope_dim=0), BAD), (dict(nope_dim=96), UNSUP),
                       (dict(value_dim=256), UNSUP)):
        assert lib.kda_latent_prefill(ref(c), ref(rows_io(**kw)), ref(b), A, 1 << 40, None) == status, kw
    for kw in (dict(n_seqs=-1), dict(max_rows=-1), dict(max_kv_rows=-1), dict(max_kv_rows=0), dict(max_new=0), dict(cu_seqlens=None),
               dict(cu_kv=None), dict(cu_kv=A + 2)):
        assert lib.kda_latent_prefill(ref(c), ref(rows_io()), ref(rows_batch(**kw)), A, 1 << 40, None) == BAD, kw
        assert lib.kda_latent_prefill_workspace_bytes(ref(c), ref(rows_io()), ref(rows_batch(**kw))) == 0
    for kw, status in ((dict(err=None), BAD), (dict(num_heads=0), BAD), (dict(rope_dim=48), UNSUP), (dict(act=7), BAD)):
        assert lib.kda_latent_prefill(ref(cache(**kw)), ref(rows_io()), ref(b), A, 1 << 40, None) == status
    assert lib.kda_latent_prefill(ref(c), None, ref(b), A, 1 << 40, None) == BAD
    for ws, n in ((None, need), (A, need - 1), (A + 64, need)):
        assert lib.kda_latent_prefill(ref(c), ref(rows_io()), ref(b), ws, n, None) == kda.KDA_ERR_WORKSPACE
    for nothing in (rows_batch(n_seqs=0), rows_batch(max_rows=0)):
        assert lib.kda_latent_prefill(ref(c), ref(rows_io()), ref(nothing), None, 0, None) == kda.KDA_OK


def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        kda.PagedLatent(2, 16, 2, 128, 32, kv_format="int4", device="cpu")
    with pytest.raises(ValueError):
        kda.PagedLatent(2, 16, 2, 128, 32, c=torch.zeros(2, 16, 64, dtype=bf))
    with pytest.raises(ValueError):
        kda.PagedLatent(2, 16, 2, 128, 32, c_scale=torch.zeros(2, 16, dtype=torch.uint8), device="cpu")
    kv = kda.PagedLatent(2, 16, 2, 128, 32, device="cpu")
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # tables on the CPU
        kda.make_latent_prefill_batch(i32, i32, 1, 1, 1)
    with pytest.raises(ValueError):  # channels not back to back
        kda.make_latent_attn_io(torch.zeros(4, 2, 256)[..., ::2], torch.zeros(4, 2, 32), torch.zeros(4, 2, 128), 0.1)
    b = batch()
    qr, out = torch.zeros(2, 2, 32, dtype=bf), torch.zeros(2, 2, 128, dtype=bf)
    for wrong in (torch.zeros(1, 2, 128, dtype=bf), torch.zeros(2, 2, 128), torch.zeros(2, 3, 128, dtype=bf)):
        with pytest.raises(ValueError):
            kda.kda_latent_attend(kv, kda.make_latent_attn_io(wrong, qr, out, 0.1), b, None)
    with pytest.raises(ValueError):  # q_r of another size than the cache's key part
        kda.kda_latent_append(kv, None, kda.make_latent_io(out[:, 0], qr[:, 0], qr[..., :16], qr[..., :16]), b)
    with pytest.raises(ValueError):
        kda.kda_latent_append(kv, kda.make_latent_params(torch.ones(64, dtype=bf)), kda.make_latent_io(out[:, 0], qr[:, 0], None, None), b)
    with pytest.raises(ValueError):
        kda.kda_latent_read(kv, b, out[:, 0], qr[:1, 0])


def test_reference_attention():
    """Hand-worked: two equal scores weigh alike, a later key is hidden, a row without keys gives zeros."""
    s = torch.zeros(2, 1, 3, dtype=torch.float64)
    v = torch.tensor([[[1.0]], [[3.0]], [[float("nan")]]], dtype=torch.float64)
    out, mag = R.attend(s, v, 0)
    assert out.flatten().tolist() == [1.0, 2.0] and mag.flatten().tolist() == [1.0, 2.0]
    out, _ = R.attend(s, v, 0, gone=(0,))
    assert out.flatten().tolist() == [0.0, 3.0]

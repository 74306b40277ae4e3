"""Host-side refusals of the paged-cache entry points and binding (no GPU), and the reference quantiser's pins."""

import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import kv_ref as R


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.lib()


A = 0x10000  # an aligned address that no host check dereferences


def cache(**kw):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, err=A, num_pages=4, page_size=16, num_heads=8, num_kv_heads=2,
             head_dim=64, act=kda.KDA_BF16, format=kda.KDA_KV_ACT)
    f.update(kw)
    return kda.kda_kv_cache(**f)


def batch(**kw):
    f = dict(cu_seqlens=A, kv_lens=A, page_table=A, n_seqs=2, table_stride=4, max_rows=2, max_new=1)
    f.update(kw)
    return kda.kda_kv_batch(**f)


def kv_io(**kw):
    f = dict(q=A, k=A, v=A, q_out=2 * A, q_stride=512, k_stride=128, v_stride=128, q_out_stride=512)
    f.update(kw)
    return kda.kda_kv_io(**f)


def attn_io(**kw):
    f = dict(q=A, out=2 * A, q_stride=512, out_stride=512, scale=0.1)
    f.update(kw)
    return kda.kda_attn_io(**f)


ref = ctypes.byref
BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
CACHES = [(dict(k=None), BAD), (dict(v=A + 8), BAD), (dict(err=None), BAD), (dict(num_pages=0), BAD),
          (dict(num_heads=7), BAD), (dict(num_kv_heads=0), BAD), (dict(act=2), BAD), (dict(format=2), BAD),
          (dict(format=kda.KDA_KV_E4M3), BAD), (dict(format=kda.KDA_KV_E4M3, k_scale=A, v_scale=A + 8), BAD), (dict(page_size=48), UNSUP), (dict(page_size=256), UNSUP),
          (dict(head_dim=96), UNSUP), (dict(num_heads=130, num_kv_heads=1), UNSUP),
          (dict(num_pages=1 << 30, num_kv_heads=8), UNSUP)]
BATCHES = [dict(n_seqs=-1), dict(max_rows=-1), dict(max_new=0), dict(max_new=-1), dict(cu_seqlens=None),
           dict(kv_lens=None), dict(page_table=None), dict(table_stride=0), dict(kv_lens=A + 2)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_bad_caches(lib, kw, status):
    c, b = cache(**kw), batch()
    assert lib.kda_kv_append(ref(c), None, ref(kv_io()), ref(b), None) == status
    assert lib.kda_kv_read(ref(c), ref(b), A, A, None) == status
    assert lib.kda_kv_attend(ref(c), ref(attn_io()), ref(b), A, 1 << 40, None) == status
    assert lib.kda_kv_attend_workspace_bytes(ref(c), ref(b)) == 0


@pytest.mark.parametrize("kw", BATCHES)
def test_bad_batches(lib, kw):
    c, b = cache(), batch(**kw)
    assert lib.kda_kv_append(ref(c), None, ref(kv_io()), ref(b), None) == BAD
    assert lib.kda_kv_read(ref(c), ref(b), A, A, None) == BAD
    assert lib.kda_kv_attend(ref(c), ref(attn_io()), ref(b), A, 1 << 40, None) == BAD
    assert lib.kda_kv_attend_workspace_bytes(ref(c), ref(b)) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(q_out=None), dict(k=None), dict(v=A + 4), dict(k_stride=120),
                                dict(v_stride=130), dict(q_stride=504), dict(q_out_stride=516),
                                dict(q_out=A, q_out_stride=520)])
def test_bad_append_rows(lib, kw):
    assert lib.kda_kv_append(ref(cache()), None, ref(kv_io(**kw)), ref(batch()), None) == BAD


def test_bad_norm_and_rotation(lib):
    freq = (ctypes.c_double * 32)(*[0.5] * 32)
    inf = (ctypes.c_double * 32)(*[float("inf")] * 32)
    for kw, status in ((dict(q_norm_w=A + 2), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
                       (dict(rot_dim=72), BAD), (dict(rot_dim=-8), BAD), (dict(rot_dim=16, inv_freq=None), BAD),
                       (dict(rot_dim=16, inv_freq=inf), BAD), (dict(interleaved=2), BAD),
                       (dict(rot_dim=12), UNSUP)):
        f = dict(q_norm_w=A, k_norm_w=A, eps=1e-5, rot_dim=64, interleaved=0, inv_freq=freq)
        f.update(kw)
        p = kda.kda_qk_params(**f)
        assert lib.kda_kv_append(ref(cache()), ref(p), ref(kv_io()), ref(batch()), None) == status, kw


def test_bad_attend_arguments(lib):
    c, b = cache(), batch()
    for kw in (dict(q=None), dict(out=A), dict(out=2 * A + 2), dict(q_stride=8), dict(out_stride=513),
               dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan"))):
        assert lib.kda_kv_attend(ref(c), ref(attn_io(**kw)), ref(b), A, 1 << 40, None) == BAD, kw
    need = lib.kda_kv_attend_workspace_bytes(ref(c), ref(b))
    assert need > 0
    for ws, n in ((None, need), (A, need - 1), (A + 64, need)):
        assert lib.kda_kv_attend(ref(c), ref(attn_io()), ref(b), ws, n, None) == kda.KDA_ERR_WORKSPACE
    assert lib.kda_kv_poll_device_error(None, None, None) == BAD
    for nothing in (batch(n_seqs=0), batch(max_rows=0)):
        assert lib.kda_kv_attend(ref(c), ref(attn_io()), ref(nothing), None, 0, None) == kda.KDA_OK
        assert lib.kda_kv_read(ref(c), ref(nothing), None, None, None) == kda.KDA_OK


def test_binding_refuses_wrong_tensors():
    with pytest.raises(ValueError):
        kda.PagedKV(2, 16, 2, 1, 16, kv_format="int4", device="cpu")
    with pytest.raises(ValueError):
        kda.PagedKV(2, 16, 2, 1, 16, k=torch.zeros(2, 1, 16, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kda.PagedKV(2, 16, 2, 1, 16, k_scale=torch.zeros(2, 1, 16, dtype=torch.uint8), device="cpu")
    kv = kda.PagedKV(2, 16, 2, 1, 16, device="cpu")
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # tables on the CPU
        kda.make_kv_batch(i32, i32[:1], i32.view(1, 2), 1, 1)
    with pytest.raises(ValueError):  # heads of a row not back to back
        kda.make_attn_io(torch.zeros(4, 2, 32)[:, :, :16], torch.zeros(4, 2, 16))
    b = batch()
    b._tensors = (i32,)
    for wrong in (torch.zeros(1, 2, 16, dtype=torch.bfloat16), torch.zeros(2, 2, 16), torch.zeros(2, 3, 16)):
        io = kda.make_attn_io(wrong, wrong.clone())
        with pytest.raises(ValueError):
            kda.kda_kv_attend(kv, io, b, None)


def test_reference_quantiser():
    """Hand-worked values of the test's own quantiser."""
    v, e = R.quantise([[448.0, 1.0, 17.0, 2.0 ** -10 * 3], [450.0, 0.0, 0.0, 0.0], [0.0] * 4, [float("inf"), 3.0, -1.0, 0.0]])
    assert e.tolist() == [127, 128, 0, 120]
    assert v[0].tolist() == [448.0, 1.0, 16.0, 2.0 ** -8]  # 17 is a tie between 16 and 18 and 3/1024 one of 2/512 and 1/512
    assert v[1].tolist() == [224.0, 0.0, 0.0, 0.0]  # 225 -> 224
    assert np.isnan(v[3][0]) and v[3][1] == 384.0 and v[3][2] == -128.0

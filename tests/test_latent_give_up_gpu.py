"""Bounded waits of the latent-attention kernels that give up, as in test_kv_give_up_gpu.py: libraries in which the two
tensor-core kernels' waits look once (or a few times) and no more.  Such a call comes back, sets KDA_DEVERR_TIMEOUT and
writes nothing behind its rows; the next call is as good as ever."""

from __future__ import annotations

import ctypes
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import latent_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

LOOKS = (1, 30, 300)
SHORT = ("kda_latent_tile", "kda_latent_prefill")  # what waits on mbarriers


@pytest.fixture(scope="module")
def short(tmp_path_factory):
    """{looks: library}"""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kda.lib()
    at = tmp_path_factory.mktemp("waits")

    def compile_one(job):
        looks, stem = job
        obj = at / f"{stem}_{looks}.o"
        subprocess.run([kbuild.nvcc(), *kbuild.ARCH, *kbuild.FLAGS, f"-DKDA_ATTEND_LOOKS={looks}", "-I", str(kbuild.INCLUDE),
                        "-I", str(kbuild.CSRC), "-c", str(kbuild.CSRC / f"{stem}.cu"), "-o", str(obj)], check=True,
                       capture_output=True)
        return job, str(obj)

    with ThreadPoolExecutor(max_workers=6) as ex:
        made = dict(ex.map(compile_one, [(n, stem) for n in LOOKS for stem in SHORT]))
    libs = {}
    for looks in LOOKS:
        so = at / f"libkda_looks_{looks}.so"
        objs = [made.get((looks, s.stem), str(kbuild.BUILD / (s.stem + ".o"))) for s in kbuild.sources()]
        subprocess.run([kbuild.nvcc(), *kbuild.ARCH, "-shared", "-o", str(so), *objs], check=True, capture_output=True)
        libs[looks] = ctypes.CDLL(str(so))
        for name in ("kda_latent_attend", "kda_latent_prefill"):
            getattr(libs[looks], name).argtypes = getattr(kda.lib(), name).argtypes
            getattr(libs[looks], name).restype = ctypes.c_int32
    return libs


def call_with(lib, name, cache, io, batch, ws):
    """One call through `lib`; the error word's flags once the stream has finished."""
    stream = torch.cuda.current_stream()
    assert getattr(lib, name)(cache.ref, ctypes.byref(io), ctypes.byref(batch), ws.data_ptr(), ws.nbytes,
                              stream.cuda_stream) == kda.KDA_OK
    assert kda.kda_stream_wait(stream, 30.0) == kda.KDA_OK
    return kda.kda_latent_poll_device_error(cache)[1]


ATTEND = [
    # new, total, heads, latent, rope, page
    ([1] * 9, [1, 2, 130, 700, 129, 63, 64, 1000, 257], 16, 512, 64, 16),
    ([1], [4000], 64, 512, 64, 64),
    ([8, 8, 0, 8], [300, 8, 5, 900], 16, 256, 32, 32),
    ([40, 1, 65], [196, 50, 65], 8, 128, 64, 128),
]


@pytest.mark.parametrize("looks", LOOKS)
@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_absorbed(short, case, fmt, looks):
    new, total, heads, latent, rope, page = ATTEND[case]
    b = R.Batch(new, total, heads, latent, rope, page, BF, fmt, seed=600 + case, fill=float("nan"), extra_rows=2)
    held = b.fill_cache()
    q = b.queries()
    out = torch.full((b.max_rows, heads, latent), 9.0, dtype=BF, device="cuda")
    scale = (128 + rope) ** -0.5
    io, ws = kda.make_latent_attn_io(*q, out, scale), b.workspace()
    for _ in range(3):
        flags = call_with(short[looks], "kda_latent_attend", b.kv, io, b.batch, ws)
        assert flags == kda.KDA_DEVERR_TIMEOUT or (flags == 0 and looks > 1)
        assert (out[b.rows:] == 9.0).all()
        if flags == 0:
            b.check_attend(q, out, held, scale)
    out.fill_(9.0)
    kda.kda_latent_attend(b.kv, io, b.batch, ws)
    b.no_error()
    b.check_attend(q, out, held, scale)
    assert (out[b.rows:] == 9.0).all()


@pytest.mark.parametrize("looks", LOOKS)
@pytest.mark.parametrize("fmt", ["act", "e4m3"])
def test_absorbed_among_absent_pages_and_odd_latents(short, fmt, looks):
    new, total = 7, 300
    b = R.Batch([new], [total], 16, 512, 64, 32, BF, fmt, seed=61)
    b.fill_cache()
    at = total - new // 2
    page, line = int(b.table[0, at // 32]), at % 32
    if fmt == "e4m3":
        b.kv.c.view(torch.uint8)[page, line, 1] = 0xFF
    else:
        b.kv.c[page, line, 1] = float("inf")
    b.dev[2][0, 2] = -1
    q = b.queries()
    outs = [torch.empty_like(q[0]) for _ in range(2)]
    ws = b.workspace()
    kda.kda_latent_attend(b.kv, kda.make_latent_attn_io(*q, outs[0], 0.07), b.batch, ws)
    assert kda.kda_latent_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_PAGE_RANGE
    io = kda.make_latent_attn_io(*q, outs[1], 0.07)
    for _ in range(3):
        flags = call_with(short[looks], "kda_latent_attend", b.kv, io, b.batch, ws)
        assert flags & kda.KDA_DEVERR_TIMEOUT or (flags == kda.KDA_DEVERR_PAGE_RANGE and looks > 1)
    kda.kda_latent_attend(b.kv, io, b.batch, ws)
    assert kda.kda_latent_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_PAGE_RANGE
    assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8))


EXPANDED = [
    # new, total, heads, nope, rope, value: sides by rows and by keys, chunks, an item without a second side
    ([300, 1, 140], [700, 50, 140], 4, 128, 64, 128),
    ([100, 7], [1200, 129], 3, 128, 64, 128),
    ([200, 77], [600, 500], 2, 64, 32, 64),
]


@pytest.mark.parametrize("looks", LOOKS)
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("case", range(len(EXPANDED)))
def test_expanded(short, case, odd, looks):
    """Odd: a value that only the last rows see is infinite, so a path that follows a list of keys is taken."""
    new, total, heads, nope, rope, value = EXPANDED[case]
    r = R.Rows(new, total, heads, nope, rope, value, BF, seed=700 + case, extra_rows=2, extra_keys=3)
    if odd:
        r.v[total[0] - 1, 0, 3] = float("inf")
    ws = r.workspace()
    r.call(ws)
    r.no_error()
    good = r.out.clone()
    for _ in range(3):
        r.wide.fill_(9.0)
        flags = call_with(short[looks], "kda_latent_prefill", r.cache, r.io, r.batch, ws)
        assert flags == kda.KDA_DEVERR_TIMEOUT or (flags == 0 and looks > 1)
        assert (r.out[r.rows:] == 9.0).all() and (r.wide[:, heads * value:] == 9.0).all()
    r.call(ws)
    r.no_error()
    assert torch.equal(r.out.view(torch.int16), good.view(torch.int16))
    if not odd:
        r.check()

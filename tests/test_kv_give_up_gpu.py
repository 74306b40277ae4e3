"""The attention kernels' bounded waits that give up.  Libraries of their own, in which the two tensor-core kernels are built
so that a wait looks once (or a few times) and no more, run calls that give up at the start or on the way.  Such a call
comes back, sets KDA_DEVERR_TIMEOUT and writes nothing behind its rows; the next call is as good as ever."""

from __future__ import annotations

import ctypes
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from hybrid_linear_attention_03_gb300 import build as kbuild
from hybrid_linear_attention_03_gb300 import kda

import kv_ref as R
from test_kv_gpu import check_attend, fill_cache

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

LOOKS = (1, 30, 300)
SHORT = ("kda_attend_few", "kda_attend_tile")  # what waits on mbarriers


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
        libs[looks].kda_kv_attend.argtypes = kda.lib().kda_kv_attend.argtypes
        libs[looks].kda_kv_attend.restype = ctypes.c_int32
    return libs


def attend_with(lib, b, io, ws):
    """One call through `lib`; the error word's flags once the stream has finished."""
    stream = torch.cuda.current_stream()
    assert lib.kda_kv_attend(b.kv.ref, ctypes.byref(io), ctypes.byref(b.batch), ws.data_ptr(), ws.nbytes,
                             stream.cuda_stream) == kda.KDA_OK
    assert kda.kda_stream_wait(stream, 30.0) == kda.KDA_OK
    return kda.kda_kv_poll_device_error(b.kv)[1]


CALLS = [
    # new, total, hq, hkv, d: one token, a verify, chunks on sides by keys and by rows, heads of 64 and 32
    ([1] * 9, [1, 2, 130, 700, 129, 63, 64, 1000, 257], 16, 2, 128),
    ([1], [4000], 8, 1, 128),
    ([8, 8, 0, 8], [300, 8, 5, 900], 16, 2, 128),
    ([300, 1, 140], [700, 50, 140], 4, 2, 128),
    ([200, 77], [600, 500], 4, 2, 64),
    ([8, 1], [600, 1], 8, 2, 32),
]


@pytest.mark.parametrize("looks", LOOKS)
@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("case", range(len(CALLS)))
def test_waits_that_give_up(short, case, fmt, looks):
    new, total, hq, hkv, d = CALLS[case]
    b = R.Batch(new, total, hq, hkv, d, 16, BF, fmt, seed=500 + case, fill=float("nan"), extra_rows=2)
    cache = fill_cache(b)
    q = b.randn(b.max_rows, hq).cuda()
    out = torch.full_like(q, 9.0)
    io, ws = kda.make_attn_io(q, out), b.workspace()
    for _ in range(3):
        flags = attend_with(short[looks], b, io, ws)
        assert flags == kda.KDA_DEVERR_TIMEOUT or (flags == 0 and looks > 1)
        assert (out[b.rows:] == 9.0).all()
        if flags == 0:
            check_attend(b, q, out, cache, d ** -0.5)
    out.fill_(9.0)
    kda.kda_kv_attend(b.kv, io, b.batch, ws)
    assert kda.kda_kv_poll_device_error(b.kv)[0] == kda.KDA_OK
    check_attend(b, q, out, cache, d ** -0.5)
    assert (out[b.rows:] == 9.0).all()


@pytest.mark.parametrize("looks", LOOKS)
@pytest.mark.parametrize("fmt", ["act", "e4m3"])
@pytest.mark.parametrize("new,hq,hkv,d", [(4, 4, 2, 128), (100, 4, 2, 128), (300, 2, 1, 64)])
def test_waits_that_give_up_among_absent_pages_and_odd_values(short, new, hq, hkv, d, fmt, looks):
    """The paths that follow a list of keys from shared memory are the ones a warp that gave up must not take."""
    total = new + 270
    b = R.Batch([new], [total], hq, hkv, d, 16, BF, fmt, seed=43)
    fill_cache(b)
    at = total - new // 2
    page, line = int(b.table[0, at // 16]), at % 16
    if fmt == "e4m3":
        b.kv.v.view(torch.uint8)[page, :, line, 1] = 0xFF
    else:
        b.kv.v[page, :, line, 1] = float("inf")
    b.dev[2][0, 2] = -1
    q = b.randn(b.rows, hq).cuda()
    outs = [torch.empty_like(q) for _ in range(2)]
    ws = b.workspace()
    kda.kda_kv_attend(b.kv, kda.make_attn_io(q, outs[0]), b.batch, ws)
    assert kda.kda_kv_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_PAGE_RANGE
    io = kda.make_attn_io(q, outs[1])
    for _ in range(3):
        flags = attend_with(short[looks], b, io, ws)
        assert flags & kda.KDA_DEVERR_TIMEOUT or (flags == kda.KDA_DEVERR_PAGE_RANGE and looks > 1)
    kda.kda_kv_attend(b.kv, io, b.batch, ws)
    assert kda.kda_kv_poll_device_error(b.kv)[1] == kda.KDA_DEVERR_PAGE_RANGE
    assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8))

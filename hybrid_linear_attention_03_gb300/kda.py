"""Thin ctypes binding of libkda (include/kda.h): argument marshalling only.

Every entry point of the C ABI has a function of the same name here.  Tensors
are torch tensors (device memory and streams come from PyTorch); each call
passes their data pointers and the current CUDA stream to the library, where
all of the work runs in the hand-written sm_103a kernels.  There is no
fallback: if ``libkda.so`` is missing the first call raises.
"""

from __future__ import annotations

import ctypes
from pathlib import Path

import torch

_LIB_PATH = Path(__file__).resolve().parent / "_build" / "libkda.so"
_LIB = None

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_SLOT_RANGE = 2
KDA_ERR_ALIAS = 3
KDA_ERR_UNSUPPORTED = 4
KDA_ERR_CUDA = 5
KDA_ERR_DEVICE = 6
KDA_ERR_WORKSPACE = 7
KDA_ERR_HOST_MEMORY = 8
KDA_ERR_TIMEOUT = 9
KDA_F32 = 0
KDA_BF16 = 1
KDA_DEVERR_SLOT_RANGE = 0x1
KDA_DEVERR_META = 0x2
KDA_DEVERR_TIMEOUT = 0x4
KDA_DEVERR_PAGE_RANGE = 0x8
KDA_KV_ACT = 0
KDA_KV_E4M3 = 1
KDA_POOL_OVERLAP_INPUTS = 0x1

# Every symbol include/kda.h declares.
EXPORTS = ("kda_state_pool_bytes", "kda_state_pool_create", "kda_state_pool_destroy", "kda_state_pool_layout",
           "kda_check_slots", "kda_decode", "kda_verify", "kda_prefill_workspace_bytes", "kda_prefill_chunked",
           "kda_state_checkpoint", "kda_poll_device_error", "kda_status_string", "kda_prefill_chunked_noalloc",
           "kda_state_slot_bytes", "kda_state_export", "kda_state_import", "kda_prefill_workspace_bytes_bound",
           "kda_prefill_chunked_dev", "kda_prefix_cache_create", "kda_prefix_cache_destroy", "kda_prefix_cache_plan",
           "kda_prefix_cache_forget", "kda_prefix_cache_get_stats", "kda_prefix_cache_saved", "kda_stream_wait",
           "kda_state_pool_set_flags", "kda_profile_start", "kda_profile_stop", "kda_state_prefetch",
           "kda_kv_append", "kda_kv_read", "kda_kv_attend_workspace_bytes", "kda_kv_attend",
           "kda_kv_poll_device_error", "kda_latent_append", "kda_latent_read", "kda_latent_attend_workspace_bytes",
           "kda_latent_attend", "kda_latent_prefill_workspace_bytes", "kda_latent_prefill", "kda_latent_poll_device_error")

# kda_kernel_kind
KERNEL_KINDS = ("step", "slot_copy", "prefill_meta", "prefill_intra", "prefill_chain", "prefill_out", "prefill_tails",
                "state_prefetch", "prefill_intra_exact", "kv_append", "kv_read", "kv_attend", "kv_combine",
                "latent_append", "latent_read", "latent_attend", "latent_prefill", "latent_combine")

KDA_NOALLOC_SCRATCH_BYTES = 64 << 20


class kda_pool_desc(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("conv_width", ctypes.c_int32), ("act", ctypes.c_int32)]


class kda_pool_layout(ctypes.Structure):
    _fields_ = [("header_offset", ctypes.c_size_t), ("state_offset", ctypes.c_size_t),
                ("state_slot_bytes", ctypes.c_size_t), ("tail_offset", ctypes.c_size_t),
                ("tail_slot_bytes", ctypes.c_size_t), ("total_bytes", ctypes.c_size_t)]


class kda_weights(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("norm_w", ctypes.c_void_p), ("eps_l2", ctypes.c_float),
                ("eps_rms", ctypes.c_float)]


class kda_io(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("beta", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class kda_ckpt_req(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_int32), ("token_pos", ctypes.c_int32), ("dst_slot", ctypes.c_int32)]


class kda_prefix_plan(ctypes.Structure):
    _fields_ = [("hit_len", ctypes.c_int32), ("hit_slot", ctypes.c_int32), ("admit_pos", ctypes.c_int32),
                ("admit_slot", ctypes.c_int32)]


class kda_prefix_cache_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("plans", "hits", "admissions", "evictions", "n_saved", "n_unsaved",
                                               "n_free")]


class kda_profile(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int64 * len(KERNEL_KINDS)), ("ms", ctypes.c_double * len(KERNEL_KINDS)),
                ("dropped", ctypes.c_int64)]


class kda_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("err", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("act", ctypes.c_int32), ("format", ctypes.c_int32)]


class kda_kv_batch(ctypes.Structure):
    _fields_ = [("cu_seqlens", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("table_stride", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


class kda_qk_params(ctypes.Structure):
    _fields_ = [("q_norm_w", ctypes.c_void_p), ("k_norm_w", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class kda_kv_io(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64)]


class kda_attn_io(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("scale", ctypes.c_float)]


class kda_latent_cache(ctypes.Structure):
    _fields_ = [("c", ctypes.c_void_p), ("c_scale", ctypes.c_void_p), ("kr", ctypes.c_void_p), ("err", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("act", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class kda_latent_params(ctypes.Structure):
    _fields_ = [("c_norm_w", ctypes.c_void_p), ("eps", ctypes.c_float), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class kda_latent_io(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("c", "kr", "q", "q_out")] + \
               [(n, ctypes.c_int64) for n in ("c_stride", "kr_stride", "q_stride", "q_head_stride", "q_out_stride",
                                              "q_out_head_stride")]


class kda_latent_attn_io(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_c", "q_r", "out")] + \
               [(n, ctypes.c_int64) for n in ("q_c_stride", "q_c_head_stride", "q_r_stride", "q_r_head_stride",
                                              "out_stride", "out_head_stride")] + [("scale", ctypes.c_float)]


class kda_latent_prefill_io(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_n", "q_r", "k", "kr", "v", "out")] + \
               [(n, ctypes.c_int64) for n in ("q_n_stride", "q_n_head_stride", "q_r_stride", "q_r_head_stride", "k_stride",
                                              "k_head_stride", "kr_stride", "v_stride", "v_head_stride", "out_stride",
                                              "out_head_stride")] + \
               [("nope_dim", ctypes.c_int32), ("value_dim", ctypes.c_int32), ("scale", ctypes.c_float)]


class kda_latent_prefill_batch(ctypes.Structure):
    _fields_ = [("cu_seqlens", ctypes.c_void_p), ("cu_kv", ctypes.c_void_p), ("n_seqs", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("max_kv_rows", ctypes.c_int32), ("max_new", ctypes.c_int32)]


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kda_status_string(status)} ({status})")


def lib_path() -> Path:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libkda.so (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not _LIB_PATH.exists():
            raise RuntimeError(f"{_LIB_PATH} is missing: build it first (python -m hybrid_linear_attention_03_gb300.build)")
        L = ctypes.CDLL(str(_LIB_PATH))
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        P = ctypes.POINTER
        L.kda_state_pool_bytes.argtypes = [P(kda_pool_desc)]
        L.kda_state_pool_bytes.restype = sz
        L.kda_state_pool_create.argtypes = [P(kda_pool_desc), vp, sz, P(vp)]
        L.kda_state_pool_create.restype = i32
        L.kda_state_pool_destroy.argtypes = [vp]
        L.kda_state_pool_destroy.restype = None
        L.kda_state_pool_set_flags.argtypes = [vp, ctypes.c_uint32]
        L.kda_state_pool_set_flags.restype = i32
        L.kda_state_pool_layout.argtypes = [vp, P(kda_pool_layout)]
        L.kda_state_pool_layout.restype = i32
        L.kda_check_slots.argtypes = [vp, vp, i32, vp, i32]
        L.kda_check_slots.restype = i32
        L.kda_decode.argtypes = [vp, P(kda_weights), P(kda_io), vp, i32, vp]
        L.kda_decode.restype = i32
        L.kda_state_prefetch.argtypes = [vp, vp, vp, i32, vp]
        L.kda_state_prefetch.restype = i32
        L.kda_verify.argtypes = [vp, P(kda_weights), P(kda_io), vp, vp, i32, i32, vp]
        L.kda_verify.restype = i32
        L.kda_prefill_workspace_bytes.argtypes = [vp, vp, i32, i32]
        L.kda_prefill_workspace_bytes.restype = sz
        L.kda_prefill_chunked.argtypes = [vp, P(kda_weights), P(kda_io), vp, vp, vp, i32, i32,
                                          P(kda_ckpt_req), i32, vp, sz, vp]
        L.kda_prefill_chunked.restype = i32
        L.kda_prefill_chunked_noalloc.argtypes = [vp, P(kda_weights), P(kda_io), vp, vp, vp, i32, i32,
                                                  P(kda_ckpt_req), i32, vp]
        L.kda_prefill_chunked_noalloc.restype = i32
        L.kda_state_checkpoint.argtypes = [vp, vp, vp, i32, vp]
        L.kda_state_checkpoint.restype = i32
        L.kda_prefill_workspace_bytes_bound.argtypes = [vp, i32, i32, i32, i32]
        L.kda_prefill_workspace_bytes_bound.restype = sz
        L.kda_prefill_chunked_dev.argtypes = [vp, P(kda_weights), P(kda_io), vp, vp, vp, i32, i32, i32, vp, i32,
                                              vp, sz, vp]
        L.kda_prefill_chunked_dev.restype = i32
        L.kda_state_slot_bytes.argtypes = [vp]
        L.kda_state_slot_bytes.restype = sz
        L.kda_state_export.argtypes = [vp, i32, vp, sz, vp]
        L.kda_state_export.restype = i32
        L.kda_state_import.argtypes = [vp, i32, vp, sz, vp]
        L.kda_state_import.restype = i32
        L.kda_poll_device_error.argtypes = [vp, vp, P(ctypes.c_uint32)]
        L.kda_poll_device_error.restype = i32
        L.kda_prefix_cache_create.argtypes = [i32, vp, i32, i32, P(vp)]
        L.kda_prefix_cache_create.restype = i32
        L.kda_prefix_cache_destroy.argtypes = [vp]
        L.kda_prefix_cache_destroy.restype = None
        L.kda_prefix_cache_plan.argtypes = [vp, vp, i32, P(kda_prefix_plan)]
        L.kda_prefix_cache_plan.restype = i32
        L.kda_prefix_cache_forget.argtypes = [vp, i32]
        L.kda_prefix_cache_forget.restype = i32
        L.kda_prefix_cache_get_stats.argtypes = [vp, P(kda_prefix_cache_stats)]
        L.kda_prefix_cache_get_stats.restype = i32
        L.kda_prefix_cache_saved.argtypes = [vp, vp, vp, i32]
        L.kda_prefix_cache_saved.restype = i32
        L.kda_stream_wait.argtypes = [vp, ctypes.c_double]
        L.kda_stream_wait.restype = i32
        L.kda_profile_start.argtypes = [i32]
        L.kda_profile_start.restype = i32
        L.kda_profile_stop.argtypes = [P(kda_profile)]
        L.kda_profile_stop.restype = i32
        L.kda_kv_append.argtypes = [P(kda_kv_cache), P(kda_qk_params), P(kda_kv_io), P(kda_kv_batch), vp]
        L.kda_kv_append.restype = i32
        L.kda_kv_read.argtypes = [P(kda_kv_cache), P(kda_kv_batch), vp, vp, vp]
        L.kda_kv_read.restype = i32
        L.kda_kv_attend_workspace_bytes.argtypes = [P(kda_kv_cache), P(kda_kv_batch)]
        L.kda_kv_attend_workspace_bytes.restype = sz
        L.kda_kv_attend.argtypes = [P(kda_kv_cache), P(kda_attn_io), P(kda_kv_batch), vp, sz, vp]
        L.kda_kv_attend.restype = i32
        L.kda_kv_poll_device_error.argtypes = [P(kda_kv_cache), vp, P(ctypes.c_uint32)]
        L.kda_kv_poll_device_error.restype = i32
        lc, lb = P(kda_latent_cache), P(kda_kv_batch)
        L.kda_latent_append.argtypes = [lc, P(kda_latent_params), P(kda_latent_io), lb, vp]
        L.kda_latent_append.restype = i32
        L.kda_latent_read.argtypes = [lc, lb, vp, ctypes.c_int64, vp, ctypes.c_int64, vp]
        L.kda_latent_read.restype = i32
        L.kda_latent_attend_workspace_bytes.argtypes = [lc, lb]
        L.kda_latent_attend_workspace_bytes.restype = sz
        L.kda_latent_attend.argtypes = [lc, P(kda_latent_attn_io), lb, vp, sz, vp]
        L.kda_latent_attend.restype = i32
        L.kda_latent_prefill_workspace_bytes.argtypes = [lc, P(kda_latent_prefill_io), P(kda_latent_prefill_batch)]
        L.kda_latent_prefill_workspace_bytes.restype = sz
        L.kda_latent_prefill.argtypes = [lc, P(kda_latent_prefill_io), P(kda_latent_prefill_batch), vp, sz, vp]
        L.kda_latent_prefill.restype = i32
        L.kda_latent_poll_device_error.argtypes = [lc, vp, P(ctypes.c_uint32)]
        L.kda_latent_poll_device_error.restype = i32
        L.kda_status_string.argtypes = [i32]
        L.kda_status_string.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


def kda_stream_wait(stream=None, timeout_s: float = 60.0) -> int:
    """Waits at most timeout_s for the stream's work; KDA_OK or KDA_ERR_TIMEOUT
    (raises on any other status)."""
    st = lib().kda_stream_wait(_stream(stream), float(timeout_s))
    if st not in (KDA_OK, KDA_ERR_TIMEOUT):
        raise KdaError(st, "kda_stream_wait")
    return st


def kda_profile_start(max_launches: int = 4096) -> None:
    """Starts timing every kernel the library launches (CUDA events on the
    launching stream) on the current device."""
    _check(lib().kda_profile_start(int(max_launches)), "kda_profile_start")


def kda_profile_stop() -> dict:
    """Stops the profile: {kind: (launches, total ms)} plus "dropped"."""
    out = kda_profile()
    _check(lib().kda_profile_stop(ctypes.byref(out)), "kda_profile_stop")
    res = {k: (int(out.launches[i]), float(out.ms[i])) for i, k in enumerate(KERNEL_KINDS)}
    res["dropped"] = int(out.dropped)
    return res


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != KDA_OK:
        raise KdaError(status, where)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dptr(t: torch.Tensor | None):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _host_i32(x):
    """A host int32 array for the C side (keeps the buffer alive in the tuple)."""
    t = torch.as_tensor(x, dtype=torch.int32).contiguous().cpu()
    return t, ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def act_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return KDA_BF16
    if dtype == torch.float32:
        return KDA_F32
    raise ValueError(f"unsupported activation dtype {dtype}")


def make_desc(num_slots, H, dk, dv, act: torch.dtype, conv_width=4) -> kda_pool_desc:
    return kda_pool_desc(num_slots, H, dk, dv, conv_width, act_code(act))


def kda_state_pool_bytes(desc: kda_pool_desc) -> int:
    return int(lib().kda_state_pool_bytes(ctypes.byref(desc)))


def kda_state_pool_create(desc: kda_pool_desc, buf: torch.Tensor) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(lib().kda_state_pool_create(ctypes.byref(desc), _dptr(buf), buf.numel() * buf.element_size(),
                                       ctypes.byref(h)), "kda_state_pool_create")
    return h


def kda_state_pool_destroy(handle) -> None:
    if handle:
        lib().kda_state_pool_destroy(handle)


def kda_state_pool_set_flags(pool: "StatePool", flags: int) -> None:
    """Launch options of the pool's decode / verify calls (KDA_POOL_* flags)."""
    _check(lib().kda_state_pool_set_flags(pool.handle, int(flags)), "kda_state_pool_set_flags")


def kda_state_pool_layout(handle) -> kda_pool_layout:
    out = kda_pool_layout()
    _check(lib().kda_state_pool_layout(handle, ctypes.byref(out)), "kda_state_pool_layout")
    return out


def make_weights(conv_w: torch.Tensor, norm_w: torch.Tensor, eps_l2=1e-6, eps_rms=1e-5) -> kda_weights:
    """The struct holds raw device pointers; it also keeps the two tensors
    alive, so their memory cannot be handed to another tensor while the
    struct is in use."""
    w = kda_weights(conv_w.data_ptr(), norm_w.data_ptr(), float(eps_l2), float(eps_rms))
    w._tensors = (conv_w, norm_w)
    return w


def make_io(inp: dict, out: torch.Tensor) -> kda_io:
    """Raw pointers to the step's arrays; the struct keeps the tensors alive."""
    io = kda_io(inp["q"].data_ptr(), inp["k"].data_ptr(), inp["v"].data_ptr(), inp["alpha"].data_ptr(),
                inp["beta"].data_ptr(), inp["gate"].data_ptr(), out.data_ptr())
    io._tensors = (inp["q"], inp["k"], inp["v"], inp["alpha"], inp["beta"], inp["gate"], out)
    return io


class StatePool:
    """A slot pool over a torch-allocated device buffer (zero-filled)."""

    def __init__(self, num_slots, H, dk, dv, act: torch.dtype = torch.bfloat16, device="cuda"):
        self.desc = make_desc(num_slots, H, dk, dv, act)
        self.act = act
        self.H, self.dk, self.dv, self.num_slots = H, dk, dv, num_slots
        self.n_ch = H * (2 * dk + dv)
        nbytes = kda_state_pool_bytes(self.desc)
        if nbytes == 0:
            raise KdaError(KDA_ERR_INVALID_ARG, "kda_state_pool_bytes")
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.handle = kda_state_pool_create(self.desc, self.buf)
        self.layout = kda_state_pool_layout(self.handle)

    def states(self) -> torch.Tensor:
        """View [num_slots][H][d_v][d_k] fp32 (S^T per head)."""
        L = self.layout
        n = self.num_slots * L.state_slot_bytes
        return self.buf[L.state_offset:L.state_offset + n].view(torch.float32).view(
            self.num_slots, self.H, self.dv, self.dk)

    def tails(self) -> torch.Tensor:
        """View [num_slots][3][n_ch] act."""
        L = self.layout
        n = self.num_slots * L.tail_slot_bytes
        return self.buf[L.tail_offset:L.tail_offset + n].view(self.act).view(self.num_slots, 3, self.n_ch)

    def error_word(self) -> torch.Tensor:
        return self.buf[0:4].view(torch.int32)

    def close(self):
        kda_state_pool_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                kda_state_pool_destroy(self.handle)
        except Exception:
            pass


def kda_check_slots(pool: StatePool, in_slots=None, out_slots=None) -> int:
    """Host-side check of slot tables; returns the kda_status (0 = ok)."""
    ti, pi = _host_i32(in_slots if in_slots is not None else [])
    to, po = _host_i32(out_slots if out_slots is not None else [])
    return int(lib().kda_check_slots(pool.handle, pi, ti.numel(), po, to.numel()))


def kda_decode(pool: StatePool, weights: kda_weights, io: kda_io, slots: torch.Tensor, B: int | None = None,
               stream=None) -> None:
    B = slots.numel() if B is None else B
    _check(lib().kda_decode(pool.handle, ctypes.byref(weights), ctypes.byref(io), _dptr(slots), int(B),
                            _stream(stream)), "kda_decode")


def kda_state_prefetch(pool: StatePool, slots: torch.Tensor, B: int | None = None, stream=None,
                       weights: kda_weights | None = None) -> None:
    """Hint: bring the slots' state and conv tail (and the weights, if given)
    into L2 ahead of a decode."""
    B = slots.numel() if B is None else B
    wp = ctypes.byref(weights) if weights is not None else None
    _check(lib().kda_state_prefetch(pool.handle, wp, _dptr(slots), int(B), _stream(stream)), "kda_state_prefetch")


def kda_verify(pool: StatePool, weights: kda_weights, io: kda_io, in_slots: torch.Tensor, snap_slots: torch.Tensor,
               B: int, T: int, stream=None) -> None:
    _check(lib().kda_verify(pool.handle, ctypes.byref(weights), ctypes.byref(io), _dptr(in_slots),
                            _dptr(snap_slots), int(B), int(T), _stream(stream)), "kda_verify")


def kda_prefill_workspace_bytes(pool: StatePool, cu_seqlens, chunk: int = 64) -> int:
    t, p = _host_i32(cu_seqlens)
    return int(lib().kda_prefill_workspace_bytes(pool.handle, p, t.numel() - 1, int(chunk)))


def kda_prefill_chunked(pool: StatePool, weights: kda_weights, io: kda_io, cu_seqlens, slots, has_initial_state,
                        chunk: int = 64, reqs=(), workspace: torch.Tensor | None = None, stream=None) -> None:
    tc, pc = _host_i32(cu_seqlens)
    ts, ps = _host_i32(slots)
    th = torch.as_tensor(has_initial_state, dtype=torch.uint8).contiguous().cpu()
    n_req = len(reqs)
    req_arr = (kda_ckpt_req * max(1, n_req))(*[kda_ckpt_req(int(a), int(b), int(c)) for a, b, c in reqs])
    ws_ptr = _dptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kda_prefill_chunked(pool.handle, ctypes.byref(weights), ctypes.byref(io), pc, ps,
                                     ctypes.c_void_p(th.data_ptr()), int(tc.numel() - 1), int(chunk),
                                     req_arr, int(n_req), ws_ptr, ws_bytes, _stream(stream)),
           "kda_prefill_chunked")


def kda_prefill_workspace_bytes_bound(pool: StatePool, n_seqs: int, max_tokens: int, n_reqs: int,
                                      chunk: int = 64) -> int:
    return int(lib().kda_prefill_workspace_bytes_bound(pool.handle, int(n_seqs), int(max_tokens), int(n_reqs),
                                                       int(chunk)))


def kda_prefill_chunked_dev(pool: StatePool, weights: kda_weights, io: kda_io, cu_seqlens: torch.Tensor,
                            slots: torch.Tensor, has_initial_state: torch.Tensor, max_tokens: int,
                            reqs: torch.Tensor | None, workspace: torch.Tensor, chunk: int = 64, stream=None) -> None:
    """kda_prefill_chunked with the metadata in device memory: cu_seqlens and
    slots int32, has_initial_state uint8, reqs int32 [n, 3] (seq, token_pos,
    dst_slot) or None, all CUDA tensors; the tables are built on the GPU."""
    for name, t, dt in (("cu_seqlens", cu_seqlens, torch.int32), ("slots", slots, torch.int32),
                        ("has_initial_state", has_initial_state, torch.uint8)):
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    n_req = 0 if reqs is None else int(reqs.shape[0])
    if reqs is not None and (not reqs.is_cuda or reqs.dtype != torch.int32 or tuple(reqs.shape[1:]) != (3,)
                             or not reqs.is_contiguous()):
        raise ValueError("reqs must be a contiguous CUDA int32 tensor of shape [n, 3]")
    _check(lib().kda_prefill_chunked_dev(pool.handle, ctypes.byref(weights), ctypes.byref(io), cu_seqlens.data_ptr(),
                                         slots.data_ptr(), has_initial_state.data_ptr(), int(cu_seqlens.numel() - 1),
                                         int(max_tokens), int(chunk), None if n_req == 0 else reqs.data_ptr(),
                                         n_req, _dptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream)),
           "kda_prefill_chunked_dev")


def kda_prefill_chunked_noalloc(pool: StatePool, weights: kda_weights, io: kda_io, cu_seqlens, slots,
                                has_initial_state, chunk: int = 64, reqs=(), stream=None) -> None:
    """kda_prefill_chunked for callers that cannot allocate device memory: the
    library's fixed 64 MiB scratch array stands in for the workspace."""
    tc, pc = _host_i32(cu_seqlens)
    ts, ps = _host_i32(slots)
    th = torch.as_tensor(has_initial_state, dtype=torch.uint8).contiguous().cpu()
    n_req = len(reqs)
    req_arr = (kda_ckpt_req * max(1, n_req))(*[kda_ckpt_req(int(a), int(b), int(c)) for a, b, c in reqs])
    _check(lib().kda_prefill_chunked_noalloc(pool.handle, ctypes.byref(weights), ctypes.byref(io), pc, ps,
                                             ctypes.c_void_p(th.data_ptr()), int(tc.numel() - 1), int(chunk),
                                             req_arr, int(n_req), _stream(stream)),
           "kda_prefill_chunked_noalloc")


def kda_state_checkpoint(pool: StatePool, src_slots, dst_slots, stream=None) -> None:
    ts, ps = _host_i32(src_slots)
    td, pd = _host_i32(dst_slots)
    if ts.numel() != td.numel():
        raise ValueError("src and dst slot lists differ in length")
    _check(lib().kda_state_checkpoint(pool.handle, ps, pd, int(ts.numel()), _stream(stream)),
           "kda_state_checkpoint")


def kda_state_slot_bytes(pool: StatePool) -> int:
    return int(lib().kda_state_slot_bytes(pool.handle))


def kda_state_export(pool: StatePool, slot: int, host: torch.Tensor, stream=None) -> None:
    """Copies slot `slot` (state, then conv tail) into the CPU uint8 tensor
    `host` (pin it for an asynchronous copy); bit-exact."""
    if host.device.type != "cpu" or not host.is_contiguous():
        raise ValueError("host must be a contiguous CPU tensor")
    _check(lib().kda_state_export(pool.handle, int(slot), host.data_ptr(), host.numel() * host.element_size(),
                                  _stream(stream)), "kda_state_export")


def kda_state_import(pool: StatePool, slot: int, host: torch.Tensor, stream=None) -> None:
    """Copies a buffer written by kda_state_export into slot `slot`; bit-exact."""
    if host.device.type != "cpu" or not host.is_contiguous():
        raise ValueError("host must be a contiguous CPU tensor")
    _check(lib().kda_state_import(pool.handle, int(slot), host.data_ptr(), host.numel() * host.element_size(),
                                  _stream(stream)), "kda_state_import")


def kda_poll_device_error(pool: StatePool, stream=None) -> tuple[int, int]:
    """Returns (status, flags); reading clears the device error word."""
    flags = ctypes.c_uint32(0)
    st = int(lib().kda_poll_device_error(pool.handle, _stream(stream), ctypes.byref(flags)))
    return st, int(flags.value)


def kda_prefix_cache_create(block: int, slots, max_tracked: int) -> ctypes.c_void_p:
    ts, ps = _host_i32(slots)
    h = ctypes.c_void_p()
    _check(lib().kda_prefix_cache_create(int(block), ps, int(ts.numel()), int(max_tracked), ctypes.byref(h)),
           "kda_prefix_cache_create")
    return h


def kda_prefix_cache_destroy(handle: ctypes.c_void_p) -> None:
    lib().kda_prefix_cache_destroy(handle)


def kda_prefix_cache_plan(handle: ctypes.c_void_p, tokens) -> tuple[int, int, int, int]:
    """(hit_len, hit_slot, admit_pos, admit_slot) for a prompt of token ids."""
    t, pt = _host_i32(tokens)
    out = kda_prefix_plan()
    _check(lib().kda_prefix_cache_plan(handle, pt, int(t.numel()), ctypes.byref(out)), "kda_prefix_cache_plan")
    return out.hit_len, out.hit_slot, out.admit_pos, out.admit_slot


def kda_prefix_cache_forget(handle: ctypes.c_void_p, slot: int) -> None:
    _check(lib().kda_prefix_cache_forget(handle, int(slot)), "kda_prefix_cache_forget")


def kda_prefix_cache_get_stats(handle: ctypes.c_void_p) -> dict:
    st = kda_prefix_cache_stats()
    _check(lib().kda_prefix_cache_get_stats(handle, ctypes.byref(st)), "kda_prefix_cache_get_stats")
    return {n: getattr(st, n) for n, _ in kda_prefix_cache_stats._fields_}


def kda_prefix_cache_saved(handle: ctypes.c_void_p) -> dict:
    """{slot: prefix length} of the saved prefixes."""
    n = lib().kda_prefix_cache_saved(handle, None, None, 0)
    lens = (ctypes.c_int32 * max(n, 1))()
    slots = (ctypes.c_int32 * max(n, 1))()
    m = lib().kda_prefix_cache_saved(handle, lens, slots, n)
    return {int(slots[i]): int(lens[i]) for i in range(m)}


class PrefixCache:
    """Owner of a kda_prefix_cache handle (destroyed with the object); the
    methods are the kda_prefix_cache_* functions above."""

    def __init__(self, block: int, slots, max_tracked: int):
        self.handle = kda_prefix_cache_create(block, slots, max_tracked)
        self.block = int(block)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _LIB is not None:
            _LIB.kda_prefix_cache_destroy(h)
            self.handle = None

    def plan(self, tokens) -> tuple[int, int, int, int]:
        return kda_prefix_cache_plan(self.handle, tokens)

    def forget(self, slot: int) -> None:
        kda_prefix_cache_forget(self.handle, slot)

    def stats(self) -> dict:
        return kda_prefix_cache_get_stats(self.handle)

    def saved(self) -> dict:
        return kda_prefix_cache_saved(self.handle)


# ---- full attention over a paged cache ------------------------------------------------


class PagedKV:
    """A paged key / value cache of one layer (a kda_kv_cache record and the
    tensors behind it).  k and v are [num_pages, num_kv_heads, page_size,
    head_dim] in ``act`` (kv_format "act") or float8_e4m3fn ("e4m3", with
    k_scale and v_scale uint8 [num_pages, num_kv_heads, page_size]); those not
    given are allocated, zero-filled, on ``device``."""

    def __init__(self, num_pages, page_size, num_heads, num_kv_heads, head_dim, act: torch.dtype = torch.bfloat16,
                 kv_format: str = "act", k=None, v=None, k_scale=None, v_scale=None, device="cuda"):
        if kv_format not in ("act", "e4m3"):
            raise ValueError(f"kv_format must be \"act\" or \"e4m3\", not {kv_format!r}")
        e4m3 = kv_format == "e4m3"
        dtype = torch.float8_e4m3fn if e4m3 else act
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        for t in (k, v, k_scale, v_scale):
            if t is not None:
                device = t.device
                break

        def pages(t, name):
            if t is None:
                return torch.zeros(shape, dtype=torch.uint8 if e4m3 else act, device=device).view(dtype)
            return _kv_tensor(t, name, dtype, shape, device)

        def scales(t, name):
            if not e4m3:
                if t is not None:
                    raise ValueError(f"{name} is for kv_format \"e4m3\"")
                return None
            if t is None:
                return torch.zeros(shape[:3], dtype=torch.uint8, device=device)
            return _kv_tensor(t, name, torch.uint8, shape[:3], device)

        self.k, self.v = pages(k, "k"), pages(v, "v")
        self.k_scale, self.v_scale = scales(k_scale, "k_scale"), scales(v_scale, "v_scale")
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.device, self.act, self.kv_format = self.k.device, act, kv_format
        self.num_pages, self.page_size, self.num_heads = num_pages, page_size, num_heads
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        self.desc = kda_kv_cache(self.k.data_ptr(), self.v.data_ptr(), _addr(self.k_scale), _addr(self.v_scale),
                                 self.err.data_ptr(), num_pages, page_size, num_heads, num_kv_heads, head_dim,
                                 act_code(act), KDA_KV_E4M3 if e4m3 else KDA_KV_ACT)
        self.ref = ctypes.byref(self.desc)
        self.q_kind = (self.device, act, num_heads, head_dim)  # of row tensors, see _kind
        self.kv_kind = (self.device, act, num_kv_heads, head_dim)
        self.norm_kind = (self.device, act, head_dim)

    def error_word(self) -> torch.Tensor:
        return self.err


def _addr(t):
    return None if t is None else t.data_ptr()


def _kv_tensor(t, name, dtype, shape, device):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != torch.device(device) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _row_stride(t, name):
    """[rows][heads][head_dim] with the heads of a row back to back; the row stride in elements."""
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be [rows, heads, head_dim] with each row's heads back to back")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] * t.shape[2])


def _kind(t):
    """What a call checks of a row tensor: (device, type, heads, head_dim); None for no tensor."""
    return None if t is None else (t.device, t.dtype, t.shape[1], t.shape[2])


def make_kv_batch(cu_seqlens: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor, max_rows: int,
                  max_new: int) -> kda_kv_batch:
    """The batch's device tables (int32: cu_seqlens [n + 1], kv_lens [n],
    page_table [n, pages]) and host bounds; the record keeps the tensors alive."""
    n = kv_lens.numel()
    for name, t, shape in (("cu_seqlens", cu_seqlens, (n + 1,)), ("kv_lens", kv_lens, (n,)),
                           ("page_table", page_table, (n,) + tuple(page_table.shape[1:]))):
        if not t.is_cuda or t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() \
                or t.device != cu_seqlens.device:
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of shape {shape}, all on one device")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seqs, pages]")
    b = kda_kv_batch(cu_seqlens.data_ptr(), kv_lens.data_ptr(), page_table.data_ptr(), n, page_table.shape[1],
                     int(max_rows), int(max_new))
    b._tensors = (cu_seqlens, kv_lens, page_table)
    b._device = cu_seqlens.device
    return b


def make_qk_params(q_norm_w: torch.Tensor | None = None, k_norm_w: torch.Tensor | None = None, eps: float = 1e-5,
                   inv_freq=(), interleaved: bool = False) -> kda_qk_params:
    """Norm weights (or None) and the rotation: inv_freq holds one frequency
    (radians per position) per rotated pair, so 2 * len(inv_freq) channels turn."""
    freq = [float(f) for f in inv_freq]
    arr = (ctypes.c_double * max(1, len(freq)))(*freq)
    p = kda_qk_params(_addr(q_norm_w), _addr(k_norm_w), float(eps), 2 * len(freq), int(bool(interleaved)),
                      ctypes.cast(arr, ctypes.POINTER(ctypes.c_double)) if freq else None)
    p._tensors = (q_norm_w, k_norm_w, arr)
    for name, w in (("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)):
        if w is not None and (w.dim() != 1 or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor [head_dim]")
    p._kinds = tuple(None if w is None else (w.device, w.dtype, w.shape[0]) for w in (q_norm_w, k_norm_w))
    return p


def make_kv_io(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, q_out: torch.Tensor | None) -> kda_kv_io:
    """Row tensors [rows, heads, head_dim] (rows may be strided); q and q_out
    may both be None (keys and values only)."""
    io = kda_kv_io(_addr(q), k.data_ptr(), v.data_ptr(), _addr(q_out), _row_stride(q, "q") if q is not None else 0,
                   _row_stride(k, "k"), _row_stride(v, "v"), _row_stride(q_out, "q_out") if q_out is not None else 0)
    io._tensors = (q, k, v, q_out)
    io._kinds = tuple(_kind(t) for t in io._tensors)
    io._rows = min(t.shape[0] for t in io._tensors if t is not None)
    return io


def make_attn_io(q: torch.Tensor, out: torch.Tensor, scale: float | None = None) -> kda_attn_io:
    """q and out [rows, num_heads, head_dim]; scale defaults to head_dim^-0.5."""
    s = float(q.shape[2]) ** -0.5 if scale is None else float(scale)
    io = kda_attn_io(q.data_ptr(), out.data_ptr(), _row_stride(q, "q"), _row_stride(out, "out"), s)
    io._tensors = (q, out)
    io._kinds = tuple(_kind(t) for t in io._tensors)
    io._rows = min(q.shape[0], out.shape[0])
    return io


def _check_rows(kv: PagedKV, batch: kda_kv_batch, where: str, names, kinds, rows) -> None:
    """The row tensors hold max_rows rows of the cache's heads, type and device."""
    for name, kind in zip(names, kinds):
        if kind is not None and kind != (kv.kv_kind if name[0] != "q" and name != "out" else kv.q_kind):
            raise ValueError(f"{where}: {name} must be a {kv.act} tensor on {kv.device} of the cache's heads and "
                             f"head_dim, not {kind}")
    if rows < batch.max_rows:
        raise ValueError(f"{where}: the batch has up to {batch.max_rows} rows, the tensors {rows}")


# The current stream's handle without a Stream object, which costs more than a launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _kv_stream(kv: PagedKV, batch: kda_kv_batch, stream, where: str) -> int:
    """The call's stream; it, the cache, the batch and the current device must be on one GPU."""
    if torch.cuda.current_device() != kv.device.index or (stream is not None and stream.device != kv.device):
        raise ValueError(f"{where}: the cache is on {kv.device}: make it the current device and use its stream")
    if batch is not None and batch._device != kv.device:
        raise ValueError(f"{where}: the batch's tables are not on {kv.device}")
    return _raw_stream(kv.device.index) if stream is None else stream.cuda_stream


def kda_kv_append(kv: PagedKV, params: kda_qk_params | None, io: kda_kv_io, batch: kda_kv_batch, stream=None) -> None:
    """Norm and rotation of q and k per head, q to q_out, k and v to their pages."""
    _check_rows(kv, batch, "kda_kv_append", ("q", "k", "v", "q_out"), io._kinds, io._rows)
    if params is not None:
        for kind in params._kinds:
            if kind is not None and kind != kv.norm_kind:
                raise ValueError(f"kda_kv_append: norm weights must be {kv.act} tensors [{kv.head_dim}] on {kv.device}")
        params = ctypes.byref(params)
    st = lib().kda_kv_append(kv.ref, params, ctypes.byref(io), ctypes.byref(batch),
                             _kv_stream(kv, batch, stream, "kda_kv_append"))
    if st != KDA_OK:
        _check(st, "kda_kv_append")


def kda_kv_read(kv: PagedKV, batch: kda_kv_batch, k_out: torch.Tensor, v_out: torch.Tensor, stream=None) -> None:
    """The batch's tokens read back from their pages into contiguous rows."""
    if k_out.dim() != 3 or v_out.dim() != 3 or not k_out.is_contiguous() or not v_out.is_contiguous():
        raise ValueError("kda_kv_read: k_out and v_out must be contiguous [rows, heads, head_dim] tensors")
    _check_rows(kv, batch, "kda_kv_read", ("k_out", "v_out"), (_kind(k_out), _kind(v_out)),
                min(k_out.shape[0], v_out.shape[0]))
    st = lib().kda_kv_read(kv.ref, ctypes.byref(batch), k_out.data_ptr(), v_out.data_ptr(),
                           _kv_stream(kv, batch, stream, "kda_kv_read"))
    if st != KDA_OK:
        _check(st, "kda_kv_read")


def kda_kv_attend_workspace_bytes(kv: PagedKV, batch: kda_kv_batch) -> int:
    return int(lib().kda_kv_attend_workspace_bytes(kv.ref, ctypes.byref(batch)))


def kda_kv_attend(kv: PagedKV, io: kda_attn_io, batch: kda_kv_batch, workspace: torch.Tensor, stream=None) -> None:
    """Causal attention of the batch's tokens over their sequences' pages."""
    _check_rows(kv, batch, "kda_kv_attend", ("q", "out"), io._kinds, io._rows)
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.device != kv.device or not workspace.is_contiguous():
            raise ValueError(f"kda_kv_attend: the workspace must be a contiguous tensor on {kv.device}")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    st = lib().kda_kv_attend(kv.ref, ctypes.byref(io), ctypes.byref(batch), ws, ws_bytes,
                             _kv_stream(kv, batch, stream, "kda_kv_attend"))
    if st != KDA_OK:
        _check(st, "kda_kv_attend")


def kda_kv_poll_device_error(kv: PagedKV, stream=None) -> tuple[int, int]:
    """Returns (status, flags) of the cache's error word; reading clears it."""
    flags = ctypes.c_uint32(0)
    st = int(lib().kda_kv_poll_device_error(kv.ref, _kv_stream(kv, None, stream, "kda_kv_poll_device_error"),
                                            ctypes.byref(flags)))
    return st, int(flags.value)


# ---- latent attention ---------------------------------------------------------------------


class PagedLatent:
    """A paged latent cache of one layer (a kda_latent_cache record and the tensors behind it).  c is [num_pages, page_size,
    latent_dim] in ``act`` (kv_format "act") or float8_e4m3fn ("e4m3", with c_scale uint8 [num_pages, page_size]), kr
    [num_pages, page_size, rope_dim] in ``act``; those not given are allocated, zero-filled, on ``device``."""

    def __init__(self, num_pages, page_size, num_heads, latent_dim, rope_dim, act: torch.dtype = torch.bfloat16,
                 kv_format: str = "act", c=None, kr=None, c_scale=None, device="cuda"):
        if kv_format not in ("act", "e4m3"):
            raise ValueError(f"kv_format must be \"act\" or \"e4m3\", not {kv_format!r}")
        e4m3 = kv_format == "e4m3"
        if not e4m3 and c_scale is not None:
            raise ValueError("c_scale is for kv_format \"e4m3\"")
        for t in (c, kr, c_scale):
            if t is not None:
                device = t.device
                break

        def made(t, name, dtype, *shape):
            if t is not None:
                return _kv_tensor(t, name, dtype, shape, device)
            raw = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
            return torch.zeros(shape, dtype=raw, device=device).view(dtype)

        self.c = made(c, "c", torch.float8_e4m3fn if e4m3 else act, num_pages, page_size, latent_dim)
        self.c_scale = made(c_scale, "c_scale", torch.uint8, num_pages, page_size) if e4m3 else None
        self.kr = made(kr, "kr", act, num_pages, page_size, rope_dim)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.device, self.act, self.kv_format = self.c.device, act, kv_format
        self.num_pages, self.page_size, self.num_heads = num_pages, page_size, num_heads
        self.latent_dim, self.rope_dim = latent_dim, rope_dim
        self.desc = kda_latent_cache(self.c.data_ptr(), _addr(self.c_scale), self.kr.data_ptr(), self.err.data_ptr(),
                                     num_pages, page_size, num_heads, latent_dim, rope_dim, act_code(act),
                                     KDA_KV_E4M3 if e4m3 else KDA_KV_ACT)
        self.ref = ctypes.byref(self.desc)
        # of row tensors, see _shape: a token's vectors, and the heads'
        self.c_kind, self.kr_kind = (self.device, act, latent_dim), (self.device, act, rope_dim)
        self.qc_kind, self.qr_kind = (self.device, act, num_heads, latent_dim), (self.device, act, num_heads, rope_dim)

    def error_word(self) -> torch.Tensor:
        return self.err


def _strides(t, name, dims):
    """Strides in elements of [rows, ..., channels] with the channels back to back (any that fits for an axis of one entry)."""
    if t.dim() != dims or t.stride(-1) != 1:
        raise ValueError(f"{name} must have {dims} axes, the last one contiguous")
    return [t.stride(i) if t.shape[i] > 1 else t.shape[-1] for i in range(dims - 1)]


def _shape(t):
    """What a call checks of a row tensor: (device, type, sizes after the rows); None for no tensor."""
    return None if t is None else (t.device, t.dtype, *t.shape[1:])


def make_latent_params(c_norm_w: torch.Tensor | None = None, eps: float = 1e-5, inv_freq=(),
                       interleaved: bool = False) -> kda_latent_params:
    """The latents' norm weight (or None) and the rotation: inv_freq holds one frequency (radians per position) per rotated
    pair, so 2 * len(inv_freq) channels of kr and q turn."""
    freq = [float(f) for f in inv_freq]
    arr = (ctypes.c_double * max(1, len(freq)))(*freq)
    if c_norm_w is not None and (c_norm_w.dim() != 1 or not c_norm_w.is_contiguous()):
        raise ValueError("c_norm_w must be a contiguous tensor [latent_dim]")
    p = kda_latent_params(_addr(c_norm_w), float(eps), 2 * len(freq), int(bool(interleaved)),
                          ctypes.cast(arr, ctypes.POINTER(ctypes.c_double)) if freq else None)
    p._tensors = (c_norm_w, arr)
    p._kind = None if c_norm_w is None else (c_norm_w.device, c_norm_w.dtype, c_norm_w.shape[0])
    return p


def make_latent_io(c: torch.Tensor, kr: torch.Tensor, q: torch.Tensor | None, q_out: torch.Tensor | None) -> kda_latent_io:
    """c [rows, latent_dim], kr [rows, rope_dim], q and q_out [rows, heads, rope_dim] (or both None: cache only), any strides
    over contiguous channels."""
    heads = [_strides(t, n, 3) if t is not None else [0, 0] for n, t in (("q", q), ("q_out", q_out))]
    io = kda_latent_io(c.data_ptr(), kr.data_ptr(), _addr(q), _addr(q_out), *_strides(c, "c", 2), *_strides(kr, "kr", 2),
                       *heads[0], *heads[1])
    io._tensors = (c, kr, q, q_out)
    io._kinds = tuple(_shape(t) for t in io._tensors)
    io._rows = min(t.shape[0] for t in io._tensors if t is not None)
    return io


def make_latent_attn_io(q_c: torch.Tensor, q_r: torch.Tensor, out: torch.Tensor, scale: float) -> kda_latent_attn_io:
    """q_c and out [rows, heads, latent_dim], q_r [rows, heads, rope_dim], any strides over contiguous channels; scale is that
    of the layer's scores, usually (nope_dim + rope_dim)^-0.5."""
    io = kda_latent_attn_io(q_c.data_ptr(), q_r.data_ptr(), out.data_ptr(), *_strides(q_c, "q_c", 3), *_strides(q_r, "q_r", 3),
                            *_strides(out, "out", 3), float(scale))
    io._tensors = (q_c, q_r, out)
    io._kinds = tuple(_shape(t) for t in io._tensors)
    io._rows = min(t.shape[0] for t in io._tensors)
    return io


def make_latent_prefill_io(q_n: torch.Tensor, q_r: torch.Tensor, k: torch.Tensor, kr: torch.Tensor, v: torch.Tensor,
                           out: torch.Tensor, scale: float | None = None) -> kda_latent_prefill_io:
    """q_n [rows, heads, nope_dim], q_r [rows, heads, rope_dim], k [kv rows, heads, nope_dim], kr [kv rows, rope_dim], v [kv
    rows, heads, value_dim], out [rows, heads, value_dim], any strides over contiguous channels; scale defaults to
    (nope_dim + rope_dim)^-0.5."""
    s = float(q_n.shape[-1] + q_r.shape[-1]) ** -0.5 if scale is None else float(scale)
    io = kda_latent_prefill_io(q_n.data_ptr(), q_r.data_ptr(), k.data_ptr(), kr.data_ptr(), v.data_ptr(), out.data_ptr(),
                               *_strides(q_n, "q_n", 3), *_strides(q_r, "q_r", 3), *_strides(k, "k", 3), *_strides(kr, "kr", 2),
                               *_strides(v, "v", 3), *_strides(out, "out", 3), k.shape[-1], v.shape[-1], s)
    io._tensors = (q_n, q_r, k, kr, v, out)
    io._kinds = tuple(_shape(t) for t in io._tensors)
    io._rows = min(t.shape[0] for t in (q_n, q_r, out))
    io._kv_rows = min(t.shape[0] for t in (k, kr, v))
    return io


def make_latent_prefill_batch(cu_seqlens: torch.Tensor, cu_kv: torch.Tensor, max_rows: int, max_kv_rows: int,
                              max_new: int) -> kda_latent_prefill_batch:
    """The expanded form's device tables (int32 [n + 1] each) and host bounds; the record keeps the tensors alive."""
    for name, t in (("cu_seqlens", cu_seqlens), ("cu_kv", cu_kv)):
        if not t.is_cuda or t.dtype != torch.int32 or t.dim() != 1 or t.numel() < 1 or t.shape != cu_seqlens.shape \
                or not t.is_contiguous() or t.device != cu_seqlens.device:
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor [n_seqs + 1], both on one device")
    b = kda_latent_prefill_batch(cu_seqlens.data_ptr(), cu_kv.data_ptr(), cu_seqlens.numel() - 1, int(max_rows),
                                 int(max_kv_rows), int(max_new))
    b._tensors = (cu_seqlens, cu_kv)
    b._device = cu_seqlens.device
    return b


def _check_kinds(where: str, names, kinds, want) -> None:
    for name, kind, w in zip(names, kinds, want):
        if kind is not None and kind != w:
            raise ValueError(f"{where}: {name} must be (device, type, sizes after the rows) {w}, not {kind}")


def _check_bound(where: str, what: str, bound: int, rows: int) -> None:
    if rows < bound:
        raise ValueError(f"{where}: the batch has up to {bound} {what}, the tensors {rows}")


def _workspace(cache, workspace, where: str):
    if workspace is None:
        return None, 0
    if workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError(f"{where}: the workspace must be a contiguous tensor on {cache.device}")
    return workspace.data_ptr(), workspace.nbytes


def kda_latent_append(cache: PagedLatent, params: kda_latent_params | None, io: kda_latent_io, batch: kda_kv_batch,
                      stream=None) -> None:
    """Norm of c and rotation of kr and q; c and kr to their pages, q to q_out."""
    where = "kda_latent_append"
    _check_kinds(where, ("c", "kr", "q", "q_out"), io._kinds, (cache.c_kind, cache.kr_kind, cache.qr_kind, cache.qr_kind))
    _check_bound(where, "rows", batch.max_rows, io._rows)
    if params is not None:
        _check_kinds(where, ("c_norm_w",), (params._kind,), (cache.c_kind,))
        params = ctypes.byref(params)
    st = lib().kda_latent_append(cache.ref, params, ctypes.byref(io), ctypes.byref(batch),
                                 _kv_stream(cache, batch, stream, where))
    if st != KDA_OK:
        _check(st, "kda_latent_append")


def kda_latent_read(cache: PagedLatent, batch: kda_kv_batch, c_out: torch.Tensor, kr_out: torch.Tensor, stream=None) -> None:
    """The batch's tokens read back from their pages: c_out [rows, latent_dim], kr_out [rows, rope_dim]."""
    where = "kda_latent_read"
    _check_kinds(where, ("c_out", "kr_out"), (_shape(c_out), _shape(kr_out)), (cache.c_kind, cache.kr_kind))
    _check_bound(where, "rows", batch.max_rows, min(c_out.shape[0], kr_out.shape[0]))
    st = lib().kda_latent_read(cache.ref, ctypes.byref(batch), c_out.data_ptr(), *_strides(c_out, "c_out", 2),
                               kr_out.data_ptr(), *_strides(kr_out, "kr_out", 2), _kv_stream(cache, batch, stream, where))
    if st != KDA_OK:
        _check(st, "kda_latent_read")


def kda_latent_attend_workspace_bytes(cache: PagedLatent, batch: kda_kv_batch) -> int:
    return int(lib().kda_latent_attend_workspace_bytes(cache.ref, ctypes.byref(batch)))


def kda_latent_attend(cache: PagedLatent, io: kda_latent_attn_io, batch: kda_kv_batch, workspace: torch.Tensor,
                      stream=None) -> None:
    """The absorbed form, causal, of the batch's tokens over their sequences' pages."""
    where = "kda_latent_attend"
    _check_kinds(where, ("q_c", "q_r", "out"), io._kinds, (cache.qc_kind, cache.qr_kind, cache.qc_kind))
    _check_bound(where, "rows", batch.max_rows, io._rows)
    st = lib().kda_latent_attend(cache.ref, ctypes.byref(io), ctypes.byref(batch), *_workspace(cache, workspace, where),
                                 _kv_stream(cache, batch, stream, where))
    if st != KDA_OK:
        _check(st, "kda_latent_attend")


def kda_latent_prefill_workspace_bytes(cache: PagedLatent, io: kda_latent_prefill_io, batch: kda_latent_prefill_batch) -> int:
    return int(lib().kda_latent_prefill_workspace_bytes(cache.ref, ctypes.byref(io), ctypes.byref(batch)))


def kda_latent_prefill(cache: PagedLatent, io: kda_latent_prefill_io, batch: kda_latent_prefill_batch,
                       workspace: torch.Tensor, stream=None) -> None:
    """The expanded form, causal, over keys and values in rows; of the cache it takes heads, rope_dim, type and error word."""
    where = "kda_latent_prefill"
    d, a, h, n, v = cache.device, cache.act, cache.num_heads, io.nope_dim, io.value_dim
    _check_kinds(where, ("q_n", "q_r", "k", "kr", "v", "out"), io._kinds,
                 ((d, a, h, n), cache.qr_kind, (d, a, h, n), cache.kr_kind, (d, a, h, v), (d, a, h, v)))
    _check_bound(where, "rows", batch.max_rows, io._rows)
    _check_bound(where, "key rows", batch.max_kv_rows, io._kv_rows)
    st = lib().kda_latent_prefill(cache.ref, ctypes.byref(io), ctypes.byref(batch), *_workspace(cache, workspace, where),
                                  _kv_stream(cache, batch, stream, where))
    if st != KDA_OK:
        _check(st, "kda_latent_prefill")


def kda_latent_poll_device_error(cache: PagedLatent, stream=None) -> tuple[int, int]:
    """Returns (status, flags) of the cache's error word; reading clears it."""
    flags = ctypes.c_uint32(0)
    st = int(lib().kda_latent_poll_device_error(cache.ref, _kv_stream(cache, None, stream, "kda_latent_poll_device_error"),
                                                ctypes.byref(flags)))
    return st, int(flags.value)

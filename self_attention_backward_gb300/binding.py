"""ctypes binding of the C ABI in ``include/psa_attn.h`` (argument marshalling only).

Every function here turns torch tensors into device pointers and sizes and
calls the C entry point of the same name; all arithmetic runs in the CUDA
library.  There is no fallback: if ``_psa_attn.so`` is missing, the first call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_psa_attn.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "psa_attn.h")

PSA_F32, PSA_BF16 = 0, 1
PSA_OK, PSA_ERR_ARG, PSA_ERR_ALIGN, PSA_ERR_UNSUPPORTED = 0, -1, -2, -3
PSA_ERR_WORKSPACE, PSA_ERR_CUDA, PSA_ERR_TIMEOUT = -4, -5, -6
PSA_ALGO_AUTO, PSA_ALGO_SIMT, PSA_ALGO_TC, PSA_ALGO_TC_2PASS = 0, 1, 2, 3

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong


class psa_attn_view(ctypes.Structure):
    """A strided view of a [B, heads, N, d] tensor (strides in elements), as in
    include/psa_attn.h."""
    _fields_ = [("base", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("pos_stride", ctypes.c_longlong), ("feat_stride", ctypes.c_longlong)]


class psa_win_shape(ctypes.Structure):
    """Sizes, mask and scale of a sliding-window attention, as in include/psa_attn.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "q_heads", "kv_heads", "Nq", "Nk", "head_dim", "window", "sinks")] + [
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class psa_rope_plan(ctypes.Structure):
    """A rotation's frequencies and pairing, as in include/psa_attn.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("head_dim", "rot_dim", "n_axes", "interleaved")] + [
        ("turn", ctypes.c_ulonglong * 64), ("axis", ctypes.c_ubyte * 64)]


class psa_win_cache(ctypes.Structure):
    """A rolling key/value cache, as in include/psa_attn.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int) for n in ("B", "kv_heads", "capacity", "head_dim", "window", "sinks", "dtype")] + [
        (n, ctypes.c_longlong) for n in ("batch_stride", "head_stride", "slot_stride")]


PSA_ROPE_SHARED, PSA_ROPE_PER_AXIS = 0, 1

_vw = ctypes.POINTER(psa_attn_view)
_sh, _pl, _ca = ctypes.POINTER(psa_win_shape), ctypes.POINTER(psa_rope_plan), ctypes.POINTER(psa_win_cache)
_SIGS = {
    "psa_attn_fwd": ([_vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp], _i),
    "psa_attn_fwd_algo": ([_vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp], _i),
    "psa_attn_bwd_workspace_bytes": ([_i, _i, _i, _i, _i], _sz),
    "psa_attn_bwd_workspace_bytes_algo": ([_i, _i, _i, _i, _i, _i], _sz),
    "psa_attn_bwd": ([_vp] * 8 + [_sz, _i, _i, _i, _i, _f, _i, _vp], _i),
    "psa_attn_bwd_algo": ([_vp] * 8 + [_sz, _i, _i, _i, _i, _f, _i, _i, _vp], _i),
    "psa_attn_bwd_noalloc": ([_vp] * 7 + [_i, _i, _i, _i, _f, _i, _vp], _i),
    "psa_attn_bwd_noalloc_max_rows": ([], ctypes.c_longlong),
    "psa_attn_bwd_host": ([_vp] * 8 + [_sz, _i, _i, _i, _i, _f, _i, _i, _i, _vp], _i),
    "psa_attn_bwd_host_buffer_bytes": ([_i, _i, _i, _i, _i, _i], _sz),
    "psa_attn_bwd_host_chunks": ([_i, _i, _i, _i, _i, _i], _i),
    "psa_attn_sync_status": ([_vp], _i),
    "psa_attn_selftest_wait_timeout": ([_vp], _i),
    "psa_attn_profile_enable": ([_i], _i),
    "psa_attn_profile_read": ([ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), _i], _i),
    "psa_attn_profile_slot_name": ([_i], ctypes.c_char_p),
    "psa_attn_last_error": ([], ctypes.c_char_p),
    "psa_attn_version": ([], _i),
    "psa_attn_bwd_ex": ([_vp, _ll, _vp, _vp, _ll, _vp, _vw, _vw, _vp, _vp, _sz, _i, _i, _i, _i, _f, _i, _i, _vp], _i),
    "psa_attn_bwd_ex_workspace_bytes": ([_vw, _vw, _i, _i, _i, _i, _i, _i], _sz),
    "psa_merge_bwd": ([_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp], _i),
    "psa_merge_attn_bwd": ([_vp] * 6 + [_vp, _sz, _i, _i, _i, _i, _i, _f, _i, _i, _vp], _i),
    "psa_merge_attn_bwd_workspace_bytes": ([_i] * 7, _sz),
    "psa_win_attn_fwd": ([_sh] + [_vw] * 4 + [_vp] * 3 + [_i, _vp], _i),
    "psa_win_attn_bwd": ([_sh] + [_vw] * 4 + [_vp] + [_vw] * 4 + [_vp] * 3 + [_sz, _i, _vp], _i),
    "psa_win_attn_bwd_workspace_bytes": ([_sh], _sz),
    "psa_rope_plan_init": ([_pl, _i, _i, _i, ctypes.POINTER(_i), ctypes.c_double, _i, _i], _i),
    "psa_rope": ([_pl, _vw, _vw, _i, _vw, _vw, _i, _i, _i, _vp, _ll, _ll, _i, _i, _vp], _i),
    "psa_win_cache_append": ([_ca, _vw, _vw, _i, _vp, _vp, _pl, _vp, _ll, _ll, _vp], _i),
    "psa_win_decode": ([_ca, _vw, _vw, _vp, _i, _vp, _f, _vp, _sz, _vp], _i),
    "psa_win_decode_workspace_bytes": ([_ca, _i], _sz),
}

_lock = threading.Lock()
_lib = None


class PsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"psa status {code}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"CUDA library {LIB_PATH} is not built; run "
                                   "`python -m self_attention_backward_gb300.build` (nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGS.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/psa_attn.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(psa_\w+)\s*\(", text)))


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return PSA_F32
    if t.dtype == torch.bfloat16:
        return PSA_BF16
    raise TypeError(f"unsupported storage dtype {t.dtype}")


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int) -> int:
    if rc != PSA_OK:
        raise PsaError(rc, psa_attn_last_error())
    return rc


def psa_attn_last_error() -> str:
    return lib().psa_attn_last_error().decode()


def psa_attn_version() -> int:
    return int(lib().psa_attn_version())


def psa_attn_fwd(packed, o_lo, o_hi, lse, B, heads, N, head_dim, scale, dtype=None, stream=None,
                 check=True, algo=PSA_ALGO_AUTO) -> int:
    dtype = _dtype_code(packed) if dtype is None else dtype
    rc = lib().psa_attn_fwd_algo(_ptr(packed), _ptr(o_lo), _ptr(o_hi), _ptr(lse), B, heads, N, head_dim,
                                 float(scale), dtype, algo, _stream(stream))
    return _check(rc) if check else rc


def psa_attn_bwd_workspace_bytes(B, heads, N, head_dim, dtype, algo=PSA_ALGO_AUTO) -> int:
    return int(lib().psa_attn_bwd_workspace_bytes_algo(B, heads, N, head_dim, dtype, algo))


def psa_attn_bwd(packed, o_lo, o_hi, lse, do_lo, do_hi, d_packed, workspace, workspace_bytes,
                 B, heads, N, head_dim, scale, dtype=None, stream=None, algo=PSA_ALGO_AUTO,
                 check=True) -> int:
    dtype = _dtype_code(packed) if dtype is None else dtype
    rc = lib().psa_attn_bwd_algo(_ptr(packed), _ptr(o_lo), _ptr(o_hi), _ptr(lse), _ptr(do_lo), _ptr(do_hi),
                                 _ptr(d_packed), _ptr(workspace), int(workspace_bytes), B, heads, N,
                                 head_dim, float(scale), dtype, algo, _stream(stream))
    return _check(rc) if check else rc


def psa_attn_bwd_noalloc(packed, o_lo, o_hi, lse, do_lo, do_hi, d_packed, B, heads, N, head_dim, scale,
                         dtype=None, stream=None, check=True) -> int:
    """Backward without a workspace argument: its scratch is a static array in
    the library (see include/psa_attn.h).  For callers that cannot allocate."""
    dtype = _dtype_code(packed) if dtype is None else dtype
    rc = lib().psa_attn_bwd_noalloc(_ptr(packed), _ptr(o_lo), _ptr(o_hi), _ptr(lse), _ptr(do_lo), _ptr(do_hi),
                                    _ptr(d_packed), B, heads, N, head_dim, float(scale), dtype, _stream(stream))
    return _check(rc) if check else rc


def psa_attn_bwd_noalloc_max_rows() -> int:
    return int(lib().psa_attn_bwd_noalloc_max_rows())


def psa_attn_bwd_host(packed, o_lo, o_hi, lse, do_lo, do_hi, d_packed, dev_buf, dev_buf_bytes,
                      B, heads, N, head_dim, scale, dtype=None, algo=PSA_ALGO_AUTO, chunks=0, stream=None,
                      check=True) -> int:
    """Backward on HOST tensors (ideally pinned), `dev_buf` a device scratch of
    psa_attn_bwd_host_buffer_bytes(...) bytes (see include/psa_attn.h)."""
    dtype = _dtype_code(packed) if dtype is None else dtype
    rc = lib().psa_attn_bwd_host(_ptr(packed), _ptr(o_lo), _ptr(o_hi), _ptr(lse), _ptr(do_lo), _ptr(do_hi),
                                 _ptr(d_packed), _ptr(dev_buf), int(dev_buf_bytes), B, heads, N, head_dim,
                                 float(scale), dtype, algo, int(chunks), _stream(stream))
    return _check(rc) if check else rc


def psa_attn_bwd_host_buffer_bytes(B, heads, N, head_dim, dtype, algo=PSA_ALGO_AUTO) -> int:
    return int(lib().psa_attn_bwd_host_buffer_bytes(B, heads, N, head_dim, dtype, algo))


def psa_attn_bwd_host_chunks(B, heads, N, head_dim, dtype, algo=PSA_ALGO_AUTO) -> int:
    return int(lib().psa_attn_bwd_host_chunks(B, heads, N, head_dim, dtype, algo))


def psa_attn_sync_status(stream=None, check=True) -> int:
    rc = lib().psa_attn_sync_status(_stream(stream))
    return _check(rc) if check else rc


def psa_attn_selftest_wait_timeout(stream=None, check=True) -> int:
    rc = lib().psa_attn_selftest_wait_timeout(_stream(stream))
    return _check(rc) if check else rc


def psa_attn_profile_enable(on: bool = True) -> int:
    return _check(lib().psa_attn_profile_enable(1 if on else 0))


def psa_attn_profile_slot_name(slot: int) -> str:
    return lib().psa_attn_profile_slot_name(slot).decode()


def psa_attn_profile_read() -> dict:
    """{slot name: (total ms, launches)} since the last read; clears the records."""
    n = 4
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int * n)()
    rc = lib().psa_attn_profile_read(ms, cnt, n)
    if rc < 0:
        raise PsaError(rc, psa_attn_last_error())
    return {psa_attn_profile_slot_name(i): (float(ms[i]), int(cnt[i])) for i in range(rc)}


# ----------------------------------------------------------------- helpers
def _torch_dtype(dtype):
    import torch
    return {PSA_F32: torch.float32, PSA_BF16: torch.bfloat16}[dtype]


def attn_fwd(packed, scale: float, stream=None, algo=PSA_ALGO_AUTO):
    """Allocates O_lo, O_hi, LSE on packed's device and runs psa_attn_fwd.

    packed: [BH, 4, N, d] CUDA tensor (fp32 or bf16).  B is taken as BH, heads 1.
    """
    import torch
    BH, four, N, d = packed.shape
    assert four == 4 and packed.is_contiguous()
    o_lo = torch.empty((BH, N, d), dtype=packed.dtype, device=packed.device)
    o_hi = torch.empty_like(o_lo)
    lse = torch.empty((BH, N), dtype=torch.float32, device=packed.device)
    psa_attn_fwd(packed, o_lo, o_hi, lse, BH, 1, N, d, scale, stream=stream, algo=algo)
    return o_lo, o_hi, lse


class BwdWorkspace:
    """A device workspace sized for psa_attn_bwd, grown on demand."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = None

    def get(self, nbytes: int):
        import torch
        if nbytes == 0:
            return None
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return self.buf


def attn_bwd(packed, o_lo, o_hi, lse, do_lo, do_hi, scale: float, d_packed=None, workspace=None,
             algo=PSA_ALGO_AUTO, stream=None):
    """Runs psa_attn_bwd; returns d_packed [BH, 4, N, d] (dQ, dK, dV_lo, dV_hi)."""
    import torch
    BH, _, N, d = packed.shape
    dt = _dtype_code(packed)
    if d_packed is None:
        d_packed = torch.empty_like(packed)
    nbytes = psa_attn_bwd_workspace_bytes(BH, 1, N, d, dt, algo)
    ws = (workspace or BwdWorkspace(packed.device)).get(nbytes)
    psa_attn_bwd(packed, o_lo, o_hi, lse, do_lo, do_hi, d_packed, ws, nbytes, BH, 1, N, d, scale,
                 dtype=dt, stream=stream, algo=algo)
    return d_packed


class HostBwd:
    """psa_attn_bwd_host for one shape: the device buffer it needs (the
    device copies of the inputs and of d_packed, and the workspace) is
    allocated once here, by torch; each call passes the host tensors (pinned
    for asynchronous copies) to the native entry point, which pipelines the
    copies in, the backward and the copy back over `chunks` groups of
    (batch*head) slices (None = the library's choice)."""

    def __init__(self, BH: int, N: int, d: int, dtype: int, device="cuda", algo=PSA_ALGO_AUTO, chunks=None):
        import torch
        self.shape = (BH, N, d)
        self.dtype, self.algo = dtype, algo
        self.chunks = 0 if chunks is None else int(chunks)
        self.buf_bytes = psa_attn_bwd_host_buffer_bytes(BH, 1, N, d, dtype, algo)
        self.buf = torch.empty(max(self.buf_bytes, 1), dtype=torch.uint8, device=device)
        es = 2 if dtype == PSA_BF16 else 4
        self._in_bytes = BH * N * (8 * d * es + 4)
        self._out_bytes = BH * N * 4 * d * es

    def h2d_bytes(self) -> int:
        return self._in_bytes

    def d2h_bytes(self) -> int:
        return self._out_bytes

    def __call__(self, packed, o_lo, o_hi, lse, do_lo, do_hi, scale: float, out, stream=None):
        BH, N, d = self.shape
        psa_attn_bwd_host(packed, o_lo, o_hi, lse, do_lo, do_hi, out, self.buf, self.buf_bytes, BH, 1, N, d,
                          scale, dtype=self.dtype, algo=self.algo, chunks=self.chunks, stream=stream)
        return out


# ----------------------------------------------------------------- strided layouts and the merge
def view_of(t) -> psa_attn_view:
    """psa_attn_view of a 4-D torch tensor [B, heads, N, d] with any strides."""
    assert t.dim() == 4
    sb, sh, sn, sj = t.stride()
    return psa_attn_view(t.data_ptr(), sb, sh, sn, sj)


def psa_attn_bwd_ex(packed, qkv_row_stride, o_lo, o_hi, o_row_stride, lse, do_lo: psa_attn_view,
                    do_hi: psa_attn_view, d_packed, workspace, workspace_bytes, B, heads, N, head_dim, scale,
                    dtype, algo=PSA_ALGO_AUTO, stream=None, check=True) -> int:
    rc = lib().psa_attn_bwd_ex(_ptr(packed), int(qkv_row_stride), _ptr(o_lo), _ptr(o_hi), int(o_row_stride),
                               _ptr(lse), ctypes.byref(do_lo), ctypes.byref(do_hi), _ptr(d_packed), _ptr(workspace),
                               int(workspace_bytes), B, heads, N, head_dim, float(scale), dtype, algo,
                               _stream(stream))
    return _check(rc) if check else rc


def psa_attn_bwd_ex_workspace_bytes(do_lo: psa_attn_view, do_hi: psa_attn_view, B, heads, N, head_dim, dtype,
                                    algo=PSA_ALGO_AUTO) -> int:
    return int(lib().psa_attn_bwd_ex_workspace_bytes(ctypes.byref(do_lo), ctypes.byref(do_hi), B, heads, N,
                                                     head_dim, dtype, algo))


def psa_merge_bwd(d_merged, d_lo, d_hi, B, heads, H, W, head_dim, dtype, stream=None, check=True) -> int:
    rc = lib().psa_merge_bwd(_ptr(d_merged), _ptr(d_lo), _ptr(d_hi), B, heads, H, W, head_dim, dtype,
                             _stream(stream))
    return _check(rc) if check else rc


def psa_merge_attn_bwd(packed, o_lo, o_hi, lse, d_merged, d_packed, workspace, workspace_bytes, B, heads, H, W,
                       head_dim, scale, dtype, algo=PSA_ALGO_AUTO, stream=None, check=True) -> int:
    rc = lib().psa_merge_attn_bwd(_ptr(packed), _ptr(o_lo), _ptr(o_hi), _ptr(lse), _ptr(d_merged), _ptr(d_packed),
                                  _ptr(workspace), int(workspace_bytes), B, heads, H, W, head_dim, float(scale),
                                  dtype, algo, _stream(stream))
    return _check(rc) if check else rc


def psa_merge_attn_bwd_workspace_bytes(B, heads, H, W, head_dim, dtype, algo=PSA_ALGO_AUTO) -> int:
    return int(lib().psa_merge_attn_bwd_workspace_bytes(B, heads, H, W, head_dim, dtype, algo))


def attn_bwd_ex(packed, d, o_lo, o_hi, lse, do_lo4, do_hi4, scale: float, heads: int, d_packed=None,
                workspace=None, algo=PSA_ALGO_AUTO, stream=None):
    """psa_attn_bwd_ex on torch tensors: packed [BH, 4, N, ld] (rows of d used),
    o_lo / o_hi [BH, N, ld_o], do_lo4 / do_hi4 any 4-D [B, heads, N, d] views
    (their torch strides are passed through).  Returns d_packed, shaped like
    packed (only the first d elements of each row are written)."""
    import torch
    BH, _, N, ld = packed.shape
    B = BH // heads
    dt = _dtype_code(packed)
    if d_packed is None:
        d_packed = torch.zeros_like(packed)
    vlo, vhi = view_of(do_lo4), view_of(do_hi4)
    nbytes = psa_attn_bwd_ex_workspace_bytes(vlo, vhi, B, heads, N, d, dt, algo)
    ws = (workspace or BwdWorkspace(packed.device)).get(nbytes)
    psa_attn_bwd_ex(packed, ld, o_lo, o_hi, o_lo.shape[-1], lse, vlo, vhi, d_packed, ws, nbytes, B, heads, N, d,
                    scale, dt, algo=algo, stream=stream)
    return d_packed


def merge_bwd(d_merged, heads: int, d: int, stream=None):
    """psa_merge_bwd: d_merged [B, 2*heads*d, H, W] -> (dO_lo, dO_hi) [B*heads, H*W, d]."""
    import torch
    B, c, H, W = d_merged.shape
    d_lo = torch.empty((B * heads, H * W, d), dtype=d_merged.dtype, device=d_merged.device)
    d_hi = torch.empty_like(d_lo)
    psa_merge_bwd(d_merged, d_lo, d_hi, B, heads, H, W, d, _dtype_code(d_merged), stream=stream)
    return d_lo, d_hi


def merge_attn_bwd(packed, o_lo, o_hi, lse, d_merged, heads: int, scale: float, d_packed=None, workspace=None,
                   algo=PSA_ALGO_AUTO, stream=None):
    """psa_merge_attn_bwd: the merge's backward fused into the attention
    backward; d_merged [B, 2*heads*d, H, W].  Returns d_packed."""
    import torch
    BH, _, N, d = packed.shape
    B, c, H, W = d_merged.shape
    dt = _dtype_code(packed)
    if d_packed is None:
        d_packed = torch.empty_like(packed)
    nbytes = psa_merge_attn_bwd_workspace_bytes(B, heads, H, W, d, dt, algo)
    ws = (workspace or BwdWorkspace(packed.device)).get(nbytes)
    psa_merge_attn_bwd(packed, o_lo, o_hi, lse, d_merged, d_packed, ws, nbytes, B, heads, H, W, d, scale, dt,
                       algo=algo, stream=stream)
    return d_packed


# ----------------------------------------------------------------- sliding-window attention, rotary positions, rolling cache
# A small call's time is this file's: checks build no message unless they fail,
# and the stream comes from torch's raw accessor.
def _bad(what: str):
    raise ValueError(what)


def _same(first, *others) -> int:
    """The dtype code of tensors that have to agree in dtype and device."""
    dtype, device = first.dtype, first.device
    for t in others:
        if t.dtype is not dtype or t.device != device:
            _bad(f"tensors differ: {dtype} on {device}, {t.dtype} on {t.device}")
    return _dtype_code(first)


def _int32(name: str, t, device, shape):
    """Pointer of a contiguous int32 tensor, or None."""
    if t is None:
        return None
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        _bad(f"{name} has to be a contiguous int32 tensor {shape} on {device}")
    return t.data_ptr()


def _lse_ptr(lse, like, device):
    import torch
    if lse.dtype is not torch.float32 or lse.shape != like or lse.device != device or not lse.is_contiguous():
        _bad(f"lse has to be a contiguous fp32 tensor {tuple(like)} on {device}")
    return lse.data_ptr()


def _launch(device, call, *args) -> None:
    """call(*args, stream) with the tensors' device current, on its current stream."""
    import torch
    i = device.index
    if i is None:
        _bad(f"tensors have to be on a CUDA device, not {device}")
    if torch._C._cuda_getDevice() == i:
        rc = call(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            rc = call(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc:
        _check(rc)


def _takes_stream(f):
    """Lets f take `stream` (a torch stream, or a handle): it is the current one while f
    runs, so that what f allocates belongs to it."""
    @functools.wraps(f)
    def on(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        import torch
        if isinstance(stream, int):
            device = next(a.device for a in args if hasattr(a, "device"))
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return on


def _view(t) -> psa_attn_view:
    return psa_attn_view(t.data_ptr(), *t.stride())


def _win_args(q, k, v, scale, window, sinks, q_lens, kv_lens):
    if q.dim() != 4 or k.dim() != 4:
        _bad("q, k, v have to be [B, heads, N, d]")
    B, Hq, Nq, d = q.shape
    B2, Hkv, Nk, d2 = k.shape
    if B2 != B or d2 != d or v.shape != k.shape:
        _bad(f"k {tuple(k.shape)}, v {tuple(v.shape)} and q {tuple(q.shape)} do not fit together")
    sh = psa_win_shape(B, Hq, Hkv, Nq, Nk, d, window, sinks, scale, _same(q, k, v))
    dev = q.device
    if dev.type != "cuda":
        _bad(f"tensors have to be on a CUDA device, not {dev}")
    return sh, _int32("q_lens", q_lens, dev, (B,)), _int32("kv_lens", kv_lens, dev, (B,))


@_takes_stream
def win_attn_fwd(q, k, v, scale: float, window: int, sinks: int, q_lens=None, kv_lens=None, out=None, lse=None,
                 algo=PSA_ALGO_AUTO):
    """Causal attention over the last `window` and the first `sinks` positions.

    q [B, Hq, Nq, d], k and v [B, Hkv, Nk, d] with any strides; q_lens, kv_lens
    int32 [B] device tensors or None.  Returns O (q's layout) and LSE
    [B, Hq, Nq].  See psa_win_attn_fwd in include/psa_attn.h."""
    import torch
    sh, ql, kl = _win_args(q, k, v, scale, window, sinks, q_lens, kv_lens)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        _bad("out has to be shaped like q")
    else:
        _same(q, out)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    _launch(q.device, lib().psa_win_attn_fwd, sh, _view(q), _view(k), _view(v), _view(out),
            _lse_ptr(lse, q.shape[:3], q.device), ql, kl, algo)
    return out, lse


@_takes_stream
def win_attn_bwd(q, k, v, o, lse, do, scale: float, window: int, sinks: int, q_lens=None, kv_lens=None, dq=None,
                 dk=None, dv=None, workspace=None, algo=PSA_ALGO_AUTO):
    """dQ, dK, dV of win_attn_fwd (o, lse: its outputs; do: the gradient in o).

    workspace: a BwdWorkspace that the caller keeps (calls that share one must not
    overlap on the GPU), or None for one of this call's own."""
    import torch
    sh, ql, kl = _win_args(q, k, v, scale, window, sinks, q_lens, kv_lens)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _same(q, o, do, dq, dk, dv)
    if o.shape != q.shape or do.shape != q.shape or dq.shape != q.shape or dk.shape != k.shape or dv.shape != k.shape:
        _bad("o, do, dq have to be shaped like q, and dk, dv like k")
    L = lib()
    nbytes = L.psa_win_attn_bwd_workspace_bytes(sh)
    ws = (BwdWorkspace(q.device) if workspace is None else workspace).get(nbytes)
    if ws is not None and ws.device != q.device:
        _bad(f"the workspace is on {ws.device}, the tensors on {q.device}")
    _launch(q.device, L.psa_win_attn_bwd, sh, _view(q), _view(k), _view(v), _view(o),
            _lse_ptr(lse, q.shape[:3], q.device), _view(do), _view(dq), _view(dk), _view(dv), ql, kl, _ptr(ws), nbytes,
            algo)
    return dq, dk, dv


class RopePlan:
    """Rotary positions with len(sections) axes (1 to 3): sections[a] pairs turn by
    axis a's position.  See psa_rope_plan in include/psa_attn.h."""

    def __init__(self, head_dim: int, sections, theta: float = 10000.0, rot_dim: int | None = None,
                 ladder=PSA_ROPE_SHARED, interleaved: bool = False):
        sections = [int(s) for s in sections]
        self.n_axes, self.head_dim = len(sections), head_dim
        self.c = psa_rope_plan()
        _check(lib().psa_rope_plan_init(self.c, head_dim, head_dim if rot_dim is None else rot_dim, self.n_axes,
                                        (ctypes.c_int * max(self.n_axes, 1))(*sections), float(theta), ladder,
                                        1 if interleaved else 0))


def _pos_args(plan: RopePlan, pos, device, B: int, N: int):
    """Pointer and strides of int32 positions [axes, B, N] or, shared by the batch,
    [axes, 1, N] or [axes, N]."""
    import torch
    if pos.dtype is not torch.int32 or pos.device != device:
        _bad(f"pos has to be an int32 tensor on {device}")
    shape, st = pos.shape, pos.stride()
    A = plan.n_axes
    if shape == (A, B, N):
        sb = st[1] if B > 1 else 0
    elif shape == (A, 1, N) or shape == (A, N):
        sb = 0
    else:
        _bad(f"pos has to be [{A}, {B}, {N}] or [{A}, {N}], not {list(shape)}")
    if N > 1 and st[-1] != 1:
        _bad("pos has to be contiguous along the rows")
    return pos.data_ptr(), st[0], sb


@_takes_stream
def rope(plan: RopePlan, q, pos, k=None, inverse: bool = False, out=None, out_k=None):
    """Rotates q [B, H, N, d] (and k [B, H2, N, d]) by the positions pos; inverse
    turns back, which is the gradient.  out / out_k may be q / k themselves."""
    import torch
    if q.dim() != 4 or q.shape[3] != plan.head_dim:
        _bad("q has to be [B, heads, N, d] with the plan's d")
    B, H, N, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        _bad("out has to be shaped like q")
    dev = q.device
    p, sa, sb = _pos_args(plan, pos, dev, B, N)
    if k is None:
        _launch(dev, lib().psa_rope, plan.c, _view(q), _view(out), H, None, None, 0, B, N, p, sa, sb,
                1 if inverse else 0, _same(q, out))
        return out
    if k.dim() != 4 or k.shape[0] != B or k.shape[2] != N or k.shape[3] != plan.head_dim:
        _bad("k and q do not fit together")
    if out_k is None:
        out_k = torch.empty_like(k)
    elif out_k.shape != k.shape:
        _bad("out_k has to be shaped like k")
    _launch(dev, lib().psa_rope, plan.c, _view(q), _view(out), H, _view(k), _view(out_k), k.shape[1], B, N, p, sa,
            sb, 1 if inverse else 0, _same(q, k, out, out_k))
    return out, out_k


class WinCache:
    """A rolling key/value cache over the caller's tensors k, v [B, Hkv, capacity,
    d] (same strides, features adjacent), with its single-token attention.  See
    psa_win_cache in include/psa_attn.h.  The workspace of decode() is kept here:
    decode() calls on one WinCache have to follow one another on the GPU."""

    def __init__(self, k, v, window: int, sinks: int):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            _bad("k and v have to be [B, Hkv, capacity, d] with the same strides")
        if k.stride(3) != 1:
            _bad("the features of a slot have to be adjacent")
        dt = _same(k, v)
        B, H, cap, d = k.shape
        self.k, self.v, self.device = k, v, k.device
        self.c = psa_win_cache(k.data_ptr(), v.data_ptr(), B, H, cap, d, window, sinks, dt, *k.stride()[:3])
        self._batch = (B,)
        self._ws = BwdWorkspace(k.device)
        self._ws_bytes: dict[int, int] = {}

    @_takes_stream
    def append(self, k_new, v_new, start, n_new=None, plan: RopePlan | None = None, pos=None) -> None:
        """Writes the positions start[b] .. start[b] + n_new[b] - 1 of every
        sequence (k_new, v_new [B, Hkv, T, d]; start, n_new int32 [B]); with a plan
        the keys are rotated by pos on the way."""
        dev, (B, Hkv, _, d) = self.device, self.k.shape
        if k_new.dim() != 4 or v_new.shape != k_new.shape:
            _bad("k_new and v_new have to be [B, Hkv, T, d] of the cache")
        B2, H2, T, d2 = k_new.shape
        if B2 != B or H2 != Hkv or d2 != d:
            _bad("k_new and v_new have to be [B, Hkv, T, d] of the cache")
        _same(self.k, k_new, v_new)
        if (plan is None) != (pos is None):
            _bad("plan and pos are given together or not at all")
        p, sa, sb = (None, 0, 0) if plan is None else _pos_args(plan, pos, dev, B, T)
        _launch(dev, lib().psa_win_cache_append, self.c, _view(k_new), _view(v_new), T,
                _int32("start", start, dev, self._batch), _int32("n_new", n_new, dev, self._batch),
                None if plan is None else plan.c, p, sa, sb)

    @_takes_stream
    def decode(self, q, lens, scale: float, out=None, lse=None):
        """Attention of q [B, Hq, d] at the positions lens - 1 (int32 [B]); returns O
        [B, Hq, d].  lse: None or an fp32 tensor [B, Hq] to fill."""
        import torch
        dev = self.device
        if q.dim() != 3 or q.shape[0] != self.k.shape[0] or q.shape[2] != self.k.shape[3]:
            _bad("q has to be [B, Hq, d] of the cache")
        if out is None:
            out = torch.empty_like(q)
        elif out.shape != q.shape:
            _bad("out has to be shaped like q")
        _same(self.k, q, out)
        if lens is None:
            _bad("lens is missing")
        H = q.shape[1]
        nbytes = self._ws_bytes.get(H)
        if nbytes is None:
            nbytes = self._ws_bytes[H] = lib().psa_win_decode_workspace_bytes(self.c, H)
        (qb, qh, qj), (ob, oh, oj) = q.stride(), out.stride()
        _launch(dev, lib().psa_win_decode, self.c, psa_attn_view(q.data_ptr(), qb, qh, 0, qj),
                psa_attn_view(out.data_ptr(), ob, oh, 0, oj), None if lse is None else _lse_ptr(lse, q.shape[:2], dev), H,
                _int32("lens", lens, dev, self._batch), scale, _ptr(self._ws.get(nbytes)), nbytes)
        return out

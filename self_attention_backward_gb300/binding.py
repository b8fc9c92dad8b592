"""ctypes binding of the C ABI in ``include/psa_attn.h`` (argument marshalling only).

Every function here turns torch tensors into device pointers and sizes and
calls the C entry point of the same name; all arithmetic runs in the CUDA
library.  There is no fallback: if ``_psa_attn.so`` is missing, the first call
raises.
"""
from __future__ import annotations

import ctypes
import operator
import os
import re
import sysconfig
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_psa_attn.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "psa_attn.h")

PSA_F32, PSA_BF16, PSA_E4M3 = 0, 1, 2
PSA_TREE_MAX = 256
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


class psa_win_scales(ctypes.Structure):
    """An 8-bit cache's scales, as in include/psa_attn.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_longlong) for n in ("batch_stride", "head_stride", "slot_stride")]


PSA_ROPE_SHARED, PSA_ROPE_PER_AXIS = 0, 1

_vw = ctypes.POINTER(psa_attn_view)
_sh, _pl, _ca = ctypes.POINTER(psa_win_shape), ctypes.POINTER(psa_rope_plan), ctypes.POINTER(psa_win_cache)
_sc = ctypes.POINTER(psa_win_scales)
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
    "psa_win_store": ([_ca, _sc, _vw, _vw, _i, _vp, _ll, _i, _vp, _vp, _pl, _vp, _ll, _ll, _i, _vp], _i),
    "psa_win_read": ([_ca, _sc, _vw, _vw, _i, _vp, _vp, _i, _vp], _i),
    "psa_win_decode_any": ([_ca, _sc, _vw, _vw, _vp, _i, _vp, _f, _vp, _sz, _i, _vp], _i),
    "psa_win_decode_any_workspace_bytes": ([_ca, _i, _i], _sz),
    "psa_win_tree_attn": ([_ca, _sc] + [_vw] * 4 + [_vp, _i, _i, _vp, _ll, _vp, _vp, _f, _vp, _sz, _i, _i, _vp], _i),
    "psa_win_tree_attn_workspace_bytes": ([_ca, _i, _i, _i], _sz),
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
# Their tensors are taken apart in C (csrc/py_bind.c): small calls take a few
# microseconds on the GPU, and marshalling them here took more.
BIND_PATH = os.path.join(PKG, "_psa_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
_bind = None


def _native():
    """The loaded C marshalling module (raises if it has not been built)."""
    global _bind
    L = lib()
    with _lock:
        if _bind is None:
            import torch
            from importlib.machinery import ExtensionFileLoader
            from importlib.util import module_from_spec, spec_from_file_location
            if not os.path.exists(BIND_PATH):
                raise RuntimeError(f"{BIND_PATH} is not built; run `python -m self_attention_backward_gb300.build`")
            spec = spec_from_file_location("_psa_bind", BIND_PATH, loader=ExtensionFileLoader("_psa_bind", BIND_PATH))
            m = module_from_spec(spec)
            spec.loader.exec_module(m)
            at = [ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
                "psa_rope", "psa_win_attn_fwd", "psa_win_attn_bwd", "psa_win_attn_bwd_workspace_bytes",
                "psa_win_cache_append", "psa_win_decode", "psa_win_store", "psa_win_read", "psa_win_decode_any",
                "psa_win_tree_attn", "psa_win_decode_any_workspace_bytes", "psa_win_tree_attn_workspace_bytes")]
            m.init(torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch._C._cuda_getDevice,
                   torch._C._cuda_getCurrentRawStream, torch.empty_like, torch.empty, *at)
            _bind = m
    return _bind


def _again(rc: int, device, call, args):
    """A call that returned a status: once more with the tensors' device current, or its error."""
    if rc == _bind.OTHER_DEVICE:
        import torch
        with torch.cuda.device(device):
            r = call(*args)
        if type(r) is not int:
            return r
        rc = r
    _check(rc)
    return rc


def _on_stream(stream, device, f, *args, **kw):
    """f with `stream` (a torch stream, or a handle) the current one, so that what f
    allocates belongs to it."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    elif stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return f(*args, **kw)


def win_attn_fwd(q, k, v, scale: float, window: int, sinks: int, q_lens=None, kv_lens=None, out=None, lse=None,
                 algo=PSA_ALGO_AUTO, stream=None):
    """Causal attention over the last `window` and the first `sinks` positions.

    q [B, Hq, Nq, d], k and v [B, Hkv, Nk, d] with any strides; q_lens, kv_lens
    int32 [B] device tensors or None.  Returns O (q's layout) and LSE
    [B, Hq, Nq].  See psa_win_attn_fwd in include/psa_attn.h."""
    if stream is not None:
        return _on_stream(stream, q.device, win_attn_fwd, q, k, v, scale, window, sinks, q_lens, kv_lens, out, lse, algo)
    m = _bind or _native()
    args = (q, k, v, scale, window, sinks, q_lens, kv_lens, out, lse, algo)
    r = m.win_fwd(*args)
    return _again(r, q.device, m.win_fwd, args) if type(r) is int else r


def win_attn_bwd(q, k, v, o, lse, do, scale: float, window: int, sinks: int, q_lens=None, kv_lens=None, dq=None,
                 dk=None, dv=None, workspace=None, algo=PSA_ALGO_AUTO, stream=None):
    """dQ, dK, dV of win_attn_fwd (o, lse: its outputs; do: the gradient in o).

    workspace: a BwdWorkspace that the caller keeps (calls that share one must not
    overlap on the GPU, and one that a graph was captured with must not grow), or
    None for one of this call's own."""
    if stream is not None:
        return _on_stream(stream, q.device, win_attn_bwd, q, k, v, o, lse, do, scale, window, sinks, q_lens, kv_lens, dq,
                          dk, dv, workspace, algo)
    m = _bind or _native()
    ws = None if workspace is None else workspace.get(m.win_bwd_bytes(q, k, v, scale, window, sinks))
    args = (q, k, v, scale, window, sinks, q_lens, kv_lens, o, lse, do, dq, dk, dv, ws, algo)
    r = m.win_bwd(*args)
    return _again(r, q.device, m.win_bwd, args) if type(r) is int else r


def _c_int(name: str, x) -> int:
    """x, refused where a C int would drop its upper bits."""
    x = operator.index(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} {x} does not fit 32 bits")
    return x


class RopePlan:
    """Rotary positions with len(sections) axes (1 to 3): sections[a] pairs turn by
    axis a's position.  See psa_rope_plan in include/psa_attn.h."""

    def __init__(self, head_dim: int, sections, theta: float = 10000.0, rot_dim: int | None = None,
                 ladder=PSA_ROPE_SHARED, interleaved: bool = False):
        sections = [_c_int("a section of", int(s)) for s in sections]
        n = len(sections)
        self.c = psa_rope_plan()
        _check(lib().psa_rope_plan_init(self.c, _c_int("head_dim", head_dim),
                                        _c_int("rot_dim", head_dim if rot_dim is None else rot_dim), n,
                                        (ctypes.c_int * max(n, 1))(*sections), float(theta), _c_int("ladder", ladder),
                                        1 if interleaved else 0))
        self.address = ctypes.addressof(self.c)


def rope(plan: RopePlan, q, pos, k=None, inverse: bool = False, out=None, out_k=None, stream=None):
    """Rotates q [B, H, N, d] (and k [B, H2, N, d]) by the int32 positions pos
    [axes, B, N] or, shared by the batch, [axes, N]; inverse turns back, which is the
    gradient.  out / out_k may be q / k themselves."""
    if stream is not None:
        return _on_stream(stream, q.device, rope, plan, q, pos, k, inverse, out, out_k)
    m = _bind or _native()
    args = (plan.address, q, pos, k, inverse, out, out_k)
    r = m.rope(*args)
    return _again(r, q.device, m.rope, args) if type(r) is int else r


class WinCache:
    """A rolling key/value cache over the caller's tensors k, v [B, Hkv, capacity,
    d] (same strides, features adjacent): fp32, bf16, or float8_e4m3fn with fp32
    scales k_scale, v_scale [B, Hkv, capacity] (same strides).  Written by append(),
    read back by read(), attended to by decode() (single tokens) and tree() (drafted
    tokens).  See psa_win_cache and psa_win_scales in include/psa_attn.h.  The
    workspace of decode() over an fp32 or bf16 cache is kept here: such calls on one
    WinCache have to follow one another on the GPU.  Those of tree() and of decode()
    over an 8-bit cache are each call's own."""

    def __init__(self, k, v, window: int, sinks: int, k_scale=None, v_scale=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v have to be [B, Hkv, capacity, d] with the same strides")
        if k.stride(3) != 1:
            raise ValueError("the features of a slot have to be adjacent")
        if k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v differ in dtype or device")
        is8 = k.dtype == torch.float8_e4m3fn
        sizes = [_c_int(n, x) for n, x in zip(("B", "Hkv", "capacity", "d", "window", "sinks"), (*k.shape, window, sinks))]
        self.k, self.v, self.device = k, v, k.device
        self.k_scale, self.v_scale = k_scale, v_scale
        self.c = psa_win_cache(k.data_ptr(), v.data_ptr(), *sizes, PSA_E4M3 if is8 else _dtype_code(k), *k.stride()[:3])
        self._at = (ctypes.addressof(self.c), k.get_device())
        # by query heads, and by them and the stream: a workspace (which a captured call holds on
        # to), its bytes and the stream that uses it, in whose order its memory is given back
        self._ws: dict[int, tuple] = {}
        self._all: dict[tuple, tuple] = {}
        self.scales = None
        if is8:
            for s in (k_scale, v_scale):
                if s is None or s.shape != k.shape[:3] or s.dtype != torch.float32 or s.device != k.device or (
                        s.stride() != k_scale.stride()):
                    raise ValueError("an 8-bit cache has fp32 scales k_scale, v_scale [B, Hkv, capacity] with the same "
                                     "strides, on its device")
            self.scales = psa_win_scales(k_scale.data_ptr(), v_scale.data_ptr(), *k_scale.stride())
        elif k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale belong to a cache in float8_e4m3fn")
        self._any = (self._at[0], ctypes.addressof(self.scales) if is8 else 0, self._at[1])
        self._dtype = torch.bfloat16 if is8 else k.dtype

    def append(self, k_new, v_new, start, n_new=None, plan: RopePlan | None = None, pos=None, stream=None, rows=None) -> None:
        """Writes the positions start[b] .. start[b] + n_new[b] - 1 of every
        sequence (k_new, v_new [B, Hkv, T, d]; start, n_new int32 [B]); with a plan
        the keys are rotated by pos (as in rope) on the way.  rows: int32 [B, R] or [R],
        the row of k_new and v_new that each position takes (an accepted path); a
        position whose row is not in 0 .. T - 1 is left as it was."""
        if stream is not None:
            return _on_stream(stream, self.device, self.append, k_new, v_new, start, n_new, plan, pos, rows=rows)
        m = _bind or _native()
        at = 0 if plan is None else plan.address
        if rows is None and self.scales is None:
            f, args = m.append, (*self._at, k_new, v_new, start, n_new, at, pos)
        else:
            f, args = m.store, (*self._any, k_new, v_new, start, n_new, at, pos, rows)
        rc = f(*args)
        if rc:
            _again(rc, self.device, f, args)

    def read(self, first, n: int, lens, dtype=None, out_k=None, out_v=None, stream=None):
        """The positions first[b] .. first[b] + n - 1 of every sequence (first, lens int32
        [B]; lens: positions appended so far) as K, V [B, Hkv, n, d] of dtype (None: the
        cache's, bf16 for an 8-bit cache); 0 where the cache does not hold a position."""
        if stream is not None:
            return _on_stream(stream, self.device, self.read, first, n, lens, dtype, out_k, out_v)
        m = _bind or _native()
        if dtype is None:
            dtype = self._dtype if out_k is None else out_k.dtype
        args = (*self._any, self.k, first, n, lens, dtype, out_k, out_v)
        r = m.read_back(*args)
        return _again(r, self.device, m.read_back, args) if type(r) is int else r

    def decode(self, q, lens, scale: float, out=None, lse=None, stream=None):
        """Attention of q [B, Hq, d] at the positions lens - 1 (int32 [B]); returns O
        [B, Hq, d].  lse: None or an fp32 tensor [B, Hq] to fill."""
        if stream is not None:
            return _on_stream(stream, self.device, self.decode, q, lens, scale, out, lse)
        m = _bind or _native()
        if self.scales is not None:
            args = (*self._any, q, lens, scale, out, lse)
            r = m.decode_any(*args)
            return _again(r, self.device, m.decode_any, args) if type(r) is int else r
        ws = self._ws.get(q.shape[1])
        if ws is not None:
            r = m.decode(*self._at, q, lens, scale, out, lse, *ws)
            if type(r) is not int or r not in (m.OTHER_DEVICE, m.OTHER_STREAM):
                return r if type(r) is not int else _check(r)
        return self._decode_here(q, lens, scale, out, lse)

    def tree(self, q, k_new, v_new, lens, scale: float, parents=None, n_new=None, out=None, lse=None, algo=PSA_ALGO_AUTO,
             stream=None):
        """Attention of T new tokens per sequence, q [B, Hq, T, d] with k_new, v_new [B, Hkv,
        T, d], over the cache's first lens positions (int32 [B]) and over each other.  parents:
        int32 [B, T] or [T], each token's parent (below it; -1: none), or None for a run of
        tokens; n_new int32 [B] or None: how many of them are there.  Returns O (q's layout).
        Over an 8-bit cache whose scales are no powers of two the tensor cores' kernel rounds
        codes times scale to bf16, algo=PSA_ALGO_SIMT does not.
        lse: None or an fp32 tensor [B, Hq, T] to fill.  The cache is not changed: see
        append(rows=...).  See psa_win_tree_attn in include/psa_attn.h."""
        if stream is not None:
            return _on_stream(stream, self.device, self.tree, q, k_new, v_new, lens, scale, parents, n_new, out, lse, algo)
        m = _bind or _native()
        args = (*self._any, q, k_new, v_new, lens, scale, parents, n_new, out, lse, algo)
        r = m.tree(*args)
        return _again(r, self.device, m.tree, args) if type(r) is int else r

    def _decode_here(self, q, lens, scale, out, lse):
        """decode() with the workspace of the current stream of the cache's device."""
        import torch
        H = q.shape[1]
        with torch.cuda.device(self.device if self.device.type == "cuda" else -1):
            at = H, torch.cuda.current_stream().cuda_stream if self.device.type == "cuda" else 0
            ws = self._all.get(at)
            if ws is None:
                n = int(lib().psa_win_decode_workspace_bytes(self.c, H))
                ws = self._all[at] = (torch.empty(n, dtype=torch.uint8, device=self.device) if n else None, n, at[1])
            self._ws[H] = ws
            r = _bind.decode(*self._at, q, lens, scale, out, lse, *ws)
        return r if type(r) is not int else _check(r)

"""Python binding of libcla.so (ctypes), with the C entry points' names.

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  If the
shared library has not been built the import of a function fails loudly;
there is no CPU fallback.

All tensors must be CUDA tensors, contiguous, with the dtype the C ABI names
(float32, or bfloat16 passed as its bit pattern; float16 too where an entry
point takes a dtype).  The window_attn_* tensors may be strided over batch,
heads and tokens.  Outputs and the workspace are allocated with torch when not
supplied.  `stream` is the stream of the call, the current one by default; what
another stream has to write first is the caller's to wait for.  That holds for
a buffer the caller makes as well, a *_ckpt function's among them: its memory
is ready for a call on another stream once that stream has waited for the
current one.  What a call allocates itself needs no such wait.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcla.so")
_lock = threading.Lock()
_lib = None

CLA_OK = 0
SELECTIVE_CKPT_CHUNK = 16


class ClaError(RuntimeError):
    def __init__(self, fn, status, message):
        super().__init__(f"{fn}: {status_string(status)}: {message}")
        self.status = status


def lib():
    """The loaded libcla.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with chunkwise_linear_attention_gb300.build.build() "
                    "(needs nvcc); there is no fallback implementation")
            L = ctypes.CDLL(LIB_PATH)
            P, I64, SZ, INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
            F = ctypes.c_float
            sig = {
                "cla_status_string": ([INT], ctypes.c_char_p),
                "cla_last_error_message": ([], ctypes.c_char_p),
                "cla_check_status": ([P, P], INT),
                "cla_selftest_wait_timeout": ([P, SZ, P], INT),
                "cla_scan_diag_workspace_size": ([I64, I64, I64], SZ),
                "cla_scan_diag_fwd": ([P, P, P, P, P, I64, I64, I64, P, SZ, P], INT),
                "cla_scan_diag_fwd_blelloch": ([P, P, P, P, P, I64, I64, I64, P, SZ, P], INT),
                "cla_scan_diag_bwd": ([P] * 9 + [I64, I64, I64, P, SZ, P], INT),
                "cla_scan_diag_fwd_noalloc": ([P, P, P, P, P, I64, I64, I64, P], INT),
                "cla_scan_diag_noalloc_check_status": ([P], INT),
                "cla_selective_scan_workspace_size": ([I64, I64, I64, I64], SZ),
                "cla_selective_scan_ckpt_elems": ([I64, I64, I64, I64], SZ),
                "cla_selective_scan_fwd": ([P] * 9 + [I64] * 4 + [P, SZ, P], INT),
                "cla_selective_scan_bwd": ([P] * 15 + [I64] * 4 + [P, SZ, P], INT),
                "cla_chunk_la_workspace_size": ([I64] * 5 + [INT], SZ),
                "cla_chunk_la_fwd": ([P] * 7 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_chunk_la_bwd": ([P] * 12 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_chunk_la_ckpt_size": ([I64] * 5 + [INT], SZ),
                "cla_chunk_la_fwd_ckpt": ([P] * 8 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_chunk_la_bwd_ckpt": ([P] * 13 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_gla_workspace_size": ([I64] * 5 + [INT], SZ),
                "cla_gla_fwd": ([P] * 7 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_gla_bwd_workspace_size": ([I64] * 5 + [INT], SZ),
                "cla_gla_bwd": ([P] * 12 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_gla_ckpt_size": ([I64] * 5 + [INT], SZ),
                "cla_gla_fwd_ckpt": ([P] * 8 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_gla_bwd_ckpt": ([P] * 13 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_decay_total": ([P, P, I64, I64, I64, P], INT),
                "cla_delta_workspace_size": ([I64] * 5 + [INT], SZ),
                "cla_delta_fwd": ([P] * 8 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_delta_bwd_workspace_size": ([I64] * 5 + [INT], SZ),
                "cla_delta_bwd": ([P] * 14 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_delta_ckpt_size": ([I64] * 5 + [INT], SZ),
                "cla_delta_fwd_ckpt": ([P] * 9 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_delta_bwd_ckpt": ([P] * 15 + [I64] * 5 + [INT, P, SZ, P], INT),
                "cla_state_compose": ([P] * 4 + [I64] * 7 + [P], INT),
                "cla_gated_scan_ckpt_elems": ([I64, I64, I64], SZ),
                "cla_gated_scan_workspace_size": ([I64, I64, I64], SZ),
                "cla_gated_scan_fwd": ([P] * 10 + [F, INT] + [I64] * 3 + [P, SZ, P], INT),
                "cla_gated_scan_bwd": ([P] * 15 + [F, INT] + [I64] * 3 + [P, SZ, P], INT),
                "cla_gated_scan_step": ([P] * 7 + [F, INT, I64, I64, P], INT),
                "cla_window_attn_workspace_size": ([I64] * 7, SZ),
                "cla_window_attn_fwd": ([P] * 6 + [F, I64, I64, INT] + [I64] * 5 + [P, P, SZ, P], INT),
                "cla_window_attn_bwd_workspace_size": ([I64] * 7, SZ),
                "cla_window_attn_bwd": ([P] * 10 + [F, I64, I64, INT] + [I64] * 5 + [P, P, SZ, P], INT),
                "cla_window_cache_write": ([P] * 5 + [I64, I64, INT] + [I64] * 4 + [P, P], INT),
                "cla_window_attn_step": ([P] * 7 + [F, I64, I64, INT] + [I64] * 4 + [P, P], INT),
                "cla_window_cache8_write": ([P] * 7 + [I64, I64, INT] + [I64] * 4 + [P, P], INT),
                "cla_window_attn_step8": ([P] * 9 + [F, I64, I64, INT] + [I64] * 4 + [P, P, SZ, P], INT),
                "cla_window_attn_step8_workspace_size": ([I64] * 6, SZ),
                "cla_qk_norm_rope_fwd": ([P] * 9 + [F, I64, INT, INT] + [I64] * 5 + [P, P], INT),
                "cla_qk_norm_rope_bwd_workspace_size": ([I64] * 5, SZ),
                "cla_qk_norm_rope_bwd": ([P] * 13 + [F, I64, INT, INT] + [I64] * 5 + [P, P, SZ, P], INT),
                "cla_delta_step": ([P] * 8 + [INT] + [I64] * 6 + [P, P], INT),
            }
            for name, (args, res) in sig.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().cla_status_string(int(status)).decode()


def last_error_message() -> str:
    return lib().cla_last_error_message().decode()


def _check(fn: str, status: int) -> None:
    if status != CLA_OK:
        raise ClaError(fn, status, last_error_message())


def _stream(stream, device=None):
    """The cudaStream_t to launch on: `stream` (a torch.cuda.Stream or a raw handle), else the
    current stream of `device` (else of the current device)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _other_stream(stream, device):
    """`stream` (a torch.cuda.Stream or a raw handle) as a torch.cuda.Stream of `device`; None if it is the current one."""
    handle = _stream(stream, device).value or 0  # refuses a stream of another device
    if handle == 1:  # cudaStreamLegacy: the device's default stream, as 0 is
        handle = 0
    if handle == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _dims(t, n, name):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")
    return tuple(t.shape)


_ALL = "all"


def _T(t, dtype, name, shape=None, strided=False):
    """A tensor argument of an entry point (None stays NULL), checked by _launch for what the
    C ABI cannot check: dtype and shape (the sizes the call passes), then device and layout.
    strided: the entry point takes the outer strides; _ALL: the last dimension's too.
    A plain tuple: a call makes up to fifteen of them."""
    return (t, dtype, name, shape, strided)


def _check_meta(t, dtype, name, shape, strided):
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_place(device, t, dtype, name, shape, strided):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's first tensor on {device}")
    if strided:  # the entry point takes the outer strides
        if t.shape[-1] > 1 and t.stride(-1) != 1 and strided is not _ALL:
            raise ValueError(f"{name} must be contiguous in its last dimension")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _nbytes(t):
    return t.numel() * t.element_size()


def _ws(nbytes, device, workspace, minimum=None):
    """A workspace of nbytes (allocated when not given); a given one needs at least `minimum`
    bytes (default nbytes) -- the entry points that take less than their size query's amount."""
    if workspace is None:
        workspace = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    need = nbytes if minimum is None else minimum
    if _nbytes(workspace) < need:
        raise ValueError(f"workspace of {_nbytes(workspace)} bytes < {need} needed")
    return workspace


def _out(t, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else t


def _own_memory(call):
    """An entry point that allocates.  Where its stream is named and not the current one, it allocates on that stream, so
    that it cannot be given a block that was freed while queued work of the current stream still uses it; what it
    returns is used on the current stream, and not given out again before that is done with it either."""
    @functools.wraps(call)
    def entry(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        device = next((a.device for a in (*args, *kw.values()) if isinstance(a, torch.Tensor)), None)
        if device is None or device.type != "cuda":
            return call(*args, stream=stream, **kw)
        on = _other_stream(stream, device)
        if on is None:
            return call(*args, stream=stream, **kw)
        current = torch.cuda.current_stream(device)
        with torch.cuda.stream(on):
            out = call(*args, stream=stream, **kw)
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(current)
        return out
    return entry


def _launch(fn, device, args, stream):
    """Calls entry point `fn` with the tensors' device current: `args` are plain values and _T
    tensor arguments, every one of which is checked (dtype and shape of all of them first)
    before its pointer is taken; raises ClaError on a non-OK status."""
    cargs, good = [], device.type == "cuda"
    for a in args:  # one quick pass; what does not pass it is looked at again for its message
        if type(a) is tuple:
            t, dtype, _, shape, strided = a
            if t is None:
                a = None
            else:
                if ((t.dtype is not dtype and dtype is not None) or (shape is not None and t.shape != shape)
                        or t.device != device or not (t.is_contiguous() or strided and (t.stride(-1) == 1 or strided is _ALL))):
                    good = False
                a = t.data_ptr()
        cargs.append(a)
    if not good:
        tensors = [a for a in args if type(a) is tuple and a[0] is not None]
        for a in tensors:
            _check_meta(*a)
        for a in tensors:
            _check_place(device, *a)
    handle = None if stream is None else _stream(stream, device)  # refuses a stream of another device
    if isinstance(stream, torch.cuda.Stream):
        # memory that was allocated on another stream is not given out again before this stream is done
        # with it; with a raw handle that is the caller's part
        for a in args:
            if type(a) is tuple and a[0] is not None:
                a[0].record_stream(stream)
    call = getattr(_lib or lib(), fn)
    index = device.index
    if index == torch._C._cuda_getDevice():
        # the current stream's handle, without the Stream object around it
        status = call(*cargs, torch._C._cuda_getCurrentRawStream(index) if handle is None else handle)
    else:
        with torch.cuda.device(device):
            status = call(*cargs, _stream(None, device) if handle is None else handle)
    if status != CLA_OK:
        _check(fn, status)


def check_status(workspace, stream=None) -> None:
    """Synchronise and raise if a kernel of the last call on `workspace` gave up a wait."""
    _launch("cla_check_status", workspace.device, (_T(workspace, None, "workspace"),), stream)


def selftest_wait_timeout(workspace, stream=None) -> None:
    """Launch the bounded-wait self-test on `workspace` (16-byte aligned, at least the
    256-byte workspace header)."""
    _launch("cla_selftest_wait_timeout", workspace.device,
            (_T(workspace, None, "workspace"), _nbytes(workspace)), stream)


# ---------------------------------------------------------------- diagonal scan
def scan_diag_workspace_size(B, T, D) -> int:
    return int(lib().cla_scan_diag_workspace_size(B, T, D))


def _scan_fwd(fn, a, b, h0, h, hT, workspace, stream, with_ws=True):
    B, T, D = _dims(a, 3, "a")
    dev = a.device
    f32 = torch.float32
    h = _out(h, (B, T, D), f32, dev)
    hT = _out(hT, (B, D), f32, dev)
    bt, bd = (B, T, D), (B, D)
    args = (_T(a, f32, "a", bt), _T(b, f32, "b", bt), _T(h0, f32, "h0", bd),
            _T(h, f32, "h", bt), _T(hT, f32, "hT", bd), B, T, D)
    if with_ws:
        ws = _ws(scan_diag_workspace_size(B, T, D), dev, workspace)
        args += (_T(ws, None, "workspace"), _nbytes(ws))
    _launch(fn, dev, args, stream)
    return h, hT


@_own_memory
def scan_diag_fwd(a, b, h0=None, *, h=None, hT=None, workspace=None, stream=None):
    """h_t = a_t h_{t-1} + b_t over axis 1 of [B, T, D] (fp32); returns (h, hT)."""
    return _scan_fwd("cla_scan_diag_fwd", a, b, h0, h, hT, workspace, stream)


@_own_memory
def scan_diag_fwd_blelloch(a, b, h0=None, *, h=None, hT=None, workspace=None, stream=None):
    """scan_diag_fwd with a Blelloch tree across the runs of a chunk (a measured
    alternative to Hillis-Steele); returns (h, hT)."""
    return _scan_fwd("cla_scan_diag_fwd_blelloch", a, b, h0, h, hT, workspace, stream)


@_own_memory
def scan_diag_fwd_noalloc(a, b, h0=None, *, h=None, hT=None, stream=None):
    """scan_diag_fwd without a workspace: the library's static scratch array
    is used (limited size; overlapping calls race).  Returns (h, hT)."""
    return _scan_fwd("cla_scan_diag_fwd_noalloc", a, b, h0, h, hT, None, stream, with_ws=False)


def scan_diag_noalloc_check_status(stream=None, device=None) -> None:
    """Synchronise and raise if the last scan_diag_fwd_noalloc on `device` gave up a wait."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        _check("cla_scan_diag_noalloc_check_status",
               lib().cla_scan_diag_noalloc_check_status(_stream(stream, dev)))


@_own_memory
def scan_diag_bwd(a, b, h0, h, dh, dhT=None, *, da=None, db=None, dh0=None, workspace=None, stream=None):
    """Adjoint of scan_diag_fwd; returns (da, db, dh0).  h: the forward's states, or None to
    recompute them from (a, b, h0) (then b is required; b may be None when h is given)."""
    B, T, D = _dims(a, 3, "a")
    dev = a.device
    f32 = torch.float32
    da = _out(da, (B, T, D), f32, dev)
    db = _out(db, (B, T, D), f32, dev)
    dh0 = _out(dh0, (B, D), f32, dev)
    ws = _ws(scan_diag_workspace_size(B, T, D), dev, workspace)
    bt, bd = (B, T, D), (B, D)
    _launch("cla_scan_diag_bwd", dev, (
        _T(a, f32, "a", bt), _T(b, f32, "b", bt), _T(h0, f32, "h0", bd), _T(h, f32, "h", bt),
        _T(dh, f32, "dh", bt), _T(dhT, f32, "dhT", bd), _T(da, f32, "da", bt),
        _T(db, f32, "db", bt), _T(dh0, f32, "dh0", bd), B, T, D,
        _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return da, db, dh0


# ---------------------------------------------------------------- selective scan
def selective_scan_workspace_size(B, T, D, N) -> int:
    return int(lib().cla_selective_scan_workspace_size(B, T, D, N))


def selective_scan_ckpt_elems(B, T, D, N) -> int:
    return int(lib().cla_selective_scan_ckpt_elems(B, T, D, N))


def _sel_ckpt_arg(ckpt, B, T, D, N):
    if ckpt is None:
        return None
    need = selective_scan_ckpt_elems(B, T, D, N)
    if ckpt.numel() < need:
        raise ValueError(f"ckpt: need at least {need} fp32 values, got {ckpt.numel()}")
    return _T(ckpt, torch.float32, "ckpt")


@_own_memory
def selective_scan_fwd(x, delta, A, Bm, Cm, h0=None, *, y=None, hT=None, ckpt=None, want_ckpt=True,
                       workspace=None, stream=None):
    """Selective scan forward; returns (y, hT, ckpt)."""
    B, T, D = _dims(x, 3, "x")
    N = _dims(A, 2, "A")[1]
    dev = x.device
    f32, bf16 = torch.float32, torch.bfloat16
    y = _out(y, (B, T, D), f32, dev)
    hT = _out(hT, (B, D, N), f32, dev)
    if ckpt is None and want_ckpt:
        ckpt = torch.empty(selective_scan_ckpt_elems(B, T, D, N), dtype=f32, device=dev)
    ws = _ws(selective_scan_workspace_size(B, T, D, N), dev, workspace)
    btd, btn, bdn = (B, T, D), (B, T, N), (B, D, N)
    _launch("cla_selective_scan_fwd", dev, (
        _T(x, bf16, "x", btd), _T(delta, f32, "delta", btd), _T(A, f32, "A", (D, N)),
        _T(Bm, bf16, "Bm", btn), _T(Cm, bf16, "Cm", btn), _T(h0, f32, "h0", bdn),
        _T(y, f32, "y", btd), _T(hT, f32, "hT", bdn), _sel_ckpt_arg(ckpt, B, T, D, N),
        B, T, D, N, _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return y, hT, ckpt


@_own_memory
def selective_scan_bwd(x, delta, A, Bm, Cm, h0, ckpt, dy, dhT=None, *, dx=None, ddelta=None, dA=None,
                       dB=None, dC=None, dh0=None, want_dA=True, want_dh0=True, workspace=None, stream=None):
    """Selective scan backward; returns (dx, ddelta, dA, dB, dC, dh0)."""
    B, T, D = _dims(x, 3, "x")
    N = _dims(A, 2, "A")[1]
    dev = x.device
    f32, bf16 = torch.float32, torch.bfloat16
    dx = _out(dx, (B, T, D), f32, dev)
    ddelta = _out(ddelta, (B, T, D), f32, dev)
    dA = _out(dA, (D, N), f32, dev) if (want_dA or dA is not None) else None
    dB = _out(dB, (B, T, N), f32, dev)
    dC = _out(dC, (B, T, N), f32, dev)
    dh0 = _out(dh0, (B, D, N), f32, dev) if (want_dh0 or dh0 is not None) else None
    ws = _ws(selective_scan_workspace_size(B, T, D, N), dev, workspace)
    btd, btn, bdn = (B, T, D), (B, T, N), (B, D, N)
    _launch("cla_selective_scan_bwd", dev, (
        _T(x, bf16, "x", btd), _T(delta, f32, "delta", btd), _T(A, f32, "A", (D, N)),
        _T(Bm, bf16, "Bm", btn), _T(Cm, bf16, "Cm", btn), _T(h0, f32, "h0", bdn),
        _sel_ckpt_arg(ckpt, B, T, D, N), _T(dy, f32, "dy", btd), _T(dhT, f32, "dhT", bdn),
        _T(dx, f32, "dx", btd), _T(ddelta, f32, "ddelta", btd), _T(dA, f32, "dA", (D, N)),
        _T(dB, f32, "dB", btn), _T(dC, f32, "dC", btn), _T(dh0, f32, "dh0", bdn),
        B, T, D, N, _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return dx, ddelta, dA, dB, dC, dh0


# ---------------------------------------------------------------- chunkwise linear attention
def chunk_la_workspace_size(B, H, T, dim_k, dim_v, chunk) -> int:
    return int(lib().cla_chunk_la_workspace_size(B, H, T, dim_k, dim_v, int(chunk)))


def chunk_la_ckpt_size(B, H, T, dim_k, dim_v, chunk) -> int:
    """Bytes of the segment-state checkpoint the forward can save for the backward."""
    return int(lib().cla_chunk_la_ckpt_size(B, H, T, dim_k, dim_v, int(chunk)))


def chunk_la_ckpt(q, v, *, chunk=64):
    """A device buffer (fp32) for the checkpoint of a forward on q [B, H, T, dk], v [.., dv]."""
    B, H, T, dk = _dims(q, 4, "q")
    n = chunk_la_ckpt_size(B, H, T, dk, v.shape[-1], chunk) // 4
    return torch.empty(max(n, 1), dtype=torch.float32, device=q.device)


def _ckpt_arg(ckpt, B, H, T, dk, dv, chunk):
    if ckpt is None:
        return None
    need = chunk_la_ckpt_size(B, H, T, dk, dv, chunk)
    if _nbytes(ckpt) < need:
        raise ValueError(f"ckpt: need at least {need} bytes, got {_nbytes(ckpt)}")
    return _T(ckpt, torch.float32, "ckpt")


@_own_memory
def chunk_la_fwd(q, k, v, log_decay, S0=None, *, chunk=64, o=None, ST=None, ckpt=None, workspace=None,
                 stream=None):
    """Chunkwise decayed linear attention forward; returns (o, ST).  With ckpt (see
    chunk_la_ckpt) it also saves the state entering each segment for chunk_la_bwd."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 4, "v")[3]
    dev = q.device
    f32, bf16 = torch.float32, torch.bfloat16
    o = _out(o, (B, H, T, dv), f32, dev)
    ST = _out(ST, (B, H, dk, dv), f32, dev)
    ws = _ws(chunk_la_workspace_size(B, H, T, dk, dv, chunk), dev, workspace)
    tk, tv, st = (B, H, T, dk), (B, H, T, dv), (B, H, dk, dv)
    args = (_T(q, bf16, "q", tk), _T(k, bf16, "k", tk), _T(v, bf16, "v", tv),
            _T(log_decay, f32, "log_decay", (B, H, T)), _T(S0, f32, "S0", st),
            _T(o, f32, "o", tv), _T(ST, f32, "ST", st))
    tail = (B, H, T, dk, dv, int(chunk), _T(ws, None, "workspace"), _nbytes(ws))
    if ckpt is None:
        _launch("cla_chunk_la_fwd", dev, args + tail, stream)
    else:
        _launch("cla_chunk_la_fwd_ckpt", dev, args + (_ckpt_arg(ckpt, B, H, T, dk, dv, chunk),) + tail,
                stream)
    return o, ST


@_own_memory
def chunk_la_bwd(q, k, v, log_decay, S0, dO, dST=None, *, chunk=64, dq=None, dk=None, dv=None,
                 dlog_decay=None, dS0=None, ckpt=None, workspace=None, stream=None):
    """Chunkwise decayed linear attention backward; returns (dq, dk, dv, dlog_decay, dS0).  ckpt:
    the checkpoint a chunk_la_fwd on the same inputs saved (its states are then not rebuilt)."""
    B, H, T, dkk = _dims(q, 4, "q")
    dvv = _dims(v, 4, "v")[3]
    dev = q.device
    f32, bf16 = torch.float32, torch.bfloat16
    dq = _out(dq, (B, H, T, dkk), f32, dev)
    dk = _out(dk, (B, H, T, dkk), f32, dev)
    dv = _out(dv, (B, H, T, dvv), f32, dev)
    dlog_decay = _out(dlog_decay, (B, H, T), f32, dev)
    dS0 = _out(dS0, (B, H, dkk, dvv), f32, dev)
    ws = _ws(chunk_la_workspace_size(B, H, T, dkk, dvv, chunk), dev, workspace)
    tk, tv, st, bht = (B, H, T, dkk), (B, H, T, dvv), (B, H, dkk, dvv), (B, H, T)
    args = (_T(q, bf16, "q", tk), _T(k, bf16, "k", tk), _T(v, bf16, "v", tv),
            _T(log_decay, f32, "log_decay", bht), _T(S0, f32, "S0", st),
            _T(dO, bf16, "dO", tv), _T(dST, f32, "dST", st), _T(dq, f32, "dq", tk),
            _T(dk, f32, "dk", tk), _T(dv, f32, "dv", tv),
            _T(dlog_decay, f32, "dlog_decay", bht), _T(dS0, f32, "dS0", st))
    tail = (B, H, T, dkk, dvv, int(chunk), _T(ws, None, "workspace"), _nbytes(ws))
    if ckpt is None:
        _launch("cla_chunk_la_bwd", dev, args + tail, stream)
    else:
        _launch("cla_chunk_la_bwd_ckpt", dev, args + (_ckpt_arg(ckpt, B, H, T, dkk, dvv, chunk),) + tail,
                stream)
    return dq, dk, dv, dlog_decay, dS0


# ---------------------------------------------------------------- gated linear attention
def gla_workspace_size(B, H, T, dim_k, dim_v, chunk=64) -> int:
    return int(lib().cla_gla_workspace_size(B, H, T, dim_k, dim_v, int(chunk)))


def gla_ckpt_size(B, H, T, dim_k, dim_v, chunk=64) -> int:
    """Bytes of the segment-state checkpoint the GLA forward can save for the backward."""
    return int(lib().cla_gla_ckpt_size(B, H, T, dim_k, dim_v, int(chunk)))


def gla_ckpt(q, v, *, chunk=64):
    """A device buffer (fp32) for the checkpoint of a gla_fwd on q [B, H, T, dk], v [.., dv]."""
    B, H, T, dk = _dims(q, 4, "q")
    n = gla_ckpt_size(B, H, T, dk, v.shape[-1], chunk) // 4
    return torch.empty(max(n, 1), dtype=torch.float32, device=q.device)


def _gla_ckpt_arg(ckpt, B, H, T, dk, dv, chunk):
    need = gla_ckpt_size(B, H, T, dk, dv, chunk)
    if _nbytes(ckpt) < need:
        raise ValueError(f"ckpt: need at least {need} bytes, got {_nbytes(ckpt)}")
    return _T(ckpt, torch.float32, "ckpt")


@_own_memory
def gla_fwd(q, k, v, log_decay, S0=None, *, chunk=64, o=None, ST=None, ckpt=None, workspace=None, stream=None):
    """Gated linear attention forward (one decay per key dimension: log_decay [B, H, T, dk]);
    returns (o, ST).  check_status(workspace) reports decays outside the kernel's range.  With
    ckpt (see gla_ckpt) it also saves the state entering every segment for gla_bwd."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 4, "v")[3]
    dev = q.device
    f32, bf16 = torch.float32, torch.bfloat16
    o = _out(o, (B, H, T, dv), f32, dev)
    ST = _out(ST, (B, H, dk, dv), f32, dev)
    ws = _ws(gla_workspace_size(B, H, T, dk, dv, chunk), dev, workspace)
    tk, tv, st = (B, H, T, dk), (B, H, T, dv), (B, H, dk, dv)
    args = (_T(q, bf16, "q", tk), _T(k, bf16, "k", tk), _T(v, bf16, "v", tv),
            _T(log_decay, f32, "log_decay", tk), _T(S0, f32, "S0", st),
            _T(o, f32, "o", tv), _T(ST, f32, "ST", st))
    tail = (B, H, T, dk, dv, int(chunk), _T(ws, None, "workspace"), _nbytes(ws))
    if ckpt is None:
        _launch("cla_gla_fwd", dev, args + tail, stream)
    else:
        _launch("cla_gla_fwd_ckpt", dev, args + (_gla_ckpt_arg(ckpt, B, H, T, dk, dv, chunk),) + tail, stream)
    return o, ST


def gla_bwd_workspace_size(B, H, T, dim_k, dim_v, chunk=64) -> int:
    return int(lib().cla_gla_bwd_workspace_size(B, H, T, dim_k, dim_v, int(chunk)))


@_own_memory
def gla_bwd(q, k, v, log_decay, S0, dO, dST=None, *, chunk=64, dq=None, dk=None, dv=None, dlog_decay=None,
            dS0=None, ckpt=None, workspace=None, stream=None):
    """Gated linear attention backward; returns (dq, dk, dv, dlog_decay [B, H, T, dk], dS0).  ckpt:
    the checkpoint a gla_fwd(..., ckpt=) on the same inputs saved (its dq traversal then starts
    from it)."""
    B, H, T, dkk = _dims(q, 4, "q")
    dvv = _dims(v, 4, "v")[3]
    dev = q.device
    f32, bf16 = torch.float32, torch.bfloat16
    dq = _out(dq, (B, H, T, dkk), f32, dev)
    dk = _out(dk, (B, H, T, dkk), f32, dev)
    dv = _out(dv, (B, H, T, dvv), f32, dev)
    dlog_decay = _out(dlog_decay, (B, H, T, dkk), f32, dev)
    dS0 = _out(dS0, (B, H, dkk, dvv), f32, dev)
    ws = _ws(gla_bwd_workspace_size(B, H, T, dkk, dvv, chunk), dev, workspace)
    tk, tv, st = (B, H, T, dkk), (B, H, T, dvv), (B, H, dkk, dvv)
    args = (_T(q, bf16, "q", tk), _T(k, bf16, "k", tk), _T(v, bf16, "v", tv),
            _T(log_decay, f32, "log_decay", tk), _T(S0, f32, "S0", st), _T(dO, bf16, "dO", tv),
            _T(dST, f32, "dST", st), _T(dq, f32, "dq", tk), _T(dk, f32, "dk", tk), _T(dv, f32, "dv", tv),
            _T(dlog_decay, f32, "dlog_decay", tk), _T(dS0, f32, "dS0", st))
    tail = (B, H, T, dkk, dvv, int(chunk), _T(ws, None, "workspace"), _nbytes(ws))
    if ckpt is None:
        _launch("cla_gla_bwd", dev, args + tail, stream)
    else:
        _launch("cla_gla_bwd_ckpt", dev, args + (_gla_ckpt_arg(ckpt, B, H, T, dkk, dvv, chunk),) + tail, stream)
    return dq, dk, dv, dlog_decay, dS0


# ---------------------------------------------------------------- state passing between slices
@_own_memory
def decay_total(log_decay, *, alpha=None, stream=None):
    """exp of the sum over the slice of log_decay: [B, H, T] -> [B, H] (one decay per head) or
    [B, H, T, dk] -> [B, H, dk] (gated)."""
    if log_decay.dim() == 3:
        B, H, T = log_decay.shape
        A, shape = 1, (B, H)
    else:
        B, H, T, A = _dims(log_decay, 4, "log_decay")
        shape = (B, H, A)
    dev = log_decay.device
    alpha = _out(alpha, shape, torch.float32, dev)
    _launch("cla_decay_total", dev, (_T(log_decay, torch.float32, "log_decay", tuple(log_decay.shape)),
                                     _T(alpha, torch.float32, "alpha", shape), B * H, T, A), stream)
    return alpha


@_own_memory
def state_compose(alphas, dSs, edge, first, count, step, *, out=None, stream=None):
    """Fold acc <- diag(alpha_j) acc + dS_j over j = first + c * step (c < count) from edge.
    alphas [P, B, H] or [P, B, H, dk]; dSs [P, B, H, dk, dv]; edge [B, H, dk, dv] or None."""
    P, B, H, dk, dv = _dims(dSs, 5, "dSs")
    A = 1 if alphas.dim() == 3 else alphas.shape[3]
    dev = dSs.device
    out = _out(out, (B, H, dk, dv), torch.float32, dev)
    st = (B, H, dk, dv)
    _launch("cla_state_compose", dev, (
        _T(alphas, torch.float32, "alphas", (P, B, H) if A == 1 else (P, B, H, A)),
        _T(dSs, torch.float32, "dSs", (P, B, H, dk, dv)), _T(edge, torch.float32, "edge", st),
        _T(out, torch.float32, "out", st), P, B * H, dk * dv, A, int(first), int(count), int(step)), stream)
    return out


# ---------------------------------------------------------------- delta rule (Gated DeltaNet)
def delta_workspace_size(B, H, T, dim_k, dim_v, chunk=64) -> int:
    return int(lib().cla_delta_workspace_size(B, H, T, dim_k, dim_v, int(chunk)))


def delta_ckpt_size(B, H, T, dim_k, dim_v, chunk=64) -> int:
    """Bytes of the checkpoint (the state entering every chunk) the forward can save for the backward."""
    return int(lib().cla_delta_ckpt_size(B, H, T, dim_k, dim_v, int(chunk)))


def delta_ckpt(q, v, *, chunk=64):
    """A device buffer (fp32) for the checkpoint of a delta_fwd on q [B, H, T, dk], v [.., dv]."""
    B, H, T, dk = _dims(q, 4, "q")
    n = delta_ckpt_size(B, H, T, dk, v.shape[-1], chunk) // 4
    return torch.empty(max(n, 1), dtype=torch.float32, device=q.device)


def _delta_ckpt_arg(ckpt, B, H, T, dk, dv, chunk):
    need = delta_ckpt_size(B, H, T, dk, dv, chunk)
    if _nbytes(ckpt) < need:
        raise ValueError(f"ckpt: need at least {need} bytes, got {_nbytes(ckpt)}")
    return _T(ckpt, torch.float32, "ckpt")


@_own_memory
def delta_fwd(q, k, v, log_decay, beta, S0=None, *, chunk=64, o=None, ST=None, ckpt=None, workspace=None,
              stream=None):
    """Delta rule with a decay per head: S_t = a_t (I - beta_t k_t^T k_t) S_{t-1} + beta_t k_t^T v_t,
    o_t = q_t S_t; log_decay, beta [B, H, T].  Returns (o, ST).  With ckpt (see delta_ckpt) it also
    saves the state entering every chunk for delta_bwd.  A given workspace needs 256 bytes; the
    size query's amount lets the chunks' (I + A)^-1 be formed beforehand, all at once."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 4, "v")[3]
    dev = q.device
    f32, bf16 = torch.float32, torch.bfloat16
    o = _out(o, (B, H, T, dv), f32, dev)
    ST = _out(ST, (B, H, dk, dv), f32, dev)
    ws = _ws(delta_workspace_size(B, H, T, dk, dv, chunk), dev, workspace, minimum=256)
    tk, tv, st, bht = (B, H, T, dk), (B, H, T, dv), (B, H, dk, dv), (B, H, T)
    args = (_T(q, bf16, "q", tk), _T(k, bf16, "k", tk), _T(v, bf16, "v", tv),
            _T(log_decay, f32, "log_decay", bht), _T(beta, f32, "beta", bht), _T(S0, f32, "S0", st),
            _T(o, f32, "o", tv), _T(ST, f32, "ST", st))
    tail = (B, H, T, dk, dv, int(chunk), _T(ws, None, "workspace"), _nbytes(ws))
    if ckpt is None:
        _launch("cla_delta_fwd", dev, args + tail, stream)
    else:
        _launch("cla_delta_fwd_ckpt", dev, args + (_delta_ckpt_arg(ckpt, B, H, T, dk, dv, chunk),) + tail, stream)
    return o, ST


def delta_bwd_workspace_size(B, H, T, dim_k, dim_v, chunk=64) -> int:
    return int(lib().cla_delta_bwd_workspace_size(B, H, T, dim_k, dim_v, int(chunk)))


@_own_memory
def delta_bwd(q, k, v, log_decay, beta, S0, dO, dST=None, *, chunk=64, dq=None, dk=None, dv=None,
              dlog_decay=None, dbeta=None, dS0=None, ckpt=None, workspace=None, stream=None):
    """Adjoint of delta_fwd (dO bf16 [B, H, T, dv]); returns (dq, dk, dv, dlog_decay, dbeta, dS0).  ckpt:
    the checkpoint a delta_fwd on the same inputs saved (the states are then not recomputed)."""
    B, H, T, dkk = _dims(q, 4, "q")
    dvv = _dims(v, 4, "v")[3]
    dev = q.device
    f32, bf16 = torch.float32, torch.bfloat16
    dq = _out(dq, (B, H, T, dkk), f32, dev)
    dk = _out(dk, (B, H, T, dkk), f32, dev)
    dv = _out(dv, (B, H, T, dvv), f32, dev)
    dlog_decay = _out(dlog_decay, (B, H, T), f32, dev)
    dbeta = _out(dbeta, (B, H, T), f32, dev)
    dS0 = _out(dS0, (B, H, dkk, dvv), f32, dev)
    need = delta_bwd_workspace_size(B, H, T, dkk, dvv, chunk)
    if ckpt is not None:  # no states in the workspace: the header and the partials only
        need = max(need - delta_ckpt_size(B, H, T, dkk, dvv, chunk), 256)
    ws = _ws(need, dev, workspace)
    tk, tv, st, bht = (B, H, T, dkk), (B, H, T, dvv), (B, H, dkk, dvv), (B, H, T)
    args = (_T(q, bf16, "q", tk), _T(k, bf16, "k", tk), _T(v, bf16, "v", tv),
            _T(log_decay, f32, "log_decay", bht), _T(beta, f32, "beta", bht), _T(S0, f32, "S0", st),
            _T(dO, bf16, "dO", tv), _T(dST, f32, "dST", st), _T(dq, f32, "dq", tk), _T(dk, f32, "dk", tk),
            _T(dv, f32, "dv", tv), _T(dlog_decay, f32, "dlog_decay", bht), _T(dbeta, f32, "dbeta", bht),
            _T(dS0, f32, "dS0", st))
    tail = (B, H, T, dkk, dvv, int(chunk), _T(ws, None, "workspace"), _nbytes(ws))
    if ckpt is None:
        _launch("cla_delta_bwd", dev, args + tail, stream)
    else:
        _launch("cla_delta_bwd_ckpt", dev, args + (_delta_ckpt_arg(ckpt, B, H, T, dkk, dvv, chunk),) + tail, stream)
    return dq, dk, dv, dlog_decay, dbeta, dS0


# ---------------------------------------------------------------- gated scan
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _dtype_code(t, name, allowed):
    if t.dtype not in allowed:
        raise ValueError(f"{name} must be one of {', '.join(map(str, allowed))}, got {t.dtype}")
    return _DTYPES[t.dtype]


def _reset_arg(reset, shape):
    """A reset mask: bool or uint8 (the C ABI reads bytes)."""
    return _T(reset, torch.bool if reset is not None and reset.dtype == torch.bool else torch.uint8, "reset", shape)


def gated_scan_workspace_size(B, T, D) -> int:
    return int(lib().cla_gated_scan_workspace_size(B, T, D))


def gated_scan_ckpt_elems(B, T, D) -> int:
    return int(lib().cla_gated_scan_ckpt_elems(B, T, D))


def gated_scan_ckpt(x):
    """A device buffer (fp32) for the checkpoint of a gated_scan_fwd on x [B, T, D]."""
    return torch.empty(max(gated_scan_ckpt_elems(*_dims(x, 3, "x")), 1), dtype=torch.float32, device=x.device)


def _gated_ckpt_arg(ckpt, B, T, D):
    need = gated_scan_ckpt_elems(B, T, D)
    if ckpt is not None and ckpt.numel() < need:
        raise ValueError(f"ckpt: need at least {need} fp32 values, got {ckpt.numel()}")
    return _T(ckpt, torch.float32, "ckpt")


@_own_memory
def gated_scan_fwd(x, rgate, igate, lam, h0=None, *, reset=None, lens=None, c=8.0, h=None, hT=None, ckpt=None,
                   workspace=None, stream=None):
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(igate_t) x_t with a = exp(-c softplus(lam) sigmoid(rgate)) over axis 1
    of [B, T, D] (fp32, bf16 or fp16); returns (h, hT).  reset [B, T]: tokens that start afresh; lens [B] int32: lengths
    of a right-padded batch.  With ckpt (see gated_scan_ckpt) it also saves states for gated_scan_bwd."""
    B, T, D = _dims(x, 3, "x")
    dev, dt, f32 = x.device, x.dtype, torch.float32
    code = _dtype_code(x, "x", _DTYPES)
    h = _out(h, (B, T, D), dt, dev)
    hT = _out(hT, (B, D), f32, dev)
    ws = _ws(gated_scan_workspace_size(B, T, D), dev, workspace)
    bt, bd = (B, T, D), (B, D)
    _launch("cla_gated_scan_fwd", dev, (
        _T(x, dt, "x", bt), _T(rgate, dt, "rgate", bt), _T(igate, dt, "igate", bt), _T(lam, f32, "lam", (D,)),
        _T(h0, f32, "h0", bd), _reset_arg(reset, (B, T)), _T(lens, torch.int32, "lens", (B,)), _T(h, dt, "h", bt),
        _T(hT, f32, "hT", bd), _gated_ckpt_arg(ckpt, B, T, D), float(c), code, B, T, D,
        _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return h, hT


@_own_memory
def gated_scan_bwd(x, rgate, igate, lam, h0, dh, dhT=None, *, reset=None, lens=None, c=8.0, dx=None, drgate=None,
                   digate=None, dlam=None, dh0=None, ckpt=None, workspace=None, stream=None):
    """Adjoint of gated_scan_fwd; returns (dx, drgate, digate, dlam, dh0).  ckpt: what a gated_scan_fwd on the same
    inputs saved, or None to rebuild the states."""
    B, T, D = _dims(x, 3, "x")
    dev, dt, f32 = x.device, x.dtype, torch.float32
    code = _dtype_code(x, "x", _DTYPES)
    bt, bd = (B, T, D), (B, D)
    dx, drgate, digate = (_out(t, bt, dt, dev) for t in (dx, drgate, digate))
    dlam = _out(dlam, (D,), f32, dev)
    dh0 = _out(dh0, bd, f32, dev)
    ws = _ws(gated_scan_workspace_size(B, T, D), dev, workspace)
    _launch("cla_gated_scan_bwd", dev, (
        _T(x, dt, "x", bt), _T(rgate, dt, "rgate", bt), _T(igate, dt, "igate", bt), _T(lam, f32, "lam", (D,)),
        _T(h0, f32, "h0", bd), _reset_arg(reset, (B, T)), _T(lens, torch.int32, "lens", (B,)),
        _gated_ckpt_arg(ckpt, B, T, D), _T(dh, dt, "dh", bt), _T(dhT, f32, "dhT", bd), _T(dx, dt, "dx", bt),
        _T(drgate, dt, "drgate", bt), _T(digate, dt, "digate", bt), _T(dlam, f32, "dlam", (D,)),
        _T(dh0, f32, "dh0", bd), float(c), code, B, T, D, _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return dx, drgate, digate, dlam, dh0


@_own_memory
def gated_scan_step(x, rgate, igate, lam, h, *, reset=None, c=8.0, y=None, stream=None):
    """One token of gated_scan_fwd for each of B sequences ([B, D]); updates the state h [B, D] fp32 in place and
    returns it rounded to x's dtype."""
    B, D = _dims(x, 2, "x")
    dt, dev, bd = x.dtype, x.device, (B, D)
    code = _dtype_code(x, "x", _DTYPES)
    y = _out(y, bd, dt, dev)
    _launch("cla_gated_scan_step", dev, (
        _T(x, dt, "x", bd), _T(rgate, dt, "rgate", bd), _T(igate, dt, "igate", bd), _T(lam, torch.float32, "lam", (D,)),
        _reset_arg(reset, (B,)), _T(h, torch.float32, "h", bd), _T(y, dt, "y", bd), float(c), code, B, D), stream)
    return y


# ---------------------------------------------------------------- sliding-window attention with sinks
_HALF = (torch.bfloat16, torch.float16)


def _strides(*tensors):
    """The tensors' outer strides as the C ABI takes them; None when all are dense."""
    for t in tensors:
        if not t.is_contiguous():
            break
    else:
        return None
    flat = ()
    for t in tensors:
        flat += t.stride()[:-1]
    return (ctypes.c_int64 * len(flat))(*flat)


def _counts(window, sinks):
    """Window and sinks as the C ABI's 64 bits hold them (ctypes would cut longer ones)."""
    out = int(window), int(sinks)
    if out != (window, sinks) or not -2 ** 63 <= min(out) <= max(out) < 2 ** 63:
        raise ValueError(f"window and sinks must be a whole number of 64 bits each, got {window} and {sinks}")
    return out


def _scale(scale, d):
    return float(d) ** -0.5 if scale is None else float(scale)


def window_attn_workspace_size(B, H, Hkv, T, d, window, sinks=0) -> int:
    return int(lib().cla_window_attn_workspace_size(B, H, Hkv, T, d, *_counts(window, sinks)))


@_own_memory
def window_attn_fwd(q, k, v, *, window, sinks=0, lens=None, scale=None, o=None, lse=None, workspace=None, stream=None):
    """Softmax attention of token t over s <= t with t - s < window or s < sinks: q [B, H, T, d], k and v
    [B, Hkv, T, d] (bf16 or fp16, d 64 or 128, H a multiple of Hkv; strided views are taken as they are).  lens [B]
    int32: lengths of a right-padded batch.  scale: d ** -0.5 when None.  Returns (o, lse [B, H, T] fp32)."""
    window, sinks = _counts(window, sinks)
    B, H, T, d = _dims(q, 4, "q")
    Hkv = _dims(k, 4, "k")[1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q, "q", _HALF)
    o = _out(o, (B, H, T, d), dt, dev)
    lse = _out(lse, (B, H, T), torch.float32, dev)
    ws = _ws(window_attn_workspace_size(B, H, Hkv, T, d, window, sinks), dev, workspace)
    hs, ks = (B, H, T, d), (B, Hkv, T, d)
    _launch("cla_window_attn_fwd", dev, (
        _T(q, dt, "q", hs, True), _T(k, dt, "k", ks, True), _T(v, dt, "v", ks, True),
        _T(lens, torch.int32, "lens", (B,)), _T(o, dt, "o", hs, True), _T(lse, torch.float32, "lse", (B, H, T)),
        _scale(scale, d), window, sinks, code, B, H, Hkv, T, d, _strides(q, k, v, o),
        _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return o, lse


def window_attn_bwd_workspace_size(B, H, Hkv, T, d, window, sinks=0) -> int:
    return int(lib().cla_window_attn_bwd_workspace_size(B, H, Hkv, T, d, *_counts(window, sinks)))


@_own_memory
def window_attn_bwd(q, k, v, o, lse, dO, *, window, sinks=0, lens=None, scale=None, dq=None, dk=None, dv=None,
                    workspace=None, stream=None):
    """Adjoint of window_attn_fwd from its outputs (o, lse) and dO; returns (dq, dk, dv)."""
    window, sinks = _counts(window, sinks)
    B, H, T, d = _dims(q, 4, "q")
    Hkv = _dims(k, 4, "k")[1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q, "q", _HALF)
    hs, ks = (B, H, T, d), (B, Hkv, T, d)
    dq = _out(dq, hs, dt, dev)
    dk, dv = _out(dk, ks, dt, dev), _out(dv, ks, dt, dev)
    ws = _ws(window_attn_bwd_workspace_size(B, H, Hkv, T, d, window, sinks), dev, workspace)
    _launch("cla_window_attn_bwd", dev, (
        _T(q, dt, "q", hs, True), _T(k, dt, "k", ks, True), _T(v, dt, "v", ks, True),
        _T(lens, torch.int32, "lens", (B,)), _T(o, dt, "o", hs, True), _T(lse, torch.float32, "lse", (B, H, T)),
        _T(dO, dt, "dO", hs, True), _T(dq, dt, "dq", hs, True), _T(dk, dt, "dk", ks, True), _T(dv, dt, "dv", ks, True),
        _scale(scale, d), window, sinks, code, B, H, Hkv, T, d, _strides(q, k, v, o, dO, dq, dk, dv),
        _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return dq, dk, dv


def window_cache_write(k, v, kcache, vcache, *, window, sinks=0, lens=None, stream=None):
    """Writes the prompts' keys and values ([B, Hkv, T, d], from position 0) into the rolling cache
    [B, Hkv, sinks + window, d] that window_attn_step reads: token p in slot p while p < sinks, else in slot
    sinks + (p - sinks) % window, the last one that falls on a slot; slots without one stay as they were."""
    window, sinks = _counts(window, sinks)
    B, Hkv, T, d = _dims(k, 4, "k")
    dev, dt = k.device, k.dtype
    code = _dtype_code(k, "k", _HALF)
    ks, cs = (B, Hkv, T, d), (B, Hkv, sinks + window, d)
    _launch("cla_window_cache_write", dev, (
        _T(k, dt, "k", ks, True), _T(v, dt, "v", ks, True), _T(lens, torch.int32, "lens", (B,)),
        _T(kcache, dt, "kcache", cs), _T(vcache, dt, "vcache", cs), window, sinks, code, B, Hkv, T, d,
        _strides(k, v)), stream)


@_own_memory
def window_attn_step(q, k, v, kcache, vcache, pos, *, window, sinks=0, scale=None, o=None, stream=None):
    """One token for each of B sequences: writes k and v [B, Hkv, d] into the rolling cache (see window_cache_write) and
    returns the attention of q [B, H, d] over what it then holds.  pos [B] int32: tokens before this one; negative: a
    row without a sequence (o is 0, its cache is left alone)."""
    window, sinks = _counts(window, sinks)
    B, H, d = _dims(q, 3, "q")
    Hkv = _dims(k, 3, "k")[1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q, "q", _HALF)
    o = _out(o, (B, H, d), dt, dev)
    cs = (B, Hkv, sinks + window, d)
    _launch("cla_window_attn_step", dev, (
        _T(q, dt, "q", (B, H, d), True), _T(k, dt, "k", (B, Hkv, d), True), _T(v, dt, "v", (B, Hkv, d), True),
        _T(kcache, dt, "kcache", cs), _T(vcache, dt, "vcache", cs), _T(pos, torch.int32, "pos", (B,)),
        _T(o, dt, "o", (B, H, d)), _scale(scale, d), window, sinks, code, B, H, Hkv, d, _strides(q, k, v)), stream)
    return o


# ---------------------------------------------------------------- the window's cache in 8 bits
WINDOW_CACHE8_BLOCK = 64


def _cache8_args(kcache, vcache, kscale, vscale, B, Hkv, d, window, sinks):
    S = sinks + window
    cs, ss = (B, Hkv, S, d), (B, Hkv, -(-S // WINDOW_CACHE8_BLOCK))
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    return (_T(kcache, e4m3, "kcache", cs), _T(vcache, e4m3, "vcache", cs), _T(kscale, f32, "kscale", ss),
            _T(vscale, f32, "vscale", ss))


def window_cache8(B, Hkv, d, *, window, sinks=0, device="cuda"):
    """An empty cache of window_cache8_write and window_attn_step8: (kcache, vcache, kscale, vscale)."""
    window, sinks = _counts(window, sinks)
    S = sinks + window
    cache = (torch.zeros(B, Hkv, S, d, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
    return (*cache, *(torch.zeros(B, Hkv, -(-S // WINDOW_CACHE8_BLOCK), dtype=torch.float32, device=device) for _ in range(2)))


def window_cache8_write(k, v, kcache, vcache, kscale, vscale, *, window, sinks=0, lens=None, stream=None):
    """window_cache_write into a cache of 8 bits: kcache and vcache [B, Hkv, sinks + window, d] float8_e4m3fn, whose numbers
    stand for themselves times a power of two for every 64 slots of a key head, kscale and vscale [B, Hkv,
    ceil((sinks + window) / 64)] fp32."""
    window, sinks = _counts(window, sinks)
    B, Hkv, T, d = _dims(k, 4, "k")
    dev, dt = k.device, k.dtype
    code = _dtype_code(k, "k", _HALF)
    ks = (B, Hkv, T, d)
    _launch("cla_window_cache8_write", dev, (
        _T(k, dt, "k", ks, True), _T(v, dt, "v", ks, True), _T(lens, torch.int32, "lens", (B,)),
        *_cache8_args(kcache, vcache, kscale, vscale, B, Hkv, d, window, sinks), window, sinks, code, B, Hkv, T, d,
        _strides(k, v)), stream)


@functools.lru_cache(maxsize=256)  # a number that the sizes fix; a step asks for it
def window_attn_step8_workspace_size(B, H, Hkv, d, window, sinks=0) -> int:
    return int(lib().cla_window_attn_step8_workspace_size(B, H, Hkv, d, *_counts(window, sinks)))


@_own_memory
def window_attn_step8(q, k, v, kcache, vcache, kscale, vscale, pos, *, window, sinks=0, scale=None, o=None, workspace=None,
                      stream=None):
    """window_attn_step over a cache of 8 bits (see window_cache8_write): k and v go into their slot, the factors of its
    block become those of what the block then holds, and q attends over what the cache then holds."""
    window, sinks = _counts(window, sinks)
    B, H, d = _dims(q, 3, "q")
    Hkv = _dims(k, 3, "k")[1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q, "q", _HALF)
    o = _out(o, (B, H, d), dt, dev)
    ws = _ws(window_attn_step8_workspace_size(B, H, Hkv, d, window, sinks), dev, workspace)
    _launch("cla_window_attn_step8", dev, (
        _T(q, dt, "q", (B, H, d), True), _T(k, dt, "k", (B, Hkv, d), True), _T(v, dt, "v", (B, Hkv, d), True),
        *_cache8_args(kcache, vcache, kscale, vscale, B, Hkv, d, window, sinks), _T(pos, torch.int32, "pos", (B,)),
        _T(o, dt, "o", (B, H, d)), _scale(scale, d), window, sinks, code, B, H, Hkv, d, _strides(q, k, v),
        _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return o


# ---------------------------------------------------------------- norm and rotation of queries and keys
def _rot(freq):
    return 0 if freq is None else 2 * _dims(freq, 1, "freq")[0]


@_own_memory
def qk_norm_rope_fwd(q, k, wq=None, wk=None, freq=None, *, pos=None, lens=None, eps=1e-6, interleaved=False, qo=None, ko=None,
                     stream=None):
    """Norm and rotation of every query and key head: x / sqrt(mean(x^2) + eps) times the weights (wq, wk [d] fp32; ones when
    None), with the first 2 len(freq) values turned by pos freq (freq [rot / 2] fp32 radians; pairs (i, i + rot / 2), or
    (2i, 2i + 1) when interleaved; None turns nothing).  q [B, H, T, d], k [B, Hkv, T, d] (fp32, bf16 or fp16; strided views
    are taken as they are); pos [B, T] int32, 0, 1, ... when None; lens [B] int32: lengths of a right-padded batch.
    Returns (qo, ko); q and k themselves may be given for them."""
    B, H, T, d = _dims(q, 4, "q")
    Hkv = _dims(k, 4, "k")[1]
    dev, dt, f32 = q.device, q.dtype, torch.float32
    code = _dtype_code(q, "q", _DTYPES)
    hs, ks, rot = (B, H, T, d), (B, Hkv, T, d), _rot(freq)
    qo, ko = _out(qo, hs, dt, dev), _out(ko, ks, dt, dev)
    _launch("cla_qk_norm_rope_fwd", dev, (
        _T(q, dt, "q", hs, True), _T(k, dt, "k", ks, True), _T(wq, f32, "wq", (d,)), _T(wk, f32, "wk", (d,)),
        _T(freq, f32, "freq", (rot // 2,)), _T(pos, torch.int32, "pos", (B, T)), _T(lens, torch.int32, "lens", (B,)),
        _T(qo, dt, "qo", hs, True), _T(ko, dt, "ko", ks, True), float(eps), rot, int(bool(interleaved)), code, B, H, Hkv, T, d,
        _strides(q, k, qo, ko)), stream)
    return qo, ko


@_own_memory
def qk_norm_rope_step(q, k, wq, wk, freq, pos, *, eps=1e-6, interleaved=False, qo=None, ko=None, stream=None):
    """qk_norm_rope_fwd for one token of each of B sequences: q [B, H, d], k [B, Hkv, d], pos [B] int32 (what
    window_attn_step takes)."""
    B, H, d = _dims(q, 3, "q")
    Hkv = _dims(k, 3, "k")[1]
    dev, dt, f32 = q.device, q.dtype, torch.float32
    code = _dtype_code(q, "q", _DTYPES)
    hs, ks, rot = (B, H, d), (B, Hkv, d), _rot(freq)
    qo, ko = _out(qo, hs, dt, dev), _out(ko, ks, dt, dev)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and qo.is_contiguous() and ko.is_contiguous()):
        # there is no stride from token to token
        strides = (ctypes.c_int64 * 12)(*q.stride()[:2], d, *k.stride()[:2], d, *qo.stride()[:2], d, *ko.stride()[:2], d)
    _launch("cla_qk_norm_rope_fwd", dev, (
        _T(q, dt, "q", hs, True), _T(k, dt, "k", ks, True), _T(wq, f32, "wq", (d,)), _T(wk, f32, "wk", (d,)),
        _T(freq, f32, "freq", (rot // 2,)), _T(pos, torch.int32, "pos", (B,)), None, _T(qo, dt, "qo", hs, True),
        _T(ko, dt, "ko", ks, True), float(eps), rot, int(bool(interleaved)), code, B, H, Hkv, 1, d, strides), stream)
    return qo, ko


@functools.lru_cache(maxsize=256)  # a number that the sizes fix
def qk_norm_rope_bwd_workspace_size(B, H, Hkv, T, d) -> int:
    return int(lib().cla_qk_norm_rope_bwd_workspace_size(B, H, Hkv, T, d))


@_own_memory
def qk_norm_rope_bwd(q, k, wq, wk, freq, dqo, dko, *, pos=None, lens=None, eps=1e-6, interleaved=False, dq=None, dk=None,
                     dwq=None, dwk=None, workspace=None, stream=None):
    """Adjoint of qk_norm_rope_fwd from its inputs; returns (dq, dk, dwq, dwk), dwq and dwk [d] fp32 (None for weights that
    are None)."""
    B, H, T, d = _dims(q, 4, "q")
    Hkv = _dims(k, 4, "k")[1]
    dev, dt, f32 = q.device, q.dtype, torch.float32
    code = _dtype_code(q, "q", _DTYPES)
    hs, ks, rot = (B, H, T, d), (B, Hkv, T, d), _rot(freq)
    dq, dk = _out(dq, hs, dt, dev), _out(dk, ks, dt, dev)
    dwq = _out(dwq, (d,), f32, dev) if wq is not None else dwq
    dwk = _out(dwk, (d,), f32, dev) if wk is not None else dwk
    ws = _ws(qk_norm_rope_bwd_workspace_size(B, H, Hkv, T, d), dev, workspace)
    _launch("cla_qk_norm_rope_bwd", dev, (
        _T(q, dt, "q", hs, True), _T(k, dt, "k", ks, True), _T(wq, f32, "wq", (d,)), _T(wk, f32, "wk", (d,)),
        _T(freq, f32, "freq", (rot // 2,)), _T(pos, torch.int32, "pos", (B, T)), _T(lens, torch.int32, "lens", (B,)),
        _T(dqo, dt, "dqo", hs, True), _T(dko, dt, "dko", ks, True), _T(dq, dt, "dq", hs, True), _T(dk, dt, "dk", ks, True),
        _T(dwq, f32, "dwq", (d,)), _T(dwk, f32, "dwk", (d,)), float(eps), rot, int(bool(interleaved)), code, B, H, Hkv, T, d,
        _strides(q, k, dqo, dko, dq, dk), _T(ws, None, "workspace"), _nbytes(ws)), stream)
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- the delta rule token by token
@_own_memory
def delta_step(q, k, v, log_decay, beta, S, *, lens=None, o=None, stream=None):
    """The recurrence of delta_fwd for a few tokens of each of B sequences, on the states S [B, H, dk, dv] fp32, which it
    updates in place: q, k [B, Hk, T, dk], v [B, H, T, dv] (fp32, bf16 or fp16; H a multiple of Hk), log_decay, beta [B, H, T]
    fp32; strided views are taken as they are.  lens [B] int32: tokens of each sequence.  Returns o [B, H, T, dv] fp32."""
    B, Hk, T, dk = _dims(q, 4, "q")
    H, dv = _dims(v, 4, "v")[1::2]
    dev, dt, f32 = q.device, q.dtype, torch.float32
    code = _dtype_code(q, "q", _DTYPES)
    o = _out(o, (B, H, T, dv), f32, dev)
    ks, gs = (B, Hk, T, dk), (B, H, T)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and log_decay.is_contiguous() and beta.is_contiguous()):
        strides = (ctypes.c_int64 * 15)(*q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *log_decay.stride(), *beta.stride())
    _launch("cla_delta_step", dev, (
        _T(q, dt, "q", ks, True), _T(k, dt, "k", ks, True), _T(v, dt, "v", (B, H, T, dv), True),
        _T(log_decay, f32, "log_decay", gs, _ALL), _T(beta, f32, "beta", gs, _ALL), _T(lens, torch.int32, "lens", (B,)),
        _T(S, f32, "S", (B, H, dk, dv)), _T(o, f32, "o", (B, H, T, dv)), code, B, H, Hk, T, dk, dv, strides), stream)
    return o

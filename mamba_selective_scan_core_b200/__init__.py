"""Python binding of the B200 Mamba mixer core library (libmamba_mixer.so).

Argument marshalling only: tensors are checked (device, dtype, shape,
contiguity), output tensors are allocated with torch when not given, and the
data pointers plus the current CUDA stream go through ctypes to the C ABI of
``include/mamba_mixer.h``.  Every step of the computation runs in the
library's kernels; there is no fallback path.  If the compiled library is
missing, loading fails with an error that says how to build it.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "MM_F32", "MM_BF16", "MixerError", "lib", "library_path", "mixer_fwd", "mixer_fwd_noalloc", "mixer_fwd_host",
    "state_update", "workspace_size", "host_workspace_size", "status_string", "abi_version", "fault_status",
    "check_status", "proj_matmul", "proj_matmul_workspace_size", "mixer_fwd_projected",
    "projected_workspace_size", "ssd_fwd", "ssd_workspace_size", "ssd_state_update", "m3_fwd", "m3_state_update", "m3_workspace_size",
    "gdr_fwd", "gdr_state_update", "gdr_workspace_size", "proj_q4", "EXPORTED_SYMBOLS",
]

MM_F32 = 0
MM_BF16 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmamba_mixer.so"
_lib = None

EXPORTED_SYMBOLS = (
    "mamba_mixer_fwd",
    "mamba_mixer_fwd_noalloc",
    "mamba_mixer_fwd_host",
    "mamba_mixer_workspace_size",
    "mamba_mixer_host_workspace_size",
    "mamba_state_update",
    "mamba_status_string",
    "mamba_mixer_abi_version",
    "mamba_mixer_fault_status",
    "mamba_check_status",
    "mamba_mixer_fwd_normed",
    "mamba_state_update_normed",
    "mamba_proj_matmul",
    "mamba_proj_matmul_workspace_size",
    "mamba_mixer_fwd_projected",
    "mamba_mixer_projected_workspace_size",
    "mamba_mixer_projected_layout",
    "mamba_ssd_fwd",
    "mamba_ssd_workspace_size",
    "mamba_ssd_state_update",
    "mamba_m3_fwd",
    "mamba_m3_workspace_size",
    "mamba_m3_state_update",
    "mamba_gdr_fwd",
    "mamba_gdr_workspace_size",
    "mamba_gdr_state_update",
    "mamba_proj_q4",
)


class MixerError(RuntimeError):
    """A non-zero mm_status returned by the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (mm_status {status})")


def library_path() -> str:
    """The library this process loads: libmamba_mixer.so, or its checked build
    libmamba_mixer_checked.so when MAMBA_MIXER_CHECKED=1 is set before the
    first call (index checks in the forward and decode kernels; an access
    outside its buffer is skipped and reported as MM_ERR_BOUNDS)."""
    if os.environ.get("MAMBA_MIXER_CHECKED") == "1":
        return os.path.join(_HERE, "libmamba_mixer_checked.so")
    return os.path.join(_HERE, _LIB_NAME)


def _declare(L):
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    L.mamba_mixer_fwd.restype = ctypes.c_int
    L.mamba_mixer_fwd.argtypes = [P] * 14 + [I64] * 5 + [ctypes.c_int, P, ctypes.c_size_t, P]
    L.mamba_mixer_fwd_noalloc.restype = ctypes.c_int
    L.mamba_mixer_fwd_noalloc.argtypes = [P] * 14 + [I64] * 5 + [ctypes.c_int, P]
    L.mamba_mixer_fwd_host.restype = ctypes.c_int
    L.mamba_mixer_fwd_host.argtypes = [P] * 14 + [I64] * 5 + [ctypes.c_int, P, ctypes.c_size_t, P, P, P]
    L.mamba_mixer_workspace_size.restype = ctypes.c_size_t
    L.mamba_mixer_workspace_size.argtypes = [I64] * 5 + [ctypes.c_int]
    L.mamba_mixer_host_workspace_size.restype = ctypes.c_size_t
    L.mamba_mixer_host_workspace_size.argtypes = [I64] * 5 + [ctypes.c_int]
    L.mamba_state_update.restype = ctypes.c_int
    L.mamba_state_update.argtypes = [P] * 13 + [I64] * 5 + [ctypes.c_int, P]
    L.mamba_status_string.restype = ctypes.c_char_p
    L.mamba_status_string.argtypes = [ctypes.c_int]
    L.mamba_mixer_abi_version.restype = ctypes.c_int
    L.mamba_mixer_abi_version.argtypes = []
    L.mamba_mixer_fault_status.restype = ctypes.c_int
    L.mamba_mixer_fault_status.argtypes = [ctypes.c_int]
    L.mamba_check_status.restype = ctypes.c_int
    L.mamba_check_status.argtypes = [P, P]
    L.mamba_mixer_fwd_normed.restype = ctypes.c_int
    L.mamba_mixer_fwd_normed.argtypes = [P] * 14 + [I64] * 5 + [ctypes.c_int, P, P, ctypes.c_float, P,
                                                                 ctypes.c_size_t, P]
    L.mamba_state_update_normed.restype = ctypes.c_int
    L.mamba_state_update_normed.argtypes = [P] * 13 + [I64] * 5 + [ctypes.c_int, P, P, ctypes.c_float, P]
    L.mamba_proj_matmul.restype = ctypes.c_int
    L.mamba_proj_matmul.argtypes = [P, P, P, I64, I64, I64, ctypes.c_int, P, ctypes.c_size_t, P]
    L.mamba_proj_matmul_workspace_size.restype = ctypes.c_size_t
    L.mamba_proj_matmul_workspace_size.argtypes = [I64, I64, I64]
    L.mamba_mixer_fwd_projected.restype = ctypes.c_int
    L.mamba_mixer_fwd_projected.argtypes = [P] * 13 + [ctypes.c_float] + [P] * 3 + [I64] * 6 + [
        ctypes.c_int, P, ctypes.c_size_t, P]
    L.mamba_mixer_projected_workspace_size.restype = ctypes.c_size_t
    L.mamba_mixer_projected_workspace_size.argtypes = [I64] * 6 + [ctypes.c_int]
    L.mamba_mixer_projected_layout.restype = ctypes.c_int
    L.mamba_mixer_projected_layout.argtypes = [I64] * 6 + [P]
    L.mamba_ssd_fwd.restype = ctypes.c_int
    L.mamba_ssd_fwd.argtypes = [P] * 11 + [I64] * 6 + [P, ctypes.c_size_t, P]
    L.mamba_ssd_workspace_size.restype = ctypes.c_size_t
    L.mamba_ssd_workspace_size.argtypes = [I64] * 6
    L.mamba_ssd_state_update.restype = ctypes.c_int
    L.mamba_ssd_state_update.argtypes = [P] * 10 + [I64] * 5 + [P]
    L.mamba_m3_fwd.restype = ctypes.c_int
    L.mamba_m3_fwd.argtypes = [P] * 15 + [I64] * 7 + [P, ctypes.c_size_t, P]
    L.mamba_m3_workspace_size.restype = ctypes.c_size_t
    L.mamba_m3_workspace_size.argtypes = [I64] * 7
    L.mamba_m3_state_update.restype = ctypes.c_int
    L.mamba_m3_state_update.argtypes = [P] * 14 + [I64] * 6 + [P]
    L.mamba_gdr_fwd.restype = ctypes.c_int
    L.mamba_gdr_fwd.argtypes = [P] * 10 + [I64] * 9 + [ctypes.c_float] * 2 + [ctypes.c_int, P, ctypes.c_size_t, P]
    L.mamba_gdr_workspace_size.restype = ctypes.c_size_t
    L.mamba_gdr_workspace_size.argtypes = [I64] * 6 + [ctypes.c_int]
    L.mamba_gdr_state_update.restype = ctypes.c_int
    L.mamba_gdr_state_update.argtypes = [P] * 9 + [I64] * 8 + [ctypes.c_float] * 2 + [ctypes.c_int, P]
    L.mamba_proj_q4.restype = ctypes.c_int
    L.mamba_proj_q4.argtypes = [P] * 5 + [I64] * 4 + [ctypes.c_int, P]
    return L


def lib():
    """The loaded C library (ctypes.CDLL).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build the CUDA library first "
                "(python -m mamba_selective_scan_core_b200.build, or __graft_entry__.build())")
        _lib = _declare(ctypes.CDLL(path))
    return _lib


def status_string(status: int) -> str:
    return lib().mamba_status_string(int(status)).decode()


def abi_version() -> int:
    return int(lib().mamba_mixer_abi_version())


def fault_status(reset: bool = False) -> int:
    """0 if no kernel gave up waiting for its bulk copies on the current
    device, else MM_ERR_TIMEOUT (11) -- or MM_ERR_BOUNDS (13) when a kernel of
    the checked build skipped an access outside its buffer; clears the word
    when reset is set."""
    return int(lib().mamba_mixer_fault_status(1 if reset else 0))


def check_status(workspace=None, stream=None) -> int:
    """Status of the last forward that ran on `workspace` (a CUDA uint8
    tensor given to mixer_fwd or mixer_fwd_host; None = the fixed scratch of
    mixer_fwd_noalloc): 0 if it completed, MM_ERR_TIMEOUT (11) if one of its
    kernels gave up a bounded wait, MM_ERR_BOUNDS (13) if the checked build
    skipped an access outside its buffer.  Waits for `stream` (default: current)."""
    import torch

    dev = workspace.device if workspace is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        return int(lib().mamba_check_status(_ptr(workspace), _stream_handle(stream)))


def _act_code(dtype):
    import torch

    if dtype == torch.bfloat16:
        return MM_BF16
    if dtype == torch.float32:
        return MM_F32
    raise TypeError(f"activation dtype must be bfloat16 or float32, got {dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype, shape, device):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _keep_alive_on(tensors, streams):
    """Tell torch's caching allocator that device tensors this module
    allocated are used by work queued on `streams` (besides the stream current
    at allocation), so their memory is not handed out again before that work
    has finished."""
    for t in tensors:
        for s in streams:
            if s is not None:
                t.record_stream(s)


def workspace_size(batch, seqlen, d_inner, d_state=16, d_conv=4, act=MM_BF16) -> int:
    return int(lib().mamba_mixer_workspace_size(batch, seqlen, d_inner, d_state, d_conv, act))


def mixer_fwd(xz, conv_w, conv_b, dt, dt_bias, A, Bm, Cm, Dskip, h0=None, conv_state_in=None, *,
              y=None, h_last=None, conv_state_out=None, workspace=None, stream=None,
              b_norm_w=None, c_norm_w=None, norm_eps=1e-6):
    """Selective-scan forward.  Shapes: xz [B,L,2D], dt [B,L,D], Bm/Cm [B,L,N]
    (act dtype: bf16 or fp32); conv_w [D,W], conv_b/dt_bias/Dskip [D], A [D,N],
    h0 [B,D,N] (fp32); conv_state_in [B,D,W-1] (act).  conv_b, Dskip, h0 and
    conv_state_in may be None.  b_norm_w / c_norm_w ([N] fp32) switch on the
    fused RMSNorm of B / C (mamba_mixer_fwd_normed).  Returns (y [B,L,D],
    h_last [B,D,N], conv_state_out [B,D,W-1]), allocating any output not
    given."""
    import torch

    act = _act_code(xz.dtype)
    Bsz, L, twoD = xz.shape
    D = twoD // 2
    N = A.shape[-1]
    W = conv_w.shape[-1]
    dev = xz.device
    f32 = torch.float32
    made = []
    _check(xz, "xz", xz.dtype, (Bsz, L, 2 * D), dev)
    _check(conv_w, "conv_w", f32, (D, W), dev)
    _check(conv_b, "conv_b", f32, (D,), dev)
    _check(dt, "dt", xz.dtype, (Bsz, L, D), dev)
    _check(dt_bias, "dt_bias", f32, (D,), dev)
    _check(A, "A", f32, (D, N), dev)
    _check(Bm, "Bm", xz.dtype, (Bsz, L, N), dev)
    _check(Cm, "Cm", xz.dtype, (Bsz, L, N), dev)
    _check(Dskip, "Dskip", f32, (D,), dev)
    _check(h0, "h0", f32, (Bsz, D, N), dev)
    _check(conv_state_in, "conv_state_in", xz.dtype, (Bsz, D, W - 1), dev)
    _check(b_norm_w, "b_norm_w", f32, (N,), dev)
    _check(c_norm_w, "c_norm_w", f32, (N,), dev)
    normed = b_norm_w is not None or c_norm_w is not None
    if y is None:
        y = torch.empty((Bsz, L, D), dtype=xz.dtype, device=dev)
        made.append(y)
    if h_last is None:
        h_last = torch.empty((Bsz, D, N), dtype=f32, device=dev)
        made.append(h_last)
    if conv_state_out is None:
        conv_state_out = torch.empty((Bsz, D, W - 1), dtype=xz.dtype, device=dev)
        made.append(conv_state_out)
    _check(y, "y", xz.dtype, (Bsz, L, D), dev)
    _check(h_last, "h_last", f32, (Bsz, D, N), dev)
    _check(conv_state_out, "conv_state_out", xz.dtype, (Bsz, D, W - 1), dev)
    ws_bytes = workspace_size(Bsz, L, D, N, W, act)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    args = (_ptr(xz), _ptr(conv_w), _ptr(conv_b), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm),
            _ptr(Dskip), _ptr(h0), _ptr(conv_state_in), _ptr(y), _ptr(h_last), _ptr(conv_state_out),
            Bsz, L, D, N, W, act)
    tail = (_ptr(workspace), workspace.numel() * workspace.element_size(), _stream_handle(stream))
    with torch.cuda.device(dev):
        if normed:
            st = lib().mamba_mixer_fwd_normed(*args, _ptr(b_norm_w), _ptr(c_norm_w), float(norm_eps), *tail)
        else:
            st = lib().mamba_mixer_fwd(*args, *tail)
    if st != 0:
        raise MixerError(st, "mamba_mixer_fwd_normed" if normed else "mamba_mixer_fwd")
    _keep_alive_on(made, (stream,))
    return y, h_last, conv_state_out


def host_workspace_size(batch, seqlen, d_inner, d_state=16, d_conv=4, act=MM_BF16) -> int:
    return int(lib().mamba_mixer_host_workspace_size(batch, seqlen, d_inner, d_state, d_conv, act))


def _check_host(t, name, dtype, shape):
    if t is None:
        return
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_side_streams = {}


def _copy_streams(dev):
    """Two side streams per device for the host path's copies (created once)."""
    import torch

    key = torch.device(dev).index
    if key not in _side_streams:
        with torch.cuda.device(dev):
            _side_streams[key] = (torch.cuda.Stream(), torch.cuda.Stream())
    return _side_streams[key]


def mixer_fwd_host(xz, conv_w, conv_b, dt, dt_bias, A, Bm, Cm, Dskip, h0=None, conv_state_in=None, *,
                   y=None, h_last=None, conv_state_out=None, workspace=None, stream=None):
    """mixer_fwd on activations in host memory (mamba_mixer_fwd_host): xz, dt,
    Bm, Cm, h0, conv_state_in and the outputs are CPU tensors (page-locked for
    the copies to overlap the compute; outputs are allocated pinned when not
    given); conv_w, conv_b, dt_bias, A, Dskip are CUDA tensors on the device
    that runs it.  Copies go on two side streams, the forward on `stream`
    (default: the current stream), which waits for the copies back: the
    outputs are valid once `stream` is synchronised."""
    import torch

    act = _act_code(xz.dtype)
    Bsz, L, twoD = xz.shape
    D = twoD // 2
    N = A.shape[-1]
    W = conv_w.shape[-1]
    dev = conv_w.device
    f32 = torch.float32
    for t, name, dtype, shape in ((xz, "xz", xz.dtype, (Bsz, L, 2 * D)), (dt, "dt", xz.dtype, (Bsz, L, D)),
                                  (Bm, "Bm", xz.dtype, (Bsz, L, N)), (Cm, "Cm", xz.dtype, (Bsz, L, N)),
                                  (h0, "h0", f32, (Bsz, D, N)),
                                  (conv_state_in, "conv_state_in", xz.dtype, (Bsz, D, W - 1))):
        _check_host(t, name, dtype, shape)
    _check(conv_w, "conv_w", f32, (D, W), dev)
    _check(conv_b, "conv_b", f32, (D,), dev)
    _check(dt_bias, "dt_bias", f32, (D,), dev)
    _check(A, "A", f32, (D, N), dev)
    _check(Dskip, "Dskip", f32, (D,), dev)
    if y is None:
        y = torch.empty((Bsz, L, D), dtype=xz.dtype).pin_memory()
    if h_last is None:
        h_last = torch.empty((Bsz, D, N), dtype=f32).pin_memory()
    if conv_state_out is None:
        conv_state_out = torch.empty((Bsz, D, W - 1), dtype=xz.dtype).pin_memory()
    _check_host(y, "y", xz.dtype, (Bsz, L, D))
    _check_host(h_last, "h_last", f32, (Bsz, D, N))
    _check_host(conv_state_out, "conv_state_out", xz.dtype, (Bsz, D, W - 1))
    ws_bytes = host_workspace_size(Bsz, L, D, N, W, act)
    made = []
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
        made.append(workspace)
    s_in, s_out = _copy_streams(dev)
    with torch.cuda.device(dev):
        st = lib().mamba_mixer_fwd_host(
            _ptr(xz), _ptr(conv_w), _ptr(conv_b), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm),
            _ptr(Dskip), _ptr(h0), _ptr(conv_state_in), _ptr(y), _ptr(h_last), _ptr(conv_state_out),
            Bsz, L, D, N, W, act, _ptr(workspace), ws_bytes, _stream_handle(stream),
            ctypes.c_void_p(s_in.cuda_stream), ctypes.c_void_p(s_out.cuda_stream))
    if st != 0:
        raise MixerError(st, "mamba_mixer_fwd_host")
    _keep_alive_on(made, (stream, s_in, s_out))
    return y, h_last, conv_state_out


def mixer_fwd_noalloc(xz, conv_w, conv_b, dt, dt_bias, A, Bm, Cm, Dskip, h0=None, conv_state_in=None, *,
                      y, h_last, conv_state_out, stream=None):
    """mixer_fwd through the entry point that takes no workspace and allocates
    nothing (its scratch is a fixed array inside the library).  The caller
    passes the output tensors; calls that overlap on the GPU race on the
    shared scratch, so serialise them."""
    import torch

    act = _act_code(xz.dtype)
    Bsz, L, twoD = xz.shape
    D = twoD // 2
    N = A.shape[-1]
    W = conv_w.shape[-1]
    dev = xz.device
    f32 = torch.float32
    for t, name, dtype, shape in (
            (xz, "xz", xz.dtype, (Bsz, L, 2 * D)), (conv_w, "conv_w", f32, (D, W)), (conv_b, "conv_b", f32, (D,)),
            (dt, "dt", xz.dtype, (Bsz, L, D)), (dt_bias, "dt_bias", f32, (D,)), (A, "A", f32, (D, N)),
            (Bm, "Bm", xz.dtype, (Bsz, L, N)), (Cm, "Cm", xz.dtype, (Bsz, L, N)), (Dskip, "Dskip", f32, (D,)),
            (h0, "h0", f32, (Bsz, D, N)), (conv_state_in, "conv_state_in", xz.dtype, (Bsz, D, W - 1)),
            (y, "y", xz.dtype, (Bsz, L, D)), (h_last, "h_last", f32, (Bsz, D, N)),
            (conv_state_out, "conv_state_out", xz.dtype, (Bsz, D, W - 1))):
        _check(t, name, dtype, shape, dev)
    with torch.cuda.device(dev):
        st = lib().mamba_mixer_fwd_noalloc(
            _ptr(xz), _ptr(conv_w), _ptr(conv_b), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm),
            _ptr(Dskip), _ptr(h0), _ptr(conv_state_in), _ptr(y), _ptr(h_last), _ptr(conv_state_out),
            Bsz, L, D, N, W, act, _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_mixer_fwd_noalloc")
    return y, h_last, conv_state_out


def state_update(x, z, dt, conv_w, conv_b, dt_bias, Dskip, A, Bm, Cm, ssm_state, conv_state, *,
                 y=None, stream=None, b_norm_w=None, c_norm_w=None, norm_eps=1e-6):
    """One-token decode step for NL stacked layers, in place on ssm_state
    [NL,B,D,N] (fp32) and conv_state [NL,B,D,W-1] (act).  x/z/dt [NL,B,D] and
    Bm/Cm [NL,B,N] in the act dtype; conv_w [NL,D,W], conv_b/dt_bias/Dskip
    [NL,D], A [NL,D,N] in fp32 (conv_b, Dskip may be None).  b_norm_w /
    c_norm_w ([NL,N] fp32) switch on the fused RMSNorm of B / C
    (mamba_state_update_normed).  Returns y [NL,B,D]."""
    import torch

    act = _act_code(x.dtype)
    NL, Bsz, D = x.shape
    N = A.shape[-1]
    W = conv_w.shape[-1]
    dev = x.device
    f32 = torch.float32
    for t, name in ((x, "x"), (z, "z"), (dt, "dt")):
        _check(t, name, x.dtype, (NL, Bsz, D), dev)
    _check(conv_w, "conv_w", f32, (NL, D, W), dev)
    for t, name in ((conv_b, "conv_b"), (dt_bias, "dt_bias"), (Dskip, "Dskip")):
        _check(t, name, f32, (NL, D), dev)
    _check(A, "A", f32, (NL, D, N), dev)
    _check(Bm, "Bm", x.dtype, (NL, Bsz, N), dev)
    _check(Cm, "Cm", x.dtype, (NL, Bsz, N), dev)
    _check(ssm_state, "ssm_state", f32, (NL, Bsz, D, N), dev)
    _check(conv_state, "conv_state", x.dtype, (NL, Bsz, D, W - 1), dev)
    _check(b_norm_w, "b_norm_w", f32, (NL, N), dev)
    _check(c_norm_w, "c_norm_w", f32, (NL, N), dev)
    normed = b_norm_w is not None or c_norm_w is not None
    made = []
    if y is None:
        y = torch.empty((NL, Bsz, D), dtype=x.dtype, device=dev)
        made.append(y)
    _check(y, "y", x.dtype, (NL, Bsz, D), dev)
    args = (_ptr(x), _ptr(z), _ptr(dt), _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), _ptr(Dskip), _ptr(A),
            _ptr(Bm), _ptr(Cm), _ptr(ssm_state), _ptr(conv_state), _ptr(y), NL, Bsz, D, N, W, act)
    with torch.cuda.device(dev):
        if normed:
            st = lib().mamba_state_update_normed(*args, _ptr(b_norm_w), _ptr(c_norm_w), float(norm_eps),
                                                 _stream_handle(stream))
        else:
            st = lib().mamba_state_update(*args, _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_state_update_normed" if normed else "mamba_state_update")
    _keep_alive_on(made, (stream,))
    return y


def proj_matmul_workspace_size(M, N, K) -> int:
    return int(lib().mamba_proj_matmul_workspace_size(M, N, K))


def proj_matmul(A, W, *, out=None, out_dtype=None, workspace=None, stream=None):
    """out = A @ W^T on the tensor cores (mamba_proj_matmul): A [M, K] and W
    [N, K] bf16 CUDA tensors, out [M, N] fp32 (default) or bf16."""
    import torch

    M, K = A.shape
    N = W.shape[0]
    dev = A.device
    _check(A, "A", torch.bfloat16, (M, K), dev)
    _check(W, "W", torch.bfloat16, (N, K), dev)
    dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=dev)
    _check(out, "out", dtype, (M, N), dev)
    code = MM_BF16 if dtype == torch.bfloat16 else MM_F32
    ws_bytes = proj_matmul_workspace_size(M, N, K)
    made = []
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    with torch.cuda.device(dev):
        st = lib().mamba_proj_matmul(_ptr(A), _ptr(W), _ptr(out), M, N, K, code, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_proj_matmul")
    _keep_alive_on(made, (stream,))
    return out


def projected_workspace_size(batch, seqlen, d_inner, dt_rank, d_state=16, d_conv=4, act=MM_BF16) -> int:
    return int(lib().mamba_mixer_projected_workspace_size(batch, seqlen, d_inner, d_state, dt_rank, d_conv, act))


def projected_intermediates(workspace, batch, seqlen, d_inner, dt_rank, d_state=16, d_conv=4):
    """Views of the intermediates a mixer_fwd_projected call left in its
    workspace (u, dt_low, Bm, Cm, dt; bf16), by mamba_mixer_projected_layout."""
    import torch

    offs = (ctypes.c_size_t * 5)()
    st = lib().mamba_mixer_projected_layout(batch, seqlen, d_inner, d_state, dt_rank, d_conv, offs)
    if st != 0:
        raise MixerError(st, "mamba_mixer_projected_layout")
    shapes = ((batch, seqlen, d_inner), (batch, seqlen, dt_rank), (batch, seqlen, d_state), (batch, seqlen, d_state),
              (batch, seqlen, d_inner))
    out = []
    for off, shp in zip(offs, shapes):
        n = 1
        for v in shp:
            n *= v
        out.append(workspace[off:off + 2 * n].view(torch.bfloat16).view(shp))
    return dict(zip(("u", "dt_low", "Bm", "Cm", "dt"), out))


def mixer_fwd_projected(xz, conv_w, conv_b, W_x, W_dt, dt_bias, A, Dskip, h0=None, conv_state_in=None, *,
                        dt_norm_w=None, b_norm_w=None, c_norm_w=None, norm_eps=1e-6, y=None, h_last=None,
                        conv_state_out=None, workspace=None, stream=None):
    """The mixer with its producers (mamba_mixer_fwd_projected): u = SiLU(conv
    x), x_proj (W_x [R + 2N, D] bf16) split into dt_low | B | C with optional
    RMSNorms (dt_norm_w [R], b_norm_w / c_norm_w [N] fp32), dt_proj (W_dt
    [D, R] bf16), then the selective scan.  bf16 activations only.  Returns
    (y, h_last, conv_state_out)."""
    import torch

    Bsz, L, twoD = xz.shape
    D = twoD // 2
    N = A.shape[-1]
    W = conv_w.shape[-1]
    R = W_dt.shape[-1]
    dev = xz.device
    f32, bf = torch.float32, torch.bfloat16
    _check(xz, "xz", bf, (Bsz, L, 2 * D), dev)
    _check(conv_w, "conv_w", f32, (D, W), dev)
    _check(conv_b, "conv_b", f32, (D,), dev)
    _check(W_x, "W_x", bf, (R + 2 * N, D), dev)
    _check(W_dt, "W_dt", bf, (D, R), dev)
    _check(dt_bias, "dt_bias", f32, (D,), dev)
    _check(A, "A", f32, (D, N), dev)
    _check(Dskip, "Dskip", f32, (D,), dev)
    _check(h0, "h0", f32, (Bsz, D, N), dev)
    _check(conv_state_in, "conv_state_in", bf, (Bsz, D, W - 1), dev)
    _check(dt_norm_w, "dt_norm_w", f32, (R,), dev)
    _check(b_norm_w, "b_norm_w", f32, (N,), dev)
    _check(c_norm_w, "c_norm_w", f32, (N,), dev)
    made = []
    if y is None:
        y = torch.empty((Bsz, L, D), dtype=bf, device=dev)
        made.append(y)
    if h_last is None:
        h_last = torch.empty((Bsz, D, N), dtype=f32, device=dev)
        made.append(h_last)
    if conv_state_out is None:
        conv_state_out = torch.empty((Bsz, D, W - 1), dtype=bf, device=dev)
        made.append(conv_state_out)
    ws_bytes = projected_workspace_size(Bsz, L, D, R, N, W)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    with torch.cuda.device(dev):
        st = lib().mamba_mixer_fwd_projected(
            _ptr(xz), _ptr(conv_w), _ptr(conv_b), _ptr(W_x), _ptr(W_dt), _ptr(dt_bias), _ptr(A), _ptr(Dskip),
            _ptr(h0), _ptr(conv_state_in), _ptr(dt_norm_w), _ptr(b_norm_w), _ptr(c_norm_w), float(norm_eps),
            _ptr(y), _ptr(h_last), _ptr(conv_state_out), Bsz, L, D, N, R, W, MM_BF16, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_mixer_fwd_projected")
    _keep_alive_on(made, (stream,))
    return y, h_last, conv_state_out



def ssd_workspace_size(batch, seqlen, heads, headdim=64, d_state=128, groups=1) -> int:
    return int(lib().mamba_ssd_workspace_size(batch, seqlen, heads, headdim, d_state, groups))


def ssd_fwd(x, z, dt, dt_bias, A, Bm, Cm, Dskip, h0=None, *, headdim=64, y=None, h_last=None, workspace=None,
            stream=None):
    """The Mamba-2 form of the scan (mamba_ssd_fwd): x, z [B,L,H*P] bf16 (z may
    be None: no gate), dt [B,L,H] bf16, dt_bias/A/Dskip [H] fp32 (dt_bias and
    Dskip may be None), Bm/Cm [B,L,G,N] bf16, h0 [B,H,P,N] fp32 or None, P =
    headdim.  Returns (y [B,L,H*P] bf16, h_last [B,H,P,N] fp32), allocating any
    output not given."""
    import torch

    bf, f32 = torch.bfloat16, torch.float32
    Bsz, L, HP = x.shape
    H = A.shape[0]
    P = int(headdim)
    G, N = Bm.shape[2], Bm.shape[3]
    if HP != H * P:
        raise ValueError(f"x has {HP} channels, expected heads x headdim = {H * P}")
    dev = x.device
    made = []
    _check(x, "x", bf, (Bsz, L, H * P), dev)
    _check(z, "z", bf, (Bsz, L, H * P), dev)
    _check(dt, "dt", bf, (Bsz, L, H), dev)
    _check(dt_bias, "dt_bias", f32, (H,), dev)
    _check(A, "A", f32, (H,), dev)
    _check(Bm, "Bm", bf, (Bsz, L, G, N), dev)
    _check(Cm, "Cm", bf, (Bsz, L, G, N), dev)
    _check(Dskip, "Dskip", f32, (H,), dev)
    _check(h0, "h0", f32, (Bsz, H, P, N), dev)
    if y is None:
        y = torch.empty((Bsz, L, H * P), dtype=bf, device=dev)
        made.append(y)
    if h_last is None:
        h_last = torch.empty((Bsz, H, P, N), dtype=f32, device=dev)
        made.append(h_last)
    _check(y, "y", bf, (Bsz, L, H * P), dev)
    _check(h_last, "h_last", f32, (Bsz, H, P, N), dev)
    ws_bytes = ssd_workspace_size(Bsz, L, H, P, N, G)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    with torch.cuda.device(dev):
        st = lib().mamba_ssd_fwd(_ptr(x), _ptr(z), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm),
                                 _ptr(Dskip), _ptr(h0), _ptr(y), _ptr(h_last), Bsz, L, H, P, N, G,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_ssd_fwd")
    _keep_alive_on(made, (stream,))
    return y, h_last


def ssd_state_update(x, z, dt, dt_bias, A, Bm, Cm, Dskip, state, *, headdim=64, y=None, stream=None):
    """One token of the Mamba-2 form (mamba_ssd_state_update), in place on
    state [B,H,P,N] fp32: x, z [B,H*P] bf16 (z may be None: no gate), dt [B,H]
    bf16, dt_bias/A/Dskip [H] fp32 (dt_bias and Dskip may be None), Bm/Cm
    [B,G,N] bf16, P = headdim.  Returns y [B,H*P] bf16, allocated if not given."""
    import torch

    bf, f32 = torch.bfloat16, torch.float32
    Bsz, HP = x.shape
    H = A.shape[0]
    P = int(headdim)
    G, N = Bm.shape[1], Bm.shape[2]
    if HP != H * P:
        raise ValueError(f"x has {HP} channels, expected heads x headdim = {H * P}")
    dev = x.device
    made = []
    _check(x, "x", bf, (Bsz, H * P), dev)
    _check(z, "z", bf, (Bsz, H * P), dev)
    _check(dt, "dt", bf, (Bsz, H), dev)
    _check(dt_bias, "dt_bias", f32, (H,), dev)
    _check(A, "A", f32, (H,), dev)
    _check(Bm, "Bm", bf, (Bsz, G, N), dev)
    _check(Cm, "Cm", bf, (Bsz, G, N), dev)
    _check(Dskip, "Dskip", f32, (H,), dev)
    _check(state, "state", f32, (Bsz, H, P, N), dev)
    if y is None:
        y = torch.empty((Bsz, H * P), dtype=bf, device=dev)
        made.append(y)
    _check(y, "y", bf, (Bsz, H * P), dev)
    with torch.cuda.device(dev):
        st = lib().mamba_ssd_state_update(_ptr(x), _ptr(z), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm),
                                          _ptr(Dskip), _ptr(state), _ptr(y), Bsz, H, P, N, G,
                                          _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_ssd_state_update")
    _keep_alive_on(made, (stream,))
    return y


def m3_workspace_size(batch, seqlen, heads, rank=1, headdim=64, d_state=16, groups=1) -> int:
    return int(lib().mamba_m3_workspace_size(batch, seqlen, rank, heads, headdim, d_state, groups))


def m3_fwd(x, z, dt, trap, dt_bias, A, theta, Bm, Cm, Dskip, h0=None, x_prev=None, B_prev=None, *,
           headdim=64, y=None, h_last=None, workspace=None, stream=None):
    """The Mamba-3 form of the scan (mamba_m3_fwd): x, z [B,L,R,H*P] bf16
    (z may be None: no gate), dt and trap [B,L,H] bf16 (trap None: 1/2),
    dt_bias/A/Dskip [H] fp32 (dt_bias and Dskip may be None), theta [H,N/2]
    fp32, Bm/Cm [B,L,R,G,N] bf16, h0 [B,H,P,N] fp32 or None, x_prev [B,R,H*P]
    and B_prev [B,R,G,N] bf16 or None, P = headdim.  Returns (y [B,L,R,H*P]
    bf16, h_last [B,H,P,N] fp32), allocating any output not given."""
    import torch

    bf, f32 = torch.bfloat16, torch.float32
    Bsz, L, R, HP = x.shape
    H = A.shape[0]
    P = int(headdim)
    G, N = Bm.shape[3], Bm.shape[4]
    if HP != H * P:
        raise ValueError(f"x has {HP} channels, expected heads x headdim = {H * P}")
    dev = x.device
    made = []
    _check(x, "x", bf, (Bsz, L, R, H * P), dev)
    _check(z, "z", bf, (Bsz, L, R, H * P), dev)
    _check(dt, "dt", bf, (Bsz, L, H), dev)
    _check(trap, "trap", bf, (Bsz, L, H), dev)
    _check(dt_bias, "dt_bias", f32, (H,), dev)
    _check(A, "A", f32, (H,), dev)
    _check(theta, "theta", f32, (H, N // 2), dev)
    _check(Bm, "Bm", bf, (Bsz, L, R, G, N), dev)
    _check(Cm, "Cm", bf, (Bsz, L, R, G, N), dev)
    _check(Dskip, "Dskip", f32, (H,), dev)
    _check(h0, "h0", f32, (Bsz, H, P, N), dev)
    _check(x_prev, "x_prev", bf, (Bsz, R, H * P), dev)
    _check(B_prev, "B_prev", bf, (Bsz, R, G, N), dev)
    if y is None:
        y = torch.empty((Bsz, L, R, H * P), dtype=bf, device=dev)
        made.append(y)
    if h_last is None:
        h_last = torch.empty((Bsz, H, P, N), dtype=f32, device=dev)
        made.append(h_last)
    _check(y, "y", bf, (Bsz, L, R, H * P), dev)
    _check(h_last, "h_last", f32, (Bsz, H, P, N), dev)
    ws_bytes = m3_workspace_size(Bsz, L, H, R, P, N, G)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    with torch.cuda.device(dev):
        st = lib().mamba_m3_fwd(_ptr(x), _ptr(z), _ptr(dt), _ptr(trap), _ptr(dt_bias), _ptr(A), _ptr(theta),
                                _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(h0), _ptr(x_prev), _ptr(B_prev), _ptr(y),
                                _ptr(h_last), Bsz, L, R, H, P, N, G, _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_m3_fwd")
    _keep_alive_on(made, (stream,))
    return y, h_last


def m3_state_update(x, z, dt, trap, dt_bias, A, theta, Bm, Cm, Dskip, state, x_prev=None, B_prev=None, *,
                    headdim=64, y=None, stream=None):
    """One token of the Mamba-3 form (mamba_m3_state_update), in place on
    state [B,H,P,N] fp32: x, z [B,R,H*P] bf16 (z may be None: no gate), dt and
    trap [B,H] bf16 (trap None: 1/2), dt_bias/A/Dskip [H] fp32 (dt_bias and
    Dskip may be None), theta [H,N/2] fp32, Bm/Cm [B,R,G,N] bf16, x_prev
    [B,R,H*P] and B_prev [B,R,G,N] bf16 (the previous token's) or None, P =
    headdim.  Returns y [B,R,H*P] bf16, allocated if not given."""
    import torch

    bf, f32 = torch.bfloat16, torch.float32
    Bsz, R, HP = x.shape
    H = A.shape[0]
    P = int(headdim)
    G, N = Bm.shape[2], Bm.shape[3]
    if HP != H * P:
        raise ValueError(f"x has {HP} channels, expected heads x headdim = {H * P}")
    dev = x.device
    made = []
    _check(x, "x", bf, (Bsz, R, H * P), dev)
    _check(z, "z", bf, (Bsz, R, H * P), dev)
    _check(dt, "dt", bf, (Bsz, H), dev)
    _check(trap, "trap", bf, (Bsz, H), dev)
    _check(dt_bias, "dt_bias", f32, (H,), dev)
    _check(A, "A", f32, (H,), dev)
    _check(theta, "theta", f32, (H, N // 2), dev)
    _check(Bm, "Bm", bf, (Bsz, R, G, N), dev)
    _check(Cm, "Cm", bf, (Bsz, R, G, N), dev)
    _check(Dskip, "Dskip", f32, (H,), dev)
    _check(state, "state", f32, (Bsz, H, P, N), dev)
    _check(x_prev, "x_prev", bf, (Bsz, R, H * P), dev)
    _check(B_prev, "B_prev", bf, (Bsz, R, G, N), dev)
    if y is None:
        y = torch.empty((Bsz, R, H * P), dtype=bf, device=dev)
        made.append(y)
    _check(y, "y", bf, (Bsz, R, H * P), dev)
    with torch.cuda.device(dev):
        st = lib().mamba_m3_state_update(_ptr(x), _ptr(z), _ptr(dt), _ptr(trap), _ptr(dt_bias), _ptr(A),
                                         _ptr(theta), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(state), _ptr(x_prev),
                                         _ptr(B_prev), _ptr(y), Bsz, R, H, P, N, G, _stream_handle(stream))
    if st != 0:
        raise MixerError(st, "mamba_m3_state_update")
    _keep_alive_on(made, (stream,))
    return y


def _check_rows(t, name, dtype, shape, device):
    """A tensor [B, L, heads, width] (or [B, heads, width]) whose tokens' rows
    are dense and evenly spaced, as a part of a wider packed tensor is.
    Returns the elements between rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    heads, width = shape[-2:]
    if (width > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != width):
        raise ValueError(f"{name} must have contiguous rows of {heads} x {width}")
    lead = [(n, s) for n, s in zip(shape[:-2], t.stride()[:-2])]
    if any(n == 0 for n, _ in lead):
        return heads * width
    stride, rows = None, 1
    for n, s in reversed(lead):
        if n > 1:
            if stride is None:
                stride = s
            elif s != rows * stride:
                raise ValueError(f"{name} must have its tokens' rows evenly spaced")
            rows *= n
    return heads * width if stride is None else stride


# The calls below are made once per layer and decoded token, where a launch
# takes a few microseconds: one expression looks at all tensors with the fewest
# calls into torch, and the checks that name what is wrong run once it fails.
def _required(t, name):
    if t is None:
        raise ValueError(f"{name} must be given")


_ERR_WORKSPACE = 9


class _Torch:
    """What the calls below need of torch and of the library, looked up once."""

    def __init__(self):
        import torch

        self.f32, self.bf16, self.u8 = torch.float32, torch.bfloat16, torch.uint8
        self.codes = {torch.float32: MM_F32, torch.bfloat16: MM_BF16}
        self.device, self.current_device = torch.cuda.device, torch.cuda.current_device
        self.on, self.current_stream = torch.cuda.stream, torch.cuda.current_stream
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
        self.lib = lib()
        # the same calls with the tensors looked at in C++ (they return None
        # where the Python below is to decide); without the module, or with one
        # compiled against another torch or Python, this alone
        from .build import calls_fit

        self.calls = None
        if calls_fit():
            try:
                from . import _calls
            except ImportError:
                return
            _calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                self.lib.mamba_gdr_fwd, self.lib.mamba_gdr_workspace_size, self.lib.mamba_gdr_state_update,
                self.lib.mamba_proj_q4)), MixerError)
            self.calls = _calls

    def empty(self, like, shape, dtype, stream, given_back=True):
        """Memory for a call that runs on `stream`: torch's allocator hands out
        what was freed on a stream to that stream while its work may still be
        running, so the memory is taken there and not on the current stream --
        which is told to the allocator where the caller gets the tensor."""
        if stream is None:
            return like.new_empty(shape, dtype=dtype)
        with self.on(stream):
            t = like.new_empty(shape, dtype=dtype)
        if given_back:
            t.record_stream(self.current_stream(t.device))
        return t


_torch_names = None


def _names():
    global _torch_names
    if _torch_names is None:
        _torch_names = _Torch()
    return _torch_names


def gdr_workspace_size(batch, seqlen, heads, headdim=128, d_state=128, groups=1, act=MM_BF16) -> int:
    return int(lib().mamba_gdr_workspace_size(batch, seqlen, heads, headdim, d_state, groups, act))


def gdr_fwd(q, k, v, dt, beta, dt_bias, A, h0=None, *, scale=None, norm_eps=1e-6, y=None, h_last=None,
            workspace=None, stream=None):
    """The gated delta rule (mamba_gdr_fwd): q, k [B,L,G,N] and v [B,L,H,P]
    (bf16 or fp32; they may be parts of one packed tensor, rows evenly spaced
    and 16-byte multiples apart), dt and beta [B,L,H] (same dtype), dt_bias/A
    [H] fp32 (dt_bias may be None), h0 [B,H,P,N] fp32 or None.  scale defaults
    to N ** -0.5; q and k are L2-normalised with norm_eps, or used as they are
    when it is 0.  Returns (y [B,L,H,P], h_last [B,H,P,N] fp32), allocating any
    output not given."""
    T = _torch_names or _names()
    if stream is None and T.calls is not None:
        out = T.calls.gdr_fwd(q, k, v, dt, beta, dt_bias, A, h0, scale, norm_eps, y, h_last, workspace)
        if out is not None:
            return out
    f32, dtype, idx = T.f32, v.dtype, v.get_device()
    act = T.codes.get(dtype)
    if act is None:
        _act_code(dtype)
    Bsz, L, H, P = v.shape
    G, N = q.shape[2:]
    tokens, keys, state = (Bsz, L, H), (Bsz, L, G, N), (Bsz, H, P, N)
    if not (idx >= 0 and q.dtype is dtype and k.dtype is dtype and q.get_device() == idx and k.get_device() == idx
            and q.shape == keys and k.shape == keys and A is not None
            and dt.shape == tokens and dt.dtype is dtype and dt.get_device() == idx and dt.is_contiguous()
            and beta.shape == tokens and beta.dtype is dtype and beta.get_device() == idx and beta.is_contiguous()
            and A.shape == (H,) and A.dtype is f32 and A.get_device() == idx and A.is_contiguous()
            and (dt_bias is None or (dt_bias.shape == (H,) and dt_bias.dtype is f32 and dt_bias.get_device() == idx
                                     and dt_bias.is_contiguous()))
            and (h0 is None or (h0.shape == state and h0.dtype is f32 and h0.get_device() == idx and h0.is_contiguous()))
            and (y is None or (y.shape == v.shape and y.dtype is dtype and y.get_device() == idx and y.is_contiguous()))
            and (h_last is None or (h_last.shape == state and h_last.dtype is f32 and h_last.get_device() == idx
                                    and h_last.is_contiguous()))):
        dev = v.device
        for t, name, want, shape in ((dt, "dt", dtype, tokens), (beta, "beta", dtype, tokens), (A, "A", f32, (H,))):
            _required(t, name)
            _check(t, name, want, shape, dev)
        for t, name, want, shape in ((dt_bias, "dt_bias", f32, (H,)), (h0, "h0", f32, state), (y, "y", dtype, (Bsz, L, H, P)),
                                     (h_last, "h_last", f32, state)):
            _check(t, name, want, shape, dev)
        for t, name, shape in ((q, "q", keys), (k, "k", keys), (v, "v", (Bsz, L, H, P))):
            _check_rows(t, name, dtype, shape, dev)
    if Bsz > 0 and L > 1:
        (qb, qs, qh, q1), (kb, ks, kh, k1), (vb, vs, vh, v1) = q.stride(), k.stride(), v.stride()
        plain = (q1 == 1 and k1 == 1 and v1 == 1 and qh == N and kh == N and vh == P
                 and qb == L * qs and kb == L * ks and vb == L * vs)
    else:
        plain = False
    if not plain:
        qs, ks, vs = (_check_rows(t, name, dtype, shape, v.device)
                      for t, name, shape in ((q, "q", keys), (k, "k", keys), (v, "v", (Bsz, L, H, P))))
    if T.current_device() != idx:
        with T.device(idx):
            return gdr_fwd(q, k, v, dt, beta, dt_bias, A, h0, scale=scale, norm_eps=norm_eps, y=y, h_last=h_last,
                           workspace=workspace, stream=stream)
    if y is None:
        y = T.empty(v, (Bsz, L, H, P), dtype, stream)
    if h_last is None:
        h_last = T.empty(v, state, f32, stream)
    while True:
        if workspace is None:
            have = max(T.lib.mamba_gdr_workspace_size(Bsz, L, H, P, N, G, act), 256)
            workspace = T.empty(v, (have,), T.u8, stream, given_back=False)
        else:
            if workspace.get_device() != idx:
                raise ValueError(f"workspace is on {workspace.device}, expected {v.device}")
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            have = workspace.nbytes
        st = T.lib.mamba_gdr_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), beta.data_ptr(),
                                 None if dt_bias is None else dt_bias.data_ptr(), A.data_ptr(),
                                 None if h0 is None else h0.data_ptr(), y.data_ptr(), h_last.data_ptr(),
                                 Bsz, L, G, H, P, N, qs, ks, vs, N ** -0.5 if scale is None else scale, norm_eps, act,
                                 workspace.data_ptr(), have, T.raw_stream(idx) if stream is None else stream.cuda_stream)
        if st == 0:
            break
        if st != _ERR_WORKSPACE or have >= T.lib.mamba_gdr_workspace_size(Bsz, L, H, P, N, G, act):
            raise MixerError(st, "mamba_gdr_fwd")
        workspace = None          # the one given is too small
    return y, h_last


def gdr_state_update(q, k, v, dt, beta, dt_bias, A, state, *, scale=None, norm_eps=1e-6, y=None, stream=None):
    """One token of the gated delta rule (mamba_gdr_state_update), in place on
    state [B,H,P,N] fp32: q, k [B,G,N] and v [B,H,P] (bf16 or fp32; rows evenly
    spaced), dt and beta [B,H], dt_bias/A [H] fp32 (dt_bias may be None).  scale
    and norm_eps as gdr_fwd.  Returns y [B,H,P], allocated if not given."""
    T = _torch_names or _names()
    if stream is None and T.calls is not None:
        out = T.calls.gdr_state_update(q, k, v, dt, beta, dt_bias, A, state, scale, norm_eps, y)
        if out is not None:
            return out
    f32, dtype, idx = T.f32, v.dtype, v.get_device()
    act = T.codes.get(dtype)
    if act is None:
        _act_code(dtype)
    Bsz, H, P = v.shape
    G, N = q.shape[1:]
    tokens, keys = (Bsz, H), (Bsz, G, N)
    if not (idx >= 0 and q.dtype is dtype and k.dtype is dtype and q.get_device() == idx and k.get_device() == idx
            and q.shape == keys and k.shape == keys and A is not None and state is not None
            and dt.shape == tokens and dt.dtype is dtype and dt.get_device() == idx and dt.is_contiguous()
            and beta.shape == tokens and beta.dtype is dtype and beta.get_device() == idx and beta.is_contiguous()
            and A.shape == (H,) and A.dtype is f32 and A.get_device() == idx and A.is_contiguous()
            and (dt_bias is None or (dt_bias.shape == (H,) and dt_bias.dtype is f32 and dt_bias.get_device() == idx
                                     and dt_bias.is_contiguous()))
            and state.shape == (Bsz, H, P, N) and state.dtype is f32 and state.get_device() == idx and state.is_contiguous()
            and (y is None or (y.shape == v.shape and y.dtype is dtype and y.get_device() == idx and y.is_contiguous()))):
        dev = v.device
        for t, name, want, shape in ((dt, "dt", dtype, tokens), (beta, "beta", dtype, tokens), (A, "A", f32, (H,)),
                                     (state, "state", f32, (Bsz, H, P, N))):
            _required(t, name)
            _check(t, name, want, shape, dev)
        _check(dt_bias, "dt_bias", f32, (H,), dev)
        _check(y, "y", dtype, (Bsz, H, P), dev)
        for t, name, shape in ((q, "q", keys), (k, "k", keys), (v, "v", (Bsz, H, P))):
            _check_rows(t, name, dtype, shape, dev)
    (qs, qh, q1), (ks, kh, k1), (vs, vh, v1) = q.stride(), k.stride(), v.stride()
    if Bsz == 1:                  # one row of each: as far apart as dense ones
        qs, ks, vs = G * N, G * N, H * P
    if not (Bsz > 0 and q1 == 1 and k1 == 1 and v1 == 1 and qh == N and kh == N and vh == P):
        qs, ks, vs = (_check_rows(t, name, dtype, shape, v.device)
                      for t, name, shape in ((q, "q", keys), (k, "k", keys), (v, "v", (Bsz, H, P))))
    if T.current_device() != idx:
        with T.device(idx):
            return gdr_state_update(q, k, v, dt, beta, dt_bias, A, state, scale=scale, norm_eps=norm_eps, y=y, stream=stream)
    if y is None:
        y = T.empty(v, (Bsz, H, P), dtype, stream)
    st = T.lib.mamba_gdr_state_update(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), beta.data_ptr(),
                                      None if dt_bias is None else dt_bias.data_ptr(), A.data_ptr(), state.data_ptr(),
                                      y.data_ptr(), Bsz, G, H, P, N, qs, ks, vs, N ** -0.5 if scale is None else scale,
                                      norm_eps, act, T.raw_stream(idx) if stream is None else stream.cuda_stream)
    if st != 0:
        raise MixerError(st, "mamba_gdr_state_update")
    return y


def proj_q4(x, W, scales, zeros=None, *, group=128, out=None, out_dtype=None, stream=None):
    """out = x W^T for a few rows x [M,K] bf16 and a weight of 4-bit numbers
    (mamba_proj_q4): W [N,K/2] uint8 (even inputs in the low four bits), scales
    and zeros [N,K/group] bf16 (zeros None: 8), weight = scale (number - zero).
    out [M,N] fp32 (default) or bf16, allocated if not given."""
    T = _torch_names or _names()
    dtype = out_dtype or (out.dtype if out is not None else T.f32)
    if stream is None and T.calls is not None and dtype in T.codes:
        made = T.calls.proj_q4(x, W, scales, zeros, group, out, dtype is T.bf16)
        if made is not None:
            return made
    bf, idx = T.bf16, x.get_device()
    M, K = x.shape
    N = W.shape[0]
    if group <= 0:
        raise ValueError(f"group must be positive, got {group}")
    code = T.codes.get(dtype)
    if code is None:
        _act_code(dtype)
    groups = (N, K // group)
    if not (idx >= 0 and x.dtype is bf and x.is_contiguous()
            and W.shape == (N, K // 2) and W.dtype is T.u8 and W.get_device() == idx and W.is_contiguous()
            and scales.shape == groups and scales.dtype is bf and scales.get_device() == idx and scales.is_contiguous()
            and (zeros is None or (zeros.shape == groups and zeros.dtype is bf and zeros.get_device() == idx
                                   and zeros.is_contiguous()))
            and (out is None or (out.shape == (M, N) and out.dtype is dtype and out.get_device() == idx
                                 and out.is_contiguous()))):
        for t, name, want, shape in ((x, "x", bf, (M, K)), (W, "W", T.u8, (N, K // 2)), (scales, "scales", bf, groups),
                                     (zeros, "zeros", bf, groups), (out, "out", dtype, (M, N))):
            _check(t, name, want, shape, x.device)
    if T.current_device() != idx:
        with T.device(idx):
            return proj_q4(x, W, scales, zeros, group=group, out=out, out_dtype=out_dtype, stream=stream)
    if out is None:
        out = T.empty(x, (M, N), dtype, stream)
    st = T.lib.mamba_proj_q4(x.data_ptr(), W.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
                             out.data_ptr(), M, N, K, group, code, T.raw_stream(idx) if stream is None else stream.cuda_stream)
    if st != 0:
        raise MixerError(st, "mamba_proj_q4")
    return out

"""MI355X (gfx950) selective state-space hot path: Python binding.

Thin ctypes marshalling over the C ABI of ``libmamba_amd.so`` (declared in
``include/mamba_amd.h``).  Every step of the computation runs in the HIP
kernels of that library; this module only checks tensor metadata, takes
device pointers and the current HIP stream, and raises on a non-OK status.
There is no CPU fallback: if the library is missing, calls raise.

Entry points (same names as the C ABI, without the ``mamba_`` prefix):
  conv1d_silu(x, w, bias=None, out=None)
  selective_scan_fwd(x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, h0=None,
                     return_last_state=False, out=None, workspace=None)
  selective_state_update(h, x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, out=None)
  selective_scan_fwd_workspace_size(B, D, L, N, dtype)
  conv1d_selective_scan_fwd(x_raw, conv_w, dt, A, Bm, Cm, conv_bias=None,
                            conv_state_in=None, return_conv_state=False, ...)
  conv1d_update(state, x, w, bias=None, out=None)
  selective_scan_bwd(x, dt, A, Bm, Cm, dout, dt_bias=None, Dskip=None, z=None, h0=None,
                     dh_last=None, workspace=None)
  selective_scan_bwd_workspace_size(B, D, L, N, dtype)
  ssd_scan_fwd(x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, h0=None,
               return_last_state=False, out=None, h_last=None)
  selective_scan_fwd_noalloc(x, dt, A, Bm, Cm, ..., out=None, h_last=None)
  rms_norm(x, weight, residual=None, eps=1e-5, out=None, residual_out=None)
  rms_norm_int8(x, weight, residual=None, eps=1e-5, out=None, scale=None, residual_out=None)
  rms_norm_bwd(dy, h, weight, dresidual_out=None, eps=1e-5, workspace=None)
  quantize_int8(x, channel_major=False, out=None, scale=None)
  int8_matmul(a, b, a_scale, b_scale, out_dtype=torch.bfloat16, out=None)
  int8_matmul_form(M, N, K, batch=1, aligned=True, flags=0)   diagnostic
  gated_scan_fwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, h0=None, reset=None, c=8.0,
                 return_last_state=False, return_checkpoints=False, out=None, ...)
  gated_scan_bwd(x, r, i, lam, dout, r_bias=None, i_bias=None, z=None, h0=None, reset=None,
                 dh_last=None, c=8.0, checkpoints=None, workspace=None)
  gated_scan_fwd_workspace_size(B, D, L)
  gated_scan_bwd_workspace_size(B, D, L, with_checkpoints=True)
  gated_state_update(h, x, r, i, lam, r_bias=None, i_bias=None, z=None, c=8.0, h_out=None, out=None)
  quantize_mxfp4(x, channel_major=False, out=None, scale=None)
  dequantize_mxfp4(q, scale, K=None, dtype=torch.bfloat16, out=None)
  mxfp4_matmul(a, b, a_scale, b_scale, out_dtype=torch.bfloat16, out=None)
  mxfp4_matmul_form(M, N, K, batch=1, flags=0)   diagnostic
  selective_scan_check(workspace)        the carry's error word (after a sync)
  set_scan_spin_limit(polls)             diagnostic bound of the carry waits
Test helper: set_carry_checks(True) checks the carry after every scan call.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libmamba_amd.so")
ABI_VERSION = 9  # MAMBA_AMD_ABI_VERSION of include/mamba_amd.h that this binding follows

MAMBA_F32 = 0
MAMBA_BF16 = 1
MAMBA_SCAN_REVERSE = 1
MAMBA_SCAN_ACCUMULATE = 2

STATUS_NAMES = {0: "MAMBA_OK", 1: "MAMBA_ERR_NULL", 2: "MAMBA_ERR_SHAPE", 3: "MAMBA_ERR_DTYPE",
                4: "MAMBA_ERR_UNSUPPORTED", 5: "MAMBA_ERR_ALIGN", 6: "MAMBA_ERR_ALIAS",
                7: "MAMBA_ERR_WORKSPACE", 8: "MAMBA_ERR_LAUNCH", 9: "MAMBA_ERR_DEVICE",
                10: "MAMBA_ERR_TIMEOUT"}

# every symbol include/mamba_amd.h declares
EXPORTED = ["mamba_status_string", "mamba_abi_version", "mamba_conv1d_silu",
            "mamba_selective_scan_fwd_workspace_size", "mamba_selective_scan_fwd",
            "mamba_selective_state_update", "mamba_selective_scan_fwd_ex",
            "mamba_conv1d_selective_scan_fwd",
            "mamba_conv1d_update", "mamba_set_scan_timing_events",
            "mamba_selective_scan_bwd_workspace_size", "mamba_selective_scan_bwd",
            "mamba_ssd_scan_fwd", "mamba_conv1d_selective_state_update",
            "mamba_selective_scan_check", "mamba_set_scan_spin_limit",
            "mamba_selective_scan_fwd_noalloc", "mamba_rms_norm", "mamba_rms_norm_int8",
            "mamba_rms_norm_bwd_workspace_size", "mamba_rms_norm_bwd", "mamba_quantize_int8",
            "mamba_int8_matmul", "mamba_int8_matmul_form",
            "mamba_gated_scan_checkpoints", "mamba_gated_scan_fwd_workspace_size",
            "mamba_gated_scan_fwd",
            "mamba_gated_scan_bwd_workspace_size", "mamba_gated_scan_bwd",
            "mamba_gated_state_update", "mamba_quantize_mxfp4", "mamba_dequantize_mxfp4",
            "mamba_mxfp4_matmul", "mamba_mxfp4_matmul_form"]

_lib = None


class MambaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load_library(path: str = LIBRARY):
    """Load libmamba_amd.so and declare its signatures (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m selective_state_space_80_amd.build`"
                           " (the HIP library is required, there is no fallback)")
    lib = ctypes.CDLL(path)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    rebuild = "rebuild it (`python -m selective_state_space_80_amd.build`)"
    # entry points are added without a new version: callers of the others need none
    missing = [name for name in EXPORTED if not hasattr(lib, name)]
    if missing:
        raise RuntimeError(f"{path} lacks {', '.join(missing)}: {rebuild}")
    lib.mamba_status_string.restype = ctypes.c_char_p
    lib.mamba_status_string.argtypes = [I32]
    lib.mamba_abi_version.restype = I32
    lib.mamba_abi_version.argtypes = []
    if lib.mamba_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{path} has ABI version {lib.mamba_abi_version()}, this binding "
                           f"follows {ABI_VERSION}: {rebuild}")
    lib.mamba_conv1d_silu.restype = I32
    lib.mamba_conv1d_silu.argtypes = [P, P, P, P, I64, I64, I64, I64, I32, P]
    lib.mamba_selective_scan_fwd_workspace_size.restype = SZ
    lib.mamba_selective_scan_fwd_workspace_size.argtypes = [I64, I64, I64, I64, I32]
    lib.mamba_selective_scan_fwd.restype = I32
    lib.mamba_selective_scan_fwd.argtypes = [P] * 12 + [SZ, I64, I64, I64, I64, I32, P]
    lib.mamba_selective_state_update.restype = I32
    lib.mamba_selective_state_update.argtypes = [P] * 10 + [I64, I64, I64, I32, ctypes.c_uint, P]
    lib.mamba_selective_scan_fwd_ex.restype = I32
    lib.mamba_selective_scan_fwd_ex.argtypes = ([P] * 12 + [SZ, I64, I64, I64, I64, I32,
                                                             ctypes.c_uint, P])
    lib.mamba_conv1d_selective_scan_fwd.restype = I32
    lib.mamba_conv1d_selective_scan_fwd.argtypes = ([P, P, P, I64] + [P] * 13 +
                                                    [SZ, I64, I64, I64, I64, I32, P])
    lib.mamba_conv1d_update.restype = I32
    lib.mamba_conv1d_update.argtypes = [P] * 5 + [I64, I64, I64, I32, P]
    lib.mamba_conv1d_selective_state_update.restype = I32
    lib.mamba_conv1d_selective_state_update.argtypes = ([P] * 5 + [I64] + [P] * 8 +
                                                        [I64, I64, I64, I32, ctypes.c_uint, P])
    lib.mamba_selective_scan_bwd_workspace_size.restype = SZ
    lib.mamba_selective_scan_bwd_workspace_size.argtypes = [I64, I64, I64, I64, I32]
    lib.mamba_selective_scan_bwd.restype = I32
    lib.mamba_selective_scan_bwd.argtypes = [P] * 21 + [SZ, I64, I64, I64, I64, I32, P]
    lib.mamba_ssd_scan_fwd.restype = I32
    lib.mamba_ssd_scan_fwd.argtypes = [P] * 11 + [I64] * 6 + [I32, P]
    lib.mamba_set_scan_timing_events.restype = None
    lib.mamba_set_scan_timing_events.argtypes = [P, P]
    lib.mamba_selective_scan_fwd_noalloc.restype = I32
    lib.mamba_selective_scan_fwd_noalloc.argtypes = [P] * 11 + [I64, I64, I64, I64, I32, P]
    lib.mamba_selective_scan_check.restype = I32
    lib.mamba_selective_scan_check.argtypes = [P, SZ, P]
    lib.mamba_set_scan_spin_limit.restype = None
    lib.mamba_set_scan_spin_limit.argtypes = [I32]
    U32, F = ctypes.c_uint, ctypes.c_float
    lib.mamba_rms_norm.restype = I32
    lib.mamba_rms_norm.argtypes = [P] * 5 + [I64, I64, F, I32, I32, P]
    lib.mamba_rms_norm_int8.restype = I32
    lib.mamba_rms_norm_int8.argtypes = [P] * 6 + [I64, I64, F, I32, I32, P]
    lib.mamba_rms_norm_bwd_workspace_size.restype = SZ
    lib.mamba_rms_norm_bwd_workspace_size.argtypes = [I64, I64]
    lib.mamba_rms_norm_bwd.restype = I32
    lib.mamba_rms_norm_bwd.argtypes = [P] * 8 + [SZ, I64, I64, F, I32, I32, P]
    lib.mamba_quantize_int8.restype = I32
    lib.mamba_quantize_int8.argtypes = [P] * 3 + [I64, I64, I64, I32, I32, P]
    lib.mamba_int8_matmul.restype = I32
    lib.mamba_int8_matmul.argtypes = [P] * 5 + [I64, I64, I64, I64, I32, U32, P]
    lib.mamba_int8_matmul_form.restype = I32
    lib.mamba_int8_matmul_form.argtypes = [I64] * 4 + [I32, U32, P, P, P]
    lib.mamba_gated_scan_checkpoints.restype = I64
    lib.mamba_gated_scan_checkpoints.argtypes = [I64]
    lib.mamba_gated_scan_fwd.restype = I32
    lib.mamba_gated_scan_fwd_workspace_size.restype = SZ
    lib.mamba_gated_scan_fwd_workspace_size.argtypes = [I64, I64, I64]
    lib.mamba_gated_scan_fwd.argtypes = [P] * 13 + [SZ, I64, I64, I64, F, I32, P]
    lib.mamba_gated_scan_bwd_workspace_size.restype = SZ
    lib.mamba_gated_scan_bwd_workspace_size.argtypes = [I64, I64, I64, I32]
    lib.mamba_gated_scan_bwd.restype = I32
    lib.mamba_gated_scan_bwd.argtypes = [P] * 21 + [SZ, I64, I64, I64, F, I32, P]
    lib.mamba_gated_state_update.restype = I32
    lib.mamba_gated_state_update.argtypes = [P] * 10 + [I64, I64, F, I32, P]
    lib.mamba_quantize_mxfp4.restype = I32
    lib.mamba_quantize_mxfp4.argtypes = [P] * 3 + [I64, I64, I64, I32, I32, P]
    lib.mamba_dequantize_mxfp4.restype = I32
    lib.mamba_dequantize_mxfp4.argtypes = [P] * 3 + [I64, I64, I32, P]
    lib.mamba_mxfp4_matmul.restype = I32
    lib.mamba_mxfp4_matmul.argtypes = [P] * 5 + [I64, I64, I64, I64, I32, U32, P]
    lib.mamba_mxfp4_matmul_form.restype = I32
    lib.mamba_mxfp4_matmul_form.argtypes = [I64] * 4 + [U32, P, P, P]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().mamba_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS_NAMES.get(int(status), "unknown")


_torch_module = None
_io_types = {}  # torch dtype -> mamba_dtype, filled when torch is first used


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _io_types.update({torch.float32: MAMBA_F32, torch.bfloat16: MAMBA_BF16})
        _torch_module = torch
    return _torch_module


def _io_dtype(t) -> int:
    _torch()
    io = _io_types.get(t.dtype)
    if io is None:
        raise TypeError(f"I/O tensors must be float32 or bfloat16, got {t.dtype}")
    return io


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, shape, dtype=None, device=None, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _workspace(workspace, need, device):
    """(the caller's workspace, or one made here; its bytes)."""
    if workspace is None:
        workspace = _torch().empty(max(need, 1), dtype=_torch().uint8, device=device)
    elif workspace.device != device:  # the kernels would write to it
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _stream(device):
    return ctypes.c_void_p(_torch().cuda.current_stream(device).cuda_stream)


def _addr(t):
    return None if t is None else t.data_ptr()


_current_raw_stream = None


def _raw_stream(t):
    """The current stream of t's GPU as an integer (raises for a CPU tensor)."""
    global _current_raw_stream
    index = t.get_device()
    if index < 0:
        raise ValueError(f"expected a tensor on a GPU, got one on {t.device}")
    if _current_raw_stream is None:
        torch = _torch()
        # the handle itself costs 0.1 us; by way of a torch.cuda.Stream object, 1.9
        _current_raw_stream = getattr(
            torch._C, "_cuda_getCurrentRawStream",
            lambda i: torch.cuda.current_stream(torch.device("cuda", i)).cuda_stream)
    return _current_raw_stream(index)


def _raise(st, where):
    if st != 0:
        raise MambaError(st, where)


def conv1d_silu(x, w, bias=None, out=None):
    """Causal depthwise conv1d + SiLU.  x [B,D,L] (f32/bf16), w [D,K] f32,
    bias [D] f32 or None.  Returns out [B,D,L] of x's dtype."""
    torch = _torch()
    lib = load_library()
    B, D, L = x.shape
    K = w.shape[1]
    _check(x, "x", (B, D, L), device=x.device)
    _check(w, "w", (D, K), torch.float32, x.device)
    _check(bias, "bias", (D,), torch.float32, x.device, optional=True)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", (B, D, L), x.dtype, x.device)
    st = lib.mamba_conv1d_silu(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), B, D, L, K,
                               _io_dtype(x), _stream(x.device))
    _raise(st, "mamba_conv1d_silu")
    return out


_carry_checks = False


def set_carry_checks(on: bool = True) -> None:
    """After every scan and backward call, wait for the stream and check the
    workspace's carry error word (raises MambaError with MAMBA_ERR_TIMEOUT).
    Each check synchronizes, so this is for tests, not for timed runs."""
    global _carry_checks
    _carry_checks = bool(on)


def selective_scan_check(workspace) -> None:
    """Wait for the workspace's stream, then raise MambaError(MAMBA_ERR_TIMEOUT)
    if a carry wait of the calls that last used it gave up (their affected
    outputs are NaN)."""
    st = load_library().mamba_selective_scan_check(_ptr(workspace),
                                                   workspace.numel() * workspace.element_size(),
                                                   _stream(workspace.device))
    _raise(st, "mamba_selective_scan_check")


def set_scan_spin_limit(polls: int) -> None:
    """Diagnostic: polls before a carry wait of later scans gives up (< 0: the
    default).  0 makes any wait not met at once give up, for failure-path tests."""
    load_library().mamba_set_scan_spin_limit(int(polls))


def _after_scan(workspace, need):
    # a check synchronizes, which a stream under graph capture cannot do
    if _carry_checks and need >= 256 and not _torch().cuda.is_current_stream_capturing():
        selective_scan_check(workspace)


def selective_scan_fwd_workspace_size(B, D, L, N, dtype=None) -> int:
    io = MAMBA_F32 if dtype is None else _io_dtype(_torch().empty(0, dtype=dtype))
    return int(load_library().mamba_selective_scan_fwd_workspace_size(B, D, L, N, io))


def selective_scan_fwd(x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, h0=None,
                       return_last_state=False, out=None, workspace=None, h_last=None,
                       reverse=False, accumulate=False):
    """Fused selective-scan forward.  x, dt, z [B,D,L]; Bm, Cm [B,L,N] (all of
    one dtype, f32 or bf16); A [D,N], dt_bias [D], Dskip [D], h0 [B,D,N] f32.
    Returns y [B,D,L] (x's dtype), and h_last [B,D,N] f32 if return_last_state.
    reverse: scan from step L-1 down to 0; accumulate: add into `out`."""
    torch = _torch()
    lib = load_library()
    B, D, L = x.shape
    N = A.shape[1]
    dev, io_t = x.device, x.dtype
    _check(x, "x", (B, D, L), io_t, dev)
    _check(dt, "dt", (B, D, L), io_t, dev)
    _check(z, "z", (B, D, L), io_t, dev, optional=True)
    _check(Bm, "Bm", (B, L, N), io_t, dev)
    _check(Cm, "Cm", (B, L, N), io_t, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(dt_bias, "dt_bias", (D,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (D,), torch.float32, dev, optional=True)
    _check(h0, "h0", (B, D, N), torch.float32, dev, optional=True)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs `out` (the tensor added to)")
        out = torch.empty_like(x)
    _check(out, "out", (B, D, L), io_t, dev)
    if return_last_state and h_last is None:
        h_last = torch.empty((B, D, N), dtype=torch.float32, device=dev)
    _check(h_last, "h_last", (B, D, N), torch.float32, dev, optional=True)
    io = _io_dtype(x)
    need = int(lib.mamba_selective_scan_fwd_workspace_size(B, D, L, N, io))
    workspace, workspace_bytes = _workspace(workspace, need, dev)
    flags = (MAMBA_SCAN_REVERSE if reverse else 0) | (MAMBA_SCAN_ACCUMULATE if accumulate else 0)
    if flags:
        st = lib.mamba_selective_scan_fwd_ex(
            _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z),
            _ptr(h0), _ptr(out), _ptr(h_last), _ptr(workspace), workspace_bytes, B, D, L, N, io,
            flags, _stream(dev))
        _raise(st, "mamba_selective_scan_fwd_ex")
    else:
        st = lib.mamba_selective_scan_fwd(
            _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z),
            _ptr(h0), _ptr(out), _ptr(h_last), _ptr(workspace), workspace_bytes, B, D, L, N,
            io, _stream(dev))
        _raise(st, "mamba_selective_scan_fwd")
    _after_scan(workspace, need)
    if return_last_state:
        return out, h_last
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20  # MAMBA_NOALLOC_SCRATCH_BYTES of include/mamba_amd.h


def selective_scan_fwd_noalloc(x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, h0=None,
                               out=None, h_last=None):
    """mamba_selective_scan_fwd_noalloc: the scan with the library's own scratch
    in place of a workspace (the C call allocates nothing; `out` / `h_last`
    given by the caller keep this wrapper allocation-free too).  Shapes whose
    workspace exceeds NOALLOC_SCRATCH_BYTES raise MAMBA_ERR_WORKSPACE.
    Returns out, or (out, h_last) when h_last is given."""
    torch = _torch()
    lib = load_library()
    B, D, L = x.shape
    N = A.shape[1]
    dev, io_t = x.device, x.dtype
    _check(x, "x", (B, D, L), io_t, dev)
    _check(dt, "dt", (B, D, L), io_t, dev)
    _check(z, "z", (B, D, L), io_t, dev, optional=True)
    _check(Bm, "Bm", (B, L, N), io_t, dev)
    _check(Cm, "Cm", (B, L, N), io_t, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(dt_bias, "dt_bias", (D,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (D,), torch.float32, dev, optional=True)
    _check(h0, "h0", (B, D, N), torch.float32, dev, optional=True)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", (B, D, L), io_t, dev)
    _check(h_last, "h_last", (B, D, N), torch.float32, dev, optional=True)
    st = lib.mamba_selective_scan_fwd_noalloc(
        _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z),
        _ptr(h0), _ptr(out), _ptr(h_last), B, D, L, N, _io_dtype(x), _stream(dev))
    _raise(st, "mamba_selective_scan_fwd_noalloc")
    return (out, h_last) if h_last is not None else out


def conv1d_selective_scan_fwd(x_raw, conv_w, dt, A, Bm, Cm, conv_bias=None, conv_state_in=None,
                              return_conv_state=False, conv_state_out=None, dt_bias=None,
                              Dskip=None, z=None, h0=None, return_last_state=False, out=None,
                              workspace=None, h_last=None):
    """conv1d (K <= 4 taps) + SiLU fused into the selective scan.  x_raw [B,D,L]
    (f32/bf16) is the raw block input; conv_w [D,K], conv_bias [D] f32;
    conv_state_in / conv_state_out [B,D,K-1] of x_raw's dtype (the raw inputs
    before t = 0 / of the last K-1 steps; out may be the same tensor as in).
    Other arguments as for selective_scan_fwd.  Returns y, then h_last if
    return_last_state, then the conv state if return_conv_state."""
    torch = _torch()
    lib = load_library()
    B, D, L = x_raw.shape
    N = A.shape[1]
    K = conv_w.shape[1]
    dev, io_t = x_raw.device, x_raw.dtype
    _check(x_raw, "x_raw", (B, D, L), io_t, dev)
    _check(conv_w, "conv_w", (D, K), torch.float32, dev)
    _check(conv_bias, "conv_bias", (D,), torch.float32, dev, optional=True)
    _check(conv_state_in, "conv_state_in", (B, D, K - 1), io_t, dev, optional=True)
    _check(dt, "dt", (B, D, L), io_t, dev)
    _check(z, "z", (B, D, L), io_t, dev, optional=True)
    _check(Bm, "Bm", (B, L, N), io_t, dev)
    _check(Cm, "Cm", (B, L, N), io_t, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(dt_bias, "dt_bias", (D,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (D,), torch.float32, dev, optional=True)
    _check(h0, "h0", (B, D, N), torch.float32, dev, optional=True)
    if out is None:
        out = torch.empty_like(x_raw)
    _check(out, "out", (B, D, L), io_t, dev)
    if return_last_state and h_last is None:
        h_last = torch.empty((B, D, N), dtype=torch.float32, device=dev)
    _check(h_last, "h_last", (B, D, N), torch.float32, dev, optional=True)
    if return_conv_state and conv_state_out is None:
        conv_state_out = torch.empty((B, D, K - 1), dtype=io_t, device=dev)
    _check(conv_state_out, "conv_state_out", (B, D, K - 1), io_t, dev, optional=True)
    io = _io_dtype(x_raw)
    need = int(lib.mamba_selective_scan_fwd_workspace_size(B, D, L, N, io))
    workspace, workspace_bytes = _workspace(workspace, need, dev)
    st = lib.mamba_conv1d_selective_scan_fwd(
        _ptr(x_raw), _ptr(conv_w), _ptr(conv_bias), K, _ptr(conv_state_in), _ptr(conv_state_out),
        _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(h0),
        _ptr(out), _ptr(h_last), _ptr(workspace), workspace_bytes, B, D, L, N, io,
        _stream(dev))
    _raise(st, "mamba_conv1d_selective_scan_fwd")
    _after_scan(workspace, need)
    res = [out]
    if return_last_state:
        res.append(h_last)
    if return_conv_state:
        res.append(conv_state_out)
    return res[0] if len(res) == 1 else tuple(res)


def conv1d_update(state, x, w, bias=None, out=None):
    """One decode step of the conv front end.  state [B,D,K-1] (x's dtype) is
    updated in place; x [B,D] f32/bf16; w [D,K], bias [D] f32.  Returns out
    [B,D] = SiLU(conv) of x's dtype."""
    torch = _torch()
    lib = load_library()
    B, D = x.shape
    K = w.shape[1]
    dev, io_t = x.device, x.dtype
    _check(x, "x", (B, D), io_t, dev)
    _check(w, "w", (D, K), torch.float32, dev)
    _check(bias, "bias", (D,), torch.float32, dev, optional=True)
    _check(state, "state", (B, D, K - 1), io_t, dev, optional=(K == 1))
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", (B, D), io_t, dev)
    st = lib.mamba_conv1d_update(_ptr(state), _ptr(x), _ptr(w), _ptr(bias), _ptr(out), B, D, K,
                                 _io_dtype(x), _stream(dev))
    _raise(st, "mamba_conv1d_update")
    return out


STEP_STREAM_STATE = 1  # MAMBA_STEP_STREAM_STATE


def _step_flags(stream_state):
    return STEP_STREAM_STATE if stream_state else 0


def selective_state_update(h, x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, out=None,
                           stream_state=False):
    """One decode step.  h [B,D,N] f32 is updated in place; x, dt, z [B,D] and
    Bm, Cm [B,N] share one dtype (f32/bf16).  Returns y [B,D] of that dtype.
    stream_state: h is loaded and stored with nontemporal hints (the same
    results), for a state that leaves the caches before its next step anyway."""
    torch = _torch()
    lib = load_library()
    B, D, N = h.shape
    dev, io_t = h.device, x.dtype
    _check(h, "h", (B, D, N), torch.float32, dev)
    _check(x, "x", (B, D), io_t, dev)
    _check(dt, "dt", (B, D), io_t, dev)
    _check(z, "z", (B, D), io_t, dev, optional=True)
    _check(Bm, "Bm", (B, N), io_t, dev)
    _check(Cm, "Cm", (B, N), io_t, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(dt_bias, "dt_bias", (D,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (D,), torch.float32, dev, optional=True)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", (B, D), io_t, dev)
    st = lib.mamba_selective_state_update(
        _ptr(h), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip),
        _ptr(z), _ptr(out), B, D, N, _io_dtype(x), _step_flags(stream_state), _stream(dev))
    _raise(st, "mamba_selective_state_update")
    return out


def conv1d_selective_state_update(h, conv_state, x_raw, conv_w, dt, A, Bm, Cm, conv_bias=None,
                                  dt_bias=None, Dskip=None, z=None, out=None, stream_state=False):
    """The block's decode step in one kernel: the conv front end's step on the
    raw input x_raw [B,D] (conv_state [B,D,K-1] of x_raw's dtype, updated in
    place; conv_w [D,K] f32 with K <= 4, conv_bias [D] f32), feeding the state
    update of h [B,D,N] f32 (in place).  Other arguments as for
    selective_state_update.  Returns y [B,D] of x_raw's dtype."""
    torch = _torch()
    lib = load_library()
    B, D, N = h.shape
    K = conv_w.shape[1]
    dev, io_t = h.device, x_raw.dtype
    _check(h, "h", (B, D, N), torch.float32, dev)
    _check(conv_state, "conv_state", (B, D, K - 1), io_t, dev, optional=K == 1)
    _check(x_raw, "x_raw", (B, D), io_t, dev)
    _check(conv_w, "conv_w", (D, K), torch.float32, dev)
    _check(conv_bias, "conv_bias", (D,), torch.float32, dev, optional=True)
    _check(dt, "dt", (B, D), io_t, dev)
    _check(z, "z", (B, D), io_t, dev, optional=True)
    _check(Bm, "Bm", (B, N), io_t, dev)
    _check(Cm, "Cm", (B, N), io_t, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(dt_bias, "dt_bias", (D,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (D,), torch.float32, dev, optional=True)
    if out is None:
        out = torch.empty_like(x_raw)
    _check(out, "out", (B, D), io_t, dev)
    st = lib.mamba_conv1d_selective_state_update(
        _ptr(h), _ptr(conv_state), _ptr(x_raw), _ptr(conv_w), _ptr(conv_bias), K, _ptr(dt),
        _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(out), B, D, N,
        _io_dtype(x_raw), _step_flags(stream_state), _stream(dev))
    _raise(st, "mamba_conv1d_selective_state_update")
    return out


def selective_scan_bwd_workspace_size(B, D, L, N, dtype=None) -> int:
    io = MAMBA_F32 if dtype is None else _io_dtype(_torch().empty(0, dtype=dtype))
    return int(load_library().mamba_selective_scan_bwd_workspace_size(B, D, L, N, io))


def selective_scan_bwd(x, dt, A, Bm, Cm, dout, dt_bias=None, Dskip=None, z=None, h0=None,
                       dh_last=None, workspace=None):
    """Backward pass of selective_scan_fwd: gradients of sum(out * dout)
    (+ sum(h_last * dh_last)) with the forward states recomputed.  Inputs as
    for selective_scan_fwd; dout [B,D,L] of x's dtype; dh_last [B,D,N] f32 or
    None.  Returns a dict: dx, ddt, dz (None without z) of x's dtype and
    shape; dA [D,N], dB, dC [B,L,N], dD, ddt_bias [D], dh0 [B,D,N], all f32."""
    torch = _torch()
    lib = load_library()
    B, D, L = x.shape
    N = A.shape[1]
    dev, io_t = x.device, x.dtype
    _check(x, "x", (B, D, L), io_t, dev)
    _check(dt, "dt", (B, D, L), io_t, dev)
    _check(z, "z", (B, D, L), io_t, dev, optional=True)
    _check(dout, "dout", (B, D, L), io_t, dev)
    _check(Bm, "Bm", (B, L, N), io_t, dev)
    _check(Cm, "Cm", (B, L, N), io_t, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(dt_bias, "dt_bias", (D,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (D,), torch.float32, dev, optional=True)
    _check(h0, "h0", (B, D, N), torch.float32, dev, optional=True)
    _check(dh_last, "dh_last", (B, D, N), torch.float32, dev, optional=True)
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"dx": torch.empty_like(x), "ddt": torch.empty_like(x),
         "dz": torch.empty_like(x) if z is not None else None,
         "dA": torch.empty((D, N), **f32), "dB": torch.empty((B, L, N), **f32),
         "dC": torch.empty((B, L, N), **f32), "dD": torch.empty((D,), **f32),
         "ddt_bias": torch.empty((D,), **f32), "dh0": torch.empty((B, D, N), **f32)}
    io = _io_dtype(x)
    need = int(lib.mamba_selective_scan_bwd_workspace_size(B, D, L, N, io))
    workspace, workspace_bytes = _workspace(workspace, need, dev)
    st = lib.mamba_selective_scan_bwd(
        _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z),
        _ptr(h0), _ptr(dout), _ptr(dh_last), _ptr(g["dx"]), _ptr(g["ddt"]), _ptr(g["dA"]),
        _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]), _ptr(g["ddt_bias"]),
        _ptr(g["dh0"]), _ptr(workspace), workspace_bytes, B, D, L, N, io, _stream(dev))
    _raise(st, "mamba_selective_scan_bwd")
    _after_scan(workspace, need)
    return g


def ssd_scan_fwd(x, dt, A, Bm, Cm, dt_bias=None, Dskip=None, z=None, h0=None,
                 return_last_state=False, out=None, h_last=None):
    """Mamba-2 form of the scan (one decay per head, B/C per group of heads) on
    the matrix cores.  x, z [B,L,H,P], dt [B,L,H], Bm, Cm [B,L,G,N] bf16;
    A, dt_bias, Dskip [H] f32; h0 [B,H,P,N] f32.  Returns y [B,L,H,P] bf16,
    and h_last [B,H,P,N] f32 if return_last_state."""
    torch = _torch()
    lib = load_library()
    B, L, H, P = x.shape
    G, N = Bm.shape[2], Bm.shape[3]
    dev, io_t = x.device, x.dtype
    _check(x, "x", (B, L, H, P), io_t, dev)
    _check(dt, "dt", (B, L, H), io_t, dev)
    _check(z, "z", (B, L, H, P), io_t, dev, optional=True)
    _check(Bm, "Bm", (B, L, G, N), io_t, dev)
    _check(Cm, "Cm", (B, L, G, N), io_t, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (H,), torch.float32, dev, optional=True)
    _check(Dskip, "Dskip", (H,), torch.float32, dev, optional=True)
    _check(h0, "h0", (B, H, P, N), torch.float32, dev, optional=True)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", (B, L, H, P), io_t, dev)
    if return_last_state and h_last is None:
        h_last = torch.empty((B, H, P, N), dtype=torch.float32, device=dev)
    _check(h_last, "h_last", (B, H, P, N), torch.float32, dev, optional=True)
    st = lib.mamba_ssd_scan_fwd(
        _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z),
        _ptr(h0), _ptr(out), _ptr(h_last), B, L, H, P, G, N, _io_dtype(x), _stream(dev))
    _raise(st, "mamba_ssd_scan_fwd")
    if return_last_state:
        return out, h_last
    return out


def _is(t, shape, dtype, index):
    """A contiguous tensor of this shape and dtype on GPU `index` (the quick
    form of _check, which says what is wrong with one that is not)."""
    return (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous())


def _rows(shape):
    if len(shape) == 2:
        return shape[0]
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return rows


def _norm_arguments(x, weight, residual, residual_out):
    """Checks shared by the two forward norms; returns (rows, D, residual's
    element type, residual_out)."""
    torch = _torch()
    shape, index = x.shape, x.get_device()
    if not shape:
        raise ValueError("x has no axis to normalise")
    D = shape[-1]
    if not (x.is_contiguous() and _is(weight, (D,), torch.float32, index)):
        _check(x, "x", shape)
        _check(weight, "weight", (D,), torch.float32, x.device)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs residual")
        return _rows(shape), D, 0, None
    res_t = residual.dtype
    if res_t is not torch.float32 and res_t is not x.dtype:
        raise TypeError(f"residual must be float32 or {x.dtype}, got {res_t}")
    if not _is(residual, shape, res_t, index):
        _check(residual, "residual", shape, device=x.device)
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    elif not _is(residual_out, shape, res_t, index):
        _check(residual_out, "residual_out", shape, res_t, x.device)
    return _rows(shape), D, _io_dtype(residual), residual_out


def rms_norm(x, weight, residual=None, eps=1e-5, out=None, residual_out=None):
    """Root-mean-square norm over the last axis with the residual's addition:
    h = x + residual, out = h / sqrt(mean(h^2) + eps) * weight.  x [..., D]
    f32/bf16; weight [D] f32; residual [..., D] f32 or x's dtype.  Returns out
    of x's dtype, and with a residual (out, residual_out): h in the residual's
    dtype (`residual_out` may be `residual` itself, updated in place)."""
    lib = load_library()
    M, D, res_t, residual_out = _norm_arguments(x, weight, residual, residual_out)
    if out is None:
        out = _torch().empty_like(x)
    else:
        _check(out, "out", x.shape, x.dtype, x.device)
    st = lib.mamba_rms_norm(x.data_ptr(), _addr(residual), weight.data_ptr(), out.data_ptr(),
                            _addr(residual_out), M, D, eps, _io_dtype(x), res_t, _raw_stream(x))
    if st:
        _raise(st, "mamba_rms_norm")
    return out if residual is None else (out, residual_out)


def rms_norm_int8(x, weight, residual=None, eps=1e-5, out=None, scale=None, residual_out=None):
    """rms_norm with its output in 8-bit integers and a scale per row (the
    left operand of int8_matmul): scale = max|y| / 127, q = round(y / scale).
    Returns (q [..., D] int8, scale [...] f32), and residual_out with a
    residual.  A row with a NaN or an infinity has scale NaN."""
    torch = _torch()
    lib = load_library()
    M, D, res_t, residual_out = _norm_arguments(x, weight, residual, residual_out)
    if out is None:
        out = torch.empty_like(x, dtype=torch.int8)
    else:
        _check(out, "out", x.shape, torch.int8, x.device)
    if scale is None:
        scale = weight.new_empty(x.shape[:-1])
    else:
        _check(scale, "scale", x.shape[:-1], torch.float32, x.device)
    st = lib.mamba_rms_norm_int8(x.data_ptr(), _addr(residual), weight.data_ptr(), out.data_ptr(),
                                 scale.data_ptr(), _addr(residual_out), M, D, eps, _io_dtype(x),
                                 res_t, _raw_stream(x))
    if st:
        _raise(st, "mamba_rms_norm_int8")
    return (out, scale) if residual is None else (out, scale, residual_out)


def rms_norm_bwd_workspace_size(M, D) -> int:
    return int(load_library().mamba_rms_norm_bwd_workspace_size(M, D))


def rms_norm_bwd(dy, h, weight, dresidual_out=None, eps=1e-5, workspace=None):
    """Gradient of rms_norm.  dy [..., D] f32/bf16; h [..., D] the stored sum
    (residual_out of the forward call, or its x where it had no residual) in
    f32 or dy's dtype; dresidual_out the gradient that reaches residual_out, of
    h's dtype, or None.  Returns a dict: dx of dy's dtype, dresidual of h's
    dtype (the same tensor as dx where the dtypes are equal), dweight [D] f32."""
    torch = _torch()
    lib = load_library()
    if dy.dim() < 1:
        raise ValueError("dy has no axis to normalise")
    shape, dev, index, h_t = dy.shape, dy.device, dy.get_device(), h.dtype
    D = shape[-1]
    if h_t != torch.float32 and h_t != dy.dtype:
        raise TypeError(f"h must be float32 or {dy.dtype}, got {h_t}")
    if not (dy.is_contiguous() and _is(h, shape, h_t, index)
            and _is(weight, (D,), torch.float32, index)):
        _check(dy, "dy", shape)
        _check(h, "h", shape, device=dev)
        _check(weight, "weight", (D,), torch.float32, dev)
    if dresidual_out is not None and not _is(dresidual_out, shape, h_t, index):
        _check(dresidual_out, "dresidual_out", shape, h_t, dev)
    M = _rows(shape)
    dx = torch.empty_like(dy)
    dresidual = None if h_t == dy.dtype else torch.empty_like(h)
    dweight = torch.empty_like(weight)
    need = lib.mamba_rms_norm_bwd_workspace_size(M, D) if workspace is None else 0
    workspace, workspace_bytes = _workspace(workspace, need, dev)
    st = lib.mamba_rms_norm_bwd(
        dy.data_ptr(), h.data_ptr(), weight.data_ptr(), _addr(dresidual_out), dx.data_ptr(),
        _addr(dresidual), dweight.data_ptr(), workspace.data_ptr(), workspace_bytes, M, D, eps,
        _io_dtype(dy), _io_dtype(h), _raw_stream(dy))
    if st:
        _raise(st, "mamba_rms_norm_bwd")
    return {"dx": dx, "dresidual": dx if dresidual is None else dresidual, "dweight": dweight}


def quantize_int8(x, channel_major=False, out=None, scale=None):
    """8-bit integers with a scale per row: scale = max|x| / 127 over the row,
    q = round(x / scale).  x [..., K] f32/bf16 -> q [..., K] int8, scale [...]
    f32 (tokens, or a weight's output channels).  channel_major: x is [B, K, L],
    as the scans write their output, and q [B, L, K], scale [B, L]."""
    torch = _torch()
    lib = load_library()
    dev, shape = x.device, x.shape
    if not x.is_contiguous():
        _check(x, "x", shape)
    if channel_major:
        if len(shape) != 3:
            raise ValueError(f"channel-major x is [B, K, L], got {tuple(shape)}")
        B, K, L = shape
        lead = (B, L)
    else:
        if len(shape) < 1:
            raise ValueError("x has no axis to quantise")
        lead, K = shape[:-1], shape[-1]
        B, L = 1, _rows(shape)
    if out is None:
        out = (x.new_empty((*lead, K), dtype=torch.int8) if channel_major
               else torch.empty_like(x, dtype=torch.int8))
    else:
        _check(out, "out", (*lead, K), torch.int8, dev)
    if scale is None:
        scale = x.new_empty(lead, dtype=torch.float32)
    else:
        _check(scale, "scale", lead, torch.float32, dev)
    st = lib.mamba_quantize_int8(x.data_ptr(), out.data_ptr(), scale.data_ptr(), B, L, K,
                                 1 if channel_major else 0, _io_dtype(x), _raw_stream(x))
    if st:
        _raise(st, "mamba_quantize_int8")
    return out, scale


INT8_SHARED_A = 1  # MAMBA_INT8_SHARED_A
INT8_SHARED_B = 2  # MAMBA_INT8_SHARED_B


def int8_matmul(a, b, a_scale, b_scale, out_dtype=None, out=None):
    """out[..., m, n] = a_scale[m] b_scale[n] sum_k a[m, k] b[n, k], summed
    exactly.  a [M, K] or [B, M, K], b [N, K] or [B, N, K] int8 (a 2-D operand
    is used by every batch of a 3-D one); scales f32 of the operands' leading
    shapes.  Returns out [M, N] or [B, M, N] of out_dtype (bfloat16, the
    default, or float32).  With tokens as `a` and a weight [N, K] as `b` it is
    a projection; with the weight as `a`, its channel-major form."""
    torch = _torch()
    lib = load_library()
    a_shape, b_shape = a.shape, b.shape
    a_dim, b_dim = len(a_shape), len(b_shape)
    if a_dim not in (2, 3) or b_dim not in (2, 3):
        raise ValueError(f"a and b are 2-D or 3-D, got {a_dim}-D and {b_dim}-D")
    M, K, N = a_shape[-2], a_shape[-1], b_shape[-2]
    if a_dim == 2 and b_dim == 2:
        batch, flags = 1, 0
        a_rows, b_rows, out_shape = (M,), (N,), (M, N)
    else:
        batch = a_shape[0] if a_dim == 3 else b_shape[0]
        flags = (INT8_SHARED_A if a_dim == 2 else 0) | (INT8_SHARED_B if b_dim == 2 else 0)
        a_rows = (M,) if a_dim == 2 else (batch, M)
        b_rows = (N,) if b_dim == 2 else (batch, N)
        out_shape = (batch, M, N)
    index, i8, f32 = a.get_device(), torch.int8, torch.float32
    if not (a.dtype is i8 and a.is_contiguous() and _is(b, (*b_rows, K), i8, index)
            and _is(a_scale, a_rows, f32, index) and _is(b_scale, b_rows, f32, index)):
        _check(a, "a", (*a_rows, K), i8)
        _check(b, "b", (*b_rows, K), i8, a.device)
        _check(a_scale, "a_scale", a_rows, f32, a.device)
        _check(b_scale, "b_scale", b_rows, f32, a.device)
    if out is None:
        out = a.new_empty(out_shape, dtype=torch.bfloat16 if out_dtype is None else out_dtype)
    else:
        _check(out, "out", out_shape, out_dtype, a.device)
    st = lib.mamba_int8_matmul(a.data_ptr(), b.data_ptr(), a_scale.data_ptr(), b_scale.data_ptr(),
                               out.data_ptr(), batch, M, N, K, _io_dtype(out), flags, _raw_stream(a))
    if st:
        _raise(st, "mamba_int8_matmul")
    return out


def int8_matmul_form(M, N, K, batch=1, aligned=True, flags=0):
    """Diagnostic: which kernel int8_matmul takes for these sizes, as (form, tiles,
    slots) of mamba_int8_matmul_form.  Needs no GPU."""
    form, tiles, slots = ctypes.c_int(), ctypes.c_int64(), ctypes.c_int()
    st = load_library().mamba_int8_matmul_form(batch, M, N, K, 1 if aligned else 0, flags, ctypes.byref(form),
                                               ctypes.byref(tiles), ctypes.byref(slots))
    if st:
        _raise(st, "mamba_int8_matmul_form")
    return form.value, tiles.value, slots.value


def _gated_arguments(x, r, i, lam, r_bias, i_bias, z, h0, reset):
    """Checks shared by the gated recurrence's calls; reset [B, L] for a scan."""
    torch = _torch()
    shape, io_t, index, f32 = x.shape, x.dtype, x.get_device(), torch.float32
    per = (shape[1],)
    if not (x.is_contiguous() and _is(r, shape, io_t, index) and _is(i, shape, io_t, index)
            and _is(lam, per, f32, index) and (r_bias is None or _is(r_bias, per, f32, index))
            and (i_bias is None or _is(i_bias, per, f32, index))
            and (z is None or _is(z, shape, io_t, index))):
        dev = x.device
        _check(x, "x", shape)
        _check(r, "r", shape, io_t, dev)
        _check(i, "i", shape, io_t, dev)
        _check(lam, "lam", per, f32, dev)
        _check(r_bias, "r_bias", per, f32, dev, optional=True)
        _check(i_bias, "i_bias", per, f32, dev, optional=True)
        _check(z, "z", shape, io_t, dev, optional=True)
    if h0 is not None and not _is(h0, shape[:2], f32, index):
        _check(h0, "h0", shape[:2], f32, x.device)
    if reset is not None:
        if reset.dtype is not torch.bool and reset.dtype is not torch.uint8:
            raise TypeError(f"reset must be bool or uint8, got {reset.dtype}")
        if not _is(reset, (shape[0], shape[2]), reset.dtype, index):
            _check(reset, "reset", (shape[0], shape[2]), device=x.device)


def gated_scan_fwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, h0=None, reset=None, c=8.0,
                   return_last_state=False, return_checkpoints=False, out=None, h_last=None,
                   checkpoints=None, workspace=None):
    """Gated linear recurrence over [B, D, L]: with v = c softplus(lam) sigmoid(r + r_bias) and
    a = exp(-v), h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i + i_bias) x, y = h or h SiLU(z).
    x, r, i, z [B,D,L] f32/bf16; lam, r_bias, i_bias [D] f32; h0 [B,D] f32; reset [B,L] bool or
    uint8: steps at which the state before is dropped (the first token of a packed sequence).
    A token with r = -inf leaves the state as it is.  Returns y of x's dtype, then h_last [B,D]
    f32 if return_last_state, then checkpoints [B,D,ceil(L/512)] f32, for gated_scan_bwd, if
    return_checkpoints."""
    torch = _torch()
    lib = load_library()
    B, D, L = x.shape
    _gated_arguments(x, r, i, lam, r_bias, i_bias, z, h0, reset)
    f32 = torch.float32
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", x.shape, x.dtype, x.device)
    if h_last is not None:
        _check(h_last, "h_last", (B, D), f32, x.device)
    elif return_last_state:
        h_last = lam.new_empty((B, D))
    if return_checkpoints or checkpoints is not None:
        kept = (B, D, lib.mamba_gated_scan_checkpoints(L))
        if checkpoints is None:
            checkpoints = lam.new_empty(kept)
        else:
            _check(checkpoints, "checkpoints", kept, f32, x.device)
    workspace_bytes = 0
    if workspace is not None:
        workspace, workspace_bytes = _workspace(workspace, 0, x.device)
    else:
        need = lib.mamba_gated_scan_fwd_workspace_size(B, D, L)
        if need:
            workspace, workspace_bytes = _workspace(None, need, x.device)
    st = lib.mamba_gated_scan_fwd(x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(),
                                  _addr(r_bias), _addr(i_bias), _addr(z), _addr(h0), _addr(reset),
                                  out.data_ptr(), _addr(h_last), _addr(checkpoints), _addr(workspace),
                                  workspace_bytes, B, D, L, c, _io_dtype(x), _raw_stream(x))
    if st:
        _raise(st, "mamba_gated_scan_fwd")
    got = (out,) + ((h_last,) if return_last_state else ()) + (
        (checkpoints,) if return_checkpoints else ())
    return out if len(got) == 1 else got


def gated_scan_fwd_workspace_size(B, D, L) -> int:
    return int(load_library().mamba_gated_scan_fwd_workspace_size(B, D, L))


def gated_scan_bwd_workspace_size(B, D, L, with_checkpoints=True) -> int:
    return int(load_library().mamba_gated_scan_bwd_workspace_size(B, D, L, 1 if with_checkpoints else 0))


def gated_scan_bwd(x, r, i, lam, dout, r_bias=None, i_bias=None, z=None, h0=None, reset=None,
                   dh_last=None, c=8.0, checkpoints=None, workspace=None):
    """Gradients of sum(y * dout) + sum(h_last * dh_last) of gated_scan_fwd.  checkpoints: as that
    call returned them (h0 is then not read), or None: its pass is run again for them.  Returns a
    dict: dx, dr, di, dz (None without z) of x's dtype; dlam, dr_bias, di_bias [D] and dh0 [B,D] f32."""
    torch = _torch()
    lib = load_library()
    B, D, L = x.shape
    _gated_arguments(x, r, i, lam, r_bias, i_bias, z, h0, reset)
    dev, index, f32 = x.device, x.get_device(), torch.float32
    if not _is(dout, x.shape, x.dtype, index):
        _check(dout, "dout", x.shape, x.dtype, dev)
    _check(dh_last, "dh_last", (B, D), f32, dev, optional=True)
    if checkpoints is not None:
        kept = (B, D, lib.mamba_gated_scan_checkpoints(L))
        if not _is(checkpoints, kept, f32, index):
            _check(checkpoints, "checkpoints", kept, f32, dev)
    g = {"dx": torch.empty_like(x), "dr": torch.empty_like(x), "di": torch.empty_like(x),
         "dz": None if z is None else torch.empty_like(x), "dlam": torch.empty_like(lam),
         "dr_bias": torch.empty_like(lam), "di_bias": torch.empty_like(lam),
         "dh0": lam.new_empty((B, D))}
    workspace_bytes = 0
    if workspace is None:
        need = lib.mamba_gated_scan_bwd_workspace_size(B, D, L, 0 if checkpoints is None else 1)
        if need:
            workspace, workspace_bytes = _workspace(None, need, dev)
    else:
        workspace, workspace_bytes = _workspace(workspace, 0, dev)
    st = lib.mamba_gated_scan_bwd(
        x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), _addr(r_bias), _addr(i_bias),
        _addr(z), _addr(h0), _addr(reset), _addr(checkpoints), dout.data_ptr(), _addr(dh_last),
        g["dx"].data_ptr(), g["dr"].data_ptr(), g["di"].data_ptr(), _addr(g["dz"]),
        g["dlam"].data_ptr(), g["dr_bias"].data_ptr(), g["di_bias"].data_ptr(), g["dh0"].data_ptr(),
        _addr(workspace), workspace_bytes, B, D, L, c, _io_dtype(x), _raw_stream(x))
    if st:
        _raise(st, "mamba_gated_scan_bwd")
    return g


def gated_state_update(h, x, r, i, lam, r_bias=None, i_bias=None, z=None, c=8.0, h_out=None, out=None):
    """One step of gated_scan_fwd (decode).  h [B,D] f32, updated in place, or left as it is with
    the new state in h_out; x, r, i, z [B,D] f32/bf16.  Returns y [B,D] of x's dtype."""
    torch = _torch()
    lib = load_library()
    shape, index, f32 = x.shape, x.get_device(), torch.float32
    B, D = shape
    if h is None or not _is(h, shape, f32, index):
        _check(h, "h", shape, f32, x.device)
    _gated_arguments(x, r, i, lam, r_bias, i_bias, z, None, None)
    if h_out is None:
        h_out = h
    elif not _is(h_out, shape, f32, index):
        _check(h_out, "h_out", shape, f32, x.device)
    if out is None:
        out = torch.empty_like(x)
    elif not _is(out, shape, x.dtype, index):
        _check(out, "out", shape, x.dtype, x.device)
    st = lib.mamba_gated_state_update(h.data_ptr(), h_out.data_ptr(), x.data_ptr(), r.data_ptr(),
                                      i.data_ptr(), lam.data_ptr(), _addr(r_bias), _addr(i_bias),
                                      _addr(z), out.data_ptr(), B, D, c, _io_dtype(x), _raw_stream(x))
    if st:
        _raise(st, "mamba_gated_state_update")
    return out


MXFP4_GROUP = 256  # elements a packed row is filled up to a multiple of: 128 bytes, 8 scales
MXFP4_SHARED_A = 1  # MAMBA_MXFP4_SHARED_A
MXFP4_SHARED_B = 2  # MAMBA_MXFP4_SHARED_B


def quantize_mxfp4(x, channel_major=False, out=None, scale=None):
    """Microscaled 4-bit floating point: along the last axis a power of two for every 32
    elements, the elements rounded to 0, .5, 1, 1.5, 2, 3, 4, 6 and a sign.  x [..., K] f32/bf16
    -> q [..., G * 128] uint8 (two elements a byte, zeros from K on) and scale [G, ..., 8] uint8
    (exponent + 127), G = ceil(K / 256).  channel_major: x is [B, K, L], as the scans write
    their output, and q [B, L, G * 128], scale [G, B, L, 8].  A block with a NaN or an infinity
    has scale NaN."""
    torch = _torch()
    lib = load_library()
    dev, shape = x.device, x.shape
    if not x.is_contiguous():
        _check(x, "x", shape)
    if channel_major:
        if len(shape) != 3:
            raise ValueError(f"channel-major x is [B, K, L], got {tuple(shape)}")
        B, K, L = shape
        lead = (B, L)
    else:
        if len(shape) < 1:
            raise ValueError("x has no axis to quantise")
        lead, K = shape[:-1], shape[-1]
        B, L = 1, _rows(shape)
    groups = -(-K // MXFP4_GROUP)
    u8 = torch.uint8
    if out is None:
        out = x.new_empty((*lead, groups * 128), dtype=u8)
    else:
        _check(out, "out", (*lead, groups * 128), u8, dev)
    if scale is None:
        scale = x.new_empty((groups, *lead, 8), dtype=u8)
    else:
        _check(scale, "scale", (groups, *lead, 8), u8, dev)
    st = lib.mamba_quantize_mxfp4(x.data_ptr(), out.data_ptr(), scale.data_ptr(), B, L, K,
                                  1 if channel_major else 0, _io_dtype(x), _raw_stream(x))
    if st:
        _raise(st, "mamba_quantize_mxfp4")
    return out, scale


def _mxfp4_operand(q, scale, name, index):
    """Checks a packed operand and its scales; returns its number of groups."""
    shape, u8 = q.shape, _torch().uint8
    if not shape or shape[-1] % 128:
        raise ValueError(f"{name} has rows of whole groups of 128 bytes, got {tuple(shape)}")
    groups = shape[-1] // 128
    want = (groups, shape[0], 8) if len(shape) == 2 else (groups, *shape[:-1], 8)
    if not (q.dtype is u8 and q.is_contiguous() and q.get_device() == index
            and _is(scale, want, u8, index)):
        _check(q, name, shape, u8)
        _check(scale, f"{name}_scale", want, u8, q.device)
        raise ValueError(f"{name} is on {q.device}, expected another device")
    return groups


def dequantize_mxfp4(q, scale, K=None, dtype=None, out=None):
    """The values of quantize_mxfp4's rows: [..., K] of dtype (bfloat16, the default, or float32).
    K: the row's elements, all of its groups' where it is not given."""
    torch = _torch()
    lib = load_library()
    groups = _mxfp4_operand(q, scale, "q", q.get_device())
    if K is None:
        K = groups * MXFP4_GROUP
    elif -(-K // MXFP4_GROUP) != groups:
        raise ValueError(f"rows of {groups} groups do not have {K} elements")
    shape = (*q.shape[:-1], K)
    if out is None:
        out = q.new_empty(shape, dtype=torch.bfloat16 if dtype is None else dtype)
    else:
        _check(out, "out", shape, dtype, q.device)
    st = lib.mamba_dequantize_mxfp4(q.data_ptr(), scale.data_ptr(), out.data_ptr(), _rows(q.shape), K,
                                    _io_dtype(out), _raw_stream(q))
    if st:
        _raise(st, "mamba_dequantize_mxfp4")
    return out


def mxfp4_matmul(a, b, a_scale, b_scale, out_dtype=None, out=None):
    """out[..., m, n] = sum_k A[m, k] B[n, k] of the values that quantize_mxfp4's rows stand for,
    summed in fp32.  a [M, G * 128] or [B, M, G * 128], b [N, G * 128] or [B, N, G * 128] uint8 (a
    2-D operand is used by every batch of a 3-D one); scales [G, M, 8] or [G, B, M, 8] and alike.
    Returns out [M, N] or [B, M, N] of out_dtype (bfloat16, the default, or float32).  With tokens
    as `a` and a weight as `b` it is a projection; with the weight as `a`, its channel-major form."""
    torch = _torch()
    lib = load_library()
    a_dim, b_dim = a.dim(), b.dim()
    if a_dim not in (2, 3) or b_dim not in (2, 3):
        raise ValueError(f"a and b are 2-D or 3-D, got {a_dim}-D and {b_dim}-D")
    index = a.get_device()
    groups = _mxfp4_operand(a, a_scale, "a", index)
    if _mxfp4_operand(b, b_scale, "b", index) != groups:
        raise ValueError(f"rows of a and b differ: {a.shape[-1]} and {b.shape[-1]} bytes")
    M, N = a.shape[-2], b.shape[-2]
    if a_dim == 2 and b_dim == 2:
        batch, flags, out_shape = 1, 0, (M, N)
    else:
        batch = a.shape[0] if a_dim == 3 else b.shape[0]
        if a_dim == b_dim and b.shape[0] != batch:
            raise ValueError(f"a has {batch} batches, b {b.shape[0]}")
        flags = (MXFP4_SHARED_A if a_dim == 2 else 0) | (MXFP4_SHARED_B if b_dim == 2 else 0)
        out_shape = (batch, M, N)
    if out is None:
        out = a.new_empty(out_shape, dtype=torch.bfloat16 if out_dtype is None else out_dtype)
    else:
        _check(out, "out", out_shape, out_dtype, a.device)
    st = lib.mamba_mxfp4_matmul(a.data_ptr(), b.data_ptr(), a_scale.data_ptr(), b_scale.data_ptr(),
                                out.data_ptr(), batch, M, N, groups * MXFP4_GROUP, _io_dtype(out), flags,
                                _raw_stream(a))
    if st:
        _raise(st, "mamba_mxfp4_matmul")
    return out


def mxfp4_matmul_form(M, N, K, batch=1, flags=0):
    """Diagnostic: which kernel mxfp4_matmul takes for these sizes, as (form, tiles, slots) of
    mamba_mxfp4_matmul_form.  Needs no GPU."""
    form, tiles, slots = ctypes.c_int(), ctypes.c_int64(), ctypes.c_int()
    st = load_library().mamba_mxfp4_matmul_form(batch, M, N, K, flags, ctypes.byref(form), ctypes.byref(tiles),
                                                ctypes.byref(slots))
    if st:
        _raise(st, "mamba_mxfp4_matmul_form")
    return form.value, tiles.value, slots.value


def set_scan_timing_events_raw(start=None, stop=None):
    """Have later scan calls from this thread record the raw hipEvent_t
    handles `start` / `stop` (ctypes.c_void_p) around their main kernel, on the
    call's stream.  None, None turns it off."""
    lib = load_library()
    if start is None or stop is None:
        lib.mamba_set_scan_timing_events(None, None)
    else:
        lib.mamba_set_scan_timing_events(start, stop)

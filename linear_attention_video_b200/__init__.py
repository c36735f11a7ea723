"""Python binding of libkda.so: the B200 (sm_100a) forward pass of the
modality-aware short convolution followed by the Kimi Delta Attention scan,
their backward pass, and the operators beside them (linear attention with a
decay per head, rotary positions, layer norm).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/kda.h``.  Tensors are torch
CUDA tensors (torch supplies device memory and streams); the functions take
the same names and arguments as the C entry points and raise ``KdaError``
when an entry point returns a non-zero status.  The C ABI receives bare
addresses and cannot see buffer sizes, so every tensor is first checked
against the problem (element count, dtype, device, contiguity); a mismatch
raises ``KdaError(KDA_ERR_INVALID_ARG)`` before anything is launched.  There
is no CPU fallback: importing this package fails if the compiled library is
missing.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libkda.so not found at {LIB_PATH}; build it with "
                      f"`python linear_attention_video_b200/build.py` (nvcc, sm_100a)")

_lib = ctypes.CDLL(LIB_PATH)

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_MISALIGNED = 0, 1, 2, 3
KDA_ERR_WORKSPACE, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_DEVICE_ASSERT, KDA_ERR_RANGE = 4, 5, 6, 7, 8
KDA_DT_BF16, KDA_DT_F32 = 0, 1
KDA_FLAG_VIS_CAUSAL_T = 1
KDA_FLAG_REUSE_RECORDS = 2
KDA_FLAG_QKV_F16 = 4
KDA_ROPE_INTERLEAVED = 1

EXPORTS = ("kda_tokens", "kda_workspace_bytes", "kda_shortconv_fwd", "kda_chunk_fwd", "kda_fwd",
           "kda_chunk_fwd_noalloc", "kda_fwd_host_workspace_bytes", "kda_fwd_host", "kda_bwd_workspace_bytes",
           "kda_bwd", "kda_rope_fwd", "kda_rope_bwd", "kda_layernorm_fwd", "kda_layernorm_bwd_workspace_bytes",
           "kda_layernorm_bwd", "kda_linear_workspace_bytes", "kda_linear_fwd", "kda_linear_bwd_workspace_bytes",
           "kda_linear_bwd", "kda_linear_step", "kda_selftest_wait_timeout", "kda_read_status", "kda_status_str",
           "kda_last_launch_count")


class kda_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("text_len", ctypes.c_int64),
                ("grid_t", ctypes.c_int32), ("grid_h", ctypes.c_int32), ("grid_w", ctypes.c_int32),
                ("text_k", ctypes.c_int32),
                ("vis_kt", ctypes.c_int32), ("vis_kh", ctypes.c_int32), ("vis_kw", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class kda_rope(ctypes.Structure):
    _fields_ = [("pairs_t", ctypes.c_int32), ("pairs_h", ctypes.c_int32), ("pairs_w", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


_vp, _sz, _i, _pp = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(kda_problem)
_lib.kda_tokens.argtypes = [_pp]
_lib.kda_tokens.restype = ctypes.c_int64
_lib.kda_workspace_bytes.argtypes = [_pp, _i]
_lib.kda_workspace_bytes.restype = _sz
_lib.kda_shortconv_fwd.argtypes = [_pp, _i] + [_vp] * 9
_lib.kda_shortconv_fwd.restype = _i
_lib.kda_chunk_fwd.argtypes = [_pp, _i] + [_vp] * 9 + [_sz, _vp]
_lib.kda_chunk_fwd.restype = _i
_lib.kda_fwd.argtypes = [_pp, _i] + [_vp] * 11 + [_sz, _vp]
_lib.kda_fwd.restype = _i
_lib.kda_chunk_fwd_noalloc.argtypes = [_pp, _i] + [_vp] * 10
_lib.kda_chunk_fwd_noalloc.restype = _i
_lib.kda_fwd_host_workspace_bytes.argtypes = [_pp, _i, ctypes.c_int32]
_lib.kda_fwd_host_workspace_bytes.restype = _sz
_lib.kda_fwd_host.argtypes = [_pp, _i] + [_vp] * 10 + [ctypes.c_int32, _vp, _sz, _vp, _vp, _vp]
_lib.kda_fwd_host.restype = _i
_lib.kda_bwd_workspace_bytes.argtypes = [_pp, _i]
_lib.kda_bwd_workspace_bytes.restype = _sz
_lib.kda_bwd.argtypes = [_pp, _i] + [_vp] * 19 + [_sz, _vp]
_lib.kda_bwd.restype = _i
_lib.kda_rope_fwd.argtypes = [_pp, ctypes.POINTER(kda_rope), _i] + [_vp] * 7
_lib.kda_rope_fwd.restype = _i
_lib.kda_rope_bwd.argtypes = _lib.kda_rope_fwd.argtypes
_lib.kda_rope_bwd.restype = _i
_lib.kda_layernorm_fwd.argtypes = [ctypes.c_int64, ctypes.c_int32, _i] + [_vp] * 3 + [ctypes.c_float] + [_vp] * 4
_lib.kda_layernorm_fwd.restype = _i
_lib.kda_layernorm_bwd_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32]
_lib.kda_layernorm_bwd_workspace_bytes.restype = _sz
_lib.kda_layernorm_bwd.argtypes = [ctypes.c_int64, ctypes.c_int32, _i] + [_vp] * 9 + [_sz, _vp]
_lib.kda_layernorm_bwd.restype = _i
_lib.kda_linear_workspace_bytes.argtypes = [_pp, _i]
_lib.kda_linear_workspace_bytes.restype = _sz
_lib.kda_linear_fwd.argtypes = [_pp, _i] + [_vp] * 9 + [_sz, _vp]
_lib.kda_linear_fwd.restype = _i
_lib.kda_linear_bwd_workspace_bytes.argtypes = [_pp, _i]
_lib.kda_linear_bwd_workspace_bytes.restype = _sz
_lib.kda_linear_bwd.argtypes = [_pp, _i] + [_vp] * 13 + [_sz, _vp]
_lib.kda_linear_bwd.restype = _i
_lib.kda_linear_step.argtypes = [_pp, _i] + [_vp] * 8
_lib.kda_linear_step.restype = _i
_lib.kda_selftest_wait_timeout.argtypes = [_pp, _i] + [_vp] * 7 + [_sz, ctypes.c_int32, ctypes.c_uint32, _vp]
_lib.kda_selftest_wait_timeout.restype = _i
_lib.kda_read_status.argtypes = [_vp, _vp]
_lib.kda_read_status.restype = _i
_lib.kda_status_str.argtypes = [_i]
_lib.kda_status_str.restype = ctypes.c_char_p
_lib.kda_last_launch_count.argtypes = []
_lib.kda_last_launch_count.restype = _i


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {kda_status_str(status)} (status {status})")
        self.status = status


def problem(B, H, d, text_len, grid, text_k=4, vis_k=(3, 3, 3), chunk=64, vis_causal_t=False,
            dv=None, reuse_records=False, qkv_f16=False) -> kda_problem:
    T, Hg, Wg = grid
    flags = ((KDA_FLAG_VIS_CAUSAL_T if vis_causal_t else 0) | (KDA_FLAG_REUSE_RECORDS if reuse_records else 0)
             | (KDA_FLAG_QKV_F16 if qkv_f16 else 0))
    return kda_problem(B, H, d, d if dv is None else dv, text_len, T, Hg, Wg, text_k,
                       vis_k[0], vis_k[1], vis_k[2], chunk, flags)


def rope(pairs, interleaved=False) -> kda_rope:
    """Rotary layout: pairs of a head turned by the (time, height, width) position, together d/2."""
    return kda_rope(*pairs, KDA_ROPE_INTERLEAVED if interleaved else 0)


def _dt(dtype) -> int:
    if dtype == torch.bfloat16:
        return KDA_DT_BF16
    if dtype == torch.float32:
        return KDA_DT_F32
    raise TypeError(f"unsupported dtype {dtype}")


# ---------------------------------------------------------------------------
# argument checks: the C ABI takes bare addresses, so sizes are checked here
# ---------------------------------------------------------------------------
def _dims(p: kda_problem):
    n = _lib.kda_tokens(ctypes.byref(p))
    if n < 0 or p.B < 1 or p.H < 1 or p.dk < 1 or p.dv < 1:
        raise KdaError(KDA_ERR_INVALID_ARG, "problem")
    return p.B, n, p.H, p.dk, p.dv


class _Args:
    """Collects the tensor arguments of one call and checks them against the problem."""

    def __init__(self, where: str, device: str = "cuda"):
        self.where, self.device, self.seen = where, device, []

    def fail(self, msg):
        raise KdaError(KDA_ERR_INVALID_ARG, f"{self.where}: {msg}")

    def add(self, name, t, numel, dtypes, device=None, at_least=False):
        if t is None or isinstance(t, int):   # optional argument absent, or a caller-managed raw address
            return self
        if not isinstance(t, torch.Tensor):
            self.fail(f"{name} must be a torch tensor")
        if numel > 0:   # zero-size arguments take any placeholder (the ABI wants a non-NULL address)
            if (t.numel() < numel) if at_least else (t.numel() != numel):
                self.fail(f"{name} has {t.numel()} elements, the problem needs {numel}")
            if t.dtype not in dtypes:
                self.fail(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if not t.is_contiguous():
            self.fail(f"{name} must be contiguous")
        self.seen.append((name, t, device or self.device))
        return self

    def check_devices(self):
        cuda = [(n, t) for n, t, dev in self.seen if dev == "cuda"]
        for n, t, dev in self.seen:
            if t.device.type != dev:
                self.fail(f"{n} must be a {dev.upper()} tensor, got {t.device}")
        if cuda:
            idx = {t.device.index for _, t in cuda}
            if len(idx) != 1:
                self.fail("device tensors on different GPUs")
            if idx.pop() != torch.cuda.current_device():
                self.fail("device tensors are not on the current CUDA device")


def _act_dtypes(p: kda_problem, dtype):
    """Element types of the convolved activations: fp16 under KDA_FLAG_QKV_F16, else the problem's."""
    return (torch.float16,) if p.flags & KDA_FLAG_QKV_F16 else (dtype,)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# the current stream's handle without a Stream object around it (3 us), where this torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != KDA_OK:
        raise KdaError(rc, where)


def kda_status_str(status: int) -> str:
    return _lib.kda_status_str(status).decode()


def kda_tokens(p: kda_problem) -> int:
    return _lib.kda_tokens(ctypes.byref(p))


def kda_workspace_bytes(p: kda_problem, dtype) -> int:
    return _lib.kda_workspace_bytes(ctypes.byref(p), _dt(dtype) if not isinstance(dtype, int) else dtype)


def kda_last_launch_count() -> int:
    return _lib.kda_last_launch_count()


def alloc_workspace(p: kda_problem, dtype, device="cuda") -> torch.Tensor:
    n = kda_workspace_bytes(p, dtype)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kda_shortconv_fwd(p, q, k, v, w_text, w_vis, q_out, k_out, v_out, stream=None):
    B, N, H, dk, dv = _dims(p)
    dt = q.dtype
    a = _Args("kda_shortconv_fwd")
    for n, t, d in (("q", q, dk), ("k", k, dk), ("v", v, dv)):
        a.add(n, t, B * N * H * d, (dt,))
    for n, t, d in (("q_out", q_out, dk), ("k_out", k_out, dk), ("v_out", v_out, dv)):
        a.add(n, t, B * N * H * d, _act_dtypes(p, dt))
    a.add("w_text", w_text, 3 * H * dk * p.text_k, (torch.float32,))
    a.add("w_vis", w_vis, 3 * H * dk * p.vis_kt * p.vis_kh * p.vis_kw, (torch.float32,))
    a.check_devices()
    _check(_lib.kda_shortconv_fwd(ctypes.byref(p), _dt(q.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(w_text),
                                  _ptr(w_vis), _ptr(q_out), _ptr(k_out), _ptr(v_out), _stream(stream)),
           "kda_shortconv_fwd")


def _scan_args(where, p, dtype, q, k, v, log_alpha, beta, o, s0, sn, workspace, nbytes, act_dtypes, host=False):
    B, N, H, dk, dv = _dims(p)
    dev = "cpu" if host else "cuda"
    a = _Args(where)
    a.add("q", q, B * N * H * dk, act_dtypes, dev).add("k", k, B * N * H * dk, act_dtypes, dev)
    a.add("v", v, B * N * H * dv, act_dtypes, dev)
    a.add("log_alpha", log_alpha, B * N * H * dk, (torch.float32,), dev)
    a.add("beta", beta, B * N * H, (dtype,), dev).add("o", o, B * N * H * dv, (dtype,), dev)
    a.add("initial_state", s0, B * H * dk * dv, (torch.float32,))
    a.add("final_state", sn, B * H * dk * dv, (torch.float32,))
    if workspace is not None and not isinstance(workspace, int):
        a.add("workspace", workspace, 1, (workspace.dtype,), at_least=True)
        if workspace.numel() * workspace.element_size() < nbytes:
            a.fail(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, fewer than the "
                   f"{nbytes} passed")
    return a


def kda_chunk_fwd(p, q, k, v, log_alpha, beta, o, workspace, initial_state=None, final_state=None,
                  stream=None, workspace_bytes=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    # the problem dtype is o's (q, k, v may be fp16 under KDA_FLAG_QKV_F16)
    _scan_args("kda_chunk_fwd", p, o.dtype, q, k, v, log_alpha, beta, o, initial_state, final_state, workspace,
               nbytes, _act_dtypes(p, o.dtype)).check_devices()
    _check(_lib.kda_chunk_fwd(ctypes.byref(p), _dt(o.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                              _ptr(beta), _ptr(initial_state), _ptr(o), _ptr(final_state), _ptr(workspace),
                              nbytes, _stream(stream)),
           "kda_chunk_fwd")


def _weight_args(a, p, w_text, w_vis):
    H, dk = p.H, p.dk
    a.add("w_text", w_text, 3 * H * dk * p.text_k, (torch.float32,))
    return a.add("w_vis", w_vis, 3 * H * dk * p.vis_kt * p.vis_kh * p.vis_kw, (torch.float32,))


def kda_fwd(p, q, k, v, log_alpha, beta, w_text, w_vis, o, workspace, initial_state=None, final_state=None,
            stream=None, workspace_bytes=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    a = _scan_args("kda_fwd", p, q.dtype, q, k, v, log_alpha, beta, o, initial_state, final_state, workspace,
                   nbytes, (q.dtype,))
    _weight_args(a, p, w_text, w_vis).check_devices()
    _check(_lib.kda_fwd(ctypes.byref(p), _dt(q.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                        _ptr(w_text), _ptr(w_vis), _ptr(initial_state), _ptr(o), _ptr(final_state),
                        _ptr(workspace), nbytes, _stream(stream)),
           "kda_fwd")


def kda_fwd_host_workspace_bytes(p: kda_problem, dtype, seg_frames: int) -> int:
    return _lib.kda_fwd_host_workspace_bytes(ctypes.byref(p), _dt(dtype), int(seg_frames))


def alloc_fwd_host_workspace(p: kda_problem, dtype, seg_frames: int, device="cuda") -> torch.Tensor:
    n = kda_fwd_host_workspace_bytes(p, dtype, seg_frames)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_fwd_host_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kda_fwd_host(p, q, k, v, log_alpha, beta, w_text, w_vis, o, workspace, seg_frames, initial_state=None,
                 final_state=None, stream=None, copy_in_stream=None, copy_out_stream=None, workspace_bytes=None):
    """kda_fwd on host tensors (q, k, v, log_alpha, beta, o on the CPU, pinned for overlap); the weights,
    the states and the workspace are on the device."""
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    a = _scan_args("kda_fwd_host", p, q.dtype, q, k, v, log_alpha, beta, o, initial_state, final_state, workspace,
                   nbytes, (q.dtype,), host=True)
    _weight_args(a, p, w_text, w_vis).check_devices()
    _check(_lib.kda_fwd_host(ctypes.byref(p), _dt(q.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                             _ptr(w_text), _ptr(w_vis), _ptr(initial_state), _ptr(o), _ptr(final_state),
                             int(seg_frames), _ptr(workspace), nbytes, _stream(stream), _stream(copy_in_stream),
                             _stream(copy_out_stream)),
           "kda_fwd_host")


def kda_chunk_fwd_noalloc(p, q, k, v, log_alpha, beta, o, initial_state=None, final_state=None,
                          device_status=None, stream=None):
    """kda_chunk_fwd without a workspace: scratch is the library's static device
    array (see include/kda.h for its limit and sharing rules)."""
    a = _scan_args("kda_chunk_fwd_noalloc", p, o.dtype, q, k, v, log_alpha, beta, o, initial_state, final_state,
                   None, 0, _act_dtypes(p, o.dtype))
    a.add("device_status", device_status, 1, (torch.int32, torch.uint32), at_least=True).check_devices()
    _check(_lib.kda_chunk_fwd_noalloc(ctypes.byref(p), _dt(o.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                      _ptr(beta), _ptr(initial_state), _ptr(o), _ptr(final_state),
                                      _ptr(device_status), _stream(stream)),
           "kda_chunk_fwd_noalloc")


def kda_bwd_workspace_bytes(p: kda_problem, dtype) -> int:
    return _lib.kda_bwd_workspace_bytes(ctypes.byref(p), _dt(dtype))


def alloc_bwd_workspace(p: kda_problem, dtype, device="cuda") -> torch.Tensor:
    n = kda_bwd_workspace_bytes(p, dtype)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kda_bwd(p, q, k, v, log_alpha, beta, w_text, w_vis, d_o, dq, dk, dv, d_log_alpha, d_beta, d_w_text, d_w_vis,
            workspace, initial_state=None, d_final_state=None, d_initial_state=None, stream=None,
            workspace_bytes=None):
    dk_, dv_ = dk, dv
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    a = _scan_args("kda_bwd", p, q.dtype, q, k, v, log_alpha, beta, d_o, initial_state, d_final_state, workspace,
                   nbytes, (q.dtype,))
    _weight_args(a, p, w_text, w_vis)
    B, N, H, dk, dv = _dims(p)
    for n, t, m in (("dq", dq, dk), ("dk", dk_, dk), ("dv", dv_, dv)):
        a.add(n, t, B * N * H * m, (q.dtype,))
    a.add("d_log_alpha", d_log_alpha, B * N * H * dk, (torch.float32,))
    a.add("d_beta", d_beta, B * N * H, (q.dtype,))
    a.add("d_w_text", d_w_text, 3 * H * dk * p.text_k, (torch.float32,))
    a.add("d_w_vis", d_w_vis, 3 * H * dk * p.vis_kt * p.vis_kh * p.vis_kw, (torch.float32,))
    a.add("d_initial_state", d_initial_state, B * H * dk * dv, (torch.float32,)).check_devices()
    _check(_lib.kda_bwd(ctypes.byref(p), _dt(q.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                        _ptr(w_text), _ptr(w_vis), _ptr(initial_state), _ptr(d_o), _ptr(d_final_state), _ptr(dq),
                        _ptr(dk_), _ptr(dv_), _ptr(d_log_alpha), _ptr(d_beta), _ptr(d_w_text), _ptr(d_w_vis),
                        _ptr(d_initial_state), _ptr(workspace), nbytes, _stream(stream)),
           "kda_bwd")


# ---------------------------------------------------------------------------
# operators beside the KDA scan: rotary positions, layer norm, linear attention with a decay per head
# ---------------------------------------------------------------------------
def _addresses(where, specs, workspace=None, nbytes=0):
    """Checks the arguments (name, tensor, elements, dtype) and returns their addresses.  A call in which all is well
    costs one short look at each tensor; anything else goes through _Args, which passes or names it."""
    out, device = [], -1
    for name, t, n, dtype in specs:
        if t is None:
            out.append(None)
            continue
        if type(t) is not torch.Tensor or not t.is_cuda or n == 0 or t.dtype is not dtype or t.numel() != n \
                or not t.is_contiguous():
            break
        if device < 0:
            device = torch.cuda.current_device()
        if t.get_device() != device:
            break
        out.append(t.data_ptr())
    else:
        if workspace is None or type(workspace) is torch.Tensor and workspace.is_cuda and workspace.is_contiguous() \
                and workspace.numel() * workspace.element_size() >= nbytes > 0 and workspace.get_device() == device:
            return out
    a = _Args(where)
    for name, t, n, dtype in specs:
        a.add(name, t, n, (dtype,))
    if workspace is not None and not isinstance(workspace, int):
        a.add("workspace", workspace, 1, (workspace.dtype,), at_least=True)
        if workspace.numel() * workspace.element_size() < nbytes:
            a.fail(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, fewer than the "
                   f"{nbytes} passed")
    a.check_devices()
    return [_ptr(t) for _, t, _, _ in specs]


def _nbytes(workspace, workspace_bytes):
    return workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes


_F32, _I32 = torch.float32, torch.int32


def _rope_call(where, call, p, r, q, k, inv_freq, q_out, k_out, positions, stream):
    B, N, H, d, _ = _dims(p)
    n, dt = B * N * H * d, q.dtype
    q_, k_, f_, pos_, qo_, ko_ = _addresses(where, (
        ("q", q, n, dt), ("k", k, n, dt), ("inv_freq", inv_freq, d // 2, _F32), ("positions", positions, B * N * 3, _I32),
        ("q_out", q_out, n, dt), ("k_out", k_out, n, dt)))
    _check(call(ctypes.byref(p), ctypes.byref(r), _dt(dt), q_, k_, f_, pos_, qo_, ko_, _stream(stream)), where)


def kda_rope_fwd(p, r, q, k, inv_freq, q_out, k_out, positions=None, stream=None):
    """Rotary positions on q and k (k and k_out may be None); q_out and k_out may be q and k."""
    _rope_call("kda_rope_fwd", _lib.kda_rope_fwd, p, r, q, k, inv_freq, q_out, k_out, positions, stream)


def kda_rope_bwd(p, r, d_q_out, d_k_out, inv_freq, dq, dk, positions=None, stream=None):
    """Gradients of q and k from those of kda_rope_fwd's outputs."""
    _rope_call("kda_rope_bwd", _lib.kda_rope_bwd, p, r, d_q_out, d_k_out, inv_freq, dq, dk, positions, stream)


def _rows_cols(where, x):
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.shape[-1] < 1:
        raise KdaError(KDA_ERR_INVALID_ARG, f"{where}: x must be a torch tensor with a last axis to normalise")
    return x.numel() // x.shape[-1], x.shape[-1]


def kda_layernorm_fwd(x, y, weight=None, bias=None, eps=1e-5, mean=None, rstd=None, stream=None):
    """Layer norm over x's last axis; weight, bias, mean and rstd are fp32 or None."""
    where, dt = "kda_layernorm_fwd", x.dtype
    rows, cols = _rows_cols(where, x)
    x_, w_, b_, y_, m_, r_ = _addresses(where, (
        ("x", x, rows * cols, dt), ("weight", weight, cols, _F32), ("bias", bias, cols, _F32), ("y", y, rows * cols, dt),
        ("mean", mean, rows, _F32), ("rstd", rstd, rows, _F32)))
    _check(_lib.kda_layernorm_fwd(rows, cols, _dt(dt), x_, w_, b_, eps, y_, m_, r_, _stream(stream)), where)


def kda_layernorm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return _lib.kda_layernorm_bwd_workspace_bytes(rows, cols)


def alloc_layernorm_bwd_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    n = kda_layernorm_bwd_workspace_bytes(rows, cols)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_layernorm_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kda_layernorm_bwd(dy, x, mean, rstd, dx, workspace, weight=None, d_weight=None, d_bias=None, stream=None,
                      workspace_bytes=None):
    """Gradients of kda_layernorm_fwd: dx, and the sums d_weight and d_bias (either may be None)."""
    where, dt = "kda_layernorm_bwd", x.dtype
    rows, cols = _rows_cols(where, x)
    n, nbytes = rows * cols, _nbytes(workspace, workspace_bytes)
    dy_, x_, w_, m_, r_, dx_, dw_, db_ = _addresses(where, (
        ("dy", dy, n, dt), ("x", x, n, dt), ("weight", weight, cols, _F32), ("mean", mean, rows, _F32),
        ("rstd", rstd, rows, _F32), ("dx", dx, n, dt), ("d_weight", d_weight, cols, _F32), ("d_bias", d_bias, cols, _F32)),
        workspace, nbytes)
    _check(_lib.kda_layernorm_bwd(rows, cols, _dt(dt), dy_, x_, w_, m_, r_, dx_, dw_, db_, _ptr(workspace), nbytes,
                                  _stream(stream)), where)


def kda_linear_workspace_bytes(p: kda_problem, dtype) -> int:
    return _lib.kda_linear_workspace_bytes(ctypes.byref(p), _dt(dtype))


def alloc_linear_workspace(p: kda_problem, dtype, device="cuda") -> torch.Tensor:
    n = kda_linear_workspace_bytes(p, dtype)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_linear_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kda_linear_bwd_workspace_bytes(p: kda_problem, dtype) -> int:
    return _lib.kda_linear_bwd_workspace_bytes(ctypes.byref(p), _dt(dtype))


def alloc_linear_bwd_workspace(p: kda_problem, dtype, device="cuda") -> torch.Tensor:
    n = kda_linear_bwd_workspace_bytes(p, dtype)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_linear_bwd_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kda_linear_fwd(p, q, k, v, log_decay, o, workspace, lengths=None, initial_state=None, final_state=None,
                   stream=None, workspace_bytes=None):
    """Linear attention with a fixed decay per head over whole sequences."""
    where, dt = "kda_linear_fwd", q.dtype
    B, N, H, d, _ = _dims(p)
    n, m, nbytes = B * N * H * d, B * H * d * d, _nbytes(workspace, workspace_bytes)
    q_, k_, v_, l_, len_, s0_, o_, sn_ = _addresses(where, (
        ("q", q, n, dt), ("k", k, n, dt), ("v", v, n, dt), ("log_decay", log_decay, H, _F32), ("lengths", lengths, B, _I32),
        ("initial_state", initial_state, m, _F32), ("o", o, n, dt), ("final_state", final_state, m, _F32)), workspace, nbytes)
    _check(_lib.kda_linear_fwd(ctypes.byref(p), _dt(dt), q_, k_, v_, l_, len_, s0_, o_, sn_, _ptr(workspace), nbytes,
                               _stream(stream)), where)


def kda_linear_bwd(p, q, k, v, log_decay, d_o, dq, dk, dv, workspace, lengths=None, initial_state=None,
                   d_final_state=None, d_initial_state=None, stream=None, workspace_bytes=None):
    """Gradients of kda_linear_fwd with respect to q, k, v and initial_state."""
    where, dt = "kda_linear_bwd", q.dtype
    B, N, H, d, _ = _dims(p)
    n, m, nbytes = B * N * H * d, B * H * d * d, _nbytes(workspace, workspace_bytes)
    q_, k_, v_, l_, len_, s0_, do_, dsn_, dq_, dk_, dv_, ds0_ = _addresses(where, (
        ("q", q, n, dt), ("k", k, n, dt), ("v", v, n, dt), ("log_decay", log_decay, H, _F32), ("lengths", lengths, B, _I32),
        ("initial_state", initial_state, m, _F32), ("d_o", d_o, n, dt), ("d_final_state", d_final_state, m, _F32),
        ("dq", dq, n, dt), ("dk", dk, n, dt), ("dv", dv, n, dt), ("d_initial_state", d_initial_state, m, _F32)),
        workspace, nbytes)
    _check(_lib.kda_linear_bwd(ctypes.byref(p), _dt(dt), q_, k_, v_, l_, len_, s0_, do_, dsn_, dq_, dk_, dv_, ds0_,
                               _ptr(workspace), nbytes, _stream(stream)), where)


def kda_linear_step(p, q, k, v, log_decay, state_in, o, state_out, stream=None):
    """One token of the recurrence for every batch item and head; state_out may be state_in."""
    where, dt = "kda_linear_step", q.dtype
    B, N, H, d, _ = _dims(p)
    n, m = B * N * H * d, B * H * d * d
    q_, k_, v_, l_, si_, o_, so_ = _addresses(where, (
        ("q", q, n, dt), ("k", k, n, dt), ("v", v, n, dt), ("log_decay", log_decay, H, _F32), ("state_in", state_in, m, _F32),
        ("o", o, n, dt), ("state_out", state_out, m, _F32)))
    _check(_lib.kda_linear_step(ctypes.byref(p), _dt(dt), q_, k_, v_, l_, si_, o_, so_, _stream(stream)), where)


def kda_selftest_wait_timeout(p, q, k, v, log_alpha, beta, o, workspace, stage, wait_us, stream=None):
    """Runs kda_chunk_fwd's kernels with one load never issued (stage 1: the block-record kernel's,
    stage 2: the state pass's) and every device wait limited to wait_us: the device status then reads
    KDA_ERR_TIMEOUT (see include/kda.h)."""
    nbytes = workspace.numel() * workspace.element_size()
    _scan_args("kda_selftest_wait_timeout", p, o.dtype, q, k, v, log_alpha, beta, o, None, None, workspace, nbytes,
               _act_dtypes(p, o.dtype)).check_devices()
    _check(_lib.kda_selftest_wait_timeout(ctypes.byref(p), _dt(o.dtype), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                          _ptr(beta), _ptr(o), _ptr(workspace), nbytes, int(stage), int(wait_us),
                                          _stream(stream)),
           "kda_selftest_wait_timeout")


def kda_read_status(workspace, stream=None) -> int:
    if isinstance(workspace, torch.Tensor) and workspace.device.type != "cuda":
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_read_status: workspace must be a CUDA tensor")
    return _lib.kda_read_status(_ptr(workspace), _stream(stream))

"""ctypes binding of libttt_b200.so (include/ttt.h).  Argument marshalling only.

Every step of the scan runs in the library's CUDA kernels; this module checks
tensor metadata, allocates outputs through torch when the caller does not pass
them, and forwards raw pointers and the current CUDA stream.  If the inputs
are CPU tensors, the call copies them to the GPU (from pinned memory), runs
the kernels and copies the outputs back: the end-to-end path.

Importing this module raises if the library has not been built: there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from contextlib import nullcontext as _nullcontext
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# TTT_B200_LIBRARY may name another build of the same library (the timeline build)
LIB_PATH = os.environ.get("TTT_B200_LIBRARY") or os.path.join(_PKG, "libttt_b200.so")

TTT_BF16, TTT_F32 = 0, 1
TTT_LN_RESIDUAL, TTT_PLAIN = 0, 1
IMPLS = {"auto": 0, "generic": 1, "tensorcore": 2, "tensorcore_split": 3, "tcgen05": 4}
_IMPL_NAMES = {0: "none", 1: "generic", 2: "tensorcore", 3: "tensorcore_split", 4: "tcgen05"}
STATUS = ["TTT_OK", "TTT_ERR_NULL", "TTT_ERR_SHAPE", "TTT_ERR_DTYPE", "TTT_ERR_ALIGN",
          "TTT_ERR_ALIAS", "TTT_ERR_UNSUPPORTED", "TTT_ERR_CUDA", "TTT_ERR_TIMEOUT", "TTT_ERR_WORKSPACE"]


class TTTError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python -m test_sequence_layers_ttt_b200.build or __graft_entry__.build())")

lib = ctypes.CDLL(LIB_PATH)
_I, _F, _P = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
lib.ttt_linear_forward.restype = _I
lib.ttt_linear_forward.argtypes = [_I] * 7 + [_F] + [_P] * 11 + [_P]
lib.ttt_linear_forward_impl.restype = _I
lib.ttt_linear_forward_impl.argtypes = [_I] * 7 + [_F] + [_P] * 11 + [_I, _P]
lib.ttt_mlp_forward.restype = _I
lib.ttt_mlp_forward.argtypes = [_I] * 7 + [_F] + [_P] * 15 + [_P]
lib.ttt_mlp_forward_impl.restype = _I
lib.ttt_mlp_forward_impl.argtypes = [_I] * 7 + [_F] + [_P] * 15 + [_I, _P]
lib.ttt_mlp_pick_impl.restype = _I
lib.ttt_mlp_pick_impl.argtypes = [_I] * 7
lib.ttt_status_string.restype = ctypes.c_char_p
lib.ttt_status_string.argtypes = [_I]
lib.ttt_abi_version.restype = _I
lib.ttt_abi_version.argtypes = []
lib.ttt_linear_pick_impl.restype = _I
lib.ttt_linear_pick_impl.argtypes = [_I] * 7
lib.ttt_linear_decode.restype = _I
lib.ttt_linear_decode.argtypes = [_I] * 8 + [_F] + [_P] * 11 + [_P]
lib.ttt_mlp_decode.restype = _I
lib.ttt_mlp_decode.argtypes = [_I] * 8 + [_F] + [_P] * 15 + [_P]
lib.ttt_mlp_decode_impl.restype = _I
lib.ttt_mlp_decode_impl.argtypes = [_I] * 8 + [_F] + [_P] * 15 + [_I, _P]
lib.ttt_linear_backward_workspace_size.restype = ctypes.c_size_t
lib.ttt_linear_backward_workspace_size.argtypes = [_I] * 5
lib.ttt_linear_backward.restype = _I
lib.ttt_linear_backward.argtypes = [_I] * 7 + [_F] + [_P] * 20 + [ctypes.c_size_t, _P]
lib.ttt_linear_backward_static.restype = _I
lib.ttt_linear_backward_static.argtypes = [_I] * 7 + [_F] + [_P] * 19 + [_P]
STATIC_WORKSPACE_BYTES = 32 << 20  # TTT_BACKWARD_STATIC_WORKSPACE_BYTES in include/ttt.h
lib.ttt_prologue_forward.restype = _I
lib.ttt_prologue_forward.argtypes = [_I] * 6 + [_F, _F, _I] + [_P] * 10 + [_P]


def linear_pick_impl(B, H, T, d, mini_batch, qkv_dtype, mode="ln") -> str:
    """Kernel family the library's AUTO dispatch runs for these arguments."""
    code = lib.ttt_linear_pick_impl(B, H, T, d, mini_batch,
                                    TTT_BF16 if qkv_dtype in ("bf16", torch.bfloat16) else TTT_F32,
                                    _mode_code(mode))
    return _IMPL_NAMES[code]


def mlp_pick_impl(B, H, T, d, hidden, mini_batch, qkv_dtype) -> str:
    """Kernel family the library's AUTO dispatch runs for these TTT-MLP arguments."""
    code = lib.ttt_mlp_pick_impl(B, H, T, d, hidden, mini_batch,
                                 TTT_BF16 if qkv_dtype in ("bf16", torch.bfloat16) else TTT_F32)
    return _IMPL_NAMES[code]


def status_string(status: int) -> str:
    return lib.ttt_status_string(status).decode()


def _check(status: int):
    if status != 0:
        raise TTTError(status, status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TTT_BF16
    if t.dtype == torch.float32:
        return TTT_F32
    raise TypeError(f"Q/K/V must be bf16 or fp32, got {t.dtype}")


def _mode_code(mode) -> int:
    if mode in ("ln", "ln_residual", TTT_LN_RESIDUAL):
        return TTT_LN_RESIDUAL
    if mode in ("plain", TTT_PLAIN):
        return TTT_PLAIN
    raise ValueError(f"unknown mode {mode!r}")


def _stream_handle(device: torch.device, stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _launch_stream(device: torch.device, stream):
    """The stream a call enqueues on, as a torch stream object."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)


class _HostRoundTrip:
    """Moves CPU inputs to the GPU and device outputs back (end-to-end path).

    The copies in, the launch and the copies back are all enqueued on the one
    stream the call launches on, so stream order alone makes the kernel see its
    inputs and the copies back see its outputs."""

    def __init__(self, tensors, stream=None):
        self.on_host = any(t is not None and t.device.type == "cpu" for t in tensors)
        self.device = torch.device("cuda", torch.cuda.current_device()) if self.on_host else None
        self.stream = _launch_stream(self.device, stream) if self.on_host else None

    def to_device(self, t):
        if t is None or not self.on_host:
            return t
        if t.device.type != "cpu":
            return t
        src = t if t.is_pinned() else t.pin_memory()
        with torch.cuda.stream(self.stream):
            return src.to(self.device, non_blocking=True)

    def to_host(self, outs):
        if not self.on_host:
            return outs
        host = []
        with torch.cuda.stream(self.stream):
            for o in outs:
                if o is None:
                    host.append(None)
                    continue
                h = torch.empty(o.shape, dtype=o.dtype, pin_memory=True)
                h.copy_(o, non_blocking=True)
                host.append(h)
        self.stream.synchronize()
        return tuple(host)


_STREAMS = {}


def _side_streams(dev: torch.device, n: int):
    key = (dev.index, n)
    if key not in _STREAMS:
        _STREAMS[key] = [torch.cuda.Stream(device=dev) for _ in range(n)]
    return _STREAMS[key]


def _head_groups(B: int, H: int, n: int):
    """(batch, first head, end head) groups of about B*H/n scans each."""
    per = max(1, -(-(B * H) // n))
    return [(b, h0, min(H, h0 + per)) for b in range(B) for h0 in range(0, H, per)]


def _pinned(t):
    return None if t is None else (t if t.is_pinned() else t.pin_memory())


def _host_pipeline(device_call, per_scan: dict, per_head: dict, out_shapes: dict, n_groups: int = 8):
    """End-to-end path for host tensors: the (batch, head) scans are independent,
    so they are cut into groups, and each group's copies in, scan and copies out
    run on their own stream; one group's transfers overlap the others' scans and
    the two copy directions overlap each other.  Results land in pinned host
    tensors; the call returns when every copy back has finished."""
    dev = torch.device("cuda", torch.cuda.current_device())
    any_t = next(t for t in per_scan.values() if t is not None)
    B, H = any_t.shape[:2]
    per_scan = {k: _pinned(t) for k, t in per_scan.items()}
    per_head = {k: _pinned(t) for k, t in per_head.items()}
    outs = {k: (None if shp is None else torch.empty(shp, dtype=torch.float32, pin_memory=True))
            for k, shp in out_shapes.items()}
    groups = _head_groups(B, H, n_groups)
    streams = _side_streams(dev, min(n_groups, len(groups)))
    current = torch.cuda.current_stream(dev)
    for s in streams:
        s.wait_stream(current)
    for i, (b, h0, h1) in enumerate(groups):
        s = streams[i % len(streams)]
        with torch.cuda.stream(s):
            args = {k: (None if t is None else t[b:b + 1, h0:h1].to(dev, non_blocking=True))
                    for k, t in per_scan.items()}
            args.update({k: (None if t is None else t[h0:h1].to(dev, non_blocking=True))
                         for k, t in per_head.items()})
            res = device_call(args, s)
            for (k, host), r in zip(outs.items(), res):
                if host is not None:
                    host[b:b + 1, h0:h1].copy_(r, non_blocking=True)
    for s in streams:
        s.synchronize()
    return tuple(outs.values())


def _on_host(*ts) -> bool:
    return all(t is None or t.device.type == "cpu" for t in ts)


def ttt_linear_forward(Q, K, V, eta, W0, b0=None, ln_gamma=None, ln_beta=None, *,
                       mini_batch: int = 16, mode="ln", ln_eps: float = 1e-6, impl: str = "auto",
                       Z=None, W_T=None, b_T=None, stream=None
                       ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """TTT-Linear forward scan (see include/ttt.h).  Returns (Z, W_T, b_T).
    Host (CPU) tensors in, host tensors out when every input is on the host."""
    if (_on_host(Q, K, V, eta, W0, b0, ln_gamma, ln_beta) and Z is None and W_T is None and b_T is None
            and stream is None and Q.dim() == 4 and Q.shape[0] * Q.shape[1] > 1 and Q.shape[2] > 0):
        B, H, T, d = Q.shape
        plain = _mode_code(mode) == TTT_PLAIN

        def run(a, s):
            return ttt_linear_forward(a["Q"], a["K"], a["V"], a["eta"], a["W0"], a["b0"], a["ln_gamma"],
                                      a["ln_beta"], mini_batch=mini_batch, mode=mode, ln_eps=ln_eps,
                                      impl=impl, stream=s)

        return _host_pipeline(run, dict(Q=Q, K=K, V=V, eta=eta, W0=W0, b0=b0),
                              dict(ln_gamma=ln_gamma, ln_beta=ln_beta),
                              dict(Z=(B, H, T, d), W_T=(B, H, d, d), b_T=None if plain else (B, H, d)))
    rt = _HostRoundTrip([Q, K, V, eta, W0], stream)
    if rt.on_host:
        stream = rt.stream
    Q, K, V, eta, W0, b0, ln_gamma, ln_beta = (
        rt.to_device(x) for x in (Q, K, V, eta, W0, b0, ln_gamma, ln_beta))
    B, H, T, d = Q.shape
    m = _mode_code(mode)
    for name, t in (("Q", Q), ("K", K), ("V", V), ("eta", eta), ("W0", W0), ("b0", b0),
                    ("ln_gamma", ln_gamma), ("ln_beta", ln_beta)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if K.shape != Q.shape or V.shape != Q.shape or K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("Q, K, V must share shape and dtype")
    if tuple(eta.shape) != (B, H, T) or tuple(W0.shape) != (B, H, d, d):
        raise ValueError("eta must be [B,H,T] and W0 [B,H,d,d]")
    dev = Q.device
    with torch.cuda.stream(rt.stream) if rt.on_host else _nullcontext():
        if Z is None:
            Z = torch.empty((B, H, T, d), dtype=torch.float32, device=dev)
        if W_T is None:
            W_T = torch.empty((B, H, d, d), dtype=torch.float32, device=dev)
        if b_T is None and m == TTT_LN_RESIDUAL:
            b_T = torch.empty((B, H, d), dtype=torch.float32, device=dev)
    st = lib.ttt_linear_forward_impl(
        B, H, T, d, int(mini_batch), _dtype_code(Q), m, float(ln_eps), _ptr(Q), _ptr(K), _ptr(V),
        _ptr(eta), _ptr(W0), _ptr(b0), _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(W_T),
        _ptr(b_T), IMPLS[impl], _stream_handle(dev, stream))
    _check(st)
    return rt.to_host((Z, W_T, b_T))


def ttt_linear_decode(Q, K, V, eta, W, b, W_mb, b_mb, ln_gamma=None, ln_beta=None, *, pos0: int,
                      mini_batch: int = 16, mode="ln", ln_eps: float = 1e-6, Z=None, stream=None
                      ) -> torch.Tensor:
    """TTT-Linear decode (see include/ttt.h): the scan continued by T tokens from
    position pos0 of a mini-batch.  W, b (running state) and W_mb, b_mb (the
    current mini-batch's start state) are CUDA tensors updated in place; the
    next call's pos0 is (pos0 + T) % mini_batch.  Returns Z."""
    m = _mode_code(mode)
    B, H, T, d = Q.shape
    for name, t in (("Q", Q), ("K", K), ("V", V), ("eta", eta), ("W", W), ("b", b), ("W_mb", W_mb),
                    ("b_mb", b_mb), ("ln_gamma", ln_gamma), ("ln_beta", ln_beta)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if K.shape != Q.shape or V.shape != Q.shape or K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("Q, K, V must share shape and dtype")
    if tuple(eta.shape) != (B, H, T) or tuple(W.shape) != (B, H, d, d) or tuple(W_mb.shape) != (B, H, d, d):
        raise ValueError("eta must be [B,H,T], W and W_mb [B,H,d,d]")
    for name, t in (("W", W), ("b", b), ("W_mb", W_mb), ("b_mb", b_mb), ("eta", eta)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    dev = Q.device
    if Z is None:
        Z = torch.empty((B, H, T, d), dtype=torch.float32, device=dev)
    st = lib.ttt_linear_decode(
        B, H, T, d, int(mini_batch), int(pos0), _dtype_code(Q), m, float(ln_eps), _ptr(Q), _ptr(K), _ptr(V),
        _ptr(eta), _ptr(W), _ptr(b), _ptr(W_mb), _ptr(b_mb), _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z),
        _stream_handle(dev, stream))
    _check(st)
    return Z


def ttt_mlp_decode(Q, K, V, eta, W1, b1, W2, b2, W1_mb, b1_mb, W2_mb, b2_mb, ln_gamma, ln_beta, *,
                   pos0: int, mini_batch: int = 16, ln_eps: float = 1e-6, impl: str = "auto", Z=None,
                   stream=None) -> torch.Tensor:
    """TTT-MLP decode (see include/ttt.h): the scan continued by T tokens from
    position pos0 of a mini-batch.  The running state (W1, b1, W2, b2) and the
    mini-batch start state (W1_mb, ...) are CUDA tensors updated in place.
    Returns Z."""
    B, H, T, d = Q.shape
    state = (W1, b1, W2, b2, W1_mb, b1_mb, W2_mb, b2_mb)
    for name, t in (("Q", Q), ("K", K), ("V", V), ("eta", eta), ("ln_gamma", ln_gamma), ("ln_beta", ln_beta),
                    *zip(("W1", "b1", "W2", "b2", "W1_mb", "b1_mb", "W2_mb", "b2_mb"), state)):
        if t is None or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if K.shape != Q.shape or V.shape != Q.shape or K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("Q, K, V must share shape and dtype")
    hidden = W1.shape[-1]
    shapes = ((B, H, d, hidden), (B, H, hidden), (B, H, hidden, d), (B, H, d)) * 2
    if tuple(eta.shape) != (B, H, T) or any(tuple(t.shape) != sh for t, sh in zip(state, shapes)):
        raise ValueError("eta must be [B,H,T]; W1 [B,H,d,hid], b1 [B,H,hid], W2 [B,H,hid,d], b2 [B,H,d]")
    if any(t.dtype != torch.float32 for t in (eta, *state)):
        raise TypeError("eta and the state must be float32")
    dev = Q.device
    if Z is None:
        Z = torch.empty((B, H, T, d), dtype=torch.float32, device=dev)
    st = lib.ttt_mlp_decode_impl(
        B, H, T, d, hidden, int(mini_batch), int(pos0), _dtype_code(Q), float(ln_eps), _ptr(Q), _ptr(K), _ptr(V),
        _ptr(eta), *(_ptr(t) for t in state), _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), IMPLS[impl],
        _stream_handle(dev, stream))
    _check(st)
    return Z


def ttt_mlp_forward(Q, K, V, eta, W1_0, b1_0, W2_0, b2_0, ln_gamma, ln_beta, *,
                    mini_batch: int = 16, ln_eps: float = 1e-6, impl: str = "auto", Z=None,
                    W1_T=None, b1_T=None, W2_T=None, b2_T=None, stream=None):
    """TTT-MLP forward scan (see include/ttt.h).  Returns (Z, W1_T, b1_T, W2_T, b2_T).
    Host (CPU) tensors in, host tensors out when every input is on the host."""
    if (_on_host(Q, K, V, eta, W1_0, b1_0, W2_0, b2_0, ln_gamma, ln_beta)
            and all(o is None for o in (Z, W1_T, b1_T, W2_T, b2_T)) and stream is None and Q.dim() == 4
            and Q.shape[0] * Q.shape[1] > 1 and Q.shape[2] > 0):
        B, H, T, d = Q.shape
        hid = W1_0.shape[-1]

        def run(a, s):
            return ttt_mlp_forward(a["Q"], a["K"], a["V"], a["eta"], a["W1_0"], a["b1_0"], a["W2_0"],
                                   a["b2_0"], a["ln_gamma"], a["ln_beta"], mini_batch=mini_batch,
                                   ln_eps=ln_eps, impl=impl, stream=s)

        return _host_pipeline(run, dict(Q=Q, K=K, V=V, eta=eta, W1_0=W1_0, b1_0=b1_0, W2_0=W2_0, b2_0=b2_0),
                              dict(ln_gamma=ln_gamma, ln_beta=ln_beta),
                              dict(Z=(B, H, T, d), W1_T=(B, H, d, hid), b1_T=(B, H, hid),
                                   W2_T=(B, H, hid, d), b2_T=(B, H, d)))
    rt = _HostRoundTrip([Q, K, V, eta, W1_0], stream)
    if rt.on_host:
        stream = rt.stream
    Q, K, V, eta, W1_0, b1_0, W2_0, b2_0, ln_gamma, ln_beta = (
        rt.to_device(x) for x in (Q, K, V, eta, W1_0, b1_0, W2_0, b2_0, ln_gamma, ln_beta))
    B, H, T, d = Q.shape
    hid = W1_0.shape[-1]
    for name, t in (("Q", Q), ("K", K), ("V", V), ("eta", eta), ("W1_0", W1_0), ("b1_0", b1_0),
                    ("W2_0", W2_0), ("b2_0", b2_0), ("ln_gamma", ln_gamma), ("ln_beta", ln_beta)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    dev = Q.device
    f32 = dict(dtype=torch.float32, device=dev)
    with torch.cuda.stream(rt.stream) if rt.on_host else _nullcontext():
        Z = torch.empty((B, H, T, d), **f32) if Z is None else Z
        W1_T = torch.empty((B, H, d, hid), **f32) if W1_T is None else W1_T
        b1_T = torch.empty((B, H, hid), **f32) if b1_T is None else b1_T
        W2_T = torch.empty((B, H, hid, d), **f32) if W2_T is None else W2_T
        b2_T = torch.empty((B, H, d), **f32) if b2_T is None else b2_T
    st = lib.ttt_mlp_forward_impl(
        B, H, T, d, hid, int(mini_batch), _dtype_code(Q), float(ln_eps), _ptr(Q), _ptr(K),
        _ptr(V), _ptr(eta), _ptr(W1_0), _ptr(b1_0), _ptr(W2_0), _ptr(b2_0), _ptr(ln_gamma),
        _ptr(ln_beta), _ptr(Z), _ptr(W1_T), _ptr(b1_T), _ptr(W2_T), _ptr(b2_T), IMPLS[impl],
        _stream_handle(dev, stream))
    _check(st)
    return rt.to_host((Z, W1_T, b1_T, W2_T, b2_T))


def linear_backward_workspace_size(B: int, H: int, T: int, d: int, mini_batch: int) -> int:
    """Bytes of device workspace ttt_linear_backward needs (see include/ttt.h)."""
    return int(lib.ttt_linear_backward_workspace_size(B, H, T, d, mini_batch))


def ttt_linear_backward(Q, K, V, eta, W0, b0, ln_gamma, ln_beta, dZ, dW_T=None, db_T=None, *,
                        mini_batch: int = 16, mode="ln", ln_eps: float = 1e-6, workspace=None, stream=None):
    """TTT-Linear layer backward (see include/ttt.h): gradients of
    sum(Z dZ) + sum(W_T dW_T) + sum(b_T db_T) with respect to the forward inputs.
    Returns (dQ, dK, dV, deta, dW0, db0, dgamma, dbeta), fp32 CUDA tensors.  The
    workspace (a CUDA byte tensor) is allocated here when not given."""
    B, H, T, d = Q.shape
    named = (("Q", Q), ("K", K), ("V", V), ("eta", eta), ("W0", W0), ("b0", b0), ("ln_gamma", ln_gamma),
             ("ln_beta", ln_beta), ("dZ", dZ), ("dW_T", dW_T), ("db_T", db_T))
    for name, t in named:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if K.shape != Q.shape or V.shape != Q.shape or K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("Q, K, V must share shape and dtype")
    if tuple(dZ.shape) != (B, H, T, d) or dZ.dtype != torch.float32:
        raise ValueError("dZ must be float32 [B,H,T,d]")
    dev = Q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dQ, dK, dV = (torch.empty((B, H, T, d), **f32) for _ in range(3))
    deta = torch.empty((B, H, T), **f32)
    dW0 = torch.empty((B, H, d, d), **f32)
    db0 = torch.empty((B, H, d), **f32)
    dgamma = torch.empty((H, d), **f32)
    dbeta = torch.empty((H, d), **f32)
    need = linear_backward_workspace_size(B, H, T, d, mini_batch)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = lib.ttt_linear_backward(
        B, H, T, d, int(mini_batch), _dtype_code(Q), _mode_code(mode), float(ln_eps), _ptr(Q), _ptr(K), _ptr(V),
        _ptr(eta), _ptr(W0), _ptr(b0), _ptr(ln_gamma), _ptr(ln_beta), _ptr(dZ), _ptr(dW_T), _ptr(db_T),
        _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(deta), _ptr(dW0), _ptr(db0), _ptr(dgamma), _ptr(dbeta),
        _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
        _stream_handle(dev, stream))
    _check(st)
    return dQ, dK, dV, deta, dW0, db0, dgamma, dbeta


def ttt_prologue_forward(x, theta_q, theta_k, theta_v, theta_lr, b_lr, *, pos0: int = 0,
                         eta_base: float = 1.0, rope_base: float = 10000.0, rotary: bool = True,
                         stream=None):
    """The layer's prologue (see include/ttt.h): Q, K, V [B,H,T,d] bf16 and eta
    [B,H,T] fp32 from x [B,T,d_model] bf16 and the bf16 weights."""
    B, T, dm = x.shape
    H, _, d = theta_q.shape
    for name, t in (("x", x), ("theta_q", theta_q), ("theta_k", theta_k), ("theta_v", theta_v),
                    ("theta_lr", theta_lr), ("b_lr", b_lr)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if any(t.dtype != torch.bfloat16 for t in (x, theta_q, theta_k, theta_v, theta_lr)) or b_lr.dtype != torch.float32:
        raise TypeError("x and the weights must be bfloat16, b_lr float32")
    dev = x.device
    Q, K, V = (torch.empty((B, H, T, d), dtype=torch.bfloat16, device=dev) for _ in range(3))
    eta = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    st = lib.ttt_prologue_forward(B, T, H, d, dm, int(pos0), float(eta_base), float(rope_base), int(bool(rotary)),
                                  _ptr(x), _ptr(theta_q), _ptr(theta_k), _ptr(theta_v), _ptr(theta_lr), _ptr(b_lr),
                                  _ptr(Q), _ptr(K), _ptr(V), _ptr(eta), _stream_handle(dev, stream))
    _check(st)
    return Q, K, V, eta


# ---------------------------------------------------------------- around the layer
_L = ctypes.c_longlong
_Z = ctypes.c_size_t
lib.ttt_rmsnorm_forward.restype = _I
lib.ttt_rmsnorm_forward.argtypes = [_I] * 4 + [_F] + [_P] * 6
lib.ttt_rmsnorm_q8_forward.restype = _I
lib.ttt_rmsnorm_q8_forward.argtypes = [_I] * 4 + [_F] + [_P] * 7
lib.ttt_rmsnorm_backward_workspace_size.restype = _Z
lib.ttt_rmsnorm_backward_workspace_size.argtypes = [_I] * 4
lib.ttt_rmsnorm_backward.restype = _I
lib.ttt_rmsnorm_backward.argtypes = [_I] * 4 + [_F] + [_P] * 7 + [_Z, _P]
lib.ttt_prologue_q8_forward.restype = _I
lib.ttt_prologue_q8_forward.argtypes = [_I] * 6 + [_F, _F, _I] + [_P] * 15 + [_P]
lib.ttt_conv_forward.restype = _I
lib.ttt_conv_forward.argtypes = [_I] * 6 + [_L] + [_P] * 7 + [_P]
lib.ttt_conv_decode.restype = _I
lib.ttt_conv_decode.argtypes = [_I] * 6 + [_L] + [_P] * 5 + [_P]
lib.ttt_conv_backward_workspace_size.restype = _Z
lib.ttt_conv_backward_workspace_size.argtypes = [_I] * 4
lib.ttt_conv_backward.restype = _I
lib.ttt_conv_backward.argtypes = [_I] * 6 + [_L] + [_P] * 12 + [_Z, _P]
lib.ttt_ssm_forward.restype = _I
lib.ttt_ssm_forward.argtypes = [_I] * 6 + [_L] * 5 + [_P] * 12 + [_P]
lib.ttt_ssm_decode.restype = _I
lib.ttt_ssm_decode.argtypes = [_I] * 6 + [_L] * 5 + [_P] * 10 + [_P]
lib.ttt_ssm_backward_workspace_size.restype = _Z
lib.ttt_ssm_backward_workspace_size.argtypes = [_I] * 4
lib.ttt_ssm_backward.restype = _I
lib.ttt_ssm_backward.argtypes = [_I] * 6 + [_L] * 5 + [_P] * 22 + [_Z, _P]


class _Launch:
    """Device and stream of one call: makes the tensors' device current and, where a stream is given, allocates
    on it, so that the caching allocator knows which stream the call's buffers are used on."""

    __slots__ = ("dev", "stream", "entered")

    def __init__(self, dev: torch.device, stream):
        self.dev, self.stream = dev, stream

    def __enter__(self):
        dev = self.dev
        self.entered = ()
        if dev.index != torch._C._cuda_getDevice():
            self.entered = (torch.cuda.device(dev),)
        if self.stream is not None:
            self.entered += (torch.cuda.stream(_launch_stream(dev, self.stream)),)
        for c in self.entered:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(dev.index)  # current_stream(dev).cuda_stream, 4 us cheaper

    def __exit__(self, *exc):
        for c in reversed(self.entered):
            c.__exit__(*exc)


def _token_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return TTT_BF16
    if t.dtype == torch.float32:
        return TTT_F32
    raise TypeError(f"{name} must be bf16 or fp32, got {t.dtype}")


def _refuse(t: torch.Tensor, name: str, shape, dtype, dev, what: str):
    if t.get_device() != dev.index:
        raise ValueError(f"{name} must be {what} on {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {what} on {dev}, got strides {t.stride()}")


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype, dev) -> Optional[int]:
    """Address of a contiguous CUDA tensor of this shape, type and device (None for None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev.index or not t.is_contiguous():
        _refuse(t, name, shape, dtype, dev, "a contiguous CUDA tensor")
    return t.data_ptr()


def _out(t: Optional[torch.Tensor], name: str, like: torch.Tensor, shape, dtype, dev):
    """An output and its address: the caller's tensor, checked, or a new one."""
    if t is None:
        # new_empty with the sizes one by one takes half the time of torch.empty with a type and a device
        t = like.new_empty(*shape) if dtype is like.dtype else like.new_empty(*shape, dtype=dtype)
        return t, t.data_ptr()
    return t, _dense(t, name, shape, dtype, dev)


def _rows(t: Optional[torch.Tensor], name: str, shape, dtype, dev):
    """(address, row stride) of token rows [B, T, width], which may be a slice of wider rows."""
    if t is None:
        return None, 0
    what = "a CUDA tensor with its elements side by side and its rows at one distance"
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev.index:
        _refuse(t, name, shape, dtype, dev, what)
    B, T, width = shape
    if t.is_contiguous():
        return t.data_ptr(), width
    sb, st, sw = t.stride()
    ld = st if T > 1 else (sb if B > 1 else width)
    if (sw != 1 and width > 1) or (B > 1 and T > 1 and sb != T * st) or (t.numel() and ld < width):
        _refuse(t, name, shape, dtype, dev, what)
    return t.data_ptr(), max(ld, width)


def _workspace(given: Optional[torch.Tensor], need: int, like: torch.Tensor):
    """A workspace of `need` bytes, the caller's or a new one, beside the fp32 tensor `like`."""
    dev = like.device
    if given is None:
        given = like.new_empty(max(need + 3, 16) // 4)
    elif given.get_device() != dev.index or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    return given, given.data_ptr(), given.numel() * given.element_size()


def _sizes(t: torch.Tensor, name: str):
    """The shape, whose sizes the library takes as C ints: ctypes would drop what passes them without a word."""
    if max(t.shape) > 0x7fffffff:
        raise ValueError(f"{name} has a size past 2^31 - 1: {list(t.shape)}")
    return t.shape


def _three(t: torch.Tensor, name: str):
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [B, T, width]")
    return _sizes(t, name)


def ttt_rmsnorm_forward(x, weight, residual=None, *, eps: float = 1e-6, y=None, h=None, stream=None):
    """Root-mean-square norm of x + residual (see include/ttt.h).  Returns (y, h): h is the residual stream, None
    where there is no residual and no h was given.  x, residual [B, T, d] bf16 or fp32, weight [d] fp32."""
    B, T, d = _three(x, "x")
    dev, dt = x.device, x.dtype
    code = _token_dtype(x, "x")
    px, pr = _dense(x, "x", (B, T, d), dt, dev), _dense(residual, "residual", (B, T, d), dt, dev)
    pw = _dense(weight, "weight", (d,), torch.float32, dev)
    with _Launch(dev, stream) as s:
        y, py = _out(y, "y", x, (B, T, d), dt, dev)
        ph = None
        if h is not None or residual is not None:
            h, ph = _out(h, "h", x, (B, T, d), dt, dev)
        _check(lib.ttt_rmsnorm_forward(B, T, d, code, eps, px, pr, pw, py, ph, s))
    return y, h


def ttt_rmsnorm_q8_forward(x, weight, residual=None, *, eps: float = 1e-6, q=None, scale=None, h=None, stream=None):
    """The norm with its output in 8 bits (see include/ttt.h).  Returns (q, scale, h): q [B, T, d] float8_e4m3fn,
    scale [B, T] fp32, h as in ttt_rmsnorm_forward."""
    B, T, d = _three(x, "x")
    dev, dt = x.device, x.dtype
    code = _token_dtype(x, "x")
    px, pr = _dense(x, "x", (B, T, d), dt, dev), _dense(residual, "residual", (B, T, d), dt, dev)
    pw = _dense(weight, "weight", (d,), torch.float32, dev)
    with _Launch(dev, stream) as s:
        q, pq = _out(q, "q", x, (B, T, d), torch.float8_e4m3fn, dev)
        scale, ps = _out(scale, "scale", weight, (B, T), torch.float32, dev)
        ph = None
        if h is not None or residual is not None:
            h, ph = _out(h, "h", x, (B, T, d), dt, dev)
        _check(lib.ttt_rmsnorm_q8_forward(B, T, d, code, eps, px, pr, pw, pq, ps, ph, s))
    return q, scale, h


def ttt_rmsnorm_backward(h, weight, dy, dh_in=None, *, eps: float = 1e-6, workspace=None, stream=None):
    """Gradient of the norm (see include/ttt.h).  Returns (dh, dweight): dh, in h's type, is the gradient of x and
    of residual alike; dh_in is the gradient that reaches h past the norm."""
    B, T, d = _three(h, "h")
    dev, dt = h.device, h.dtype
    code = _token_dtype(h, "h")
    ph, pg = _dense(h, "h", (B, T, d), dt, dev), _dense(dy, "dy", (B, T, d), dt, dev)
    pi = _dense(dh_in, "dh_in", (B, T, d), dt, dev)
    pw = _dense(weight, "weight", (d,), torch.float32, dev)
    with _Launch(dev, stream) as s:
        dh, dw = torch.empty_like(h), torch.empty_like(weight)
        workspace, pws, n = _workspace(workspace, lib.ttt_rmsnorm_backward_workspace_size(B, T, d, code), weight)
        _check(lib.ttt_rmsnorm_backward(B, T, d, code, eps, ph, pw, pg, pi, dh.data_ptr(), dw.data_ptr(), pws, n, s))
    return dh, dw


def prologue_q8_weights(theta):
    """Weights of ttt_prologue_q8_forward, laid out once: theta [H, d_model, d] (as ttt_prologue_forward takes it) or
    theta_lr [H, d_model] to (e4m3 [H, d, d_model] or [H, d_model], fp32 scale [H, d] or [H])."""
    rows = theta.float() if theta.dim() == 2 else theta.float().transpose(1, 2)
    scale = (rows.abs().amax(-1) / 448.0).clamp_min(2.0 ** -100)
    return (rows / scale[..., None]).to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


def ttt_prologue_q8_forward(x, scale_x, theta_q, scale_q, theta_k, scale_k, theta_v, scale_v, theta_lr, scale_lr, b_lr,
                            *, pos0: int = 0, eta_base: float = 1.0, rope_base: float = 10000.0, rotary: bool = True,
                            out=None, stream=None):
    """The layer's prologue from 8-bit operands (see include/ttt.h): x and scale_x as ttt_rmsnorm_q8_forward returns
    them, each weight and its scale as prologue_q8_weights does.  Returns Q, K, V [B, H, T, d] bf16 and eta [B, H, T]
    fp32 (the tensors of `out` where given)."""
    B, T, dm = _three(x, "x")
    if theta_q.dim() != 3:
        raise ValueError("theta_q must be [H, d, d_model]")
    H, d, _ = _sizes(theta_q, "theta_q")
    pos0 = int(pos0)
    if not -2 ** 31 <= pos0 < 2 ** 31:
        raise ValueError(f"pos0 must lie within 32 bits, got {pos0}")
    dev, f8, f32 = x.device, torch.float8_e4m3fn, torch.float32
    ptrs = [_dense(x, "x", (B, T, dm), f8, dev), _dense(scale_x, "scale_x", (B, T), f32, dev)]
    for name, w, sc in (("q", theta_q, scale_q), ("k", theta_k, scale_k), ("v", theta_v, scale_v)):
        ptrs += [_dense(w, "theta_" + name, (H, d, dm), f8, dev), _dense(sc, "scale_" + name, (H, d), f32, dev)]
    ptrs += [_dense(theta_lr, "theta_lr", (H, dm), f8, dev), _dense(scale_lr, "scale_lr", (H,), f32, dev),
             _dense(b_lr, "b_lr", (H,), f32, dev)]
    with _Launch(dev, stream) as s:
        if out is None:
            out = [b_lr.new_empty(B, H, T, d, dtype=torch.bfloat16) for _ in range(3)]
            out.append(b_lr.new_empty(B, H, T))
        Q, K, V, eta = out
        for name, o in (("Q", Q), ("K", K), ("V", V)):
            ptrs.append(_dense(o, name, (B, H, T, d), torch.bfloat16, dev))
        ptrs.append(_dense(eta, "eta", (B, H, T), f32, dev))
        _check(lib.ttt_prologue_q8_forward(B, T, H, d, dm, pos0, float(eta_base), float(rope_base),
                                           int(bool(rotary)), *ptrs, s))
    return Q, K, V, eta


def _silu_code(activation) -> int:
    if activation not in ("silu", None):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    return int(activation == "silu")


def _conv_args(x, weight, bias, state, lengths, state_name="state0"):
    B, T, C = _three(x, "x")
    if weight.dim() != 2:
        raise ValueError("weight must be [C, width]")
    W = _sizes(weight, "weight")[1]
    dev, dt = x.device, x.dtype
    code = _token_dtype(x, "x")
    px, ld = _rows(x, "x", (B, T, C), dt, dev)
    pw = _dense(weight, "weight", (C, W), torch.float32, dev)
    pb = _dense(bias, "bias", (C,), torch.float32, dev)
    ps = _dense(state, state_name, (B, W - 1, C), dt, dev)
    pl = _dense(lengths, "lengths", (B,), torch.int32, dev)
    return (B, T, C, W, code), ld, (px, pw, pb, ps, pl)


def ttt_conv_forward(x, weight, bias=None, state0=None, *, lengths=None, activation="silu", y=None, state_T=None,
                     stream=None):
    """Short causal depthwise convolution (see include/ttt.h).  x [B, T, C] bf16 or fp32 (a slice of wider rows will
    do), weight [C, width] fp32, state0 [B, width - 1, C]: the rows before x.  Returns (y, state_T): the last
    width - 1 rows of each sequence, to go on from."""
    shape, ld, (px, pw, pb, ps, pl) = _conv_args(x, weight, bias, state0, lengths)
    B, T, C, W, _ = shape
    dev, dt = x.device, x.dtype
    with _Launch(dev, stream) as s:
        y, py = _out(y, "y", x, (B, T, C), dt, dev)
        state_T, pt = _out(state_T, "state_T", x, (B, W - 1, C), dt, dev)
        _check(lib.ttt_conv_forward(*shape, _silu_code(activation), ld, px, pw, pb, ps, pl, py, pt, s))
    return y, state_T


def ttt_conv_decode(x, weight, bias, state, *, activation="silu", y=None, stream=None):
    """The convolution continued by x's tokens (see include/ttt.h); state [B, width - 1, C] is updated in place.
    Returns y."""
    if state is None:
        raise ValueError("state must be a contiguous CUDA tensor")
    shape, ld, (px, pw, pb, ps, _) = _conv_args(x, weight, bias, state, None, "state")
    B, T, C, W, _ = shape
    dev, dt = x.device, x.dtype
    with _Launch(dev, stream) as s:
        y, py = _out(y, "y", x, (B, T, C), dt, dev)
        _check(lib.ttt_conv_decode(*shape, _silu_code(activation), ld, px, pw, pb, ps, py, s))
    return y


def ttt_conv_backward(x, weight, bias, dy, state0=None, dstate_T=None, *, lengths=None, activation="silu",
                      workspace=None, stream=None):
    """Gradient of the convolution (see include/ttt.h).  Returns (dx, dweight, dbias, dstate0); dbias is None where
    bias is, dstate0 where state0 is."""
    shape, ld, (px, pw, pb, ps, pl) = _conv_args(x, weight, bias, state0, lengths)
    B, T, C, W, code = shape
    dev, dt = x.device, x.dtype
    pg = _dense(dy, "dy", (B, T, C), dt, dev)
    pt = _dense(dstate_T, "dstate_T", (B, W - 1, C), dt, dev)
    with _Launch(dev, stream) as s:
        dx, dw = x.new_empty(B, T, C), torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        d0 = None if state0 is None else torch.empty_like(state0)
        workspace, pws, n = _workspace(workspace, lib.ttt_conv_backward_workspace_size(B, T, C, W), weight)
        _check(lib.ttt_conv_backward(*shape, _silu_code(activation), ld, px, pw, pb, ps, pl, pg, pt, dx.data_ptr(),
                                     dw.data_ptr(), _ptr(db), _ptr(d0), pws, n, s))
    return dx, dw, db, d0


def _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, h_name="h0"):
    B, T, C = _three(u, "u")
    if A.dim() != 2:
        raise ValueError("A must be [C, N]")
    N = _sizes(A, "A")[1]
    dev, ty, f32 = u.device, u.dtype, torch.float32
    code = _token_dtype(u, "u")
    pu, lu = _rows(u, "u", (B, T, C), ty, dev)
    pd, ld = _rows(dt, "dt", (B, T, C), ty, dev)
    pB, lB = _rows(Bm, "Bm", (B, T, N), ty, dev)
    pC, lC = _rows(Cm, "Cm", (B, T, N), ty, dev)
    pz, lz = _rows(z, "z", (B, T, C), ty, dev)
    pbias = _dense(dt_bias, "dt_bias", (C,), f32, dev)
    pA, pD = _dense(A, "A", (C, N), f32, dev), _dense(D, "D", (C,), f32, dev)
    ph = _dense(h0, h_name, (B, C, N), f32, dev)
    pl = _dense(lengths, "lengths", (B,), torch.int32, dev)
    return (B, T, C, N, code), (lu, ld, lB, lC, lz), (pu, pd, pbias, pA, pB, pC, pD, pz, ph, pl)


def ttt_ssm_forward(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, *, lengths=None, dt_softplus: bool = True,
                    y=None, h_T=None, stream=None):
    """Selective state space scan (see include/ttt.h).  u, dt, z [B, T, C] and Bm, Cm [B, T, N], bf16 or fp32 (slices
    of wider rows will do); A [C, N], D, dt_bias [C], h0 [B, C, N] fp32.  Returns (y, h_T)."""
    shape, lds, ptrs = _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths)
    B, T, C, N, _ = shape
    dev = u.device
    with _Launch(dev, stream) as s:
        y, py = _out(y, "y", u, (B, T, C), u.dtype, dev)
        h_T, ph = _out(h_T, "h_T", A, (B, C, N), torch.float32, dev)
        _check(lib.ttt_ssm_forward(*shape, int(bool(dt_softplus)), *lds, *ptrs, py, ph, s))
    return y, h_T


def ttt_ssm_decode(u, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, *, dt_softplus: bool = True, y=None, stream=None):
    """The scan continued by u's tokens (see include/ttt.h); h [B, C, N] is updated in place.  Returns y."""
    if h is None:
        raise ValueError("h must be a contiguous CUDA tensor")
    shape, lds, ptrs = _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, h, None, "h")
    B, T, C, N, _ = shape
    dev = u.device
    with _Launch(dev, stream) as s:
        y, py = _out(y, "y", u, (B, T, C), u.dtype, dev)
        _check(lib.ttt_ssm_decode(*shape, int(bool(dt_softplus)), *lds, *ptrs[:-1], py, s))
    return y


def ttt_ssm_backward(u, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, h0=None, dh_T=None, *, lengths=None,
                     dt_softplus: bool = True, workspace=None, stream=None):
    """Gradient of the scan (see include/ttt.h), from its inputs and dy [B, T, C], dh_T [B, C, N].  Returns (du, ddt,
    dA, dB, dC, dD, dz, ddt_bias, dh0): token rows in u's type, the rest fp32; None for an input that is None."""
    shape, lds, ptrs = _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths)
    B, T, C, N, _ = shape
    dev, f32 = u.device, torch.float32
    pg = _dense(dy, "dy", (B, T, C), u.dtype, dev)
    pt = _dense(dh_T, "dh_T", (B, C, N), f32, dev)
    with _Launch(dev, stream) as s:
        du, ddt = u.new_empty(B, T, C), u.new_empty(B, T, C)
        dz = None if z is None else u.new_empty(B, T, C)
        dA = torch.empty_like(A)
        dB, dC = A.new_empty(B, T, N), A.new_empty(B, T, N)
        dD = None if D is None else torch.empty_like(D)
        dbias = None if dt_bias is None else torch.empty_like(dt_bias)
        dh0 = None if h0 is None else torch.empty_like(h0)
        workspace, pws, n = _workspace(workspace, lib.ttt_ssm_backward_workspace_size(B, T, C, N), A)
        _check(lib.ttt_ssm_backward(*shape, int(bool(dt_softplus)), *lds, *ptrs, pg, pt, du.data_ptr(), ddt.data_ptr(),
                                    dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _ptr(dD), _ptr(dz), _ptr(dbias),
                                    _ptr(dh0), pws, n, s))
    return du, ddt, dA, dB, dC, dD, dz, dbias, dh0

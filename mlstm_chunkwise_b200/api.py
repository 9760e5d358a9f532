"""Python binding of the C ABI (argument marshalling only).

Every computation runs in the CUDA kernels of ``libmlstm_fw.so``; this module
allocates outputs and workspace with PyTorch on the inputs' device, passes raw
pointers and torch's current stream, and raises ``MlstmError`` on a non-OK
status.  Inputs must be CUDA tensors: there is no CPU path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import _lib
from ._lib import MlstmError  # noqa: F401  (re-export)

_DT = {torch.float32: _lib.DT_F32, torch.bfloat16: _lib.DT_BF16}
_GATE = {"exp": _lib.GATE_EXP, "sigmoid": _lib.GATE_SIGMOID,
         "sigmoid_plain": _lib.GATE_SIGMOID_PLAIN}
_ALGO = {"auto": _lib.ALGO_AUTO, "simt": _lib.ALGO_SIMT, "tc": _lib.ALGO_TC,
         "tc_fused": _lib.ALGO_TC_FUSED}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    # the raw handle: a Stream object costs as much as a launch
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if device.index is None else device.index)


def _check_tensor(name, t, dtype, shape, device):
    if t is None or (t.shape == shape and t.dtype is dtype and t.is_contiguous() and
                     t.get_device() == device.index):  # -1 off the GPU
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _written(*tensors):
    """Raises the versions of the caller's tensors that a call wrote in place:
    autograd then refuses a backward that kept them from before."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


_written_one = torch.autograd.graph.increment_version  # half a microsecond less


def _upstream(grad):
    """An upstream gradient as the kernels take it: autograd may hand on a view with
    strides, or a slice that starts off a 16-byte boundary."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def workspace_size(B, NH, T, DK, DV, chunk_size, dtype=torch.bfloat16, algo="auto") -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.lib().mlstm_fw_workspace_size(B, NH, T, DK, DV, chunk_size, _DT[dtype],
                                                  _ALGO[algo], ctypes.byref(n)),
               "mlstm_fw_workspace_size")
    return int(n.value)


def substep_workspace_size(B, NH, T, DK, DV, chunk_size, dtype=torch.bfloat16,
                           algo="auto") -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.lib().mlstm_fw_substep_workspace_size(B, NH, T, DK, DV, chunk_size, _DT[dtype],
                                                          _ALGO[algo], ctypes.byref(n)),
               "mlstm_fw_substep_workspace_size")
    return int(n.value)


def _shapes(Q, V):
    B, NH, T, DK = Q.shape
    DV = V.shape[-1]
    return B, NH, T, DK, DV


def _check_common(Q, K, V, i_pre, f_pre):
    if Q.dim() != 4:
        raise ValueError("Q must be [B, NH, T, DK]")
    B, NH, T, DK, DV = _shapes(Q, V)
    dev = Q.device
    dt = Q.dtype
    if dt not in _DT:
        raise ValueError(f"unsupported dtype {dt} (float32 or bfloat16)")
    _check_tensor("Q", Q, dt, (B, NH, T, DK), dev)
    _check_tensor("K", K, dt, (B, NH, T, DK), dev)
    _check_tensor("V", V, dt, (B, NH, T, DV), dev)
    _check_tensor("i_pre", i_pre, torch.float32, (B, NH, T), dev)
    _check_tensor("f_pre", f_pre, torch.float32, (B, NH, T), dev)
    return B, NH, T, DK, DV, dev, dt


def _check_state(C0, n0, m0, B, NH, DK, DV, dev):
    if (C0 is None) != (n0 is None) or (C0 is None) != (m0 is None):
        raise ValueError("C0, n0 and m0 must be given together")
    _check_tensor("C0", C0, torch.float32, (B, NH, DK, DV), dev)
    _check_tensor("n0", n0, torch.float32, (B, NH, DK), dev)
    _check_tensor("m0", m0, torch.float32, (B, NH), dev)


def mlstm_fw(Q, K, V, i_pre, f_pre, C0=None, n0=None, m0=None, *, chunk_size: int = 64,
             gate_mode: str = "exp", algo: str = "auto", return_last_states: bool = True,
             workspace: torch.Tensor | None = None, out: dict | None = None):
    """mLSTM forward pass on the GPU.

    Q, K [B,NH,T,DK] and V [B,NH,T,DV] (float32 or bfloat16, same dtype);
    i_pre, f_pre [B,NH,T] float32; optional initial state C0 [B,NH,DK,DV],
    n0 [B,NH,DK], m0 [B,NH] float32.  Returns ``H`` or ``(H, (C_T, n_T, m_T))``.
    ``out`` may hold preallocated ``H``/``C_T``/``n_T``/``m_T``; ``workspace``
    a uint8 CUDA tensor of at least ``workspace_size(...)`` bytes.
    """
    B, NH, T, DK, DV, dev, dt = _check_common(Q, K, V, i_pre, f_pre)
    _check_state(C0, n0, m0, B, NH, DK, DV, dev)
    out = {} if out is None else out
    H = out.get("H")
    if H is None:
        H = torch.empty((B, NH, T, DV), dtype=dt, device=dev)
    _check_tensor("H", H, dt, (B, NH, T, DV), dev)
    C_T = n_T = m_T = None
    if return_last_states:
        C_T = out.get("C_T")
        n_T = out.get("n_T")
        m_T = out.get("m_T")
        if C_T is None:
            C_T = torch.empty((B, NH, DK, DV), dtype=torch.float32, device=dev)
        if n_T is None:
            n_T = torch.empty((B, NH, DK), dtype=torch.float32, device=dev)
        if m_T is None:
            m_T = torch.empty((B, NH), dtype=torch.float32, device=dev)
    ws_bytes = workspace_size(B, NH, T, DK, DV, chunk_size, dt, algo)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    elif workspace.numel() < ws_bytes or not workspace.is_cuda:
        raise ValueError(f"workspace must be a CUDA uint8 tensor of >= {ws_bytes} bytes")
    st = _lib.lib().mlstm_fw(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(i_pre), _ptr(f_pre), _ptr(C0), _ptr(n0), _ptr(m0),
        _ptr(H), _ptr(C_T), _ptr(n_T), _ptr(m_T), B, NH, T, DK, DV, chunk_size, _DT[dt],
        _GATE[gate_mode], _ALGO[algo], _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(st, "mlstm_fw")
    if out:
        _written(out.get("H"), *(out.get(n) for n in ("C_T", "n_T", "m_T") if return_last_states))
    if return_last_states:
        return H, (C_T, n_T, m_T)
    return H


def mlstm_bw(Q, K, V, i_pre, f_pre, dH, C0=None, n0=None, m0=None, *, chunk_size: int = 64,
             gate_mode: str = "exp"):
    """Gradients of a loss L(H) of the forward output, given dH = dL/dH.

    Inputs as ``mlstm_fw``.  Returns a dict with dQ, dK, dV (input dtype),
    di_pre, df_pre [B,NH,T] and, when an initial state is given, dC0, dn0,
    dm0 (float32).  bf16 inputs with d_qk of 128 or 256 (a d_v the tensor-core
    forward takes, T >= 128) run on the tensor cores in 128-token chunks,
    whatever ``chunk_size`` is; everything else on fp32 CUDA-core kernels.
    """
    B, NH, T, DK, DV, dev, dt = _check_common(Q, K, V, i_pre, f_pre)
    _check_state(C0, n0, m0, B, NH, DK, DV, dev)
    _check_tensor("dH", dH, dt, (B, NH, T, DV), dev)
    out = {"dQ": torch.empty_like(Q), "dK": torch.empty_like(K), "dV": torch.empty_like(V),
           "di_pre": torch.empty_like(i_pre), "df_pre": torch.empty_like(f_pre)}
    if C0 is not None:
        out.update(dC0=torch.empty_like(C0), dn0=torch.empty_like(n0), dm0=torch.empty_like(m0))
    n = ctypes.c_size_t(0)
    _lib.check(_lib.lib().mlstm_bw_workspace_size(B, NH, T, DK, DV, chunk_size, _DT[dt],
                                                  ctypes.byref(n)), "mlstm_bw_workspace_size")
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=dev)
    st = _lib.lib().mlstm_bw(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(i_pre), _ptr(f_pre), _ptr(C0), _ptr(n0), _ptr(m0),
        _ptr(dH), _ptr(out["dQ"]), _ptr(out["dK"]), _ptr(out["dV"]), _ptr(out["di_pre"]),
        _ptr(out["df_pre"]), _ptr(out.get("dC0")), _ptr(out.get("dn0")), _ptr(out.get("dm0")),
        B, NH, T, DK, DV, chunk_size, _DT[dt], _GATE[gate_mode], _ptr(ws), ws.numel(),
        _stream(dev))
    _lib.check(st, "mlstm_bw")
    return out


def train_sizes(B, NH, T, DK, DV, dtype=torch.bfloat16):
    """Bytes of the saved buffer and of the two calls' workspaces of the
    training pair, or None when the shape has no training path (it needs the
    tensor-core backward: bf16, d_qk 128 or 256, d_v 128 or a multiple of 256
    up to 1024, T >= 128)."""
    sv, fw, bw = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = _lib.lib().mlstm_train_sizes(B, NH, T, DK, DV, _DT[dtype], ctypes.byref(sv),
                                      ctypes.byref(fw), ctypes.byref(bw))
    if st == _lib.ERR_UNSUPPORTED:
        return None
    _lib.check(st, "mlstm_train_sizes")
    return int(sv.value), int(fw.value), int(bw.value)


def mlstm_fw_train(Q, K, V, i_pre, f_pre, C0=None, n0=None, m0=None, *, gate_mode: str = "exp"):
    """The forward pass of ``mlstm_fw`` (128-token chunks on the tensor cores)
    that also keeps what ``mlstm_bw_saved`` needs.  Returns ``(H, (C_T, n_T,
    m_T), saved)``; ``saved`` is an opaque uint8 tensor.  Raises
    ``MlstmError`` (unsupported) outside the shapes of ``train_sizes``."""
    B, NH, T, DK, DV, dev, dt = _check_common(Q, K, V, i_pre, f_pre)
    _check_state(C0, n0, m0, B, NH, DK, DV, dev)
    sizes = train_sizes(B, NH, T, DK, DV, dt)
    if sizes is None:
        raise MlstmError(_lib.ERR_UNSUPPORTED, "mlstm_fw_train")
    sv_bytes, fw_bytes, _ = sizes
    H = torch.empty((B, NH, T, DV), dtype=dt, device=dev)
    C_T = torch.empty((B, NH, DK, DV), dtype=torch.float32, device=dev)
    n_T = torch.empty((B, NH, DK), dtype=torch.float32, device=dev)
    m_T = torch.empty((B, NH), dtype=torch.float32, device=dev)
    saved = torch.empty(sv_bytes, dtype=torch.uint8, device=dev)
    ws = torch.empty(max(fw_bytes, 1), dtype=torch.uint8, device=dev)
    _lib.check(_lib.lib().mlstm_fw_train(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(i_pre), _ptr(f_pre), _ptr(C0), _ptr(n0), _ptr(m0),
        _ptr(H), _ptr(C_T), _ptr(n_T), _ptr(m_T), _ptr(saved), saved.numel(), B, NH, T, DK, DV,
        _DT[dt], _GATE[gate_mode], _ptr(ws), ws.numel(), _stream(dev)), "mlstm_fw_train")
    return H, (C_T, n_T, m_T), saved


def mlstm_bw_saved(Q, K, V, i_pre, f_pre, H, saved, dH, C0=None, n0=None, m0=None, *,
                   gate_mode: str = "exp"):
    """``mlstm_bw`` from the output and the saved buffer of ``mlstm_fw_train``
    (same inputs) instead of a recomputed forward.  Returns the same dict."""
    B, NH, T, DK, DV, dev, dt = _check_common(Q, K, V, i_pre, f_pre)
    _check_state(C0, n0, m0, B, NH, DK, DV, dev)
    _check_tensor("H", H, dt, (B, NH, T, DV), dev)
    _check_tensor("dH", dH, dt, (B, NH, T, DV), dev)
    sizes = train_sizes(B, NH, T, DK, DV, dt)
    if sizes is None:
        raise MlstmError(_lib.ERR_UNSUPPORTED, "mlstm_bw_saved")
    _, _, bw_bytes = sizes
    out = {"dQ": torch.empty_like(Q), "dK": torch.empty_like(K), "dV": torch.empty_like(V),
           "di_pre": torch.empty_like(i_pre), "df_pre": torch.empty_like(f_pre)}
    if C0 is not None:
        out.update(dC0=torch.empty_like(C0), dn0=torch.empty_like(n0), dm0=torch.empty_like(m0))
    ws = torch.empty(max(bw_bytes, 1), dtype=torch.uint8, device=dev)
    _lib.check(_lib.lib().mlstm_bw_saved(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(i_pre), _ptr(f_pre), _ptr(C0), _ptr(n0), _ptr(m0),
        _ptr(H), _ptr(saved), saved.numel(), _ptr(dH), _ptr(out["dQ"]), _ptr(out["dK"]),
        _ptr(out["dV"]), _ptr(out["di_pre"]), _ptr(out["df_pre"]), _ptr(out.get("dC0")),
        _ptr(out.get("dn0")), _ptr(out.get("dm0")), B, NH, T, DK, DV, _DT[dt],
        _GATE[gate_mode], _ptr(ws), ws.numel(), _stream(dev)), "mlstm_bw_saved")
    return out


def mlstm_step(q, k, v, i_pre, f_pre, C, n, m, *, gate_mode: str = "exp", h=None):
    """One token of the recurrence for every (b, h), in place on the state.

    q, k [B,NH,DK] and v [B,NH,DV] (float32 or bfloat16, same dtype); i_pre,
    f_pre [B,NH] float32; C [B,NH,DK,DV], n [B,NH,DK], m [B,NH] float32 CUDA
    tensors holding the state before the token, overwritten with the state
    after it.  Returns h [B,NH,DV] in the input dtype (``h`` may be given).
    """
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError("q, k must be [B,NH,DK] and v [B,NH,DV] with the same B, NH")
    B, NH, DK = q.shape
    DV = v.shape[2]
    dt, dev = q.dtype, q.device
    if dt not in _DT or k.dtype != dt or v.dtype != dt:
        raise ValueError("q, k, v must share a dtype of float32 or bfloat16")
    for name, t in (("i_pre", i_pre), ("f_pre", f_pre), ("m", m)):
        _check_tensor(name, t, torch.float32, (B, NH), dev)
    _check_tensor("C", C, torch.float32, (B, NH, DK, DV), dev)
    _check_tensor("n", n, torch.float32, (B, NH, DK), dev)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, dt, tuple(t.shape), dev)
    given = h
    if h is None:
        h = torch.empty((B, NH, DV), dtype=dt, device=dev)
    _check_tensor("h", h, dt, (B, NH, DV), dev)
    st = _lib.lib().mlstm_step(_ptr(q), _ptr(k), _ptr(v), _ptr(i_pre), _ptr(f_pre), _ptr(C),
                               _ptr(n), _ptr(m), _ptr(h), B, NH, DK, DV, _DT[dt],
                               _GATE[gate_mode], _stream(dev))
    _lib.check(st, "mlstm_step")
    _written(C, n, m, given)
    return h


def mlstm_fw_chunk_states(K, V, i_pre, f_pre, C0=None, n0=None, m0=None, *, chunk_size: int = 64,
                          gate_mode: str = "exp", algo: str = "auto"):
    """Recurrent half: states entering every chunk and the final state.

    Returns (C_states [B,NH,NC,DK,DV], n_states [B,NH,NC,DK], m_states
    [B,NH,NC+1], (C_T, n_T, m_T)).
    """
    B, NH, T, DK, DV, dev, dt = _check_common(K, K, V, i_pre, f_pre)
    _check_state(C0, n0, m0, B, NH, DK, DV, dev)
    NC = (T + chunk_size - 1) // chunk_size
    C_states = torch.empty((B, NH, NC, DK, DV), dtype=torch.float32, device=dev)
    n_states = torch.empty((B, NH, NC, DK), dtype=torch.float32, device=dev)
    m_states = torch.empty((B, NH, NC + 1), dtype=torch.float32, device=dev)
    C_T = torch.empty((B, NH, DK, DV), dtype=torch.float32, device=dev)
    n_T = torch.empty((B, NH, DK), dtype=torch.float32, device=dev)
    m_T = torch.empty((B, NH), dtype=torch.float32, device=dev)
    ws = torch.empty(max(substep_workspace_size(B, NH, T, DK, DV, chunk_size, dt, algo), 1),
                     dtype=torch.uint8, device=dev)
    st = _lib.lib().mlstm_fw_chunk_states(
        _ptr(K), _ptr(V), _ptr(i_pre), _ptr(f_pre), _ptr(C0), _ptr(n0), _ptr(m0), _ptr(C_states),
        _ptr(n_states), _ptr(m_states), _ptr(C_T), _ptr(n_T), _ptr(m_T), B, NH, T, DK, DV,
        chunk_size, _DT[dt], _GATE[gate_mode], _ALGO[algo], _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "mlstm_fw_chunk_states")
    return C_states, n_states, m_states, (C_T, n_T, m_T)


def mlstm_fw_parallel(Q, K, V, i_pre, f_pre, C_states, n_states, m0=None, *,
                      chunk_size: int = 64, gate_mode: str = "exp", algo: str = "auto"):
    """Parallel half: (H, n_out, m_out) from the chunk states."""
    B, NH, T, DK, DV, dev, dt = _check_common(Q, K, V, i_pre, f_pre)
    NC = (T + chunk_size - 1) // chunk_size
    _check_tensor("C_states", C_states, torch.float32, (B, NH, NC, DK, DV), dev)
    _check_tensor("n_states", n_states, torch.float32, (B, NH, NC, DK), dev)
    _check_tensor("m0", m0, torch.float32, (B, NH), dev)
    H = torch.empty((B, NH, T, DV), dtype=dt, device=dev)
    n_out = torch.empty((B, NH, T), dtype=torch.float32, device=dev)
    m_out = torch.empty((B, NH, T), dtype=torch.float32, device=dev)
    ws = torch.empty(max(substep_workspace_size(B, NH, T, DK, DV, chunk_size, dt, algo), 1),
                     dtype=torch.uint8, device=dev)
    st = _lib.lib().mlstm_fw_parallel(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(i_pre), _ptr(f_pre), _ptr(m0), _ptr(C_states),
        _ptr(n_states), _ptr(H), _ptr(n_out), _ptr(m_out), B, NH, T, DK, DV, chunk_size, _DT[dt],
        _GATE[gate_mode], _ALGO[algo], _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "mlstm_fw_parallel")
    return H, n_out, m_out


def last_device_error(device=None) -> int:
    """Synchronises the current stream and returns (and clears) the device
    error status (``_lib.OK``, ``_lib.ERR_TIMEOUT``, ...)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return int(_lib.lib().mlstm_last_device_error(_stream(dev)))


def set_watchdog(max_polls: int) -> None:
    _lib.lib().mlstm_set_watchdog(int(max_polls))


def watchdog_selftest(device=None) -> None:
    """Enqueues the failure-detection self-test (one bounded wait that nothing
    satisfies) on the current stream; the next ``last_device_error`` returns
    ``_lib.ERR_TIMEOUT``."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _lib.check(_lib.lib().mlstm_watchdog_selftest(_stream(dev)), "mlstm_watchdog_selftest")


class _MlstmChunkwise(torch.autograd.Function):
    """Differentiable mLSTM.  Where the training pair exists (``train_sizes``)
    and ``recompute`` is off, the forward is ``mlstm_fw_train`` and the
    backward ``mlstm_bw_saved`` (about 1 GB kept per 7B-shaped call, no
    recomputation); otherwise the forward is ``mlstm_fw`` and the backward
    ``mlstm_bw``, which recomputes what it needs from the inputs.  Gradients
    flow from H only; the returned final state carries none."""

    @staticmethod
    def forward(ctx, Q, K, V, i_pre, f_pre, C0, n0, m0, chunk_size, gate_mode, algo, recompute):
        saved = None
        if not recompute and algo == "auto" and Q.is_cuda and Q.dtype in _DT and \
                train_sizes(Q.shape[0], Q.shape[1], Q.shape[2], Q.shape[3], V.shape[-1],
                            Q.dtype) is not None:
            H, (C_T, n_T, m_T), saved = mlstm_fw_train(Q, K, V, i_pre, f_pre, C0, n0, m0,
                                                       gate_mode=gate_mode)
        else:
            H, (C_T, n_T, m_T) = mlstm_fw(Q, K, V, i_pre, f_pre, C0, n0, m0,
                                          chunk_size=chunk_size, gate_mode=gate_mode, algo=algo)
        if saved is not None:
            ctx.save_for_backward(Q, K, V, i_pre, f_pre, C0, n0, m0, H, saved)
        else:
            ctx.save_for_backward(Q, K, V, i_pre, f_pre, C0, n0, m0)
        ctx.cfg = (chunk_size, gate_mode, saved is not None)
        ctx.mark_non_differentiable(C_T, n_T, m_T)
        return H, C_T, n_T, m_T

    @staticmethod
    def backward(ctx, dH, dC_T, dn_T, dm_T):
        chunk_size, gate_mode, kept = ctx.cfg
        if kept:
            Q, K, V, i_pre, f_pre, C0, n0, m0, H, saved = ctx.saved_tensors
            g = mlstm_bw_saved(Q, K, V, i_pre, f_pre, H, saved, _upstream(dH), C0, n0, m0,
                               gate_mode=gate_mode)
        else:
            Q, K, V, i_pre, f_pre, C0, n0, m0 = ctx.saved_tensors
            g = mlstm_bw(Q, K, V, i_pre, f_pre, _upstream(dH), C0, n0, m0,
                         chunk_size=chunk_size, gate_mode=gate_mode)
        return (g["dQ"], g["dK"], g["dV"], g["di_pre"], g["df_pre"], g.get("dC0"), g.get("dn0"),
                g.get("dm0"), None, None, None, None)


def mlstm_chunkwise(Q, K, V, i_pre, f_pre, C0=None, n0=None, m0=None, *, chunk_size: int = 64,
                    gate_mode: str = "exp", algo: str = "auto", recompute: bool = False):
    """mLSTM forward pass that autograd can differentiate.

    Same arguments and shapes as ``mlstm_fw``; returns ``(H, (C_T, n_T, m_T))``.
    The gradient of a loss on H reaches Q, K, V, both gate pre-activations and
    the initial state; the final state is returned without a gradient path.
    Where the training pair exists (bf16, d_qk 128 or 256, T >= 128; see
    ``train_sizes``) the forward keeps the chunk states and per-token
    normalisers for the backward (128-token chunks, whatever ``chunk_size``
    says); ``recompute=True`` keeps nothing and recomputes them in the
    backward instead (less memory, a slower backward).
    """
    H, C_T, n_T, m_T = _MlstmChunkwise.apply(Q, K, V, i_pre, f_pre, C0, n0, m0, chunk_size,
                                             gate_mode, algo, recompute)
    return H, (C_T, n_T, m_T)


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------
_HERE = contextlib.nullcontext()


def _on(device):
    """Makes ``device`` current for a call (launches go to its stream)."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _check_gated_delta(Q, K, V, g, beta, C0, T_dims):
    """Shapes of a gated delta rule call; T_dims is (T,) or () for one token."""
    n = 3 + len(T_dims)
    if Q.dim() != n or V.dim() != n:
        raise ValueError("Q must be [B, NHK, T, DK] and V [B, NH, T, DV]" if T_dims else
                         "q must be [B, NHK, DK] and v [B, NH, DV]")
    B, NHK, DK = Q.shape[0], Q.shape[1], Q.shape[-1]
    NH, DV = V.shape[1], V.shape[-1]
    dt, dev = Q.dtype, Q.device
    if dt not in _DT:
        raise ValueError(f"unsupported dtype {dt} (float32 or bfloat16)")
    if NHK < 1 or NH % NHK != 0:
        raise ValueError(f"the {NH} heads of V must be a multiple of the {NHK} heads of Q and K")
    _check_tensor("Q", Q, dt, (B, NHK, *T_dims, DK), dev)
    _check_tensor("K", K, dt, (B, NHK, *T_dims, DK), dev)
    _check_tensor("V", V, dt, (B, NH, *T_dims, DV), dev)
    _check_tensor("g", g, torch.float32, (B, NH, *T_dims), dev)
    _check_tensor("beta", beta, torch.float32, (B, NH, *T_dims), dev)
    _check_tensor("C0" if T_dims else "C", C0, torch.float32, (B, NH, DK, DV), dev)
    return B, NHK, NH, DK, DV, dev, dt


@functools.lru_cache(maxsize=1024)  # sizes alone decide it
def gated_delta_workspace_size(B, NHK, NH, T, DK, DV, dtype=torch.bfloat16, algo="auto",
                               backward=False) -> int:
    """Bytes of workspace of ``gated_delta_fw`` (or, ``backward``, of
    ``gated_delta_bw``)."""
    n = ctypes.c_size_t(0)
    _lib.check(_lib.lib().mlstm_gated_delta_workspace_size(
        B, NHK, NH, T, DK, DV, _DT[dtype], _ALGO[algo], int(backward), ctypes.byref(n)),
        "mlstm_gated_delta_workspace_size")
    return int(n.value)


def gated_delta_fw(Q, K, V, g, beta, C0=None, *, scale: float | None = None, algo: str = "auto",
                   return_last_state: bool = True, workspace: torch.Tensor | None = None,
                   out: dict | None = None):
    """Gated delta rule forward pass on the GPU: for every (b, head) and token,

        C_t = e^{g_t} C_{t-1} + beta_t k_t (v_t - e^{g_t} C_{t-1}^T k_t)^T
        h_t = scale * C_t^T q_t

    Q, K [B,NHK,T,DK] and V [B,NH,T,DV] (float32 or bfloat16, same dtype), NHK
    dividing NH: head n of V reads head n // (NH // NHK) of Q and K.  g (log
    decay, <= 0; -inf forgets the state) and beta [B,NH,T] float32; optional
    initial state C0 [B,NH,DK,DV] float32.  ``scale`` defaults to 1/sqrt(DK).
    Padded tokens with g = beta = 0 (and finite q, k, v) leave the state as it
    was.  A reset at the first token forgets C0 whatever it holds; elsewhere an
    infinity or a NaN reaches all of its head from its chunk on (64 or 128 tokens),
    behind resets and padding too.  Returns ``(H, C_T)``, or ``H`` without
    ``return_last_state``.  ``out`` may hold preallocated ``H`` / ``C_T`` (C_T may
    be C0 itself); ``workspace`` a uint8 CUDA tensor of at least
    ``gated_delta_workspace_size(...)`` bytes.  ``algo``: "auto", "simt" (fp32 on
    the CUDA cores: what "auto" takes for float32, DK above 128, or DK or DV that
    are no multiples of 8; 3 to 7 times the time) or "tc".
    """
    if Q.dim() != 4:
        raise ValueError("Q must be [B, NHK, T, DK] and V [B, NH, T, DV]")
    T = Q.shape[2]
    B, NHK, NH, DK, DV, dev, dt = _check_gated_delta(Q, K, V, g, beta, C0, (T,))
    out = {} if out is None else out
    given = H, C_T = out.get("H"), out.get("C_T") if return_last_state else None
    if H is None:
        H = torch.empty_like(V)
    else:
        _check_tensor("H", H, dt, (B, NH, T, DV), dev)
    if C_T is None and return_last_state:
        C_T = g.new_empty((B, NH, DK, DV))
    else:
        _check_tensor("C_T", C_T, torch.float32, (B, NH, DK, DV), dev)
    ws_bytes = gated_delta_workspace_size(B, NHK, NH, T, DK, DV, dt, algo)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    elif workspace.dtype != torch.uint8 or workspace.numel() < ws_bytes or \
            workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a uint8 tensor of >= {ws_bytes} bytes on {dev}")
    with _on(dev):
        st = _lib.lib().mlstm_gated_delta_fw(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(g), _ptr(beta), _ptr(C0), _ptr(H), _ptr(C_T), B, NHK,
            NH, T, DK, DV, DK ** -0.5 if scale is None else float(scale), _DT[dt], _ALGO[algo],
            _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(st, "mlstm_gated_delta_fw")
    if out:
        _written(*given)
    return (H, C_T) if return_last_state else H


def _gated_delta_grads(Q, K, V, g, beta, dH, C0, dC_T):
    """Checks the upstream gradients and allocates the gradients."""
    _check_tensor("dH", dH, Q.dtype, tuple(V.shape), Q.device)
    _check_tensor("dC_T", dC_T, torch.float32, (*V.shape[:2], Q.shape[3], V.shape[3]), Q.device)
    out = {"dQ": torch.empty_like(Q), "dK": torch.empty_like(K), "dV": torch.empty_like(V),
           "dg": torch.empty_like(g), "dbeta": torch.empty_like(beta)}
    if C0 is not None:
        out["dC0"] = torch.empty_like(C0)
    return out


def gated_delta_bw(Q, K, V, g, beta, dH, C0=None, dC_T=None, *, scale: float | None = None,
                   algo: str = "auto"):
    """Gradients of a loss on ``gated_delta_fw``'s H (dH, in the input dtype)
    and, with ``dC_T`` [B,NH,DK,DV] float32, on its final state.  Returns a dict
    with dQ, dK (summed over the value heads that share them) and dV in the
    input dtype, dg and dbeta float32 and, when C0 is given, dC0 float32.  The
    forward is recomputed from the inputs."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, NHK, T, DK] and V [B, NH, T, DV]")
    T = Q.shape[2]
    B, NHK, NH, DK, DV, dev, dt = _check_gated_delta(Q, K, V, g, beta, C0, (T,))
    out = _gated_delta_grads(Q, K, V, g, beta, dH, C0, dC_T)
    n = gated_delta_workspace_size(B, NHK, NH, T, DK, DV, dt, algo, backward=True)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _lib.lib().mlstm_gated_delta_bw(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(g), _ptr(beta), _ptr(C0), _ptr(dH), _ptr(dC_T),
            _ptr(out["dQ"]), _ptr(out["dK"]), _ptr(out["dV"]), _ptr(out["dg"]),
            _ptr(out["dbeta"]), _ptr(out.get("dC0")), B, NHK, NH, T, DK, DV,
            DK ** -0.5 if scale is None else float(scale), _DT[dt], _ALGO[algo], _ptr(ws),
            ws.numel(), _stream(dev))
    _lib.check(st, "mlstm_gated_delta_bw")
    return out


@functools.lru_cache(maxsize=1024)
def gated_delta_train_sizes(B, NHK, NH, T, DK, DV, dtype=torch.bfloat16):
    """Bytes of the saved buffer and of the two calls' workspaces of the
    training pair, or None where it does not exist (it needs the tensor-core
    gradients: bf16, DK up to 128, DK and DV multiples of 8, at least 64 tokens
    over all heads)."""
    sv, fw, bw = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = _lib.lib().mlstm_gated_delta_train_sizes(B, NHK, NH, T, DK, DV, _DT[dtype],
                                                  ctypes.byref(sv), ctypes.byref(fw),
                                                  ctypes.byref(bw))
    if st == _lib.ERR_UNSUPPORTED:
        return None
    _lib.check(st, "mlstm_gated_delta_train_sizes")
    return int(sv.value), int(fw.value), int(bw.value)


def gated_delta_fw_train(Q, K, V, g, beta, C0=None, *, scale: float | None = None):
    """The forward pass of ``gated_delta_fw`` that also keeps what
    ``gated_delta_bw_saved`` needs.  Returns ``(H, C_T, saved)``; ``saved`` is
    an opaque uint8 tensor (about 2.1 KB per token and head at DK = DV = 128).
    Raises ``MlstmError`` (unsupported) outside the shapes of
    ``gated_delta_train_sizes``."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, NHK, T, DK] and V [B, NH, T, DV]")
    T = Q.shape[2]
    B, NHK, NH, DK, DV, dev, dt = _check_gated_delta(Q, K, V, g, beta, C0, (T,))
    sizes = gated_delta_train_sizes(B, NHK, NH, T, DK, DV, dt)
    if sizes is None:
        raise MlstmError(_lib.ERR_UNSUPPORTED, "mlstm_gated_delta_fw_train")
    H = torch.empty_like(V)
    C_T = torch.empty((B, NH, DK, DV), dtype=torch.float32, device=dev)
    saved = torch.empty(sizes[0], dtype=torch.uint8, device=dev)
    ws = torch.empty(sizes[1], dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _lib.lib().mlstm_gated_delta_fw_train(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(g), _ptr(beta), _ptr(C0), _ptr(H), _ptr(C_T),
            _ptr(saved), sizes[0], B, NHK, NH, T, DK, DV,
            DK ** -0.5 if scale is None else float(scale), _DT[dt], _ptr(ws), sizes[1],
            _stream(dev))
    _lib.check(st, "mlstm_gated_delta_fw_train")
    return H, C_T, saved


def gated_delta_bw_saved(Q, K, V, g, beta, saved, dH, C0=None, dC_T=None, *,
                         scale: float | None = None):
    """``gated_delta_bw`` from the saved buffer of ``gated_delta_fw_train``
    (same inputs and scale) instead of a recomputed forward.  Returns the same
    dict."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, NHK, T, DK] and V [B, NH, T, DV]")
    T = Q.shape[2]
    B, NHK, NH, DK, DV, dev, dt = _check_gated_delta(Q, K, V, g, beta, C0, (T,))
    sizes = gated_delta_train_sizes(B, NHK, NH, T, DK, DV, dt)
    if sizes is None:
        raise MlstmError(_lib.ERR_UNSUPPORTED, "mlstm_gated_delta_bw_saved")
    _check_tensor("saved", saved, torch.uint8, (sizes[0],), dev)
    out = _gated_delta_grads(Q, K, V, g, beta, dH, C0, dC_T)
    ws = torch.empty(sizes[2], dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _lib.lib().mlstm_gated_delta_bw_saved(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(g), _ptr(beta), _ptr(saved), sizes[0], _ptr(dH),
            _ptr(dC_T), _ptr(out["dQ"]), _ptr(out["dK"]), _ptr(out["dV"]), _ptr(out["dg"]),
            _ptr(out["dbeta"]), _ptr(out.get("dC0")), B, NHK, NH, T, DK, DV,
            DK ** -0.5 if scale is None else float(scale), _DT[dt], _ptr(ws), sizes[2],
            _stream(dev))
    _lib.check(st, "mlstm_gated_delta_bw_saved")
    return out


def gated_delta_step(q, k, v, g, beta, C, *, scale: float | None = None, h=None):
    """One token of ``gated_delta_fw`` for every (b, head), in place on the
    state: q, k [B,NHK,DK], v [B,NH,DV], g, beta [B,NH] float32, C [B,NH,DK,DV]
    float32 (overwritten; a g of -inf forgets it whatever it holds).  Returns h
    [B,NH,DV] in the input dtype (``h`` may be given)."""
    B, NHK, NH, DK, DV, dev, dt = _check_gated_delta(q, k, v, g, beta, C, ())
    given = h
    if h is None:
        h = torch.empty_like(v)
    else:
        _check_tensor("h", h, dt, (B, NH, DV), dev)
    with _on(dev):
        st = _lib.lib().mlstm_gated_delta_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(C), _ptr(h), B, NHK, NH, DK, DV,
            DK ** -0.5 if scale is None else float(scale), _DT[dt], _stream(dev))
    _lib.check(st, "mlstm_gated_delta_step")
    _written_one(C)
    if given is not None:
        _written_one(given)
    return h


class _GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, g, beta, C0, scale, algo, recompute):
        saved = None
        if not recompute and algo == "auto" and Q.dim() == 4 and V.dim() == 4 and \
                Q.dtype in _DT and \
                gated_delta_train_sizes(Q.shape[0], Q.shape[1], V.shape[1], Q.shape[2],
                                        Q.shape[3], V.shape[3], Q.dtype) is not None:
            H, C_T, saved = gated_delta_fw_train(Q, K, V, g, beta, C0, scale=scale)
        else:
            H, C_T = gated_delta_fw(Q, K, V, g, beta, C0, scale=scale, algo=algo)
        ctx.save_for_backward(Q, K, V, g, beta, C0, saved)
        ctx.cfg = (scale, algo)
        ctx.set_materialize_grads(False)
        return H, C_T

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dH, dC_T):
        if dH is None and dC_T is None:
            return (None,) * 9
        Q, K, V, g, beta, C0, saved = ctx.saved_tensors
        scale, algo = ctx.cfg
        dH = torch.zeros_like(V) if dH is None else _upstream(dH)
        dC_T = None if dC_T is None else _upstream(dC_T)
        if saved is not None:
            d = gated_delta_bw_saved(Q, K, V, g, beta, saved, dH, C0, dC_T, scale=scale)
        else:
            d = gated_delta_bw(Q, K, V, g, beta, dH, C0, dC_T, scale=scale, algo=algo)
        return (d["dQ"], d["dK"], d["dV"], d["dg"], d["dbeta"], d.get("dC0"), None, None, None)


def gated_delta_chunkwise(Q, K, V, g, beta, C0=None, *, scale: float | None = None,
                          algo: str = "auto", recompute: bool = False):
    """``gated_delta_fw`` that autograd can differentiate: returns ``(H, C_T)``;
    gradients of losses on H and on C_T reach Q, K, V, g, beta and C0.  Where
    the training pair exists (``gated_delta_train_sizes``) the forward keeps
    about 2.1 KB per token and head (DK = DV = 128) for the backward;
    ``recompute=True`` keeps the inputs alone and recomputes the forward.  Where
    nothing will be differentiated (``torch.no_grad()``, no input that requires a
    gradient) it is ``gated_delta_fw``.
    (Capture of a backward pass into a CUDA graph: as with any autograd
    function, not while an eager graph holds the same leaves; differentiate
    ``x.detach()``.)"""
    # asked here: inside the function an input's requires_grad says nothing of no_grad()
    if not torch.is_grad_enabled() or \
            not any(t is not None and t.requires_grad for t in (Q, K, V, g, beta, C0)):
        return gated_delta_fw(Q, K, V, g, beta, C0, scale=scale, algo=algo)
    return _GatedDelta.apply(Q, K, V, g, beta, C0, scale, algo, recompute)


# ---------------------------------------------------------------------------
# layer norm of the cell output
# ---------------------------------------------------------------------------
def _check_head_norm(X, weight, bias):
    if X.dim() != 4:
        raise ValueError("X must be [B, NH, T, D]")
    B, NH, T, D = X.shape
    if X.dtype not in _DT:
        raise ValueError(f"unsupported dtype {X.dtype} (float32 or bfloat16)")
    _check_tensor("X", X, X.dtype, (B, NH, T, D), X.device)
    _check_tensor("weight", weight, torch.float32, (NH, D), X.device)
    _check_tensor("bias", bias, torch.float32, (NH, D), X.device)
    return B, NH, T, D, X.device, X.dtype


def head_norm_fw(X, weight, bias=None, *, eps: float = 1e-5, out: torch.Tensor | None = None):
    """Layer norm of the cell output X [B,NH,T,D] (float32 or bfloat16) over D
    per (token, head), with weight and optional bias [NH,D] float32, laid out
    token-major for an output projection.  Returns ``(Y [B,T,NH*D], mean, rstd
    [B,NH,T] float32)``.  With NH = 1 it is the layer norm of B*T rows."""
    B, NH, T, D, dev, dt = _check_head_norm(X, weight, bias)
    if out is None:
        Y = X.new_empty((B, T, NH * D))
    else:
        Y = out
        _check_tensor("out", Y, dt, (B, T, NH * D), dev)
    mean = weight.new_empty((B, NH, T))
    rstd = torch.empty_like(mean)
    with _on(dev):
        st = _lib.lib().mlstm_head_norm_fw(_ptr(X), _ptr(weight), _ptr(bias), _ptr(Y), _ptr(mean),
                                           _ptr(rstd), B, NH, T, D, float(eps), _DT[dt],
                                           _stream(dev))
    _lib.check(st, "mlstm_head_norm_fw")
    if out is not None:
        _written(out)
    return Y, mean, rstd


@functools.lru_cache(maxsize=1024)
def _head_norm_workspace(B, NH, T, D, dtype) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.lib().mlstm_head_norm_bw_workspace_size(B, NH, T, D, _DT[dtype],
                                                            ctypes.byref(n)),
               "mlstm_head_norm_bw_workspace_size")
    return max(int(n.value), 1)


def head_norm_bw(X, dY, weight, mean, rstd, *, bias: bool = True):
    """Gradients of a loss on ``head_norm_fw``'s Y, from dY [B,T,NH*D] and the
    forward's mean and rstd: a dict with dX (input dtype), dweight and, with
    ``bias``, dbias [NH,D] float32 (summed in a fixed order)."""
    B, NH, T, D, dev, dt = _check_head_norm(X, weight, None)
    _check_tensor("dY", dY, dt, (B, T, NH * D), dev)
    _check_tensor("mean", mean, torch.float32, (B, NH, T), dev)
    _check_tensor("rstd", rstd, torch.float32, (B, NH, T), dev)
    out = {"dX": torch.empty_like(X), "dweight": torch.empty_like(weight)}
    if bias:
        out["dbias"] = torch.empty_like(weight)
    ws = torch.empty(_head_norm_workspace(B, NH, T, D, dt), dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _lib.lib().mlstm_head_norm_bw(
            _ptr(X), _ptr(dY), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(out["dX"]),
            _ptr(out["dweight"]), _ptr(out.get("dbias")), B, NH, T, D, _DT[dt], _ptr(ws),
            ws.numel(), _stream(dev))
    _lib.check(st, "mlstm_head_norm_bw")
    return out


class _HeadNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, weight, bias, eps):
        Y, mean, rstd = head_norm_fw(X, weight, bias, eps=eps)
        ctx.save_for_backward(X, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        X, weight, mean, rstd = ctx.saved_tensors
        d = head_norm_bw(X, _upstream(dY), weight, mean, rstd, bias=ctx.has_bias)
        return d["dX"], d["dweight"], d.get("dbias"), None


def head_norm(X, weight, bias=None, *, eps: float = 1e-5):
    """``head_norm_fw`` that autograd can differentiate; returns Y.  (Capture of a
    backward pass: as ``gated_delta_chunkwise``.)"""
    return _HeadNorm.apply(X, weight, bias, eps)

"""Binding of linear attention with a decay per head (the gdn_linear_* entry
points of include/gdn.h): S_t = lam S_{t-1} + v_t k_t^T, o_t = scale S_t q_t,
lam = exp(log_decay[h]).  Argument marshalling only, as the package's other
calls.  log_decay is a constant of the layer: there is no gradient for it."""
from __future__ import annotations

import contextlib

import torch

from . import DTYPE, GdnError, _check, _ptr, library

F32, I32 = torch.float32, torch.int32


@contextlib.contextmanager
def _on(dev, stream):
    """The device of the tensors and the stream of the call made current, so
    that outputs and workspaces allocated for it belong to that stream; yields
    the stream's handle."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream(dev).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _shapes(name, q, k, v, log_decay):
    """Checks q, k, v and log_decay; (rows, Hqk, Hv, Dk, Dv, dtype, device)."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"{name} runs on CUDA tensors only")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"{name}: q and v must have three dimensions")
    rows, Hqk, Dk = q.shape
    Hv, Dv = v.shape[1], v.shape[2]
    if q.dtype not in DTYPE:
        raise ValueError(f"unsupported io dtype {q.dtype}")
    _check(q, "q", (rows, Hqk, Dk), q.dtype, dev)
    _check(k, "k", (rows, Hqk, Dk), q.dtype, dev)
    _check(v, "v", (rows, Hv, Dv), q.dtype, dev)
    _check(log_decay, "log_decay", (Hv,), F32, dev)
    return rows, Hqk, Hv, Dk, Dv, q.dtype, dev


def _sequences(cu_seqlens, dev):
    if cu_seqlens is None:
        return 1
    N = cu_seqlens.shape[0] - 1
    _check(cu_seqlens, "cu_seqlens", (N + 1,), I32, dev)
    return N


def _flag(error_flag, dev):
    if error_flag is not None:
        _check(error_flag, "error_flag", tuple(error_flag.shape), I32, dev)


def _scratch(workspace, need, dev):
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous, on {dev}")
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def gdn_linear_prefill_workspace_bytes(N, T, Hqk, Hv, Dk, Dv, dtype=torch.bfloat16):
    """Scratch bytes gdn_linear_prefill and gdn_linear_prefill_slots need."""
    return int(library().gdn_linear_prefill_workspace_bytes(N, T, Hqk, Hv, Dk, Dv, DTYPE[dtype]))


def gdn_linear_prefill_backward_workspace_bytes(N, T, Hqk, Hv, Dk, Dv, dtype=torch.bfloat16):
    """Scratch bytes gdn_linear_prefill_backward needs."""
    return int(library().gdn_linear_prefill_backward_workspace_bytes(N, T, Hqk, Hv, Dk, Dv,
                                                                     DTYPE[dtype]))


def gdn_linear_prefill(q, k, v, log_decay, initial_state=None, cu_seqlens=None, *, scale=1.0, o=None,
                       final_state=None, output_final_state=True, workspace=None, error_flag=None,
                       stream=None):
    """Linear attention over a packed batch: q, k [T,Hqk,Dk], v [T,Hv,Dv] (bf16 or
    fp32); log_decay [Hv] fp32, <= 0; initial_state [N,Hv,Dv,Dk] fp32 or None;
    cu_seqlens int32 [N+1] or None.  Returns (o [T,Hv,Dv], final_state or None);
    ``final_state`` may be ``initial_state`` (in place)."""
    lib = library()
    T, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_prefill", q, k, v, log_decay)
    N = _sequences(cu_seqlens, dev)
    if initial_state is not None:
        _check(initial_state, "initial_state", (N, Hv, Dv, Dk), F32, dev)
    _flag(error_flag, dev)
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty((T, Hv, Dv), dtype=dt, device=dev)
        _check(o, "o", (T, Hv, Dv), dt, dev)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, Hv, Dv, Dk), dtype=F32, device=dev)
        if final_state is not None:
            _check(final_state, "final_state", (N, Hv, Dv, Dk), F32, dev)
        workspace, ws_bytes = _scratch(
            workspace, lib.gdn_linear_prefill_workspace_bytes(N, T, Hqk, Hv, Dk, Dv, DTYPE[dt]), dev)
        rc = lib.gdn_linear_prefill(_ptr(q), _ptr(k), _ptr(v), DTYPE[dt], _ptr(log_decay), scale,
                                    _ptr(initial_state), _ptr(cu_seqlens), N, T, Hqk, Hv, Dk, Dv,
                                    _ptr(o), _ptr(final_state), _ptr(workspace), ws_bytes,
                                    _ptr(error_flag), st)
    if rc != 0:
        raise GdnError(rc, "gdn_linear_prefill")
    return o, final_state


def gdn_linear_prefill_slots(q, k, v, log_decay, state_pool, slot_idx, reset=None, cu_seqlens=None, *,
                             scale=1.0, o=None, workspace=None, error_flag=None, stream=None):
    """gdn_linear_prefill whose sequence n starts from ``state_pool[slot_idx[n]]``
    ([num_slots,Hv,Dv,Dk] fp32, updated in place), or from zeros when ``reset[n]``
    is nonzero; slot_idx (distinct) and reset int32 [N].  Returns o."""
    lib = library()
    T, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_prefill_slots", q, k, v, log_decay)
    N, S = _sequences(cu_seqlens, dev), state_pool.shape[0]
    _check(state_pool, "state_pool", (S, Hv, Dv, Dk), F32, dev)
    _check(slot_idx, "slot_idx", (N,), I32, dev)
    if reset is not None:
        _check(reset, "reset", (N,), I32, dev)
    _flag(error_flag, dev)
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty((T, Hv, Dv), dtype=dt, device=dev)
        _check(o, "o", (T, Hv, Dv), dt, dev)
        workspace, ws_bytes = _scratch(
            workspace, lib.gdn_linear_prefill_workspace_bytes(N, T, Hqk, Hv, Dk, Dv, DTYPE[dt]), dev)
        rc = lib.gdn_linear_prefill_slots(_ptr(q), _ptr(k), _ptr(v), DTYPE[dt], _ptr(log_decay), scale,
                                          _ptr(state_pool), S, _ptr(slot_idx), _ptr(reset),
                                          _ptr(cu_seqlens), N, T, Hqk, Hv, Dk, Dv, _ptr(o),
                                          _ptr(workspace), ws_bytes, _ptr(error_flag), st)
    if rc != 0:
        raise GdnError(rc, "gdn_linear_prefill_slots")
    return o


def gdn_linear_prefill_backward(do, q, k, v, log_decay, initial_state=None, cu_seqlens=None, *,
                                dfinal_state=None, scale=1.0, dq=None, dk=None, dv=None,
                                dinitial_state=None, output_dinitial_state=False, workspace=None,
                                error_flag=None, stream=None):
    """Gradients of gdn_linear_prefill: ``do`` [T,Hv,Dv] is o's, ``dfinal_state``
    [N,Hv,Dv,Dk] (or None) the final state's, the rest as in the forward call.
    Returns (dq, dk, dv, dinitial_state); the last is None unless asked for
    (``output_dinitial_state``, or a tensor, which may be ``dfinal_state``)."""
    lib = library()
    T, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_prefill_backward", q, k, v, log_decay)
    N = _sequences(cu_seqlens, dev)
    _check(do, "do", (T, Hv, Dv), dt, dev)
    for x, name in ((initial_state, "initial_state"), (dfinal_state, "dfinal_state")):
        if x is not None:
            _check(x, name, (N, Hv, Dv, Dk), F32, dev)
    _flag(error_flag, dev)
    with _on(dev, stream) as st:
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        _check(dq, "dq", (T, Hqk, Dk), dt, dev)
        _check(dk, "dk", (T, Hqk, Dk), dt, dev)
        _check(dv, "dv", (T, Hv, Dv), dt, dev)
        if dinitial_state is None and output_dinitial_state:
            dinitial_state = torch.empty((N, Hv, Dv, Dk), dtype=F32, device=dev)
        if dinitial_state is not None:
            _check(dinitial_state, "dinitial_state", (N, Hv, Dv, Dk), F32, dev)
        workspace, ws_bytes = _scratch(
            workspace,
            lib.gdn_linear_prefill_backward_workspace_bytes(N, T, Hqk, Hv, Dk, Dv, DTYPE[dt]), dev)
        rc = lib.gdn_linear_prefill_backward(
            _ptr(do), _ptr(q), _ptr(k), _ptr(v), DTYPE[dt], _ptr(log_decay), scale,
            _ptr(initial_state), _ptr(dfinal_state), _ptr(cu_seqlens), N, T, Hqk, Hv, Dk, Dv, _ptr(dq),
            _ptr(dk), _ptr(dv), _ptr(dinitial_state), _ptr(workspace), ws_bytes, _ptr(error_flag), st)
    if rc != 0:
        raise GdnError(rc, "gdn_linear_prefill_backward")
    return dq, dk, dv, dinitial_state


def gdn_linear_decode_step(q, k, v, log_decay, state, *, scale=1.0, o=None, error_flag=None,
                           stream=None):
    """One token of N sequences, in place on ``state`` [N,Hv,Dv,Dk] fp32: q, k
    [N,Hqk,Dk], v [N,Hv,Dv] (bf16 or fp32), log_decay [Hv].  Returns o [N,Hv,Dv]."""
    lib = library()
    N, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_decode_step", q, k, v, log_decay)
    _check(state, "state", (N, Hv, Dv, Dk), F32, dev)
    _flag(error_flag, dev)
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty((N, Hv, Dv), dtype=dt, device=dev)
        _check(o, "o", (N, Hv, Dv), dt, dev)
        rc = lib.gdn_linear_decode_step(_ptr(q), _ptr(k), _ptr(v), DTYPE[dt], _ptr(log_decay), scale,
                                        _ptr(state), N, Hqk, Hv, Dk, Dv, _ptr(o), _ptr(error_flag), st)
    if rc != 0:
        raise GdnError(rc, "gdn_linear_decode_step")
    return o


def gdn_linear_decode_step_slots(q, k, v, log_decay, state_pool, slot_idx, reset=None, *, scale=1.0,
                                 o=None, error_flag=None, stream=None):
    """gdn_linear_decode_step whose entry n uses ``state_pool[slot_idx[n]]``
    ([num_slots,Hv,Dv,Dk] fp32, updated in place), from zeros when ``reset[n]``
    is nonzero; slot_idx (distinct) and reset int32 [N].  Returns o."""
    lib = library()
    N, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_decode_step_slots", q, k, v, log_decay)
    S = state_pool.shape[0]
    _check(state_pool, "state_pool", (S, Hv, Dv, Dk), F32, dev)
    _check(slot_idx, "slot_idx", (N,), I32, dev)
    if reset is not None:
        _check(reset, "reset", (N,), I32, dev)
    _flag(error_flag, dev)
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty((N, Hv, Dv), dtype=dt, device=dev)
        _check(o, "o", (N, Hv, Dv), dt, dev)
        rc = lib.gdn_linear_decode_step_slots(_ptr(q), _ptr(k), _ptr(v), DTYPE[dt], _ptr(log_decay),
                                              scale, _ptr(state_pool), S, _ptr(slot_idx), _ptr(reset),
                                              N, Hqk, Hv, Dk, Dv, _ptr(o), _ptr(error_flag), st)
    if rc != 0:
        raise GdnError(rc, "gdn_linear_decode_step_slots")
    return o

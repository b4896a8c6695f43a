"""Binding of linear attention with a decay per head (the gdn_linear_* entry
points of include/gdn.h): S_t = lam S_{t-1} + v_t k_t^T, o_t = scale S_t q_t,
lam = exp(log_decay[h]).  Argument marshalling only, as the package's other
calls.  log_decay is a constant of the layer: there is no gradient for it."""
from __future__ import annotations

import torch

from . import DTYPE, GdnError, _check, library

F32, I32 = torch.float32, torch.int32
# as torch.cuda.current_device() and torch.cuda.current_stream(i).cuda_stream give them
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _need(t, name, shape, dtype, dev):
    """_check without building its messages: these calls are made per token and
    layer, and an elaborate check of every argument costs more than the launch."""
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != dev
            or not t.is_contiguous()):
        _check(t, name, shape, dtype, dev)


def _at(t):
    """The address of a tensor, or None."""
    return None if t is None else t.data_ptr()


def _run(dev, stream, call):
    """call(handle) with the tensors' device and the call's stream current, so that
    outputs and workspaces it allocates belong to that stream."""
    if stream is None:
        if _device() == dev.index:  # (the public calls build objects, 2 us of a call's 13)
            return call(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return call(_raw_stream(dev.index))
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _raise(rc, name):
    if rc != 0:
        raise GdnError(rc, name)


def _shapes(name, q, k, v, log_decay):
    """Checks q, k, v and log_decay; (rows, Hqk, Hv, Dk, Dv, dtype, device)."""
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError(f"{name} runs on CUDA tensors only")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"{name}: q and v must have three dimensions")
    rows, Hqk, Dk = q.shape
    _, Hv, Dv = v.shape
    if dt not in DTYPE:
        raise ValueError(f"unsupported io dtype {dt}")
    _need(q, "q", (rows, Hqk, Dk), dt, dev)
    _need(k, "k", (rows, Hqk, Dk), dt, dev)
    _need(v, "v", (rows, Hv, Dv), dt, dev)
    _need(log_decay, "log_decay", (Hv,), F32, dev)
    return rows, Hqk, Hv, Dk, Dv, dt, dev


def _sequences(cu_seqlens, dev):
    if cu_seqlens is None:
        return 1
    N = cu_seqlens.shape[0] - 1
    _need(cu_seqlens, "cu_seqlens", (N + 1,), I32, dev)
    return N


def _flag(error_flag, dev):
    if error_flag is not None:
        _need(error_flag, "error_flag", tuple(error_flag.shape), I32, dev)


def _slots(state_pool, slot_idx, reset, N, Hv, Dv, Dk, dev):
    S = state_pool.shape[0]
    _need(state_pool, "state_pool", (S, Hv, Dv, Dk), F32, dev)
    _need(slot_idx, "slot_idx", (N,), I32, dev)
    if reset is not None:
        _need(reset, "reset", (N,), I32, dev)
    return S


def _output(t, name, shape, dtype, dev):
    """`t`, checked, or a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, name, shape, dtype, dev)
    return t


def _scratch(workspace, need, dev):
    """(address, bytes, tensor) of the workspace, or of a new one."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous, on {dev}")
    if workspace is None:
        return None, 0, None
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


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
        _need(initial_state, "initial_state", (N, Hv, Dv, Dk), F32, dev)
    _flag(error_flag, dev)
    sizes = (N, T, Hqk, Hv, Dk, Dv)

    def call(st):
        out = _output(o, "o", (T, Hv, Dv), dt, dev)
        final = final_state
        if final is not None or output_final_state:
            final = _output(final, "final_state", (N, Hv, Dv, Dk), F32, dev)
        ws, n, _keep = _scratch(workspace, lib.gdn_linear_prefill_workspace_bytes(*sizes, DTYPE[dt]), dev)
        _raise(lib.gdn_linear_prefill(_at(q), _at(k), _at(v), DTYPE[dt], _at(log_decay), scale,
                                      _at(initial_state), _at(cu_seqlens), *sizes, _at(out), _at(final), ws,
                                      n, _at(error_flag), st), "gdn_linear_prefill")
        return out, final

    return _run(dev, stream, call)


def gdn_linear_prefill_slots(q, k, v, log_decay, state_pool, slot_idx, reset=None, cu_seqlens=None, *,
                             scale=1.0, o=None, workspace=None, error_flag=None, stream=None):
    """gdn_linear_prefill whose sequence n starts from ``state_pool[slot_idx[n]]``
    ([num_slots,Hv,Dv,Dk] fp32, updated in place), or from zeros when ``reset[n]``
    is nonzero; slot_idx (distinct) and reset int32 [N].  Returns o."""
    lib = library()
    T, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_prefill_slots", q, k, v, log_decay)
    N = _sequences(cu_seqlens, dev)
    S = _slots(state_pool, slot_idx, reset, N, Hv, Dv, Dk, dev)
    _flag(error_flag, dev)
    sizes = (N, T, Hqk, Hv, Dk, Dv)

    def call(st):
        out = _output(o, "o", (T, Hv, Dv), dt, dev)
        ws, n, _keep = _scratch(workspace, lib.gdn_linear_prefill_workspace_bytes(*sizes, DTYPE[dt]), dev)
        _raise(lib.gdn_linear_prefill_slots(_at(q), _at(k), _at(v), DTYPE[dt], _at(log_decay), scale,
                                            _at(state_pool), S, _at(slot_idx), _at(reset), _at(cu_seqlens),
                                            *sizes, _at(out), ws, n, _at(error_flag), st),
               "gdn_linear_prefill_slots")
        return out

    return _run(dev, stream, call)


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
    _need(do, "do", (T, Hv, Dv), dt, dev)
    for x, name in ((initial_state, "initial_state"), (dfinal_state, "dfinal_state")):
        if x is not None:
            _need(x, name, (N, Hv, Dv, Dk), F32, dev)
    _flag(error_flag, dev)
    sizes = (N, T, Hqk, Hv, Dk, Dv)

    def call(st):
        gq = _output(dq, "dq", (T, Hqk, Dk), dt, dev)
        gk = _output(dk, "dk", (T, Hqk, Dk), dt, dev)
        gv = _output(dv, "dv", (T, Hv, Dv), dt, dev)
        gs = dinitial_state
        if gs is not None or output_dinitial_state:
            gs = _output(gs, "dinitial_state", (N, Hv, Dv, Dk), F32, dev)
        ws, n, _keep = _scratch(
            workspace, lib.gdn_linear_prefill_backward_workspace_bytes(*sizes, DTYPE[dt]), dev)
        _raise(lib.gdn_linear_prefill_backward(_at(do), _at(q), _at(k), _at(v), DTYPE[dt], _at(log_decay),
                                               scale, _at(initial_state), _at(dfinal_state), _at(cu_seqlens),
                                               *sizes, _at(gq), _at(gk), _at(gv), _at(gs), ws, n,
                                               _at(error_flag), st), "gdn_linear_prefill_backward")
        return gq, gk, gv, gs

    return _run(dev, stream, call)


def gdn_linear_decode_step(q, k, v, log_decay, state, *, scale=1.0, o=None, error_flag=None,
                           stream=None):
    """One token of N sequences, in place on ``state`` [N,Hv,Dv,Dk] fp32: q, k
    [N,Hqk,Dk], v [N,Hv,Dv] (bf16 or fp32), log_decay [Hv].  Returns o [N,Hv,Dv]."""
    lib = library()
    N, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_decode_step", q, k, v, log_decay)
    _need(state, "state", (N, Hv, Dv, Dk), F32, dev)
    _flag(error_flag, dev)

    def call(st):
        out = _output(o, "o", (N, Hv, Dv), dt, dev)
        _raise(lib.gdn_linear_decode_step(_at(q), _at(k), _at(v), DTYPE[dt], _at(log_decay), scale,
                                          _at(state), N, Hqk, Hv, Dk, Dv, _at(out), _at(error_flag), st),
               "gdn_linear_decode_step")
        return out

    return _run(dev, stream, call)


def gdn_linear_decode_step_slots(q, k, v, log_decay, state_pool, slot_idx, reset=None, *, scale=1.0,
                                 o=None, error_flag=None, stream=None):
    """gdn_linear_decode_step whose entry n uses ``state_pool[slot_idx[n]]``
    ([num_slots,Hv,Dv,Dk] fp32, updated in place), from zeros when ``reset[n]``
    is nonzero; slot_idx (distinct) and reset int32 [N].  Returns o."""
    lib = library()
    N, Hqk, Hv, Dk, Dv, dt, dev = _shapes("gdn_linear_decode_step_slots", q, k, v, log_decay)
    S = _slots(state_pool, slot_idx, reset, N, Hv, Dv, Dk, dev)
    _flag(error_flag, dev)

    def call(st):
        out = _output(o, "o", (N, Hv, Dv), dt, dev)
        _raise(lib.gdn_linear_decode_step_slots(_at(q), _at(k), _at(v), DTYPE[dt], _at(log_decay), scale,
                                                _at(state_pool), S, _at(slot_idx), _at(reset), N, Hqk, Hv,
                                                Dk, Dv, _at(out), _at(error_flag), st),
               "gdn_linear_decode_step_slots")
        return out

    return _run(dev, stream, call)

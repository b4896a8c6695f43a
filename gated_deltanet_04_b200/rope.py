"""Binding of the query/key norm with rotation (gdn_qk_norm_rope and its backward
pass, include/gdn.h): RMS norm of every (token, head) row, then the rotation of
its first dimensions by the token's positions.  Argument marshalling only."""
from __future__ import annotations

import ctypes

import torch

from . import DTYPE, library
from .linear import F32, I32, _at, _need, _output, _raise, _run, _scratch


def _rows(x, name, T, D, dtype, dev):
    """Checks x [T, H, D], dense within a token; (H, elements from token to token)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.device != dev or x.dtype != dtype:
        raise ValueError(f"{name} is {x.dtype} on {x.device}, expected {dtype} on {dev}")
    if x.dim() != 3 or x.shape[0] != T or x.shape[2] != D:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected ({T}, heads, {D})")
    H = x.shape[1]
    step, head, one = x.stride()
    if x.numel() and (one != 1 or (H > 1 and head != D)):
        raise ValueError(f"{name} must be contiguous within a token")
    return H, step if T > 1 else H * D


def _setup(name, xq, xk, positions, inv_freq, wq, wk, sections):
    dev, dt = xq.device, xq.dtype
    if dev.type != "cuda":
        raise ValueError(f"{name} runs on CUDA tensors only")
    if dt not in DTYPE:
        raise ValueError(f"unsupported io dtype {dt}")
    if xq.dim() != 3:
        raise ValueError(f"{name}: xq must have three dimensions")
    T, _, D = xq.shape
    Hq, sq = _rows(xq, "xq", T, D, dt, dev)
    Hk, sk = _rows(xk, "xk", T, D, dt, dev) if xk is not None else (0, 0)
    if wq is not None:
        _need(wq, "wq", (D,), F32, dev)
    if wk is not None:
        _need(wk, "wk", (D,), F32, dev)
    rot = axes = 0
    sec = None
    if (inv_freq is None) != (positions is None):
        raise ValueError("positions and inv_freq come together")
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0]
        _need(inv_freq, "inv_freq", (rot // 2,), F32, dev)
        axes = positions.shape[0] if positions.dim() == 2 else 1
        _need(positions, "positions", (axes, T) if positions.dim() == 2 else (T,), I32, dev)
        if sections is not None:
            if len(sections) != axes:
                raise ValueError(f"{len(sections)} sections for {axes} position axes")
            sec = (ctypes.c_int32 * axes)(*sections)
    return dev, dt, T, Hq, Hk, D, sq, sk, rot, axes, sec


def gdn_qk_norm_rope(xq, xk=None, positions=None, inv_freq=None, *, wq=None, wk=None, eps=1e-6,
                     sections=None, interleaved=False, q=None, k=None, stream=None):
    """RMS norm of every head row of xq [T,Hq,D] and xk [T,Hk,D] (or None), times
    wq, wk [D] fp32 (or None), then the rotation of the first 2 * len(inv_freq)
    dimensions: frequency i turns its pair by positions * inv_freq[i].  positions
    int32 [T], or [axes,T] with ``sections``, the frequencies of each axis in
    order; without them the norm alone.  xq and xk (bf16 or fp32) may be parts of
    one projection: dense within a token, any stride between tokens that is a
    multiple of 16 bytes.  ``interleaved``: pairs (2i, 2i+1) instead of
    (i, i + rot/2).  Returns (q, k), contiguous; k is None without xk."""
    lib = library()
    dev, dt, T, Hq, Hk, D, sq, sk, rot, axes, sec = _setup("gdn_qk_norm_rope", xq, xk, positions,
                                                           inv_freq, wq, wk, sections)

    def call(st):
        zq = _output(q, "q", (T, Hq, D), dt, dev)
        zk = None if xk is None else _output(k, "k", (T, Hk, D), dt, dev)
        _raise(lib.gdn_qk_norm_rope(_at(xq), _at(xk), DTYPE[dt], sq, sk, _at(wq), _at(wk), eps,
                                    _at(positions), axes, sec, _at(inv_freq), rot, int(interleaved), T, Hq,
                                    Hk, D, _at(zq), _at(zk), st), "gdn_qk_norm_rope")
        return zq, zk

    return _run(dev, stream, call)


def gdn_qk_norm_rope_backward(dq, dk, xq, xk=None, positions=None, inv_freq=None, *, wq=None, wk=None,
                              eps=1e-6, sections=None, interleaved=False, dxq=None, dxk=None,
                              output_dweights=True, workspace=None, stream=None):
    """Gradients of gdn_qk_norm_rope: dq [T,Hq,D], dk [T,Hk,D] (None without xk)
    are its outputs', the rest as in the forward call.  Returns (dxq, dxk, dwq,
    dwk); dxq and dxk may be given as parts of one gradient tensor; dwq, dwk
    [D] fp32 are the gradients of the weights (of ones where none were given),
    None with ``output_dweights=False``."""
    lib = library()
    dev, dt, T, Hq, Hk, D, sq, sk, rot, axes, sec = _setup("gdn_qk_norm_rope_backward", xq, xk,
                                                           positions, inv_freq, wq, wk, sections)
    _need(dq, "dq", (T, Hq, D), dt, dev)
    if xk is not None:
        _need(dk, "dk", (T, Hk, D), dt, dev)

    def call(st):
        gq = torch.empty((T, Hq, D), dtype=dt, device=dev) if dxq is None else dxq
        h, dsq = _rows(gq, "dxq", T, D, dt, dev)
        if h != Hq:
            raise ValueError(f"dxq has {h} heads, expected {Hq}")
        gk, dsk = None, 0
        if xk is not None:
            gk = torch.empty((T, Hk, D), dtype=dt, device=dev) if dxk is None else dxk
            h, dsk = _rows(gk, "dxk", T, D, dt, dev)
            if h != Hk:
                raise ValueError(f"dxk has {h} heads, expected {Hk}")
        dwq = dwk = None
        if output_dweights:
            dwq = torch.empty(D, dtype=F32, device=dev)
            dwk = None if xk is None else torch.empty(D, dtype=F32, device=dev)
        ws, n, _keep = _scratch(
            workspace, lib.gdn_qk_norm_rope_backward_workspace_bytes(D) if output_dweights else 0, dev)
        _raise(lib.gdn_qk_norm_rope_backward(
            _at(dq), None if xk is None else _at(dk), _at(xq), _at(xk), DTYPE[dt], sq, sk, _at(wq), _at(wk),
            eps, _at(positions), axes, sec, _at(inv_freq), rot, int(interleaved), T, Hq, Hk, D, _at(gq),
            _at(gk), dsq, dsk, _at(dwq), _at(dwk), ws, n, st), "gdn_qk_norm_rope_backward")
        return gq, gk, dwq, dwk

    return _run(dev, stream, call)

"""Operators around the gated delta rule, over the C ABI (include/gdn.h):

    y, final = causal_conv1d(x, weight, bias, activation, initial_state, output_final_state, cu_seqlens)
    y        = causal_conv1d_update(x, conv_state, weight, bias, activation)        # state in place
    y, final = chunk_selective_scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, ...)
    y, final = recurrent_selective_scan(x, dt, A, B, C, D, ..., initial_state, final_state)
    y        = layer_norm(x, weight, bias, gate, eps, center, gate_first)

each with its two stages (`_fwd`, `_bwd`) for custom training loops. The first and the last
are the steps in front of and behind a recurrence (q, k, v through the short convolution;
the output through the gated norm); the scan is the sibling recurrence with the same
[N, H, K, V] fp32 state and no delta correction.

Tensors are bf16 or fp32. The token inputs (x, B, C, dt, the convolution's x) may be slices
of a wider tensor: any token stride with the rest contiguous is passed on as it is; what
the library cannot address (a broken inner layout, a base or, for the scan, a token stride
off a 16-byte boundary) is copied first. This module only marshals arguments, as api.py.
"""
from __future__ import annotations

import ctypes
import torch
from torch.autograd.function import once_differentiable

from . import _binding as _b
from .api import _DTYPES, _ptr, _stream

_F32 = torch.float32


class _on:
    """Makes `dev` current for a launch (cheaply, where it already is)."""

    def __init__(self, dev):
        self.guard = None if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


def _check(dev, want):
    """Every tensor the library reads or writes: {name: (tensor or None, shape, dtype)}."""
    for name, (t, shape, dtype) in want.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _cuda(x, name="x"):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.device.type != "cuda":
        raise ValueError(f"inputs must be CUDA tensors (got {x.device}); the library has no CPU path")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    return x.device


def _dense(t):
    """Contiguous and 16-byte aligned (a copy where it is not)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _in_place(name, t):
    if not t.is_contiguous() or t.data_ptr() % 16:
        raise ValueError(f"{name} is written in place: it must be contiguous and 16-byte aligned")


def _tokens(t, width, step=1, align=16):
    """(tensor, token stride in elements) of a [B, T, ...] input whose tokens are `width`
    contiguous elements, a constant stride apart that is a multiple of `step`."""
    B, T = t.shape[0], t.shape[1]
    n, ok = 1, True
    for size, st in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
        ok &= size == 1 or st == n
        n *= size
    st = width if B * T <= 1 else t.stride(0) if T == 1 else t.stride(1)
    if T > 1 and B > 1:
        ok &= t.stride(0) == T * st
    if ok and st >= width and st % step == 0 and t.data_ptr() % align == 0:
        return t, st
    return (t.contiguous() if not t.is_contiguous() else t.clone()), width


def _packed(cu_seqlens, B, dev):
    """(device offsets or None, number of packed sequences, number of sequences)."""
    if cu_seqlens is None:
        return None, 0, B
    if cu_seqlens.dim() != 1 or cu_seqlens.dtype not in (torch.int32, torch.int64) or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D integer tensor of at least two offsets")
    if B != 1:
        raise ValueError("a packed batch (cu_seqlens) must have B == 1")
    cu = cu_seqlens.to(device=dev, dtype=torch.int32).contiguous()
    return cu, cu.numel() - 1, cu.numel() - 1


# ------------------------------------------------------------------ convolution
def _conv(x, weight, bias, activation, cu_seqlens):
    dev = _cuda(x)
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, C], got {tuple(x.shape)}")
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    B, T, C = x.shape
    if weight.dim() != 2 or not 2 <= weight.shape[1] <= 4:
        raise ValueError(f"weight must be [C, W] with W in 2..4, got {tuple(weight.shape)}")
    W = weight.shape[1]
    cu, ns, N = _packed(cu_seqlens, B, dev)
    _check(dev, {"weight": (weight, (C, W), x.dtype), "bias": (bias, (C,), x.dtype)})
    x, st = _tokens(x, C)
    P = _b.gdn_conv_problem(B, T, C, W, ns, None if cu is None else cu.data_ptr(), _DTYPES[x.dtype],
                            activation is not None, st)
    return dev, x, _dense(weight), _dense(bias), P, cu, (N, W - 1, C)


def causal_conv1d_fwd(x, weight, bias=None, activation=None, initial_state=None, output_final_state=True,
                      cu_seqlens=None):
    """Short causal depthwise convolution. x [B, T, C], weight [C, W] (W in 2..4), bias [C],
    states [N, W-1, C] (the inputs before the first and up to the last token, oldest first),
    all of one dtype; activation None or "silu". Returns (y, final_state or None)."""
    dev, x, weight, bias, P, cu, state = _conv(x, weight, bias, activation, cu_seqlens)
    _check(dev, {"initial_state": (initial_state, state, x.dtype)})
    initial_state = _dense(initial_state)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    fin = torch.empty(state, dtype=x.dtype, device=dev) if output_final_state else None
    with _on(dev):
        rc = _b.lib().gdn_conv_fwd(ctypes.byref(P), _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(y),
                                   _ptr(fin), _stream(dev))
    _b.check("gdn_conv_fwd", rc)
    return y, fin


def causal_conv1d_bwd(x, weight, bias, dy, dfinal=None, activation=None, initial_state=None, cu_seqlens=None):
    """Returns (dx, dweight, dbias or None, dinitial_state or None)."""
    dev, x, weight, bias, P, cu, state = _conv(x, weight, bias, activation, cu_seqlens)
    _check(dev, {"initial_state": (initial_state, state, x.dtype), "dy": (dy, x.shape, x.dtype),
                 "dfinal": (dfinal, state, x.dtype)})
    initial_state, dy, dfinal = _dense(initial_state), _dense(dy), _dense(dfinal)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw = torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    ds = torch.empty_like(initial_state) if initial_state is not None else None
    n = _b.lib().gdn_conv_bwd_workspace_size(ctypes.byref(P))
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    with _on(dev):
        rc = _b.lib().gdn_conv_bwd(ctypes.byref(P), _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(dy),
                                   _ptr(dfinal), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ds), _ptr(ws), n, _stream(dev))
    _b.check("gdn_conv_bwd", rc)
    return dx, dw, db, ds


def causal_conv1d_update(x, conv_state, weight, bias=None, activation=None):
    """The next few tokens of every sequence: x [B, T, C]; conv_state [B, W-1, C] is updated
    in place. Returns y [B, T, C]."""
    dev, x, weight, bias, P, _, state = _conv(x, weight, bias, activation, None)
    _check(dev, {"conv_state": (conv_state, state, x.dtype)})
    if conv_state is None:
        raise ValueError("conv_state is required")
    _in_place("conv_state", conv_state)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    with _on(dev):
        rc = _b.lib().gdn_conv_update(ctypes.byref(P), _ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(y),
                                      _stream(dev))
    _b.check("gdn_conv_update", rc)
    return y


class _Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, activation, output_final_state, cu):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, initial_state, cu)
        ctx.activation = activation
        return causal_conv1d_fwd(x, weight, bias, activation, initial_state, output_final_state, cu)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, weight, bias, h0, cu = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy
        dx, dw, db, ds = causal_conv1d_bwd(x, weight, bias, dy, dfinal, ctx.activation, h0, cu)
        return dx, dw, db, ds, None, None, None


def causal_conv1d(x, weight, bias=None, activation=None, initial_state=None, output_final_state=False,
                  cu_seqlens=None):
    """High-level call: (y, final_state or None), differentiable w.r.t. x, weight, bias and
    initial_state."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias, initial_state)):
        return _Conv.apply(x, weight, bias, initial_state, activation, output_final_state, cu_seqlens)
    return causal_conv1d_fwd(x, weight, bias, activation, initial_state, output_final_state, cu_seqlens)


# ------------------------------------------------------------------------- scan
class _Scan:
    """One scan call's checked inputs and its problem description."""

    def __init__(self, x, dt, A, B, C, D, dt_bias, dt_softplus, h0, cu_seqlens):
        dev = self.dev = _cuda(x)
        if x.dim() != 4 or B.dim() != 4:
            raise ValueError(f"x and B must be [B, T, H, D], got {tuple(x.shape)} and {tuple(B.shape)}")
        b, T, H, V = x.shape
        G, K = B.shape[2], B.shape[3]
        if dt.dtype not in (x.dtype, _F32):
            raise TypeError(f"dt has dtype {dt.dtype}, expected {x.dtype} or {_F32}")
        self.cu, ns, N = _packed(cu_seqlens, b, dev)
        self.state = (N, H, K, V)
        _check(dev, {"B": (B, (b, T, G, K), x.dtype), "C": (C, (b, T, G, K), x.dtype), "dt": (dt, (b, T, H), dt.dtype),
                     "A": (A, (H,), _F32), "D": (D, (H,), _F32), "dt_bias": (dt_bias, (H,), _F32),
                     "initial_state": (h0, self.state, _F32)})
        step = 16 // x.element_size()
        self.x, xs = _tokens(x, H * V, step)
        self.B, bs = _tokens(B, G * K, step)
        self.C, cs = _tokens(C, G * K, step)
        self.dt, ds = _tokens(dt, H, 1, dt.element_size())
        self.A, self.D, self.dt_bias, self.h0 = _dense(A), _dense(D), _dense(dt_bias), _dense(h0)
        self.P = _b.gdn_scan_problem(b, T, G, H, K, V, ns, None if self.cu is None else self.cu.data_ptr(),
                                     _DTYPES[x.dtype], _DTYPES[dt.dtype], bool(dt_softplus), xs, bs, cs, ds)

    def ref(self):
        return ctypes.byref(self.P)

    def inputs(self):
        return (_ptr(self.x), _ptr(self.dt), _ptr(self.A), _ptr(self.B), _ptr(self.C), _ptr(self.D), _ptr(self.dt_bias),
                _ptr(self.h0))

    def empty(self, like):
        return torch.empty(like.shape, dtype=like.dtype, device=self.dev)

    def bytes(self, n):
        return torch.empty(n, dtype=torch.uint8, device=self.dev)


def chunk_selective_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                             output_final_state=True, cu_seqlens=None, save_for_backward=False):
    """Selective state space scan over prompts. x [B, T, H, V], dt [B, T, H] (fp32 or x's
    dtype), A, D, dt_bias [H] fp32, B and C [B, T, G, K] (H a multiple of G), states
    [N, H, K, V] fp32. Returns (y, final_state or None, saved or None)."""
    s = _Scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens)
    L = _b.lib()
    y = s.empty(x)
    fin = torch.empty(s.state, dtype=_F32, device=s.dev) if output_final_state else None
    with _on(s.dev):
        saved = s.bytes(L.gdn_scan_saved_size(s.ref())) if save_for_backward else None
        n = L.gdn_scan_fwd_workspace_size(s.ref())
        ws = s.bytes(n) if n else None
        rc = L.gdn_scan_fwd(s.ref(), *s.inputs(), _ptr(y), _ptr(fin), _ptr(saved), _ptr(ws), n, _stream(s.dev))
    _b.check("gdn_scan_fwd", rc)
    return y, fin, saved


def chunk_selective_scan_bwd(x, dt, A, B, C, D, dt_bias, dt_softplus, saved, dy, dht=None, initial_state=None,
                             cu_seqlens=None):
    """Returns (dx, ddt, dA, dB, dC, dD, ddt_bias, dh0); dD, ddt_bias None where the input is.
    `saved` is what the forward kept, or None (recomputed)."""
    s = _Scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens)
    L = _b.lib()
    _check(s.dev, {"dy": (dy, x.shape, x.dtype), "dht": (dht, s.state, _F32)})
    dy, dht = _dense(dy), _dense(dht)
    dx, ddt, dB, dC, dA = s.empty(x), s.empty(dt), s.empty(B), s.empty(C), s.empty(A)
    dD = s.empty(D) if D is not None else None
    db = s.empty(dt_bias) if dt_bias is not None else None
    dh0 = torch.empty(s.state, dtype=_F32, device=s.dev)
    with _on(s.dev):
        if saved is not None:
            _check(s.dev, {"saved": (saved, saved.shape, torch.uint8)})
            need = L.gdn_scan_saved_size(s.ref())
            if saved.numel() < need:
                raise ValueError(f"saved holds {saved.numel()} bytes, the problem needs {need}")
        n = L.gdn_scan_bwd_workspace_size(s.ref())
        ws = s.bytes(n)
        rc = L.gdn_scan_bwd(s.ref(), *s.inputs(), _ptr(saved if saved is not None and saved.numel() else None), _ptr(dy),
                            _ptr(dht), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(db), _ptr(dh0),
                            _ptr(ws), n, _stream(s.dev))
    _b.check("gdn_scan_bwd", rc)
    return dx, ddt, dA, dB, dC, dD, db, dh0


def recurrent_selective_scan(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                             final_state=None, cu_seqlens=None):
    """Token by token, for a few tokens per sequence (decoding). Returns (y, final_state);
    `final_state` may be `initial_state` itself (updated in place)."""
    s = _Scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens)
    _check(s.dev, {"final_state": (final_state, s.state, _F32)})
    if final_state is None:
        final_state = torch.empty(s.state, dtype=_F32, device=s.dev)
    else:
        _in_place("final_state", final_state)
    y = s.empty(x)
    with _on(s.dev):
        rc = _b.lib().gdn_scan_step(s.ref(), *s.inputs(), _ptr(y), _ptr(final_state), _stream(s.dev))
    _b.check("gdn_scan_step", rc)
    return y, final_state


class _ChunkScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, dt_bias, dt_softplus, h0, output_final_state, cu):
        ctx.set_materialize_grads(False)
        y, fin, saved = chunk_selective_scan_fwd(x, dt, A, B, C, D, dt_bias, dt_softplus, h0, output_final_state, cu,
                                                 save_for_backward=True)
        ctx.save_for_backward(x, dt, A, B, C, D, dt_bias, h0, saved, cu)
        ctx.dt_softplus = dt_softplus
        return y, fin

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, dt, A, B, C, D, dt_bias, h0, saved, cu = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy
        dx, ddt, dA, dB, dC, dD, db, dh0 = chunk_selective_scan_bwd(x, dt, A, B, C, D, dt_bias, ctx.dt_softplus, saved, dy,
                                                                    dht, h0, cu)
        return dx, ddt, dA, dB, dC, dD, db, None, dh0 if h0 is not None else None, None, None


def chunk_selective_scan(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                         output_final_state=False, cu_seqlens=None):
    """High-level call: (y, final_state or None), differentiable w.r.t. every tensor but
    cu_seqlens."""
    if torch.is_grad_enabled() and any(
            t is not None and t.requires_grad for t in (x, dt, A, B, C, D, dt_bias, initial_state)):
        return _ChunkScan.apply(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, output_final_state, cu_seqlens)
    y, fin, _ = chunk_selective_scan_fwd(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, output_final_state,
                                         cu_seqlens)
    return y, fin


# ------------------------------------------------------------------- layer norm
def _norm(x, weight, bias, gate, eps, center, gate_first):
    dev = _cuda(x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have a last axis to normalise, got {tuple(x.shape)}")
    if weight.dtype not in (x.dtype, _F32):
        raise TypeError(f"weight has dtype {weight.dtype}, expected {x.dtype} or {_F32}")
    if gate_first and gate is None:
        raise ValueError("gate_first needs a gate")
    D = x.shape[-1]
    _check(dev, {"weight": (weight, (D,), weight.dtype), "bias": (bias, (D,), weight.dtype), "gate": (gate, x.shape, x.dtype)})
    P = _b.gdn_norm_problem(x.numel() // D, D, _DTYPES[x.dtype], _DTYPES[weight.dtype], bool(center), bool(gate_first),
                            float(eps))
    return dev, _dense(x), _dense(weight), _dense(bias), _dense(gate), P


def layer_norm_fwd(x, weight, bias=None, gate=None, eps=1e-5, center=True, gate_first=False):
    """Layer norm over the last axis (RMS norm without `center`), with an optional silu gate on
    its output, or on its input with `gate_first`. x, gate [..., D]; weight, bias [D] (fp32 or
    x's dtype). Returns (y, stats); stats [rows, 2] fp32 is the backward's."""
    dev, x, weight, bias, gate, P = _norm(x, weight, bias, gate, eps, center, gate_first)
    y = torch.empty_like(x)
    stats = torch.empty((P.rows, 2), dtype=_F32, device=dev)
    with _on(dev):
        rc = _b.lib().gdn_norm_fwd(ctypes.byref(P), _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(y), _ptr(stats),
                                   _stream(dev))
    _b.check("gdn_norm_fwd", rc)
    return y, stats


def layer_norm_bwd(x, weight, bias, gate, dy, stats, eps=1e-5, center=True, gate_first=False):
    """Returns (dx, dweight, dbias or None, dgate or None)."""
    dev, x, weight, bias, gate, P = _norm(x, weight, bias, gate, eps, center, gate_first)
    _check(dev, {"dy": (dy, x.shape, x.dtype), "stats": (stats, (P.rows, 2), _F32)})
    dy, stats = _dense(dy), _dense(stats)
    dx, dw = torch.empty_like(x), torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    dg = torch.empty_like(gate) if gate is not None else None
    with _on(dev):
        n = _b.lib().gdn_norm_bwd_workspace_size(ctypes.byref(P))
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        rc = _b.lib().gdn_norm_bwd(ctypes.byref(P), _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(dy), _ptr(stats),
                                   _ptr(dx), _ptr(dw), _ptr(db), _ptr(dg), _ptr(ws), n, _stream(dev))
    _b.check("gdn_norm_bwd", rc)
    return dx, dw, db, dg


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, eps, center, gate_first):
        y, stats = layer_norm_fwd(x, weight, bias, gate, eps, center, gate_first)
        ctx.save_for_backward(x, weight, bias, gate, stats)
        ctx.form = (eps, center, gate_first)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, gate, stats = ctx.saved_tensors
        return *layer_norm_bwd(x, weight, bias, gate, dy, stats, *ctx.form), None, None, None


def layer_norm(x, weight, bias=None, gate=None, eps=1e-5, center=True, gate_first=False):
    """High-level call: y, differentiable w.r.t. x, weight, bias and gate."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias, gate)):
        return _Norm.apply(x, weight, bias, gate, eps, center, gate_first)
    return layer_norm_fwd(x, weight, bias, gate, eps, center, gate_first)[0]

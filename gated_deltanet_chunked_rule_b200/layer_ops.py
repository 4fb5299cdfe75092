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

from ctypes import byref

import torch
from torch.autograd.function import once_differentiable

from . import _binding as _b
from .api import _DTYPES, _recorded, _written

_F32 = torch.float32
_Tensor = torch.Tensor
_empty_like = torch.empty_like


def _call(dev, name, *args):
    """Launches with `dev` current, on its current stream (the last argument)."""
    fn = getattr(_b.lib(), name)
    index = dev.index
    if index == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        _b.check(name, rc)


def _size(dev, name, P):
    """A size query with `dev` current."""
    fn = getattr(_b.lib(), name)
    if dev.index == torch.cuda.current_device():
        return fn(byref(P))
    with torch.cuda.device(dev):
        return fn(byref(P))


def _p(t):
    return None if t is None else t.data_ptr()


def _check(dev, *want):
    """Every tensor the library reads or writes: (name, tensor or None, shape, dtype)."""
    for name, t, shape, dtype in want:
        if t is None or (t.__class__ is _Tensor and t.dtype is dtype and t.device == dev and t.shape == shape):
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _empty(like):
    """Contiguous, of like's shape (empty_like keeps a slice's strides, and takes half as long)."""
    return _empty_like(like) if like.is_contiguous() else like.new_empty(like.shape)


def _cuda(x, name="x"):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
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
    if t.is_contiguous():
        return (t if t.data_ptr() % align == 0 else t.clone()), width
    shape, stride = t.shape, t.stride()
    B, T = shape[0], shape[1]
    n, ok = 1, True
    for i in range(len(shape) - 1, 1, -1):
        ok &= shape[i] == 1 or stride[i] == n
        n *= shape[i]
    st = width if B * T <= 1 else stride[0] if T == 1 else stride[1]
    if T > 1 and B > 1:
        ok &= stride[0] == T * st
    if ok and st >= width and st % step == 0 and t.data_ptr() % align == 0:
        return t, st
    return t.contiguous(), width


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
    _check(dev, ("weight", weight, (C, W), x.dtype), ("bias", bias, (C,), x.dtype))
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
    _check(dev, ("initial_state", initial_state, state, x.dtype))
    initial_state = _dense(initial_state)
    y = _empty(x)
    fin = x.new_empty(state) if output_final_state else None
    _call(dev, "gdn_conv_fwd", byref(P), x.data_ptr(), _p(weight), _p(bias), _p(initial_state), y.data_ptr(), _p(fin))
    return y, fin


def causal_conv1d_bwd(x, weight, bias, dy, dfinal=None, activation=None, initial_state=None, cu_seqlens=None):
    """Returns (dx, dweight, dbias or None, dinitial_state or None)."""
    dev, x, weight, bias, P, cu, state = _conv(x, weight, bias, activation, cu_seqlens)
    _check(dev, ("initial_state", initial_state, state, x.dtype), ("dy", dy, x.shape, x.dtype),
           ("dfinal", dfinal, state, x.dtype))
    initial_state, dy, dfinal = _dense(initial_state), _dense(dy), _dense(dfinal)
    dx = _empty(x)
    dw = torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    ds = torch.empty_like(initial_state) if initial_state is not None else None
    n = _size(dev, "gdn_conv_bwd_workspace_size", P)
    ws = x.new_empty(n, dtype=torch.uint8)
    _call(dev, "gdn_conv_bwd", byref(P), x.data_ptr(), _p(weight), _p(bias), _p(initial_state), _p(dy), _p(dfinal),
          dx.data_ptr(), dw.data_ptr(), _p(db), _p(ds), ws.data_ptr(), n)
    return dx, dw, db, ds


def causal_conv1d_update(x, conv_state, weight, bias=None, activation=None):
    """The next few tokens of every sequence: x [B, T, C]; conv_state [B, W-1, C] is updated
    in place. Returns y [B, T, C]. Not recorded by autograd."""
    dev, x, weight, bias, P, _, state = _conv(x, weight, bias, activation, None)
    _check(dev, ("conv_state", conv_state, state, x.dtype))
    if conv_state is None:
        raise ValueError("conv_state is required")
    _in_place("conv_state", conv_state)
    y = _empty(x)
    _call(dev, "gdn_conv_update", byref(P), x.data_ptr(), _p(weight), _p(bias), conv_state.data_ptr(), y.data_ptr())
    _written(conv_state)
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
    if _recorded(x, weight, bias, initial_state):
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
        _check(dev, ("B", B, (b, T, G, K), x.dtype), ("C", C, (b, T, G, K), x.dtype), ("dt", dt, (b, T, H), dt.dtype),
               ("A", A, (H,), _F32), ("D", D, (H,), _F32), ("dt_bias", dt_bias, (H,), _F32),
               ("initial_state", h0, self.state, _F32))
        step = 16 // x.element_size()
        self.x, xs = _tokens(x, H * V, step)
        self.B, bs = _tokens(B, G * K, step)
        self.C, cs = _tokens(C, G * K, step)
        self.dt, ds = _tokens(dt, H, 1, dt.element_size())
        self.A, self.D, self.dt_bias, self.h0 = _dense(A), _dense(D), _dense(dt_bias), _dense(h0)
        self.P = _b.gdn_scan_problem(b, T, G, H, K, V, ns, None if self.cu is None else self.cu.data_ptr(),
                                     _DTYPES[x.dtype], _DTYPES[dt.dtype], bool(dt_softplus), xs, bs, cs, ds)

    def inputs(self):
        return (byref(self.P), self.x.data_ptr(), self.dt.data_ptr(), self.A.data_ptr(), self.B.data_ptr(), self.C.data_ptr(),
                _p(self.D), _p(self.dt_bias), _p(self.h0))

    def bytes(self, n):
        return self.x.new_empty(n, dtype=torch.uint8)

    def states(self):
        return self.x.new_empty(self.state, dtype=_F32)


def chunk_selective_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                             output_final_state=True, cu_seqlens=None, save_for_backward=False):
    """Selective state space scan over prompts. x [B, T, H, V], dt [B, T, H] (fp32 or x's
    dtype), A, D, dt_bias [H] fp32, B and C [B, T, G, K] (H a multiple of G), states
    [N, H, K, V] fp32. Returns (y, final_state or None, saved or None)."""
    s = _Scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens)
    y = _empty(x)
    fin = s.states() if output_final_state else None
    saved = s.bytes(_size(s.dev, "gdn_scan_saved_size", s.P)) if save_for_backward else None
    n = _size(s.dev, "gdn_scan_fwd_workspace_size", s.P)
    ws = s.bytes(n) if n else None
    _call(s.dev, "gdn_scan_fwd", *s.inputs(), y.data_ptr(), _p(fin), _p(saved), _p(ws), n)
    return y, fin, saved


def chunk_selective_scan_bwd(x, dt, A, B, C, D, dt_bias, dt_softplus, saved, dy, dht=None, initial_state=None,
                             cu_seqlens=None):
    """Returns (dx, ddt, dA, dB, dC, dD, ddt_bias, dh0); dD, ddt_bias None where the input is.
    `saved` is what the forward kept, or None (recomputed)."""
    s = _Scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens)
    _check(s.dev, ("dy", dy, x.shape, x.dtype), ("dht", dht, s.state, _F32))
    dy, dht = _dense(dy), _dense(dht)
    dx, ddt, dB, dC, dA = _empty(x), _empty(dt), _empty(B), _empty(C), _empty(A)
    dD = _empty(D) if D is not None else None
    db = _empty(dt_bias) if dt_bias is not None else None
    dh0 = s.states()
    need = 0
    if saved is not None:
        _check(s.dev, ("saved", saved, saved.shape, torch.uint8))
        need = _size(s.dev, "gdn_scan_saved_size", s.P)
        if saved.numel() < need:
            raise ValueError(f"saved holds {saved.numel()} bytes, the problem needs {need}")
        if not need:
            saved = None
    n = _size(s.dev, "gdn_scan_bwd_workspace_size", s.P) - need  # no room to form again what is kept
    ws = s.bytes(n)
    _call(s.dev, "gdn_scan_bwd", *s.inputs(), _p(_dense(saved)), dy.data_ptr(), _p(dht), dx.data_ptr(), ddt.data_ptr(),
          dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _p(dD), _p(db), dh0.data_ptr(), ws.data_ptr(), n)
    return dx, ddt, dA, dB, dC, dD, db, dh0


def recurrent_selective_scan(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                             final_state=None, cu_seqlens=None):
    """Token by token, for a few tokens per sequence (decoding). Returns (y, final_state);
    `final_state` may be `initial_state` itself (updated in place). Not recorded by autograd."""
    s = _Scan(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens)
    _check(s.dev, ("final_state", final_state, s.state, _F32))
    given = final_state
    if final_state is None:
        final_state = s.states()
    else:
        _in_place("final_state", final_state)
    y = _empty(x)
    _call(s.dev, "gdn_scan_step", *s.inputs(), y.data_ptr(), final_state.data_ptr())
    _written(given)
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
    if _recorded(x, dt, A, B, C, D, dt_bias, initial_state):
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
    _check(dev, ("weight", weight, (D,), weight.dtype), ("bias", bias, (D,), weight.dtype), ("gate", gate, x.shape, x.dtype))
    P = _b.gdn_norm_problem(x.numel() // D, D, _DTYPES[x.dtype], _DTYPES[weight.dtype], bool(center), bool(gate_first),
                            float(eps))
    return dev, _dense(x), _dense(weight), _dense(bias), _dense(gate), P


def layer_norm_fwd(x, weight, bias=None, gate=None, eps=1e-5, center=True, gate_first=False):
    """Layer norm over the last axis (RMS norm without `center`), with an optional silu gate on
    its output, or on its input with `gate_first`. x, gate [..., D]; weight, bias [D] (fp32 or
    x's dtype). Returns (y, stats); stats [rows, 2] fp32 is the backward's."""
    dev, x, weight, bias, gate, P = _norm(x, weight, bias, gate, eps, center, gate_first)
    y = torch.empty_like(x)
    stats = x.new_empty((P.rows, 2), dtype=_F32)
    _call(dev, "gdn_norm_fwd", byref(P), x.data_ptr(), weight.data_ptr(), _p(bias), _p(gate), y.data_ptr(), stats.data_ptr())
    return y, stats


def layer_norm_bwd(x, weight, bias, gate, dy, stats, eps=1e-5, center=True, gate_first=False):
    """Returns (dx, dweight, dbias or None, dgate or None)."""
    dev, x, weight, bias, gate, P = _norm(x, weight, bias, gate, eps, center, gate_first)
    _check(dev, ("dy", dy, x.shape, x.dtype), ("stats", stats, (P.rows, 2), _F32))
    dy, stats = _dense(dy), _dense(stats)
    dx, dw = torch.empty_like(x), torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    dg = torch.empty_like(gate) if gate is not None else None
    n = _size(dev, "gdn_norm_bwd_workspace_size", P)
    ws = x.new_empty(n, dtype=torch.uint8)
    _call(dev, "gdn_norm_bwd", byref(P), x.data_ptr(), weight.data_ptr(), _p(bias), _p(gate), dy.data_ptr(), stats.data_ptr(),
          dx.data_ptr(), dw.data_ptr(), _p(db), _p(dg), ws.data_ptr(), n)
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
    if _recorded(x, weight, bias, gate):
        return _Norm.apply(x, weight, bias, gate, eps, center, gate_first)
    return layer_norm_fwd(x, weight, bias, gate, eps, center, gate_first)[0]

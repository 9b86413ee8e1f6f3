"""The operators around the scans: thin bindings of the stateless entry points of include/ttt.h.

:func:`qk_norm_rope` makes the queries and keys of the TTT-Linear family and of
:func:`gated_scan` from a projection's output; :func:`gated_scan` is the fast weight with a forget
gate (:func:`gated_scan_step` its one-token form); :func:`gated_ffn` makes the keys of the In-Place
scan. Each has its gradients in a call of its own (``*_backward``).

Tensors are checked before the call as in the rest of the package: element type, shape, the current
device, and strides (rows of the last dimension dense, so that views of a projection's output are
taken as they lie). A tensor that fails raises ValueError and nothing is launched; what the library
refuses raises TTTError. Outputs and workspaces that a call makes are allocated on the stream it
runs on. Every call can be captured into a CUDA graph.
"""

from __future__ import annotations

import contextlib
import ctypes
from functools import lru_cache

import torch

from . import abi
from .abi import check

__all__ = ["qk_norm_rope", "qk_norm_rope_backward", "rope_frequencies", "gated_scan", "gated_scan_backward",
           "gated_scan_step", "gated_ffn", "gated_ffn_backward"]

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_BF16, _F32, _F64, _I64, _I32 = torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32

NORMS = {"none": abi.TTT_NORM_NONE, None: abi.TTT_NORM_NONE, "rms": abi.TTT_NORM_RMS, "l2": abi.TTT_NORM_L2}
LAYOUTS = {"half": abi.TTT_ROPE_HALF, "interleaved": abi.TTT_ROPE_INTERLEAVED}
SCALINGS = {"none": abi.TTT_ROPE_SCALE_NONE, None: abi.TTT_ROPE_SCALE_NONE, "linear": abi.TTT_ROPE_SCALE_LINEAR,
            "ntk": abi.TTT_ROPE_SCALE_NTK, "yarn": abi.TTT_ROPE_SCALE_YARN}
ACTIVATIONS = {"silu": abi.TTT_ACT_SILU, "gelu": abi.TTT_ACT_GELU}


def _choice(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: expected one of {sorted(k for k in table if k)}, got {key!r}") from None


def _refuse(t, name, want, dev):
    got = f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}" if isinstance(t, torch.Tensor) else repr(t)
    raise ValueError(f"{name}: expected {want} on cuda:{dev}, got {got}")


def _rows(t, name, dtype, shape, dev, last=True):
    """Address of ``t`` once it has this type, shape and device, and (``last``) a dense last dimension."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or (last and t.stride(-1) != 1 and shape[-1] > 1)):
        _refuse(t, name, f"{tuple(shape)} {dtype}" + (" with a dense last dimension" if last else ""), dev)
    return t.data_ptr()


def _dense(t, name, dtype, shape, dev):
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, name, f"contiguous {tuple(shape)} {dtype}", dev)
    return t.data_ptr()


def _strides(shape, stride):
    """(batch, head, token) strides of a [batch, heads, tokens, ...] tensor; dimensions of one
    element are never stepped over, whatever stride they carry."""
    return tuple(s if n > 1 else 0 for n, s in zip(shape[:3], stride[:3]))


def _place(stream, dev):
    """The raw stream a call runs on, and a context in which torch allocates on that stream."""
    if stream is None:
        return (_raw(dev) if _raw is not None else torch.cuda.current_stream().cuda_stream) or None, None
    return stream.cuda_stream or None, torch.cuda.stream(stream)


_nothing = contextlib.nullcontext()


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---- queries and keys ---------------------------------------------------------------------


@lru_cache(maxsize=256)
def _qk_desc(io, batch, hq, hk, width, rot, norm, layout, eps, magnitude, tokens, position0, pos_stride, *strides):
    d = abi.ttt_qk_desc(io, batch, hq, hk, width, rot, norm, layout, eps, magnitude, tokens, position0, pos_stride,
                        *(abi.ttt_strides(*s) for s in strides))
    return d


_qk_workspaces = lru_cache(maxsize=256)(lambda dev, *key: abi.load().ttt_qk_norm_rope_workspace(ctypes.byref(_qk_desc(*key))))


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, trained=0.0, beta_fast=32.0, beta_slow=1.0):
    """ttt_rope_frequencies: (fp64 tensor [rot/2] of radians per position on the current device,
    magnitude), for contexts ``factor`` times the ``trained`` length with ``scaling`` "none",
    "linear", "ntk" or "yarn"."""
    out = (ctypes.c_double * max(1, int(rot) // 2))()
    magnitude = ctypes.c_float()
    check(abi.load().ttt_rope_frequencies(int(rot), float(base), _choice(SCALINGS, scaling, "scaling"), float(factor),
                                          float(trained), float(beta_fast), float(beta_slow),
                                          ctypes.addressof(out), ctypes.addressof(magnitude)))
    return torch.tensor(list(out), dtype=_F64, device=torch.device("cuda", _current_device())), magnitude.value


def _qk_args(q, k, positions, freqs, q_weight, k_weight, dev):
    x = q if q is not None else k
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.dtype not in (_BF16, _F32):
        _refuse(x, "q" if q is not None else "k", "[batch, heads, tokens, width] torch.bfloat16 or torch.float32", dev)
    batch, _, tokens, width = x.shape
    hq, hk = 0 if q is None else q.shape[1], 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            _refuse(k, "k", "[batch, heads, tokens, width]", dev)
        hk = k.shape[1]
    rot = 0
    if freqs is not None:
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            _refuse(freqs, "freqs", "[rot/2] torch.float64", dev)
        rot = 2 * freqs.shape[0]
    pos_stride = 0
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.shape not in ((tokens,), (batch, tokens)):
            _refuse(positions, "positions", f"[{tokens}] or [{batch}, {tokens}] torch.int64", dev)
        if positions.dim() == 2:
            pos_stride = tokens
    ptrs = (_dense(q_weight, "q_weight", _F32, (width,), dev), _dense(k_weight, "k_weight", _F32, (width,), dev),
            None if positions is None else _dense(positions, "positions", _I64, positions.shape, dev),
            None if rot == 0 else _dense(freqs, "freqs", _F64, (rot // 2,), dev))
    return x.dtype, batch, hq, hk, tokens, width, rot, pos_stride, ptrs


def qk_norm_rope(q, k, *, positions=None, freqs=None, magnitude=1.0, norm="rms", eps=1e-6, layout="half",
                 q_weight=None, k_weight=None, position0=0, out=None, stream=None):
    """ttt_qk_norm_rope: the norm ("rms", "l2" or "none") of each query and key head and its rotary
    position in one pass. ``q`` [batch, q_heads, tokens, width] and ``k`` [batch, k_heads, tokens,
    width], bf16 or fp32, any strides with a dense last dimension (a transposed view of a
    token-major projection, say); one of them may be None. ``positions`` int64 [tokens] or [batch,
    tokens] (default: ``position0`` + t); ``freqs`` and ``magnitude`` from :func:`rope_frequencies`
    (None: no rotation); the first 2·len(freqs) values of each row are rotated, in pairs by
    ``layout`` "half" or "interleaved". ``q_weight``, ``k_weight`` fp32 [width] (RMS). Returns (q, k),
    dense [batch, heads, tokens, width] or the pair ``out`` (which may be the inputs)."""
    dev = _current_device()
    dtype, batch, hq, hk, tokens, width, rot, pos_stride, ptrs = _qk_args(q, k, positions, freqs, q_weight, k_weight, dev)
    raw, ctx = _place(stream, dev)
    qs, ks = (batch, hq, tokens, width), (batch, hk, tokens, width)
    pq = None if q is None else _rows(q, "q", dtype, qs, dev)
    pk = None if k is None else _rows(k, "k", dtype, ks, dev)
    if out is None:
        with ctx or _nothing:
            qo = None if q is None else torch.empty(qs, dtype=dtype, device=q.device)
            ko = None if k is None else torch.empty(ks, dtype=dtype, device=k.device)
    else:
        qo, ko = out
        if (qo is None) != (q is None) or (ko is None) != (k is None):
            raise ValueError("out: expected a tensor for each of q and k that is given")
    pqo = None if qo is None else _rows(qo, "out[0]", dtype, qs, dev)
    pko = None if ko is None else _rows(ko, "out[1]", dtype, ks, dev)
    sq = (0, 0, 0) if q is None else _strides(qs, q.stride())
    sk = (0, 0, 0) if k is None else _strides(ks, k.stride())
    so = (0, 0, 0) if qo is None else _strides(qs, qo.stride())
    sp = (0, 0, 0) if ko is None else _strides(ks, ko.stride())
    d = _qk_desc(1 if dtype is _BF16 else 0, batch, hq, hk, width, rot, _choice(NORMS, norm, "norm"),
                 _choice(LAYOUTS, layout, "layout"), float(eps), float(magnitude), tokens, int(position0),
                 pos_stride, sq, sk, so, sp, (0, 0, 0), (0, 0, 0))
    check(abi.load().ttt_qk_norm_rope(ctypes.byref(d), pq, pk, *ptrs, pqo, pko, raw))
    return qo, ko


def qk_norm_rope_backward(dq_out, dk_out, q, k, *, positions=None, freqs=None, magnitude=1.0, norm="rms", eps=1e-6,
                          layout="half", q_weight=None, k_weight=None, position0=0, stream=None):
    """ttt_qk_norm_rope_backward: (dq, dk, dq_weight, dk_weight) from the gradients of the outputs and
    the inputs of :func:`qk_norm_rope`; dq and dk are dense, the weights' gradients fp32 [width]
    (None for a weight that is None). With norm "none" ``q`` and ``k`` are not read."""
    dev = _current_device()
    dtype, batch, hq, hk, tokens, width, rot, pos_stride, ptrs = _qk_args(
        dq_out, dk_out, positions, freqs, q_weight, k_weight, dev)
    raw, ctx = _place(stream, dev)
    qs, ks = (batch, hq, tokens, width), (batch, hk, tokens, width)
    kind = _choice(NORMS, norm, "norm")
    none = (0, 0, 0)
    grads, outs, xs, places = [], [], [], []
    with ctx or _nothing:
        for g, x, shape, name in ((dq_out, q, qs, "q"), (dk_out, k, ks, "k")):
            if g is None:
                if x is not None:
                    raise ValueError(f"{name}: given without the gradient of its output")
                grads.append(None), outs.append(None), xs.append(None), places.append((none, none, none))
                continue
            grads.append(_rows(g, f"d{name}_out", dtype, shape, dev))
            read = kind != abi.TTT_NORM_NONE
            xs.append(_rows(x, name, dtype, shape, dev) if read else None)
            y = torch.empty(shape, dtype=dtype, device=g.device)
            outs.append(y)
            places.append((_strides(shape, x.stride()) if read else none, _strides(shape, g.stride()),
                           _strides(shape, y.stride())))
        dqw = None if q_weight is None else torch.empty(width, dtype=_F32, device=q_weight.device)
        dkw = None if k_weight is None else torch.empty(width, dtype=_F32, device=k_weight.device)
        key = (1 if dtype is _BF16 else 0, batch, hq, hk, width, rot, kind, _choice(LAYOUTS, layout, "layout"), float(eps),
               float(magnitude), tokens, int(position0), pos_stride, places[0][0], places[1][0], places[0][1],
               places[1][1], places[0][2], places[1][2])
        d = _qk_desc(*key)
        nbytes = _qk_workspaces(dev, *key) if dqw is not None or dkw is not None else 0
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_qk_norm_rope_backward(ctypes.byref(d), *grads, *xs, *ptrs, _ptr(outs[0]), _ptr(outs[1]), _ptr(dqw), _ptr(dkw),
                                               _ptr(ws), nbytes, raw))
    return outs[0], outs[1], dqw, dkw


# ---- the gated scan -------------------------------------------------------------------------


@lru_cache(maxsize=256)
def _scan_desc(batch, heads, tokens, scale, *strides):
    return abi.ttt_gated_scan_desc(batch, heads, tokens, scale, *(abi.ttt_strides(*s) for s in strides))


_scan_workspaces = lru_cache(maxsize=256)(lambda dev, *key: abi.load().ttt_gated_scan_workspace(ctypes.byref(_scan_desc(*key))))
_scan_back_workspaces = lru_cache(maxsize=256)(
    lambda dev, *key: abi.load().ttt_gated_scan_backward_workspace(ctypes.byref(_scan_desc(*key))))


def _scan_shape(q, dims, dev):
    if not isinstance(q, torch.Tensor) or q.dim() != dims or q.shape[-1] != 64:
        _refuse(q, "q", "[batch, heads, tokens, 64] torch.bfloat16" if dims == 4 else "[batch, heads, 64] torch.bfloat16",
                dev)
    return q.shape


def gated_scan(q, k, v, g, *, scale=1.0, initial=None, out=None, final=None, stream=None):
    """ttt_gated_scan: S_t = e^{g_t}·S_{t-1} + k_tᵀ·v_t, o_t = scale·q_t·S_t per (sequence, head). ``q``,
    ``k``, ``v`` bf16 [batch, heads, tokens, 64] (any strides, dense rows), ``g`` fp32 [batch, heads,
    tokens] (any strides; natural logarithms, -inf forgets everything before its token). Returns
    (o, state): o in ``out`` or a new dense tensor; the state after the last token, fp32 [batch,
    heads, 64, 64], in ``final`` (which may be ``initial``) or a new tensor."""
    dev = _current_device()
    shape = _scan_shape(q, 4, dev)
    batch, heads, tokens, _ = shape
    st = (batch, heads, 64, 64)
    raw, ctx = _place(stream, dev)
    pq, pk, pv = (_rows(t, n, _BF16, shape, dev) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    pg = _rows(g, "g", _F32, shape[:3], dev, last=False)
    pi = _dense(initial, "initial", _F32, st, dev)
    with ctx or _nothing:
        if out is None:
            out = torch.empty(shape, dtype=_BF16, device=q.device)
        if final is None:
            final = torch.empty(st, dtype=_F32, device=q.device)
        key = (batch, heads, tokens, float(scale), _strides(shape, q.stride()), _strides(shape, k.stride()),
               _strides(shape, v.stride()), _strides(shape, out.stride()), _strides(shape, g.stride()))
        nbytes = _scan_workspaces(dev, *key)
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_gated_scan(ctypes.byref(_scan_desc(*key)), pq, pk, pv, pg, pi, _rows(out, "out", _BF16, shape, dev),
                                    _dense(final, "final", _F32, st, dev), _ptr(ws), nbytes, raw))
    return out, final


def gated_scan_backward(do, q, k, v, g, *, scale=1.0, initial=None, dfinal=None, stream=None):
    """ttt_gated_scan_backward: (dq, dk, dv, dg, dinitial) from the gradient ``do`` of the outputs and
    ``dfinal`` of the final state (None: zero). All are dense; dinitial is None where ``initial``
    is."""
    dev = _current_device()
    shape = _scan_shape(q, 4, dev)
    batch, heads, tokens, _ = shape
    st = (batch, heads, 64, 64)
    raw, ctx = _place(stream, dev)
    pd, pq, pk, pv = (_rows(t, n, _BF16, shape, dev) for t, n in ((do, "do"), (q, "q"), (k, "k"), (v, "v")))
    pg = _rows(g, "g", _F32, shape[:3], dev, last=False)
    pi, pf = _dense(initial, "initial", _F32, st, dev), _dense(dfinal, "dfinal", _F32, st, dev)
    key = (batch, heads, tokens, float(scale), _strides(shape, q.stride()), _strides(shape, k.stride()),
           _strides(shape, v.stride()), _strides(shape, do.stride()), _strides(shape, g.stride()))
    with ctx or _nothing:
        dq, dk, dv = (torch.empty(shape, dtype=_BF16, device=q.device) for _ in range(3))
        dg = torch.empty(shape[:3], dtype=_F32, device=q.device)
        di = None if initial is None else torch.empty(st, dtype=_F32, device=q.device)
        nbytes = _scan_back_workspaces(dev, *key)
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_gated_scan_backward(ctypes.byref(_scan_desc(*key)), pd, pq, pk, pv, pg, pi, pf, dq.data_ptr(), dk.data_ptr(),
                                             dv.data_ptr(), dg.data_ptr(), _ptr(di), _ptr(ws), nbytes, raw))
    return dq, dk, dv, dg, di


def gated_scan_step(state, q, k, v, g, *, scale=1.0, out=None, stream=None):
    """ttt_gated_scan_step: one token of every sequence. ``state`` fp32 [batch, heads, 64, 64] is updated
    in place; ``q``, ``k``, ``v`` bf16 [batch, heads, 64], ``g`` fp32 [batch, heads] (any strides, dense
    rows). Returns o, bf16 [batch, heads, 64]."""
    dev = _current_device()
    shape = _scan_shape(q, 3, dev)
    batch, heads, _ = shape
    raw, ctx = _place(stream, dev)
    pq, pk, pv = (_rows(t, n, _BF16, shape, dev) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    pg = _rows(g, "g", _F32, shape[:2], dev, last=False)
    if state is None:
        _refuse(state, "state", f"contiguous {(batch, heads, 64, 64)} {_F32}", dev)
    ps = _dense(state, "state", _F32, (batch, heads, 64, 64), dev)
    if out is None:
        with ctx or _nothing:
            out = torch.empty(shape, dtype=_BF16, device=q.device)
    two = lambda t: (t.stride(0) if batch > 1 else 0, t.stride(1) if heads > 1 else 0, 0)  # noqa: E731
    d = _scan_desc(batch, heads, 1, float(scale), two(q), two(k), two(v), two(out), two(g))
    check(abi.load().ttt_gated_scan_step(ctypes.byref(d), pq, pk, pv, pg, ps, _rows(out, "out", _BF16, shape, dev), raw))
    return out


# ---- the gated feed-forward block -------------------------------------------------------------


def _ffn_shape(x, w_gate, dev):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _refuse(x, "x", "[tokens, d] torch.bfloat16", dev)
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        _refuse(w_gate, "w_gate", "[f, d] torch.bfloat16", dev)
    return x.shape[0], x.shape[1], w_gate.shape[0]


def gated_ffn(x, w_gate, w_up, *, activation="silu", save=False, out=None, status=None, stream=None):
    """ttt_gated_ffn: z = act(x·w_gateᵀ) ⊙ (x·w_upᵀ), the In-Place scan's keys. ``x`` bf16 [tokens, d],
    ``w_gate`` and ``w_up`` bf16 [f, d], contiguous; ``activation`` "silu" or "gelu". Returns z [tokens,
    f], or with ``save`` (z, gate, up) with the pre-activations that :func:`gated_ffn_backward` takes.
    ``status`` (int32 device tensor of one element, optional) is set to 0, or to TTT_ERR_TIMEOUT if
    a bounded device-side wait ran out."""
    dev = _current_device()
    T, d, f = _ffn_shape(x, w_gate, dev)
    raw, ctx = _place(stream, dev)
    px, pg, pu = (_dense(x, "x", _BF16, (T, d), dev), _dense(w_gate, "w_gate", _BF16, (f, d), dev),
                  _dense(w_up, "w_up", _BF16, (f, d), dev))
    act = _choice(ACTIVATIONS, activation, "activation")
    gate = up = None
    with ctx or _nothing:
        if out is None:
            out = torch.empty((T, f), dtype=_BF16, device=x.device)
        if save:
            gate, up = torch.empty_like(out), torch.empty_like(out)
    check(abi.load().ttt_gated_ffn(px, pg, pu, T, d, f, act, _dense(out, "out", _BF16, (T, f), dev), _ptr(gate), _ptr(up),
                                   _dense(status, "status", _I32, (1,), dev), raw))
    return (out, gate, up) if save else out


_ffn_workspaces = lru_cache(maxsize=256)(lambda dev, *key: abi.load().ttt_gated_ffn_backward_workspace(*key))


def gated_ffn_backward(dz, x, w_gate, w_up, gate, up, *, activation="silu", need_dx=True, need_dw=True, status=None,
                       stream=None):
    """ttt_gated_ffn_backward: (dx, dw_gate, dw_up) from the gradient ``dz`` of z and the kept
    pre-activations ``gate`` and ``up``, all bf16 and contiguous; ``need_dx`` or ``need_dw`` false
    leaves those out (None)."""
    dev = _current_device()
    T, d, f = _ffn_shape(x, w_gate, dev)
    raw, ctx = _place(stream, dev)
    act = _choice(ACTIVATIONS, activation, "activation")
    pz, pga, pup = (_dense(t, n, _BF16, (T, f), dev) for t, n in ((dz, "dz"), (gate, "gate"), (up, "up")))
    px, pg, pu = (_dense(x, "x", _BF16, (T, d), dev), _dense(w_gate, "w_gate", _BF16, (f, d), dev),
                  _dense(w_up, "w_up", _BF16, (f, d), dev))
    with ctx or _nothing:
        dx = torch.empty((T, d), dtype=_BF16, device=x.device) if need_dx else None
        dwg, dwu = (torch.empty((f, d), dtype=_BF16, device=x.device) if need_dw else None for _ in range(2))
        nbytes = _ffn_workspaces(dev, T, d, f)
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_gated_ffn_backward(pz, px, pg, pu, pga, pup, T, d, f, act, _ptr(dx), _ptr(dwg), _ptr(dwu), _ptr(ws),
                                            nbytes, _dense(status, "status", _I32, (1,), dev), raw))
    return dx, dwg, dwu

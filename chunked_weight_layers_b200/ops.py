"""The operators around the scans: thin bindings of the stateless entry points of include/ttt.h.

:func:`qk_norm_rope` makes the queries and keys of the TTT-Linear family and of
:func:`gated_scan` from a projection's output; :func:`gated_scan` is the fast weight with a forget
gate (:func:`gated_scan_step` its one-token form); :func:`gated_ffn` makes the keys of the In-Place
scan. Each has its gradients in a call of its own (``*_backward``).

Tensors are checked before the call as in the rest of the package: element type, shape, the current
device, and strides. Rows of the last dimension are dense and start on 16-byte boundaries; the other
dimensions may lie in any order, so that views of a projection's output are taken as they are. An input
may repeat rows along a dimension (stride 0, as expand() makes), an output may not; tokens of a gated
scan have rows of their own. A tensor that fails raises ValueError and nothing is launched; what the
library refuses (alignment, strides, sizes out of its range) raises TTTError. Outputs and workspaces
that a call makes are allocated on the stream it runs on. Every call can be captured into a CUDA graph.
A call whose bounded device-side waits ran out leaves its outputs incomplete: it says so in ``status``
where that is given, and otherwise through :func:`poll_operators`.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import abi
from .abi import check

__all__ = ["qk_norm_rope", "qk_norm_rope_backward", "rope_frequencies", "gated_scan", "gated_scan_backward",
           "gated_scan_step", "gated_ffn", "gated_ffn_backward", "poll_operators"]

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
    """Checks that ``t`` has this type, shape and device, and (``last``) a dense last dimension."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or (last and t.stride(-1) != 1 and shape[-1] > 1)):
        _refuse(t, name, f"{tuple(shape)} {dtype}" + (" with a dense last dimension" if last else ""), dev)


def _dense(t, name, dtype, shape, dev):
    """Checks that ``t`` is a contiguous tensor of this type, shape and device."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, name, f"contiguous {tuple(shape)} {dtype}", dev)


def _dense_or_none(t, *how):
    if t is not None:
        _dense(t, *how)


def _strides(shape, stride):
    """(batch, head, token) strides of a [batch, heads, tokens, ...] tensor; dimensions of one
    element are never stepped over, whatever stride they carry."""
    return tuple(s if n > 1 else 0 for n, s in zip(shape[:3], stride[:3]))


# Checking every tensor of a call and filling its descriptor costs more host time than a small
# call's kernel takes. What both depend on is the tensors' metadata (shape, strides, type, device) and
# the options alone, so a call whose metadata has been checked before takes the descriptor and
# workspace size made then; addresses are read, and their alignment checked, at every call.


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


class _Plans(dict):
    """Checked calls by their metadata; emptied when it has grown past ``most``."""

    most = 1024

    def find(self, key):
        try:
            return self.get(key)
        except TypeError:  # an option that cannot be hashed: the checks will name it
            return None

    def keep(self, key, plan):
        if len(self) >= self.most:
            self.clear()
        self[key] = plan
        return plan


def _place(stream, dev):
    """The raw stream a call runs on, and a context in which torch allocates on that stream."""
    if stream is None:
        return (_raw(dev) if _raw is not None else torch.cuda.current_stream().cuda_stream) or None, _nothing
    return stream.cuda_stream or None, torch.cuda.stream(stream)


_nothing = contextlib.nullcontext()


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev)) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    """A new dense tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def poll_operators():
    """ttt_operators_poll: synchronises the device and raises TTTError if a bounded wait ran out, since the
    last poll, in a call on it that was given no ``status``."""
    check(abi.load().ttt_operators_poll())


# ---- queries and keys ---------------------------------------------------------------------


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


_qk_plans, _qk_back_plans = _Plans(), _Plans()


def _qk_call(q, k, positions, freqs, q_weight, k_weight, norm, layout, eps, magnitude, position0, dev):
    """Checks what the two calls share and returns (descriptor without strides, dtype, q's shape, k's shape);
    ``q`` and ``k`` stand for the tensors that give the shapes."""
    x, name = (q, "q") if q is not None else (k, "k")
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.dtype not in (_BF16, _F32):
        _refuse(x, name, "[batch, heads, tokens, width] torch.bfloat16 or torch.float32", dev)
    batch, _, tokens, width = x.shape
    hq, hk = 0 if q is None else q.shape[1], 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            _refuse(k, "k", "[batch, heads, tokens, width]", dev)
        hk = k.shape[1]
    rot, pos_stride = 0, 0
    if freqs is not None:
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            _refuse(freqs, "freqs", "[rot/2] torch.float64", dev)
        rot = 2 * freqs.shape[0]
        _dense(freqs, "freqs", _F64, freqs.shape, dev)
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.shape not in ((tokens,), (batch, tokens)):
            _refuse(positions, "positions", f"[{tokens}] or [{batch}, {tokens}] torch.int64", dev)
        _dense(positions, "positions", _I64, positions.shape, dev)
        if positions.dim() == 2:
            pos_stride = tokens
    _dense_or_none(q_weight, "q_weight", _F32, (width,), dev)
    _dense_or_none(k_weight, "k_weight", _F32, (width,), dev)
    d = abi.ttt_qk_desc(1 if x.dtype is _BF16 else 0, batch, hq, hk, width, rot, _choice(NORMS, norm, "norm"),
                        _choice(LAYOUTS, layout, "layout"), eps, magnitude, tokens, position0, pos_stride)
    return d, x.dtype, (batch, hq, tokens, width), (batch, hk, tokens, width)


def _set(d, field, shape, t):
    if t is not None:
        setattr(d, field, abi.ttt_strides(*_strides(shape, t.stride())))


def _freqs_ptr(freqs):
    return freqs.data_ptr() if freqs is not None and freqs.numel() else None


def qk_norm_rope(q, k, *, positions=None, freqs=None, magnitude=1.0, norm="rms", eps=1e-6, layout="half",
                 q_weight=None, k_weight=None, position0=0, out=None, stream=None):
    """ttt_qk_norm_rope: the norm ("rms", "l2" or "none") of each query and key head and its rotary
    position in one pass. ``q`` [batch, q_heads, tokens, width] and ``k`` [batch, k_heads, tokens,
    width], bf16 or fp32, rows as the module says (a transposed view of a token-major projection, say); one of
    them may be None, and an empty batch or no tokens is a no-op. ``positions`` int64 [tokens] or [batch,
    tokens] (default: ``position0`` + t); ``freqs`` and ``magnitude`` from :func:`rope_frequencies`
    (None: no rotation); the first 2·len(freqs) values of each row are rotated, in pairs by
    ``layout`` "half" or "interleaved". ``q_weight``, ``k_weight`` fp32 [width] (RMS). Returns (q, k),
    dense [batch, heads, tokens, width] or the pair ``out`` (which may be the inputs)."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    eps, magnitude, position0 = float(eps), float(magnitude), int(position0)
    try:
        key = (dev, _meta(q), _meta(k), _meta(positions), _meta(freqs), _meta(q_weight), _meta(k_weight), norm, layout, eps,
               magnitude, position0, None if out is None else (_meta(out[0]), _meta(out[1])))
    except (AttributeError, TypeError, IndexError):  # something that is no tensor: the checks will name it
        key = None
    d = _qk_plans.find(key) if key is not None else None
    if d is None:
        d, dtype, qs, ks = _qk_call(q, k, positions, freqs, q_weight, k_weight, norm, layout, eps, magnitude, position0, dev)
        qo, ko = out if out is not None else (q, k)
        if (qo is None) != (q is None) or (ko is None) != (k is None):
            raise ValueError("out: expected a tensor for each of q and k that is given")
        for x, y, shape, n, i in ((q, qo, qs, "q", 0), (k, ko, ks, "k", 1)):
            if x is not None:
                _rows(x, n, dtype, shape, dev)
                _rows(y, f"out[{i}]", dtype, shape, dev)
                _set(d, n, shape, x)
                _set(d, n + "_out", shape, y if out is not None else torch.empty(shape, device="meta"))
        if key is not None:
            _qk_plans.keep(key, d)
    if out is None:
        with ctx:
            out = (None if q is None else _like(q), None if k is None else _like(k))
    qo, ko = out
    check(abi.load().ttt_qk_norm_rope(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
                                      _freqs_ptr(freqs), _ptr(qo), _ptr(ko), raw))
    return qo, ko


def qk_norm_rope_backward(dq_out, dk_out, q, k, *, positions=None, freqs=None, magnitude=1.0, norm="rms", eps=1e-6,
                          layout="half", q_weight=None, k_weight=None, position0=0, stream=None):
    """ttt_qk_norm_rope_backward: (dq, dk, dq_weight, dk_weight) from the gradients of the outputs and
    the inputs of :func:`qk_norm_rope`; dq and dk are dense, the weights' gradients fp32 [width]
    (None for a weight that is None). With norm "none" ``q`` and ``k`` are not read."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    eps, magnitude, position0 = float(eps), float(magnitude), int(position0)
    try:
        key = (dev, _meta(dq_out), _meta(dk_out), _meta(q), _meta(k), _meta(positions), _meta(freqs), _meta(q_weight),
               _meta(k_weight), norm, layout, eps, magnitude, position0)
    except AttributeError:
        key = None
    plan = _qk_back_plans.find(key) if key is not None else None
    if plan is None:
        d, dtype, qs, ks = _qk_call(dq_out, dk_out, positions, freqs, q_weight, k_weight, norm, layout, eps, magnitude,
                                    position0, dev)
        read = d.norm != abi.TTT_NORM_NONE
        for g, x, shape, n in ((dq_out, q, qs, "q"), (dk_out, k, ks, "k")):
            if g is None:
                if x is not None:
                    raise ValueError(f"{n}: given without the gradient of its output")
                continue
            _rows(g, f"d{n}_out", dtype, shape, dev)
            _set(d, n + "_out", shape, g)
            _set(d, n + "_grad", shape, torch.empty(shape, device="meta"))
            if read:
                _rows(x, n, dtype, shape, dev)
                _set(d, n, shape, x)
        gains = q_weight is not None or k_weight is not None
        plan = d, read, abi.load().ttt_qk_norm_rope_workspace(ctypes.byref(d)) if gains else 0
        if key is not None:
            _qk_back_plans.keep(key, plan)
    d, read, nbytes = plan
    with ctx:
        dq = None if dq_out is None else _like(dq_out)
        dk = None if dk_out is None else _like(dk_out)
        dqw = None if q_weight is None else _like(q_weight)
        dkw = None if k_weight is None else _like(k_weight)
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_qk_norm_rope_backward(
        ctypes.byref(d), _ptr(dq_out), _ptr(dk_out), _ptr(q) if read else None, _ptr(k) if read else None, _ptr(q_weight),
        _ptr(k_weight), _ptr(positions), _freqs_ptr(freqs), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(ws), nbytes, raw))
    return dq, dk, dqw, dkw


# ---- the gated scan -------------------------------------------------------------------------


_scan_plans, _scan_back_plans, _step_plans = _Plans(), _Plans(), _Plans()


def _scan_shape(q, dims, dev):
    if not isinstance(q, torch.Tensor) or q.dim() != dims or q.shape[-1] != 64:
        _refuse(q, "q", "[batch, heads, tokens, 64] torch.bfloat16" if dims == 4 else "[batch, heads, 64] torch.bfloat16",
                dev)
    return q.shape


def _scan_desc(shape, scale, q, k, v, o, g):
    """The descriptor of a call; ``o`` may be None (a dense tensor)."""
    o = torch.empty(shape, device="meta") if o is None else o
    if len(shape) == 3:  # one token
        two = lambda t: (*_strides(shape[:2], t.stride()[:2]), 0)  # noqa: E731
        return abi.ttt_gated_scan_desc(shape[0], shape[1], 1, scale, *(abi.ttt_strides(*two(t)) for t in (q, k, v, o, g)))
    return abi.ttt_gated_scan_desc(shape[0], shape[1], shape[2], scale,
                                   *(abi.ttt_strides(*_strides(shape, t.stride())) for t in (q, k, v, o, g)))


def gated_scan(q, k, v, g, *, scale=1.0, initial=None, out=None, final=None, status=None, stream=None):
    """ttt_gated_scan: S_t = e^{g_t}·S_{t-1} + k_tᵀ·v_t, o_t = scale·q_t·S_t per (sequence, head). ``q``,
    ``k``, ``v`` bf16 [batch, heads, tokens, 64] (rows as the module says; at least one sequence and head, tokens
    may be 0), ``g`` fp32 [batch, heads, tokens] (any strides; natural logarithms, -inf forgets everything
    before its token). All tokens must hold finite numbers, padding too (0 · NaN is NaN). Returns (o, state): o
    in ``out`` or a new dense tensor; the state after the last token, fp32 [batch, heads, 64, 64], in ``final``
    (which may be ``initial``) or a new tensor. ``status`` as for :func:`gated_ffn`."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    scale = float(scale)  # a plain number: the key must not hold a tensor, whose value may change
    try:
        key = (dev, _meta(q), _meta(k), _meta(v), _meta(g), _meta(initial), _meta(out), _meta(final), _meta(status), scale)
    except AttributeError:  # something that is no tensor: the checks will name it
        key = None
    plan = _scan_plans.find(key) if key is not None else None
    if plan is None:
        shape = _scan_shape(q, 4, dev)
        st = (shape[0], shape[1], 64, 64)
        for t, n in ((q, "q"), (k, "k"), (v, "v")) + (((out, "out"),) if out is not None else ()):
            _rows(t, n, _BF16, shape, dev)
        _rows(g, "g", _F32, shape[:3], dev, last=False)
        _dense_or_none(initial, "initial", _F32, st, dev)
        _dense_or_none(final, "final", _F32, st, dev)
        _dense_or_none(status, "status", _I32, (1,), dev)
        d = _scan_desc(shape, scale, q, k, v, out, g)
        plan = d, st, abi.load().ttt_gated_scan_workspace(ctypes.byref(d))
        if key is not None:
            _scan_plans.keep(key, plan)
    d, st, nbytes = plan
    with ctx:
        if out is None:
            out = _like(q)
        if final is None:
            final = torch.empty(st, dtype=_F32, device=q.device)
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_gated_scan(ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(initial),
                                    out.data_ptr(), final.data_ptr(), _ptr(ws), nbytes, _ptr(status), raw))
    return out, final


def gated_scan_backward(do, q, k, v, g, *, scale=1.0, initial=None, dfinal=None, status=None, stream=None):
    """ttt_gated_scan_backward: (dq, dk, dv, dg, dinitial) from the gradient ``do`` of the outputs and
    ``dfinal`` of the final state (None: zero). All are dense; dinitial is None where ``initial``
    is."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    scale = float(scale)  # a plain number: the key must not hold a tensor, whose value may change
    try:
        key = (dev, _meta(do), _meta(q), _meta(k), _meta(v), _meta(g), _meta(initial), _meta(dfinal), _meta(status), scale)
    except AttributeError:
        key = None
    plan = _scan_back_plans.find(key) if key is not None else None
    if plan is None:
        shape = _scan_shape(q, 4, dev)
        st = (shape[0], shape[1], 64, 64)
        for t, n in ((do, "do"), (q, "q"), (k, "k"), (v, "v")):
            _rows(t, n, _BF16, shape, dev)
        _rows(g, "g", _F32, shape[:3], dev, last=False)
        _dense_or_none(initial, "initial", _F32, st, dev)
        _dense_or_none(dfinal, "dfinal", _F32, st, dev)
        _dense_or_none(status, "status", _I32, (1,), dev)
        d = _scan_desc(shape, scale, q, k, v, do, g)
        plan = d, abi.load().ttt_gated_scan_backward_workspace(ctypes.byref(d))
        if key is not None:
            _scan_back_plans.keep(key, plan)
    d, nbytes = plan
    with ctx:
        dq, dk, dv, dg = _like(q), _like(k), _like(v), _like(g)
        di = None if initial is None else _like(initial)
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_gated_scan_backward(
        ctypes.byref(d), do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(initial), _ptr(dfinal),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), _ptr(di), _ptr(ws), nbytes, _ptr(status), raw))
    return dq, dk, dv, dg, di


def gated_scan_step(state, q, k, v, g, *, scale=1.0, out=None, stream=None):
    """ttt_gated_scan_step: one token of every sequence. ``state`` fp32 [batch, heads, 64, 64] is updated
    in place; ``q``, ``k``, ``v`` bf16 [batch, heads, 64] (rows as the module says), ``g`` fp32 [batch, heads] (any
    strides). Returns o, bf16 [batch, heads, 64]."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    scale = float(scale)  # a plain number: the key must not hold a tensor, whose value may change
    try:
        key = (dev, _meta(state), _meta(q), _meta(k), _meta(v), _meta(g), _meta(out), scale)
    except AttributeError:
        key = None
    d = _step_plans.find(key) if key is not None else None
    if d is None:
        shape = _scan_shape(q, 3, dev)
        for t, n in ((q, "q"), (k, "k"), (v, "v")) + (((out, "out"),) if out is not None else ()):
            _rows(t, n, _BF16, shape, dev)
        _rows(g, "g", _F32, shape[:2], dev, last=False)
        _dense(state, "state", _F32, (shape[0], shape[1], 64, 64), dev)
        d = _scan_desc(shape, scale, q, k, v, out, g)
        if key is not None:
            _step_plans.keep(key, d)
    if out is None:
        with ctx:
            out = _like(q)
    check(abi.load().ttt_gated_scan_step(ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                         state.data_ptr(), out.data_ptr(), raw))
    return out


# ---- the gated feed-forward block -------------------------------------------------------------


_ffn_plans, _ffn_back_plans = _Plans(), _Plans()


def _ffn_shape(x, w_gate, w_up, dev):
    for t, n, want in ((x, "x", "[tokens, d]"), (w_gate, "w_gate", "[f, d]"), (w_up, "w_up", "[f, d]")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            _refuse(t, n, want + " torch.bfloat16", dev)
    T, d, f = x.shape[0], x.shape[1], w_gate.shape[0]
    _dense(x, "x", _BF16, (T, d), dev)
    _dense(w_gate, "w_gate", _BF16, (f, d), dev)
    _dense(w_up, "w_up", _BF16, (f, d), dev)
    return T, d, f


def gated_ffn(x, w_gate, w_up, *, activation="silu", save=False, out=None, status=None, stream=None):
    """ttt_gated_ffn: z = act(x·w_gateᵀ) ⊙ (x·w_upᵀ), the In-Place scan's keys. ``x`` bf16 [tokens, d],
    ``w_gate`` and ``w_up`` bf16 [f, d], contiguous; ``activation`` "silu" or "gelu". Returns z [tokens,
    f], or with ``save`` (z, gate, up) with the pre-activations that :func:`gated_ffn_backward` takes.
    ``status`` (int32 device tensor of one element, optional) is set to 0, or to TTT_ERR_TIMEOUT if
    a bounded device-side wait ran out (without it :func:`poll_operators` tells)."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    try:
        key = (dev, _meta(x), _meta(w_gate), _meta(w_up), _meta(out), _meta(status), activation)
    except AttributeError:  # something that is no tensor: the checks will name it
        key = None
    plan = _ffn_plans.find(key) if key is not None else None
    if plan is None:
        T, d, f = _ffn_shape(x, w_gate, w_up, dev)
        _dense_or_none(out, "out", _BF16, (T, f), dev)
        _dense_or_none(status, "status", _I32, (1,), dev)
        plan = T, d, f, _choice(ACTIVATIONS, activation, "activation")
        if key is not None:
            _ffn_plans.keep(key, plan)
    T, d, f, act = plan
    gate = up = None
    with ctx:
        if out is None:
            out = x.new_empty((T, f))
        if save:
            gate, up = torch.empty_like(out), torch.empty_like(out)
    check(abi.load().ttt_gated_ffn(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), T, d, f, act, out.data_ptr(), _ptr(gate),
                                   _ptr(up), _ptr(status), raw))
    return (out, gate, up) if save else out


def gated_ffn_backward(dz, x, w_gate, w_up, gate, up, *, activation="silu", need_dx=True, need_dw=True, status=None,
                       stream=None):
    """ttt_gated_ffn_backward: (dx, dw_gate, dw_up) from the gradient ``dz`` of z and the kept
    pre-activations ``gate`` and ``up``, all bf16 and contiguous; ``need_dx`` or ``need_dw`` false
    leaves those out (None)."""
    dev = _current_device()
    raw, ctx = _place(stream, dev)
    try:
        key = (dev, _meta(dz), _meta(x), _meta(w_gate), _meta(w_up), _meta(gate), _meta(up), _meta(status), activation)
    except AttributeError:
        key = None
    plan = _ffn_back_plans.find(key) if key is not None else None
    if plan is None:
        T, d, f = _ffn_shape(x, w_gate, w_up, dev)
        for t, n in ((dz, "dz"), (gate, "gate"), (up, "up")):
            _dense(t, n, _BF16, (T, f), dev)
        _dense_or_none(status, "status", _I32, (1,), dev)
        plan = (T, d, f, _choice(ACTIVATIONS, activation, "activation"), abi.load().ttt_gated_ffn_backward_workspace(T, d, f))
        if key is not None:
            _ffn_back_plans.keep(key, plan)
    T, d, f, act, nbytes = plan
    with ctx:
        dx = torch.empty_like(x) if need_dx else None
        dwg, dwu = (torch.empty_like(w_gate) if need_dw else None for _ in range(2))
        ws = _workspace(nbytes, dev)
    check(abi.load().ttt_gated_ffn_backward(
        dz.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), gate.data_ptr(), up.data_ptr(), T, d, f, act, _ptr(dx),
        _ptr(dwg), _ptr(dwu), _ptr(ws), nbytes, _ptr(status), raw))
    return dx, dwg, dwu

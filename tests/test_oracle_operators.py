"""The operators' oracles against closed forms and central differences."""

import math

import numpy as np
import pytest

from oracle import operators as op


def _difference(f, x, dy, h=1e-6):
    """d<f(x), dy>/dx by central differences."""
    out = np.zeros_like(x)
    flat, res = x.reshape(-1), out.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + h
        up = np.sum(f() * dy)
        flat[i] = keep - h
        down = np.sum(f() * dy)
        flat[i] = keep
        res[i] = (up - down) / (2 * h)
    return out


@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_rope_gradients(norm, layout):
    r = np.random.default_rng(1)
    x, dy = r.standard_normal((2, 2, 3, 8)), r.standard_normal((2, 2, 3, 8))
    w = r.standard_normal(8) if norm == "rms" else None
    pos = r.integers(0, 100, (2, 3))
    how = dict(magnitude=1.2, norm=norm, eps=1e-3, layout=layout, weight=w)
    f = lambda: op.norm_rope(x, pos, [0.7, 0.1], **how)  # noqa: E731
    dx, dw = op.norm_rope_backward(dy, x, pos, [0.7, 0.1], **how)
    # Differences with h = 1e-6: h² times the third derivative, and 2^-53 / h of rounding: 1e-8 or so.
    assert np.max(np.abs(dx - _difference(f, x, dy))) < 1e-7
    if w is not None:
        assert np.max(np.abs(dw - _difference(f, w, dy))) < 1e-7


def test_rotation_keeps_lengths_and_angles():
    """Without norm the rotation is orthogonal and depends on position differences alone."""
    r = np.random.default_rng(2)
    x = r.standard_normal((1, 2, 1, 16))
    f = 10000.0 ** (-np.arange(8) / 8.0)
    at = lambda p: op.norm_rope(x, [[p]], f, norm="none")  # noqa: E731
    assert np.allclose(np.linalg.norm(at(12345), axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    dot = lambda a, b: np.sum(at(a)[0, 0] * at(b)[0, 1])  # noqa: E731
    assert abs(dot(7, 3) - dot(1007, 1003)) < 1e-10


def test_gated_scan_closed_forms():
    r = np.random.default_rng(3)
    q, k, v = (r.standard_normal((1, 2, 9, 64)) for _ in range(3))
    # Gates of zero: the plain sum of outer products. Gates of -inf: each token alone.
    o, S, _ = op.gated_scan(q, k, v, np.zeros((1, 2, 9)), 0.5)
    assert np.allclose(S, np.einsum("bhta,bhtc->bhac", k, v))
    assert np.allclose(o[:, :, -1], 0.5 * np.einsum("bha,bhac->bhc", q[:, :, -1], S))
    o, S, _ = op.gated_scan(q, k, v, np.full((1, 2, 9), -np.inf), 1.0)
    assert np.allclose(o, np.sum(q * k, -1, keepdims=True) * v)
    assert np.allclose(S, k[:, :, -1, :, None] * v[:, :, -1, None, :])


def test_gated_scan_gradients():
    r = np.random.default_rng(4)
    B, H, T, D = 1, 1, 4, 64
    q, k, v, do = (r.standard_normal((B, H, T, D)) for _ in range(4))
    g = -r.random((B, H, T))
    S0, dS = r.standard_normal((B, H, D, D)), r.standard_normal((B, H, D, D))
    got = op.gated_scan_backward(do, q, k, v, g, 0.3, S0, dS)

    def loss():
        o, S, _ = op.gated_scan(q, k, v, g, 0.3, S0)
        return np.concatenate([o.reshape(-1), S.reshape(-1)])

    dy = np.concatenate([do.reshape(-1), dS.reshape(-1)])
    for x, d in ((q, got[0]), (k, got[1]), (v, got[2]), (g, got[3])):
        assert np.max(np.abs(d - _difference(loss, x, dy))) < 1e-5 * max(1.0, np.max(np.abs(d)))
    part = S0[0, 0, :2]  # a part of the initial state is enough
    assert np.max(np.abs(got[4][0, 0, :2] - _difference(loss, part, dy))) < 1e-5 * np.max(np.abs(got[4]))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_ffn_gradients(kind):
    r = np.random.default_rng(5)
    x, wg, wu, dz = (r.standard_normal(s) for s in ((3, 6), (5, 6), (5, 6), (3, 5)))
    _, g, u = op.gated_ffn(x, wg, wu, kind)
    dx, dwg, dwu, _, _ = op.gated_ffn_backward(dz, x, wg, wu, g, u, kind)
    f = lambda: op.gated_ffn(x, wg, wu, kind)[0]  # noqa: E731
    for t, d in ((x, dx), (wg, dwg), (wu, dwu)):
        assert np.max(np.abs(d - _difference(f, t, dz))) < 1e-7
    a, _ = op.activation(np.array([0.0, 30.0, -30.0]), kind)
    assert a[0] == 0 and abs(a[1] - 30) < 1e-9 and abs(a[2]) < 1e-9
    assert math.isclose(op.activation(np.array([1.0]), "silu")[0][0], 1 / (1 + math.exp(-1)))

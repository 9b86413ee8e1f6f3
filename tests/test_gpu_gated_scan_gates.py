"""The gated scan where gates are extreme: many document starts before a document, and heads that forget
nearly all at each token.

dg is fp32 and made of sums over pairs m_ij = A_ij·(q_i·k_j), i >= t > j. With q·k and do·v sums of 64
products of bf16 numbers, each off by at most 64 steps of 2^-23 of its terms' size, a decay off by 2^-21
(the gates in base-2 units and their sums, for the few units that the pairs here span, and the
exponential's 2^-22), and three products, a pair is off by at most 2^-16 + 2^-20 of |q|·|k|·|do|·|v|. A
token's sum is a difference of sums over the chunk's pairs, in which 27 fp32 additions follow one
another at most: 2 · 27 · 2^-24 < 2^-18 of all the chunk's pairs."""

import math

import numpy as np
import pytest
import torch

from oracle import operators as op
from tests._util import to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


def _pairs(q, k, v, do, g, scale):
    """|m_ij| of one (sequence, head) with i > j, and with i = j, from the absolute values of the rows."""
    w = np.zeros((len(g), len(g)))
    for j in range(len(g)):
        w[j:, j] = np.exp(np.cumsum(np.concatenate([[0.0], g[j + 1:]])))
    a = [np.abs(t) for t in (q, k, v, do)]
    m = scale * w * (a[0] @ a[1].T) * (a[3] @ a[2].T)
    return np.tril(m, -1), np.diag(m)


@pytest.mark.parametrize("before", ["resets", "tokens"])
@pytest.mark.parametrize("at", [33, 64, 96])
def test_a_document_after_many_short_ones(cwl, before, at):
    """A document's gradients do not depend on how many documents started before it in its chunk."""
    r = torch.Generator().manual_seed(at)
    q, k, v, do = (torch.rand((1, 2, 128, 64), generator=r).bfloat16() for _ in range(4))
    g = -0.01 * torch.rand((1, 2, 128), generator=r)
    if before == "resets":
        g[:, :, :at] = -math.inf
    g[:, :, at] = -math.inf
    c = [t.cuda() for t in (do, q, k, v, g)]
    got = to_np(cwl.gated_scan_backward(*c, scale=0.125)[3])
    n = [to_np(t) for t in (q, k, v, do, g)]
    want = op.gated_scan_backward(n[3], *n[:3], n[4], 0.125)[3]
    for h in range(2):
        off, own = _pairs(*(t[0, h] for t in n), 0.125)
        for t in range(at + 1, 128):
            bound = (2.0 ** -16 + 2.0 ** -20) * off[t:, :t].sum() + 2.0 ** -18 * (off.sum() + own.sum())
            assert abs(got[0, h, t] - want[0, h, t]) <= bound, (h, t, got[0, h, t], want[0, h, t], bound)


@pytest.mark.parametrize("strength", [8.0, 12.0, 16.0, 20.0])
@pytest.mark.parametrize("T", [40, 128, 300])
@pytest.mark.parametrize("initial", [False, True])
def test_small_gates_keep_their_gradients(cwl, strength, T, initial):
    """Every head forgets nearly all at each token: dg is e^-strength of a token's own pair, and is right
    relative to itself. Its parts from beyond the chunk come from states and operands of 2^-16, so 2^-15
    of the terms; where gates are -20 the nearest pair's decay spans 29 base-2 units, which their sums
    give to 2^-18."""
    r = torch.Generator().manual_seed(int(strength) + T)
    q, k, v, do = (torch.randn((1, 2, T, 64), generator=r).bfloat16() for _ in range(4))
    g = -strength - 0.5 * torch.rand((1, 2, T), generator=r)
    S0, dS = (torch.randn((1, 2, 64, 64), generator=r) if initial else None for _ in range(2))
    c = [t.cuda() if t is not None else None for t in (do, q, k, v, g, S0, dS)]
    got = to_np(cwl.gated_scan_backward(*c[:5], scale=0.125, initial=c[5], dfinal=c[6])[3])
    n = [to_np(t) if t is not None else None for t in (do, q, k, v, g, S0, dS)]
    a = [np.abs(t) if t is not None and i != 4 else t for i, t in enumerate(n)]
    want = op.gated_scan_backward(*n[:5], 0.125, *n[5:])[3]
    top = op.gated_scan_backward(*a[:5], 0.125, *a[5:])[3]
    for h in range(2):
        for t0 in range(0, T, 128):
            e = slice(t0, min(T, t0 + 128))
            off, _ = _pairs(n[1][0, h, e], n[2][0, h, e], n[3][0, h, e], n[0][0, h, e], n[4][0, h, e], 0.125)
            bound = (2.0 ** -15 + 2.0 ** -18) * top[0, h, e] + 2.0 ** -18 * off.sum()
            err = np.abs(got[0, h, e] - want[0, h, e])
            assert np.all(err <= bound), f"{np.max(err / bound):.3g} x the bound"

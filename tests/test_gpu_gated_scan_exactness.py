"""The gated scan's fp32 outputs keep fp32 factors: the states, their gradients and the gates' gradients.

The values here are the ones that two bf16 numbers hold worst: R = 0.5 + 2^-10 + 2^-18 rounds to 0.5, the
rest to 2^-10, and 2^-18 is left, 7.6e-6 of R. A state that takes its products' factors as two bf16 numbers
is off by that in every term alike. All terms are positive, so the tolerances are relative to the result.

A state's weights are e^g in fp32: the gate in base-2 units and its product are off by 2^-23 of an exponent
of about one, the exponential by 2^-22. A chunk's sum takes 24 matrix instructions, of which the last eight
hold nearly all of it; each may lose a step of 2^-23. That and an addition a chunk make 1.4e-6, and chunks
before count half each and add 3e-7 each of their half: below 2^-19 = 1.9e-6.

A gate's gradient is a sum of 4096 products (of 64 sums of 64): 33 additions in a row, 12 matrix
instructions and 9 more additions of 2^-24 or, for the instructions, 2^-23: below 2^-18 = 3.8e-6."""

import math

import numpy as np
import pytest
import torch

from oracle import operators as op
from tests._util import to_np

pytestmark = pytest.mark.gpu
R = 0.5 + 2.0 ** -10 + 2.0 ** -18


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


def _ones(T, value=1.0):
    return torch.full((1, 1, T, 64), value).bfloat16()


@pytest.mark.parametrize("T", [128, 384, 1300, 6000, 11200])
def test_states(cwl, T):
    """One chunk, one segment, few and many segments; each chunk's last gate is log R, the others 0."""
    k, v, q = _ones(T), _ones(T), _ones(T, 0.0)
    g = torch.zeros((1, 1, T))
    g[:, :, 127::128] = math.log(R)
    _, S = cwl.gated_scan(q.cuda(), k.cuda(), v.cuda(), g.cuda())
    want, factor = 0.0, np.exp(np.asarray(g[0, 0].double()))
    for f in factor:
        want = f * want + 1.0
    assert np.all(np.abs(to_np(S) - want) <= 2.0 ** -19 * want), np.max(np.abs(to_np(S) / want - 1))


@pytest.mark.parametrize("T", [128, 384, 1300, 6000, 11200])
def test_gradients_of_the_initial_state(cwl, T):
    """The same in reverse: each chunk's first gate is log R."""
    q, do, k = _ones(T), _ones(T), _ones(T, 0.0)
    g = torch.zeros((1, 1, T))
    g[:, :, ::128] = math.log(R)
    S0 = torch.zeros((1, 1, 64, 64))
    dS0 = cwl.gated_scan_backward(*(t.cuda() for t in (do, q, k, k, g)), initial=S0.cuda())[4]
    want, factor = 0.0, np.exp(np.asarray(g[0, 0].double()))
    for f in factor[::-1]:
        want = f * (want + 1.0)
    assert np.all(np.abs(to_np(dS0) - want) <= 2.0 ** -19 * want), np.max(np.abs(to_np(dS0) / want - 1))


@pytest.mark.parametrize("case", ["both states", "outputs of the initial state", "keys of the final gradient"])
def test_gradients_of_gates(cwl, case):
    T = 2
    q, k, v, do = (_ones(T, 0.0) for _ in range(4))
    S0 = dS = torch.zeros((1, 1, 64, 64))
    if case == "both states":
        S0, dS = torch.full((1, 1, 64, 64), R), torch.ones((1, 1, 64, 64))
    elif case == "outputs of the initial state":
        S0, q, do = torch.full((1, 1, 64, 64), R), _ones(T), _ones(T)
    else:
        dS, k, v = torch.full((1, 1, 64, 64), R), _ones(T), _ones(T)
    g = torch.zeros((1, 1, T))
    x = (do, q, k, v, g)
    got = to_np(cwl.gated_scan_backward(*(t.cuda() for t in x), initial=S0.cuda(), dfinal=dS.cuda())[3])
    want = op.gated_scan_backward(*(to_np(t) for t in x), 1.0, to_np(S0), to_np(dS))[3]
    assert np.all(np.abs(got - want) <= 2.0 ** -18 * np.abs(want)), np.max(np.abs(got / np.maximum(want, 1e-30) - 1))
    assert np.any(want > 0)

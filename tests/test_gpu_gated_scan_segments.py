"""The gated scan against the oracle around its chunks of 128 tokens, its blocks of 32, and its segments:
more than eight of a sequence, which one launch combines in order, and more than sixteen, which it takes
in rounds. Gates here are so mild that a state reaches across segments. Tolerances as derived in
test_gpu_gated_scan.py: a bf16 output is off by at most 2^-8 of itself and of its terms' size, an fp32
one by 2^-15 of its terms' size, dg also by 64 roundings of the largest sum that it is a difference of."""

import numpy as np
import pytest
import torch

import tests.test_gpu_gated_scan as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


def _both(cwl, x, scale):
    c = base._cuda(x)
    o, S = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=scale, initial=c["S0"])
    base._check_forward(o, S, x, scale)
    got = cwl.gated_scan_backward(c["do"], c["q"], c["k"], c["v"], c["g"], scale=scale, initial=c["S0"], dfinal=c["dS"])
    base._check_backward(got, x, scale)
    return o, S, got


@pytest.mark.parametrize("T", [31, 32, 33, 96, 127, 128, 255, 256, 257, 384, 512])
@pytest.mark.parametrize("initial", [False, True])
def test_around_chunks_and_blocks(cwl, T, initial):
    _both(cwl, base._inputs(1, 2, T, 500 + T, "documents", initial=initial), 0.125)


@pytest.mark.parametrize("H,T,documents", [(2, 6000, True), (1, 6000, False), (1, 88 * 128, False), (1, 88 * 128 - 37, True)])
def test_many_segments(cwl, H, T, documents):
    """Ten segments of five chunks (the last of two), and 22 of four."""
    x = base._inputs(1, H, T, 7 * T + H)
    r = torch.Generator().manual_seed(T)
    x["g"] = -2e-3 * torch.rand((1, H, T), generator=r)
    if documents:
        x["g"][:, :, [T // 3, T // 2 + 77]] = -np.inf
    _, S, got = _both(cwl, x, 0.125)
    # Into another buffer than the initial state's or over it: the same.
    c = base._cuda(x)
    o2, S2 = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"], final=c["S0"])
    assert S2 is c["S0"] and torch.equal(S2, S)
    again = cwl.gated_scan_backward(*(base._cuda(x)[n] for n in ("do", "q", "k", "v", "g")), scale=0.125,
                                    initial=x["S0"].cuda(), dfinal=c["dS"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))

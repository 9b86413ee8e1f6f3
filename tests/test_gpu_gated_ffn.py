"""GPU parity of the gated feed-forward block and its gradients.

Tolerances: products of bf16 operands summed in fp32 (2^-24 per term of the sum of absolute values A;
2^-18·A is asked, the activation's fp32 arithmetic with it), outputs rounded to bf16 once, 2^-8 of
the value. Backward, dG and dU are rounded to bf16 before they are operands: 2^-8 of each term."""

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


def _case(T, d, f, seed):
    r = torch.Generator().manual_seed(seed)
    x = torch.randn((T, d), generator=r).bfloat16()
    wg, wu = ((torch.randn((f, d), generator=r) * d ** -0.5).bfloat16() for _ in range(2))
    dz = torch.randn((T, f), generator=r).bfloat16()
    return x, wg, wu, dz


def _near(got, ref, slack, name):
    err, bound = np.abs(to_np(got) - ref), slack + 2.0 ** -8 * np.abs(ref) + 1e-30
    assert np.all(err <= bound), f"{name}: {np.max(err / bound):.3g} x the bound"


def _check_forward(got, x, wg, wu, kind):
    z, g, u = (to_np(t) if t is not None else None for t in got)
    rz, rg, ru = op.gated_ffn(to_np(x), to_np(wg), to_np(wu), kind)
    ag, au = np.abs(to_np(x)) @ np.abs(to_np(wg)).T, np.abs(to_np(x)) @ np.abs(to_np(wu)).T
    if g is not None:
        _near(g, rg, 2.0 ** -18 * ag, "gate")
        _near(u, ru, 2.0 ** -18 * au, "up")
    # |act'| stays below 1.13; act's own fp32 error is some 2^-21 of |g|.
    act = op.activation(rg, kind)[0]
    _near(z, rz, 2.0 ** -18 * (1.13 * ag * np.abs(ru) + np.abs(act) * au + np.abs(rg * ru)) , "z")


SIZES = [(1, 64, 64), (1, 2560, 200), (2, 8, 8), (3, 72, 24), (8, 40, 136), (9, 264, 1000), (16, 512, 48), (17, 104, 120),
         (31, 1000, 56), (32, 264, 264), (33, 264, 264), (64, 136, 72), (127, 520, 392), (128, 64, 128), (257, 328, 136),
         (300, 200, 520), (513, 72, 1032)]


@pytest.mark.parametrize("T,d,f", SIZES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward(cwl, T, d, f, kind):
    x, wg, wu, _ = _case(T, d, f, T + d + f)
    z, g, u = cwl.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), activation=kind, save=True)
    _check_forward((z, g, u), x, wg, wu, kind)
    assert torch.equal(z, cwl.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), activation=kind))


@pytest.mark.parametrize("T,d,f", SIZES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward(cwl, T, d, f, kind):
    x, wg, wu, dz = _case(T, d, f, T + d + f + 1)
    g, u = ((x.float() @ w.float().t()).bfloat16() for w in (wg, wu))
    c = [t.cuda() for t in (dz, x, wg, wu, g, u)]
    got = cwl.gated_ffn_backward(*c, activation=kind)
    dx, dwg, dwu, dg, du = op.gated_ffn_backward(*(to_np(t) for t in (dz, x, wg, wu, g, u)), kind)
    r = 2.0 ** -8 + 2.0 ** -17
    a, b, X = np.abs(dg), np.abs(du), np.abs(to_np(x))
    # act' has fp32 terms of up to |dz·u| where it nearly cancels.
    c0 = 2.0 ** -18 * np.abs(to_np(dz)) * (np.abs(to_np(u)) + 1)
    _near(got[0], dx, (r * a + c0) @ np.abs(to_np(wg)) + (r * b + c0) @ np.abs(to_np(wu)), "dx")
    _near(got[1], dwg, (r * a + c0).T @ X, "dw_gate")
    _near(got[2], dwu, (r * b + c0).T @ X, "dw_up")
    again = cwl.gated_ffn_backward(*c, activation=kind)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    part = cwl.gated_ffn_backward(*c, activation=kind, need_dw=False)
    assert part[1] is None and part[2] is None and torch.equal(part[0], got[0])
    part = cwl.gated_ffn_backward(*c, activation=kind, need_dx=False)
    assert part[0] is None and torch.equal(part[1], got[1]) and torch.equal(part[2], got[2])


def test_large_and_persistent(cwl):
    """More tiles than SM pairs (each pair runs several, with both accumulators), odd edges."""
    T, d, f = 2051, 584, 2312
    x, wg, wu, dz = (t.cuda() for t in _case(T, d, f, 3))
    z, g, u = cwl.gated_ffn(x, wg, wu, save=True)
    X, G, U, Wg, Wu = (t.double() for t in (x, g, u, wg, wu))
    ref = torch.nn.functional.silu(X @ Wg.T) * (X @ Wu.T)
    # Two norms: random signs make the roundings' errors at most 2^-8 of the whole.
    assert (z.double() - ref).norm() <= 2.0 ** -8 * ref.norm()
    dx, dwg, dwu = cwl.gated_ffn_backward(dz, x, wg, wu, g, u)
    s = torch.sigmoid(G)
    dG, dU = dz.double() * U * s * (1 + G * (1 - s)), dz.double() * G * s
    for got, want in ((dx, dG @ Wg + dU @ Wu), (dwg, dG.T @ X), (dwu, dU.T @ X)):
        assert (got.double() - want).norm() <= 2.0 ** -8 * want.norm()
        # No element is far off: a misplaced tile edge would show here.
        assert (got.double() - want).abs().max() <= 2.0 ** -5 * want.abs().max()
    assert (z.double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() * 1.01


@pytest.mark.parametrize("T,d,f", [(T, d, f) for T in (17, 48, 65, 113, 128, 129, 160, 161) for d, f in
                                   ((8, 9480), (584, 1224), (200, 9608), (72, 20000))]
                         + [(T, 1032, 9480) for T in (8, 9, 15, 16)] + [(T, 4104, 9480) for T in (1, 2, 8)])
def test_some_tens_of_tokens(cwl, T, d, f):
    """Around the changes of form: one k-block and several rounds of the ring, a last tile with few rows,
    more rows than one tile an SM takes."""
    x, wg, wu, _ = _case(T, d, f, T + f)
    z, g, u = cwl.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), save=True)
    _check_forward((z, g, u), x, wg, wu, "silu")
    big = torch.full((T + 3, f), 7.0, device="cuda", dtype=torch.bfloat16)
    cwl.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), out=big[:T])
    assert torch.equal(big[:T], z) and torch.all(big[T:] == 7.0)


def test_a_token_stays_its_own(cwl):
    """A NaN in one token's row reaches no other token."""
    for T, f in ((3, 200), (40, 200), (40, 9480), (300, 200)):
        x, wg, wu, _ = (t.cuda() for t in _case(T, 136, f, 8))
        want = cwl.gated_ffn(x, wg, wu)
        x[T // 2] = float("nan")
        got = cwl.gated_ffn(x, wg, wu)
        rest = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(got[rest], want[rest]) and torch.isnan(got[T // 2]).all()


def test_outputs_stay_inside(cwl):
    """Rows of a larger buffer behind the call's tokens are left as they were."""
    for T in (5, 40, 300):
        x, wg, wu, _ = (t.cuda() for t in _case(T, 136, 200, 4))
        big = torch.full((T + 9, 200), 7.0, device="cuda", dtype=torch.bfloat16)
        cwl.gated_ffn(x, wg, wu, out=big[:T])
        assert torch.all(big[T:] == 7.0)


def test_no_tokens(cwl):
    x, wg, wu, dz = (t.cuda() for t in _case(4, 64, 72, 5))
    assert cwl.gated_ffn(x[:0], wg, wu).shape == (0, 72)
    dx, dwg, dwu = cwl.gated_ffn_backward(dz[:0], x[:0], wg, wu, dz[:0], dz[:0])
    assert dx.shape == (0, 64) and torch.all(dwg == 0) and torch.all(dwu == 0)


@pytest.mark.parametrize("T", [7, 200])
def test_captured_and_replayed(cwl, T):
    x, wg, wu, dz = (t.cuda() for t in _case(T, 264, 520, 6))
    call = lambda: (*cwl.gated_ffn(x, wg, wu, save=True), *cwl.gated_ffn_backward(dz, x, wg, wu, dz, dz))  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    x.mul_(0.5), dz.add_(1)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_streams_and_status(cwl):
    x, wg, wu, dz = (t.cuda() for t in _case(300, 264, 520, 7))
    status = torch.full((1,), 9, device="cuda", dtype=torch.int32)
    want = cwl.gated_ffn(x, wg, wu, status=status)
    assert int(status) == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [cwl.gated_ffn_backward(dz, x, wg, wu, dz, dz, stream=s) for _ in range(3)]
    b = [cwl.gated_ffn_backward(dz, x, wg, wu, dz, dz, status=status) for _ in range(3)]
    c = [cwl.gated_ffn(x, wg, wu, stream=s) for _ in range(2)]
    torch.cuda.synchronize()
    assert int(status) == 0 and all(torch.equal(t, want) for t in c)
    for got in a + b:
        assert all(torch.equal(p, q) for p, q in zip(got, a[0]))


def test_refusals(cwl):
    x, wg, wu, dz = (t.cuda() for t in _case(4, 64, 72, 8))
    for args, word in (((x.float(), wg, wu), "x"), ((x, wg[:, :32], wu), "w_gate"), ((x, wg, wu[:8]), "w_up"),
                       ((x, wg.t(), wu), "w_gate"), ((x.cpu(), wg, wu), "x")):
        with pytest.raises(ValueError, match=word):
            cwl.gated_ffn(*args)
    with pytest.raises(ValueError, match="activation"):
        cwl.gated_ffn(x, wg, wu, activation="relu")
    y = torch.zeros((4, 60), device="cuda", dtype=torch.bfloat16)
    w = torch.zeros((72, 60), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(cwl.TTTError, match="multiples of 8"):
        cwl.gated_ffn(y, w, w)
    with pytest.raises(ValueError, match="gate"):
        cwl.gated_ffn_backward(dz, x, wg, wu, dz[:2], dz)

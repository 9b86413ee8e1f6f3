"""GPU parity of the gated scan, its gradients and its one-token form against the float64 oracle.

Tolerances, from the roundings on the way. Half a step of bf16 is 2^-8 of the value. An output o
is a sum of products with one factor rounded to bf16 (P, or the copy of the state), rounded once
more at the end: off by at most 2^-8·(|o| + A), A the same sum with every term's absolute value
(the oracle run on absolute values). The same holds for dq, dk, dv. States, dS0 and dg are fp32 and
every product that feeds them keeps its factors to 2^-16: off by at most 2^-15·A, and by the rounding
of the gates' sums, which enters the exponent: 2^-24 of the largest sum within a chunk of 64, in
base-2 units with gates counted from -150, over the six steps of a sum and the subtraction."""

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


def _inputs(B, H, T, seed, gates="mild", initial=True):
    r = torch.Generator().manual_seed(seed)
    x = {n: torch.randn((B, H, T, 64), generator=r).bfloat16() for n in ("q", "k", "v", "do")}
    g = torch.nn.functional.logsigmoid(3 + torch.randn((B, H, T), generator=r))
    if gates == "documents":
        for b in range(B):
            at = torch.randint(0, T, (3,), generator=r)
            g[b][:, at] = -math.inf
    elif gates == "strong":
        g = -30 * torch.rand((B, H, T), generator=r)
    elif gates == "zero":
        g = torch.zeros((B, H, T))
    elif gates == "gone":
        g = torch.full((B, H, T), -math.inf)
    elif gates == "edge":  # each side of the value whose factor is 0 in fp32
        g = torch.where(torch.rand((B, H, T), generator=r) < 0.1, torch.tensor(-103.9), g)
        g = torch.where(torch.rand((B, H, T), generator=r) < 0.1, torch.tensor(-104.1), g)
    x["g"] = g
    x["S0"] = torch.randn((B, H, 64, 64), generator=r) if initial else None
    x["dS"] = torch.randn((B, H, 64, 64), generator=r) if initial else None
    return x


def _cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def _np(x):
    return {n: None if t is None else to_np(t) for n, t in x.items()}


def _abs(x):
    return {n: None if t is None else (t if n == "g" else np.abs(t)) for n, t in x.items()}


def _gate_error(g):
    """Bound on the relative error that the gates' sums leave in a decay."""
    x = np.maximum(np.asarray(g, np.float64) / math.log(2.0), -150.0)
    T = x.shape[-1]
    pad = -T % 64
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (pad,))], -1).reshape(x.shape[:-1] + (-1, 64))
    return 8 * 2.0 ** -24 * math.log(2.0) * np.max(np.abs(np.cumsum(x, -1)))


def _near(got, ref, bound, name):
    got, ref = to_np(got), np.asarray(ref)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g} x the bound"


def _check_forward(o, S, x, scale):
    n = _np(x)
    ro, rS, _ = op.gated_scan(n["q"], n["k"], n["v"], n["g"], scale, n["S0"])
    a = _abs(n)
    ao, aS, _ = op.gated_scan(a["q"], a["k"], a["v"], a["g"], scale, a["S0"])
    e = _gate_error(n["g"])
    _near(o, ro, 2.0 ** -8 * (np.abs(ro) + ao) + e * ao + 1e-30, "o")
    _near(S, rS, (2.0 ** -15 + e) * aS + 1e-30, "state")


def _check_backward(got, x, scale):
    n, a = _np(x), _abs(_np(x))
    ref = op.gated_scan_backward(n["do"], n["q"], n["k"], n["v"], n["g"], scale, n["S0"], n["dS"])
    top = op.gated_scan_backward(a["do"], a["q"], a["k"], a["v"], a["g"], scale, a["S0"], a["dS"])
    e = _gate_error(n["g"])
    for i, name in enumerate(("dq", "dk", "dv")):
        _near(got[i], ref[i], 2.0 ** -8 * (np.abs(ref[i]) + top[i]) + e * top[i] + 1e-30, name)
    # dg is the difference of sums over the chunk, each of at most 64 of the terms of its largest.
    gone = n["g"] < -104
    assert np.all(to_np(got[3])[gone] == 0)
    most = np.max(top[3] + np.sum(a["q"] * top[0], -1) + np.sum(a["k"] * top[1], -1), -1, keepdims=True)
    _near(got[3], np.where(gone, 0, ref[3]), (2.0 ** -15 + e) * top[3] + 64 * 2.0 ** -22 * most + 1e-30, "dg")
    if n["S0"] is not None:
        _near(got[4], ref[4], (2.0 ** -15 + e) * top[4] + 1e-30, "dS0")
    else:
        assert got[4] is None


SIZES = [(1, 1, 1), (2, 3, 2), (1, 2, 15), (3, 1, 63), (1, 2, 64), (2, 2, 65), (1, 3, 129), (2, 1, 300), (1, 1, 1111)]


@pytest.mark.parametrize("B,H,T", SIZES)
@pytest.mark.parametrize("initial", [False, True])
def test_forward_sizes(cwl, B, H, T, initial):
    x = _inputs(B, H, T, 100 + T, initial=initial)
    c = _cuda(x)
    o, S = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"])
    _check_forward(o, S, x, 0.125)


@pytest.mark.parametrize("B,H,T", SIZES)
@pytest.mark.parametrize("initial", [False, True])
def test_backward_sizes(cwl, B, H, T, initial):
    x = _inputs(B, H, T, 200 + T, initial=initial)
    c = _cuda(x)
    got = cwl.gated_scan_backward(c["do"], c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"], dfinal=c["dS"])
    _check_backward(got, x, 0.125)


@pytest.mark.parametrize("gates", ["documents", "strong", "zero", "gone", "edge"])
@pytest.mark.parametrize("T", [70, 517])
def test_gates(cwl, gates, T):
    x = _inputs(2, 2, T, 300 + T, gates)
    c = _cuda(x)
    o, S = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=1.0, initial=c["S0"])
    _check_forward(o, S, x, 1.0)
    got = cwl.gated_scan_backward(c["do"], c["q"], c["k"], c["v"], c["g"], scale=1.0, initial=c["S0"], dfinal=c["dS"])
    _check_backward(got, x, 1.0)


def test_documents_do_not_leak(cwl):
    """A gate of -inf starts a document: its outputs are those of the document alone, whatever came
    before, and no gradient crosses."""
    x = _cuda(_inputs(1, 2, 256, 5, "documents"))
    x["g"][:, :, 100] = -math.inf
    run = lambda y: cwl.gated_scan(y["q"], y["k"], y["v"], y["g"], initial=y["S0"])  # noqa: E731
    o, S = run(x)
    y = {n: t.clone() for n, t in x.items()}
    y["k"][:, :, :100] *= -3
    y["v"][:, :, :100] += 1
    y["S0"] *= 7
    o2, S2 = run(y)
    assert torch.equal(o[:, :, 100:], o2[:, :, 100:]) and torch.equal(S, S2)
    do = x["do"].clone()
    do[:, :, :100] = 0
    dq, dk, dv, dg, dS0 = cwl.gated_scan_backward(do, x["q"], x["k"], x["v"], x["g"], initial=x["S0"], dfinal=x["dS"])
    for t in (dq, dk, dv):
        assert torch.all(t[:, :, :100] == 0)
    assert torch.all(dS0 == 0) and torch.all(dg[:, :, 100] == 0)


@pytest.mark.parametrize("many", [(8, 64, 200), (1, 500, 70)])
def test_more_pairs_than_the_gpu_holds(cwl, many):
    """As many (sequence, head) pairs as need no segments: forward, backward, and the same bits
    twice."""
    x = _inputs(*many, 6)
    c = _cuda(x)
    o, S = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"])
    some = {n: t[:1, 3:5] for n, t in x.items()}
    _check_forward(o[:1, 3:5], S[:1, 3:5], some, 0.125)
    back = lambda: cwl.gated_scan_backward(c["do"], c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"],  # noqa: E731
                                           dfinal=c["dS"])
    got = back()
    _check_backward([t[:1, 3:5] for t in got], some, 0.125)
    assert all(torch.equal(a, b) for a, b in zip(got, back()))
    assert torch.equal(o, cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"])[0])


def test_long_sequence_in_segments(cwl):
    """One pair, 33 chunks and a rest: many segments, the last one shorter."""
    x = _inputs(1, 1, 33 * 64 + 7, 7, "documents")
    c = _cuda(x)
    o, S = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"])
    _check_forward(o, S, x, 0.125)
    got = cwl.gated_scan_backward(c["do"], c["q"], c["k"], c["v"], c["g"], scale=0.125, initial=c["S0"], dfinal=c["dS"])
    _check_backward(got, x, 0.125)


def test_continued_calls_are_one_scan(cwl):
    x = _inputs(2, 2, 320, 8)
    c = _cuda(x)
    state, parts = c["S0"].clone(), []
    for a, b in ((0, 64), (64, 65), (65, 257), (257, 320)):
        o, state = cwl.gated_scan(*(c[n][:, :, a:b] for n in ("q", "k", "v", "g")), scale=0.125, initial=state, final=state)
        parts.append(o)
    _check_forward(torch.cat(parts, 2), state, x, 0.125)


@pytest.mark.parametrize("T", [1024 + 5, 16 * 1024])
def test_final_state_over_the_initial_one(cwl, T):
    """``final`` may be ``initial`` with one, few and many segments."""
    x = _cuda(_inputs(1, 3, T, 17))
    o, S = cwl.gated_scan(x["q"], x["k"], x["v"], x["g"], initial=x["S0"])
    for _ in range(3):
        s = x["S0"].clone()
        o2, s2 = cwl.gated_scan(x["q"], x["k"], x["v"], x["g"], initial=s, final=s)
        assert s2 is s and torch.equal(o, o2) and torch.equal(S, s)


@pytest.mark.parametrize("T", [1, 77])
def test_layouts(cwl, T):
    """Token-major views, packed projections, gates [batch, tokens, heads], an output inside a larger
    buffer, and keys shared by all heads (stride 0)."""
    x = _inputs(2, 3, T, 9)
    c = _cuda(x)
    want, S = cwl.gated_scan(c["q"], c["k"], c["v"], c["g"], initial=c["S0"])
    packed = torch.stack([c["q"], c["k"], c["v"]], 2).permute(0, 3, 2, 1, 4).contiguous()  # [B, T, 3, H, 64]
    q, k, v = (packed[:, :, i].transpose(1, 2) for i in range(3))
    g = c["g"].transpose(1, 2).contiguous().transpose(1, 2)
    big = torch.full((2, T + 3, 5, 72), 7.0, device="cuda", dtype=torch.bfloat16)
    out = big[:, 1:T + 1, 1:4, 8:].transpose(1, 2)
    o, S2 = cwl.gated_scan(q, k, v, g, initial=c["S0"], out=out)
    assert o is out and torch.equal(out, want) and torch.equal(S, S2)
    rest = big.clone()
    rest[:, 1:T + 1, 1:4, 8:] = 7.0
    assert torch.all(rest == 7.0), "values outside the output were written"
    do = c["do"].transpose(1, 2).contiguous().transpose(1, 2)
    a = cwl.gated_scan_backward(do, q, k, v, g, initial=c["S0"], dfinal=c["dS"])
    b = cwl.gated_scan_backward(c["do"], c["q"], c["k"], c["v"], c["g"], initial=c["S0"], dfinal=c["dS"])
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    shared = c["k"][:, :1].expand(2, 3, T, 64)
    o1, _ = cwl.gated_scan(c["q"], shared, c["v"], c["g"])
    o2, _ = cwl.gated_scan(c["q"], shared.contiguous(), c["v"], c["g"])
    assert torch.equal(o1, o2)


def test_steps_are_the_scan(cwl):
    x = _inputs(2, 3, 40, 10, "documents")
    c = _cuda(x)
    state, parts = c["S0"].clone(), []
    for t in range(40):
        parts.append(cwl.gated_scan_step(state, *(c[n][:, :, t] for n in ("q", "k", "v", "g")), scale=0.125))
    n, a = _np(x), _abs(_np(x))
    ro, rS, _ = op.gated_scan(n["q"], n["k"], n["v"], n["g"], 0.125, n["S0"])
    ao, aS, _ = op.gated_scan(a["q"], a["k"], a["v"], a["g"], 0.125, a["S0"])
    # fp32 throughout: two roundings a step and expf's two units, over 40 steps; o rounded to bf16.
    _near(state, rS, 40 * 6 * 2.0 ** -24 * aS + 1e-30, "state")
    _near(torch.stack(parts, 2), ro, 2.0 ** -8 * np.abs(ro) + (40 * 6 + 80) * 2.0 ** -24 * ao + 1e-30, "o")


def test_step_layout(cwl):
    x = _cuda(_inputs(3, 2, 4, 11))
    packed = torch.stack([x["q"], x["k"], x["v"]], 2).permute(0, 3, 2, 1, 4).contiguous()
    s1, s2 = x["S0"].clone(), x["S0"].clone()
    a = cwl.gated_scan_step(s1, *(x[n][:, :, 2].contiguous() for n in ("q", "k", "v", "g")))
    out = torch.zeros((3, 2, 4, 64), device="cuda", dtype=torch.bfloat16)
    b = cwl.gated_scan_step(s2, *(packed[:, 2, i] for i in range(3)), x["g"][:, :, 2], out=out[:, :, 1])
    assert torch.equal(a, b) and torch.equal(s1, s2) and torch.all(out[:, :, [0, 2, 3]] == 0)


def test_no_tokens(cwl):
    x = _cuda(_inputs(2, 2, 4, 12))
    e = {n: t[:, :, :0] for n, t in x.items() if n in ("q", "k", "v", "g", "do")}
    o, S = cwl.gated_scan(e["q"], e["k"], e["v"], e["g"], initial=x["S0"])
    assert o.shape == (2, 2, 0, 64) and torch.equal(S, x["S0"])
    assert torch.all(cwl.gated_scan(e["q"], e["k"], e["v"], e["g"])[1] == 0)
    got = cwl.gated_scan_backward(e["do"], e["q"], e["k"], e["v"], e["g"], initial=x["S0"], dfinal=x["dS"])
    assert got[0].numel() == 0 and torch.equal(got[4], x["dS"])


def test_captured_and_replayed(cwl):
    """Captured calls (the first ones of their sizes) replay on new inputs; two graphs keep
    workspaces of their own."""
    xs = [_cuda(_inputs(1, 2, 400, s)) for s in (13, 14)]
    buf = {n: t.clone() for n, t in xs[0].items()}
    call = lambda b: (*cwl.gated_scan(b["q"], b["k"], b["v"], b["g"], initial=b["S0"]),  # noqa: E731
                      *cwl.gated_scan_backward(b["do"], b["q"], b["k"], b["v"], b["g"], initial=b["S0"], dfinal=b["dS"]))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = call(buf)
        graphs.append((gr, got))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for x in xs:
        for n in buf:
            buf[n].copy_(x[n])
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        want = call(x)
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams(cwl):
    """A call given another stream runs there, its workspace and outputs allocated there."""
    x = _cuda(_inputs(1, 2, 700, 15))
    want = cwl.gated_scan_backward(x["do"], x["q"], x["k"], x["v"], x["g"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [cwl.gated_scan_backward(x["do"], x["q"], x["k"], x["v"], x["g"], stream=s) for _ in range(3)]
    b = [cwl.gated_scan_backward(x["do"], x["q"], x["k"], x["v"], x["g"]) for _ in range(3)]
    torch.cuda.synchronize()
    for got in a + b:
        assert all(torch.equal(p, r) for p, r in zip(got[:4], want[:4]))


def test_refusals(cwl):
    x = _cuda(_inputs(2, 2, 8, 16))
    q, k, v, g = x["q"], x["k"], x["v"], x["g"]
    for bad, word in (((q.float(), k, v, g), "q"), ((q, k[:, :1], v, g), "k"), ((q, k, v[..., :32], g), "v"),
                      ((q, k, v, g.bfloat16()), "g"), ((q.cpu(), k, v, g), "q"),
                      ((q.transpose(2, 3).contiguous().transpose(2, 3), k, v, g), "q")):
        with pytest.raises(ValueError, match=word):
            cwl.gated_scan(*bad)
    with pytest.raises(ValueError, match="initial"):
        cwl.gated_scan(q, k, v, g, initial=x["S0"].transpose(2, 3))
    odd = torch.zeros((2, 2, 8, 68), device="cuda", dtype=torch.bfloat16)[..., :64]
    with pytest.raises(cwl.TTTError, match="16-byte"):
        cwl.gated_scan(odd, k, v, g)
    one = torch.zeros((2, 1, 8, 64), device="cuda", dtype=torch.bfloat16).expand(2, 2, 8, 64)
    with pytest.raises(cwl.TTTError, match="overlap"):
        cwl.gated_scan(q, k, v, g, out=one)
    with pytest.raises(ValueError, match="state"):
        cwl.gated_scan_step(None, q[:, :, 0], k[:, :, 0], v[:, :, 0], g[:, :, 0])

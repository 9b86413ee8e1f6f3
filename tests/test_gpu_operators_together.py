"""The operators as one layer uses them, next to the scans: queries and keys from a projection through
qk_norm_rope into the TTT-Linear scan and the gated scan, and the feed-forward block's output into the
In-Place scan, forward and back, captured into a graph as a whole.

Each stage is compared on the stage before's own output, so the tolerances are those of the stages."""

import numpy as np
import pytest
import torch

from oracle import inplace as oinp
from oracle import linear as olin
from oracle import operators as op
from tests._util import rel_err, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


B, T, H, D = 2, 192, 3, 64


def _projection(seed):
    r = torch.Generator().manual_seed(seed)
    x = torch.randn((B, T, 3 * H, D), generator=r).bfloat16().cuda()  # queries, keys, values of each token
    w = [(1 + 0.1 * torch.randn(D, generator=r)).cuda() for _ in range(2)]
    return [x[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3)], w


def test_norm_rope_into_the_scans(cwl):
    (q, k, v), w = _projection(1)
    freqs, magnitude = cwl.rope_frequencies(D, scaling="yarn", factor=4.0, trained=4096)
    how = dict(freqs=freqs, magnitude=magnitude, norm="rms", q_weight=w[0], k_weight=w[1], position0=700)
    Q, K = cwl.qk_norm_rope(q, k, **how)
    # Rounded once each from fp32: 2^-8 of the value, which is below 2^-7 of the largest.
    pos = np.broadcast_to(700 + np.arange(T), (B, T))
    ref = op.norm_rope(to_np(q), pos, to_np(freqs), magnitude, "rms", 1e-6, "half", to_np(w[0]))
    assert rel_err(Q, ref) < 2.0 ** -7

    # Into the TTT-Linear scan (dense values; keys scaled to unit length as its step size wants).
    _, Ku = cwl.qk_norm_rope(None, K, norm="l2")
    V = v.contiguous()
    W0 = torch.zeros((B, H, D, D), device="cuda")
    st = cwl.FastWeightState(cwl.config("linear", batch=B, heads=H, chunk=16, eta=1.0), W0)
    O = torch.empty_like(Q)
    st.chunk_scan(Ku, V, Q, out=O)
    torch.cuda.synchronize()
    st.poll()
    Oref, _, _ = olin.ttt_linear_scan(Ku.cpu(), V.cpu(), Q.cpu(), W0.cpu(), 1.0, 16)
    assert rel_err(O, Oref) < 2e-2  # the scan's own tolerance
    st.close()

    # And into the gated scan, values as the projection left them.
    g = torch.nn.functional.logsigmoid(torch.randn((B, T, H), device="cuda") + 4).transpose(1, 2)
    o, S = cwl.gated_scan(Q, K, v, g, scale=D ** -0.5)
    ro, rS, _ = op.gated_scan(to_np(Q), to_np(K), to_np(v), to_np(g), D ** -0.5)
    ao, aS, _ = op.gated_scan(np.abs(to_np(Q)), np.abs(to_np(K)), np.abs(to_np(v)), to_np(g), D ** -0.5)
    assert np.all(np.abs(to_np(o) - ro) <= 2.0 ** -8 * (np.abs(ro) + ao) + 1e-4 * ao)
    assert np.all(np.abs(to_np(S) - rS) <= 2.0 ** -14 * aS)

    # One more token, from the state the scan left.
    more = torch.randn((B, H, D), device="cuda").bfloat16()
    step = cwl.gated_scan_step(S, more, more, more, g[:, :, 0], scale=D ** -0.5)
    m = to_np(more)
    S1 = np.exp(to_np(g[:, :, 0]))[..., None, None] * rS + m[..., :, None] * m[..., None, :]
    assert rel_err(step, D ** -0.5 * np.einsum("bha,bhac->bhc", m, S1)) < 2.0 ** -7


def test_gradients_through_the_layer(cwl):
    """The gradient of <dO, o> in the projection, through the gated scan and the norm, against the
    oracles' chain, and against differences of the oracles along one direction."""
    (q, k, v), w = _projection(2)
    freqs, _ = cwl.rope_frequencies(D)
    how = dict(freqs=freqs, norm="rms", q_weight=w[0], k_weight=w[1])
    g = torch.nn.functional.logsigmoid(torch.randn((B, H, T), device="cuda") + 3)
    dO = torch.randn((B, H, T, D), device="cuda").bfloat16()
    Q, K = cwl.qk_norm_rope(q, k, **how)
    dQ, dK, dv, dg, none = cwl.gated_scan_backward(dO, Q, K, v, g, scale=D ** -0.5)
    assert none is None
    dq, dk, dwq, dwk = cwl.qk_norm_rope_backward(dQ, dK, q, k, **how)

    pos = np.broadcast_to(np.arange(T), (B, T))
    f, wq, wk = to_np(freqs), to_np(w[0]), to_np(w[1])
    q0, k0, v0, g0, d0 = (to_np(t) for t in (q, k, v, g, dO))
    rQ, rK = op.norm_rope(q0, pos, f, weight=wq), op.norm_rope(k0, pos, f, weight=wk)
    rdQ, rdK, rdv, rdg, _ = op.gated_scan_backward(d0, rQ, rK, v0, g0, D ** -0.5)
    rdq, rdwq = op.norm_rope_backward(rdQ, q0, pos, f, weight=wq)
    rdk, rdwk = op.norm_rope_backward(rdK, k0, pos, f, weight=wk)
    # Q and K, one factor of each product, dQ and dK and the results are rounded to bf16: at most five
    # roundings of 2^-8 in a row, with signs of their own, so that as a whole they stay below their sum.
    for got, want in ((dq, rdq), (dk, rdk), (dv, rdv), (dg, rdg), (dwq, rdwq), (dwk, rdwk)):
        got = to_np(got)
        assert np.linalg.norm(got - want) <= 5 * 2.0 ** -8 * np.linalg.norm(want)

    r = np.random.default_rng(3)
    h = 1e-5
    along = [r.standard_normal(t.shape) for t in (q0, k0, v0, g0)]

    def loss(s):
        Qs, Ks = op.norm_rope(q0 + s * along[0], pos, f, weight=wq), op.norm_rope(k0 + s * along[1], pos, f, weight=wk)
        return np.sum(op.gated_scan(Qs, Ks, v0 + s * along[2], g0 + s * along[3], D ** -0.5)[0] * d0)

    slope = (loss(h) - loss(-h)) / (2 * h)
    parts = [np.sum(to_np(d) * a) for d, a in zip((dq, dk, dv, dg), along)]
    size = np.sqrt(sum(np.sum(to_np(d) ** 2) for d in (dq, dk, dv, dg)))
    # The directions are independent normal: an error e in the gradient moves the slope by |e| or so; six
    # times that, and the differences' own h²  of the third derivative.
    assert abs(sum(parts) - slope) <= 6 * 5 * 2.0 ** -8 * size


def test_feed_forward_into_the_in_place_scan(cwl):
    r = torch.Generator().manual_seed(4)
    d, f, tokens = 256, 384, 512
    x = torch.randn((tokens, d), generator=r).bfloat16().cuda()
    wg, wu = ((torch.randn((f, d), generator=r) * d ** -0.5).bfloat16().cuda() for _ in range(2))
    W0 = (torch.randn((d, f), generator=r) * f ** -0.5).cuda()
    Vhat = torch.randn((tokens, d), generator=r).bfloat16().cuda()
    Z = cwl.gated_ffn(x, wg, wu)
    rz, _, _ = op.gated_ffn(to_np(x), to_np(wg), to_np(wu))
    assert rel_err(Z, rz) < 2.0 ** -7
    eta = 1e-3
    st = cwl.FastWeightState(cwl.config("inplace", io_dtype=1, d_key=f, d_val=d, chunk=128, eta=eta), W0)
    O = torch.empty((tokens, d), device="cuda", dtype=torch.bfloat16)
    st.chunk_scan(Z, Vhat, out=O)
    torch.cuda.synchronize()
    st.poll()
    Oref, _ = oinp.inplace_scan(Z.cpu(), Vhat.cpu(), W0.cpu(), eta, 128)
    assert rel_err(O, Oref) < 2e-2  # the scan's own tolerance
    st.close()


def test_a_layer_in_one_graph(cwl):
    """The whole chain captured once and replayed on new tokens, the state carried on the device."""
    xs = [_projection(s)[0] for s in (5, 6)]
    w = _projection(7)[1]
    freqs, _ = cwl.rope_frequencies(D)
    g = torch.nn.functional.logsigmoid(torch.randn((B, H, T), device="cuda") + 3)
    buf = [t.clone() for t in xs[0]]
    pos = torch.arange(T, device="cuda")
    S = torch.zeros((B, H, D, D), device="cuda")

    def layer(b, S, pos):
        Q, K = cwl.qk_norm_rope(b[0], b[1], positions=pos, freqs=freqs, q_weight=w[0], k_weight=w[1])
        return cwl.gated_scan(Q, K, b[2], g, initial=S, final=S)[0]

    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o = layer(buf, S, pos)
    S.zero_()
    want_S, got = torch.zeros_like(S), []
    for i, x in enumerate(xs):
        for b, t in zip(buf, x):
            b.copy_(t)
        pos.copy_(torch.arange(i * T, (i + 1) * T))
        gr.replay()
        torch.cuda.synchronize()
        want = layer(x, want_S, torch.arange(i * T, (i + 1) * T, device="cuda"))
        assert torch.equal(o, want) and torch.equal(S, want_S)


def test_numbers_given_as_tensors_are_read_at_every_call(cwl):
    """A scale, epsilon or magnitude held in a tensor may change between calls."""
    (q, k, v), _ = _projection(8)
    g = torch.zeros((B, H, T), device="cuda")
    scale, eps = torch.tensor(1.0), torch.tensor(1e-6)
    a, _ = cwl.gated_scan(q, k, v, g, scale=scale)
    x, _ = cwl.qk_norm_rope(q, None, eps=eps)
    scale.fill_(2.0), eps.fill_(3.0)
    b, _ = cwl.gated_scan(q, k, v, g, scale=scale)
    y, _ = cwl.qk_norm_rope(q, None, eps=eps)
    assert torch.equal(b, cwl.gated_scan(q, k, v, g, scale=2.0)[0]) and not torch.equal(a, b)
    assert torch.equal(y, cwl.qk_norm_rope(q, None, eps=3.0)[0]) and not torch.equal(x, y)


_FIRST_CALLS = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import chunked_weight_layers_b200 as cwl
r = torch.Generator().manual_seed(1)
rnd = lambda *s: torch.randn(s, generator=r).bfloat16().cuda()
q, k, v, do = (rnd(1, 2, 900, 64) for _ in range(4))
g = -torch.rand((1, 2, 900), generator=r).cuda()
f, _ = cwl.rope_frequencies(64)
S = torch.zeros((1, 2, 64, 64), device="cuda")
x, wg, wu, dz = rnd(300, 128), rnd(200, 128), rnd(200, 128), rnd(300, 200)
torch.cuda.synchronize()
def calls():
    Q, K = cwl.qk_norm_rope(q, k, freqs=f)
    return [*cwl.gated_scan(Q, K, v, g), *cwl.gated_scan_backward(do, Q, K, v, g)[:4],
            *cwl.qk_norm_rope_backward(do, do, q, k, freqs=f)[:2], cwl.gated_ffn(x[:3], wg, wu),
            *cwl.gated_ffn(x, wg, wu, save=True), *cwl.gated_ffn_backward(dz, x, wg, wu, dz, dz)]
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    got = calls()
    step = cwl.gated_scan_step(S, q[:, :, 0], k[:, :, 0], v[:, :, 0], g[:, :, 0])
gr.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
assert S.abs().sum() > 0 and torch.isfinite(step.float()).all()
del gr
print("captured")
"""


def test_first_calls_of_a_process_are_captured(tmp_path):
    """Nothing needs a call outside a capture first: a new process captures each operator's first call."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-500:] + r.stderr[-1500:]

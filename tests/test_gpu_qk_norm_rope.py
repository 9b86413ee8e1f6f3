"""GPU parity of the norm of queries and keys with rotary positions, and its gradients.

Tolerances: the arithmetic is fp32 (norms, sines and sums to some 2^-21 of the row's largest terms;
2^-18 is asked), a bf16 output is rounded once, 2^-8 of the value. Gains' gradients are sums of fp32
products: 2^-18 of the sum of absolute values."""

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


def _case(B, T, hq, hk, D, rot, seed, dtype=torch.bfloat16, start=0, norm="rms"):
    r = torch.Generator().manual_seed(seed)
    q, dq = (torch.randn((B, hq, T, D), generator=r).to(dtype) for _ in range(2))
    k, dk = (torch.randn((B, hk, T, D), generator=r).to(dtype) for _ in range(2))
    pos = start + torch.randint(0, 3000, (B, T), generator=r)
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1)) if rot else None
    w = [1 + 0.2 * torch.randn(D, generator=r) for _ in range(2)] if norm == "rms" else [None, None]
    return q, k, dq, dk, pos, f, w


def _c(t):
    return None if t is None else t.cuda()


def _row_max(x):
    return np.max(np.abs(x), -1, keepdims=True)


def _near(got, ref, slack, dtype, name):
    ref = np.asarray(ref)
    bound = slack + (2.0 ** -8 * np.abs(ref) if dtype is torch.bfloat16 else 0)
    err = np.abs(to_np(got) - ref)
    assert np.all(err <= bound), f"{name}: {np.max(err / np.maximum(bound, 1e-300)):.3g} x the bound"


CASES = [  # B, T, q heads, k heads, width, rot
    (1, 1, 1, 1, 64, 64), (2, 5, 3, 1, 64, 32), (1, 33, 8, 2, 128, 64), (3, 7, 2, 2, 96, 96), (1, 9, 1, 4, 96, 48),
    (2, 3, 2, 1, 256, 256), (1, 4, 2, 2, 8, 0), (1, 130, 4, 4, 64, 0), (2, 2, 1, 1, 48, 16), (1, 3, 2, 1, 200, 176),
]


@pytest.mark.parametrize("B,T,hq,hk,D,rot", CASES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parity(cwl, B, T, hq, hk, D, rot, layout, norm, dtype):
    q, k, dq, dk, pos, f, w = _case(B, T, hq, hk, D, rot, D + rot + T, dtype, norm=norm)
    how = dict(magnitude=1.25, norm=norm, eps=1e-5, layout=layout)
    gpu = dict(how, positions=pos.cuda(), freqs=_c(f), q_weight=_c(w[0]), k_weight=_c(w[1]))
    got = cwl.qk_norm_rope(q.cuda(), k.cuda(), **gpu)
    back = cwl.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), **gpu)
    for i, (x, dy, name) in enumerate(((q, dq, "q"), (k, dk, "k"))):
        one = dict(how, weight=None if w[i] is None else to_np(w[i]))
        fr = None if f is None else to_np(f)
        ref = op.norm_rope(to_np(x), pos.numpy(), fr, **one)
        _near(got[i], ref, 2.0 ** -18 * _row_max(ref), dtype, name)
        dx, dw = op.norm_rope_backward(to_np(dy), to_np(x), pos.numpy(), fr, **one)
        # dx is a difference: its terms are as large as the rotated gradient over the norm.
        size = op._norm(to_np(x), norm, 1e-5)
        terms = 2 * _row_max(to_np(dy)) * 1.25 * (1 if w[i] is None else float(w[i].abs().max())) / size
        terms = terms * (1 + _row_max(to_np(x) / size) ** 2)
        _near(back[i], dx, 2.0 ** -18 * terms, dtype, "d" + name)
        if dw is None:
            assert back[2 + i] is None
        else:
            most = np.sum(np.abs(to_np(x) / size) * 2 * 1.25 * _row_max(to_np(dy)), axis=(0, 1, 2))
            _near(back[2 + i], dw, 2.0 ** -18 * most, torch.float32, "dw" + name)


def test_views_of_a_projection_and_in_place(cwl):
    """Token-major views of one projection are read as they lie; outputs may be the inputs."""
    B, T, hq, hk, D = 2, 19, 4, 2, 64
    r = torch.Generator().manual_seed(1)
    x = torch.randn((B, T, hq + hk + 1, D), generator=r).bfloat16().cuda()
    q, k = x[:, :, :hq].transpose(1, 2), x[:, :, hq:hq + hk].transpose(1, 2)
    f, m = cwl.rope_frequencies(64)
    assert m == 1.0
    want = cwl.qk_norm_rope(q.contiguous(), k.contiguous(), freqs=f, position0=11)
    got = cwl.qk_norm_rope(q, k, freqs=f, position0=11)
    assert got[0].is_contiguous() and all(torch.equal(a, b) for a, b in zip(got, want))
    dy = torch.randn_like(q), torch.randn_like(k)
    a = cwl.qk_norm_rope_backward(*dy, q, k, freqs=f, position0=11)
    b = cwl.qk_norm_rope_backward(*(t.contiguous() for t in dy), q.contiguous(), k.contiguous(), freqs=f, position0=11)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    last = x[:, :, -1].clone()
    cwl.qk_norm_rope(q, k, freqs=f, position0=11, out=(q, k))
    assert all(torch.equal(s, t) for s, t in zip((q, k), want)) and torch.equal(x[:, :, -1], last)


def test_one_side_alone(cwl):
    q, k, dq, dk, pos, f, w = _case(2, 6, 3, 2, 64, 64, 3)
    args = dict(positions=pos.cuda(), freqs=f.cuda())
    both = cwl.qk_norm_rope(q.cuda(), k.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda(), **args)
    qo, none = cwl.qk_norm_rope(q.cuda(), None, q_weight=w[0].cuda(), **args)
    assert none is None and torch.equal(qo, both[0])
    none, ko = cwl.qk_norm_rope(None, k.cuda(), k_weight=w[1].cuda(), **args)
    assert none is None and torch.equal(ko, both[1])
    full = cwl.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda(), **args)
    part = cwl.qk_norm_rope_backward(None, dk.cuda(), None, k.cuda(), k_weight=w[1].cuda(), **args)
    assert part[0] is None and part[2] is None and torch.equal(part[1], full[1])
    assert torch.allclose(part[3], full[3], rtol=1e-5, atol=1e-5)


def test_far_positions(cwl):
    """Positions where a 32-bit angle has lost its fraction, and negative ones."""
    q, k, _, _, pos, f, _ = _case(1, 40, 2, 1, 64, 64, 4, torch.float32, norm="none")
    for start in (10 ** 6, 2 ** 31 + 5, -10 ** 7):
        p = pos + start
        got = cwl.qk_norm_rope(q.cuda(), k.cuda(), positions=p.cuda(), freqs=f.cuda(), norm="none")
        ref = op.norm_rope(to_np(q), p.numpy(), to_np(f), norm="none")
        # The 64-bit angle itself is off by 2^-53 of it on either side.
        _near(got[0], ref, (2.0 ** -18 + 4 * 2.0 ** -53 * abs(start)) * _row_max(ref), torch.float32, "q")
    a = cwl.qk_norm_rope(q.cuda(), k.cuda(), position0=100000, freqs=f.cuda())
    b = cwl.qk_norm_rope(q.cuda(), k.cuda(), positions=torch.arange(100000, 100040).cuda(), freqs=f.cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_of_zeros_and_infinities(cwl):
    x = torch.zeros((1, 1, 4, 64), device="cuda", dtype=torch.bfloat16)
    x[0, 0, 1, 3] = float("inf")
    x[0, 0, 2, 3] = float("nan")
    x[0, 0, 3] = 1
    f, _ = cwl.rope_frequencies(32)
    y, _ = cwl.qk_norm_rope(x, None, freqs=f, norm="rms")
    assert torch.all(y[0, 0, 0] == 0) and torch.isnan(y[0, 0, 2]).any()
    assert torch.isfinite(y[0, 0, 3]).all()
    # Without norm, values past the rotated part pass through as they are.
    x[0, 0, 0, 40] = float("inf")
    y, _ = cwl.qk_norm_rope(x, None, freqs=f, norm="none")
    assert torch.equal(y[0, 0, 0], x[0, 0, 0])


def test_no_epsilon(cwl):
    """eps 0: finite rows stay finite, and so do the gains' gradients with heads left over."""
    q, k, dq, dk, pos, f, w = _case(1, 3, 3, 1, 64, 64, 8)
    args = dict(positions=pos.cuda(), freqs=f.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda(), eps=0.0)
    got = cwl.qk_norm_rope(q.cuda(), k.cuda(), **args)
    ref = op.norm_rope(to_np(q), pos.numpy(), to_np(f), eps=0.0, weight=to_np(w[0]))
    _near(got[0], ref, 2.0 ** -18 * _row_max(ref), torch.bfloat16, "q")
    back = cwl.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), **args)
    assert all(torch.isfinite(t).all() for t in back)


def test_many_rows_and_repeated_bits(cwl):
    """More rows than the GPU holds threads for, against torch in 64 bits; the gains' gradients come
    out the same every time."""
    B, T, H, D = 2, 3001, 12, 64
    q, k, dq, dk, pos, f, w = _case(B, T, H, H, D, 64, 5)
    args = dict(positions=pos.cuda(), freqs=f.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda())
    got = cwl.qk_norm_rope(q.cuda(), k.cuda(), **args)
    ref = op.norm_rope(to_np(q), pos.numpy(), to_np(f), weight=to_np(w[0]))
    _near(got[0], ref, 2.0 ** -18 * _row_max(ref), torch.bfloat16, "q")
    a = cwl.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), **args)
    b = cwl.qk_norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), **args)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    _, dw = op.norm_rope_backward(to_np(dk), to_np(k), pos.numpy(), to_np(f), weight=to_np(w[1]))
    most = np.sum(np.abs(to_np(k)) * 4, axis=(0, 1, 2))
    _near(a[3], dw, 2.0 ** -18 * most, torch.float32, "dk_weight")


def test_frequencies(cwl):
    f, m = cwl.rope_frequencies(64, 500000.0)
    i = torch.arange(32, dtype=torch.float64)
    assert torch.allclose(f.cpu(), 500000.0 ** (-i / 32), rtol=1e-14)
    lin, _ = cwl.rope_frequencies(64, 500000.0, "linear", 8.0)
    assert torch.allclose(lin * 8, f, rtol=1e-14)
    ntk, _ = cwl.rope_frequencies(64, scaling="ntk", factor=4.0)
    plain, _ = cwl.rope_frequencies(64)
    # The first pair keeps its frequency, the last is divided by the factor.
    assert ntk[0] == 1 and abs(float(ntk[-1] * 4 / plain[-1]) - 1) < 1e-12
    yarn, m = cwl.rope_frequencies(64, scaling="yarn", factor=4.0, trained=32768)
    assert abs(m - (0.1 * np.log(4.0) + 1)) < 1e-6
    ratio = (yarn / plain).cpu()
    assert ratio[0] == 1 and abs(float(ratio[-1]) - 0.25) < 1e-12 and torch.all(ratio[1:] <= ratio[:-1] + 1e-12)


def test_no_tokens(cwl):
    q = torch.zeros((2, 3, 0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    assert cwl.qk_norm_rope(q, q, q_weight=w)[0].shape == q.shape
    back = cwl.qk_norm_rope_backward(q, q, q, q, q_weight=w, k_weight=w)
    assert torch.all(back[2] == 0) and torch.all(back[3] == 0)


def test_captured_and_replayed(cwl):
    q, k, dq, dk, pos, f, w = _case(2, 50, 4, 2, 64, 64, 6)
    b = [t.cuda() for t in (q, k, dq, dk, pos)]
    args = dict(freqs=f.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda())
    call = lambda: (*cwl.qk_norm_rope(b[0], b[1], positions=b[4], **args),  # noqa: E731
                    *cwl.qk_norm_rope_backward(b[2], b[3], b[0], b[1], positions=b[4], **args))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    b[0].mul_(2), b[2].add_(1), b[4].add_(77)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, call()))


def test_refusals(cwl):
    q, k, _, _, pos, f, w = _case(2, 6, 3, 2, 64, 64, 7)
    q, k, pos, f, w = q.cuda(), k.cuda(), pos.cuda(), f.cuda(), w[0].cuda()
    for args, how, word in (((q, k.float()), {}, "k"), ((q.cpu(), k), {}, "q"), ((q, k[:, :, :5]), {}, "k"),
                            ((q, k), dict(positions=pos.int()), "positions"), ((q, k), dict(positions=pos[:, :5]), "positions"),
                            ((q, k), dict(freqs=f.float()), "freqs"), ((q, k), dict(q_weight=w[:32]), "q_weight"),
                            ((q, k), dict(norm="layer"), "norm"), ((q, k), dict(layout="third"), "layout"),
                            ((None, None), {}, "k")):
        with pytest.raises(ValueError, match=word):
            cwl.qk_norm_rope(*args, **how)
    for how, word in ((dict(norm="l2", q_weight=w), "RMS"), (dict(freqs=f[:20]), "multiple of 16"), (dict(eps=-1.0), "eps"),
                      (dict(freqs=torch.ones(40, device="cuda", dtype=torch.float64)), "multiple of 16")):
        with pytest.raises(cwl.TTTError, match=word):
            cwl.qk_norm_rope(q, k, **how)
    with pytest.raises(cwl.TTTError, match="overlap"):
        cwl.qk_norm_rope(q, k, out=(q[:, :1].expand(2, 3, 6, 64), k))
    with pytest.raises(cwl.TTTError, match="factor"):
        cwl.rope_frequencies(64, factor=0.5)

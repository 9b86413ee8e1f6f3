"""The norm's backward pass where a token's heads are cut into two parts and where they are not: the
gradients of a token do not depend on how many tokens the call has, nor on what other heads it has."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


@pytest.mark.parametrize("T", [4737, 9473, 10000, 14300, 19000, 33200, 57000])
@pytest.mark.parametrize("hq,hk", [(8, 8), (7, 6), (4, 4)])
def test_parts_of_the_heads(cwl, T, hq, hk):
    r = torch.Generator(device="cuda").manual_seed(T + hq)
    q, k, dq, dk = (torch.randn((1, h, T, 64), generator=r, device="cuda").bfloat16() for h in (hq, hk, hq, hk))
    w = [1 + 0.1 * torch.randn(64, generator=r, device="cuda") for _ in range(2)]
    freqs, _ = cwl.rope_frequencies(64)
    how = dict(freqs=freqs, q_weight=w[0], k_weight=w[1])
    got = cwl.qk_norm_rope_backward(dq, dk, q, k, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, cwl.qk_norm_rope_backward(dq, dk, q, k, **how)))
    # Stretches of 500 tokens and single heads, which are never cut, row by row the same bits.
    at = [0, T // 2, T - 500]
    gains = [torch.zeros(64, device="cuda", dtype=torch.float64) for _ in range(2)]
    for i, (x, dx, out, h) in enumerate(((q, dq, got[0], hq), (k, dk, got[1], hk))):
        for t in at:
            e = slice(t, t + 500)
            part = cwl.qk_norm_rope_backward(dx[:, h - 1:, e], None, x[:, h - 1:, e], None, position0=t, freqs=freqs, q_weight=w[i])
            assert torch.equal(part[0], out[:, h - 1:, e])
        # The gains: the sum over all rows in 64 bits of the turned-back gradient times the unit row. Each
        # term is fp32 with some 16 roundings, and a CTA's sums follow one another at most 2 · 5 rounds of
        # eight rows long before the double sum: below 2^-17 of the terms' size.
        angle = torch.arange(T, device="cuda").double()[:, None] * freqs
        c, s = torch.cos(angle), torch.sin(angle)
        d = dx[0].double()
        back = torch.cat([d[..., :32] * c + d[..., 32:] * s, d[..., 32:] * c - d[..., :32] * s], -1)
        n = x[0].double()
        n = n / (n.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        gains[i] = (back * n).sum((0, 1))
        size = (back.abs() * n.abs()).sum((0, 1))
        assert torch.all((got[2 + i].double() - gains[i]).abs() <= 2.0 ** -17 * size)

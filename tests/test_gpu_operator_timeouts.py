"""Bounded waits of the operators around the scans that run out, without a GPU fault.

TTT_OPT_INJECT_STALL makes the next call never load its second tile (or k-block), so that the kernels'
waits for it give up after the limit (5 ms here), wind down and return. The call without a status word
is then reported by poll_operators, once; one with a status word reports there and nowhere else; and the
same call made again gives the same bits as before, so the kernels had freed their tensor memory."""

import pytest
import torch

pytestmark = pytest.mark.gpu
LIMIT_NS = 5_000_000


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


@pytest.fixture()
def short_limit(cwl):
    lib = cwl.abi.load()
    cwl.abi.check(lib.ttt_operators_set_option(cwl.abi.TTT_OPT_WAIT_LIMIT_NS, LIMIT_NS))
    yield lambda: cwl.abi.check(lib.ttt_operators_set_option(cwl.abi.TTT_OPT_INJECT_STALL, 1))
    cwl.abi.check(lib.ttt_operators_set_option(cwl.abi.TTT_OPT_INJECT_STALL, 0))
    cwl.abi.check(lib.ttt_operators_set_option(cwl.abi.TTT_OPT_WAIT_LIMIT_NS, 2_000_000_000))


def _scan(cwl, H, T, back):
    r = torch.Generator(device="cuda").manual_seed(T)
    q, k, v, do = (torch.randn((1, H, T, 64), generator=r, device="cuda").bfloat16() for _ in range(4))
    g = -0.1 * torch.rand((1, H, T), generator=r, device="cuda")
    if back:
        return lambda **how: cwl.gated_scan_backward(do, q, k, v, g, **how)[:4]
    return lambda **how: cwl.gated_scan(q, k, v, g, **how)


def _ffn(cwl, T, d, f, back):
    r = torch.Generator(device="cuda").manual_seed(T + f)
    x, wg, wu, z = (torch.randn(s, generator=r, device="cuda").bfloat16() for s in ((T, d), (f, d), (f, d), (T, f)))
    if back:
        return lambda **how: cwl.gated_ffn_backward(z, x, wg, wu, z, z, **how)
    return lambda **how: cwl.gated_ffn(x, wg, wu, save=True, **how)


CASES = {
    "scan": lambda cwl: _scan(cwl, 2, 300, False),
    "scan in segments": lambda cwl: _scan(cwl, 2, 1300, False),
    "scan backward": lambda cwl: _scan(cwl, 2, 300, True),
    "scan backward in segments": lambda cwl: _scan(cwl, 2, 1300, True),
    "block, pairs": lambda cwl: _ffn(cwl, 300, 520, 520, False),
    "block, rows": lambda cwl: _ffn(cwl, 40, 264, 9480, False),
    "block backward": lambda cwl: _ffn(cwl, 300, 264, 520, True),
}


@pytest.mark.parametrize("name", CASES)
def test_a_wait_runs_out(cwl, short_limit, name):
    call = CASES[name](cwl)
    want = call()
    cwl.poll_operators()
    short_limit()
    call()
    with pytest.raises(cwl.TTTError, match="wait ran out") as e:
        cwl.poll_operators()
    assert e.value.status == cwl.abi.TTT_ERR_TIMEOUT
    cwl.poll_operators()  # the poll that told it cleared it
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    status = torch.zeros(1, device="cuda", dtype=torch.int32)
    short_limit()
    call(status=status)
    assert int(status) == cwl.abi.TTT_ERR_TIMEOUT
    cwl.poll_operators()
    assert all(torch.equal(a, b) for a, b in zip(call(status=status), want)) and int(status) == 0


def test_calls_without_a_second_tile_keep_the_injection(cwl, short_limit):
    short_limit()
    few = _ffn(cwl, 8, 264, 520, False)
    few()
    _scan(cwl, 2, 100, False)()
    cwl.poll_operators()
    _scan(cwl, 2, 300, False)()
    with pytest.raises(cwl.TTTError, match="wait ran out"):
        cwl.poll_operators()

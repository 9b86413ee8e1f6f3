"""Refusals of the operators' C entry points, which come before any device call, and the host-side
frequencies: no GPU needed. Addresses here are never dereferenced."""

import ctypes
import math

import pytest

A = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def lib():
    from chunked_weight_layers_b200 import abi, build
    build.build()
    return abi.load()


@pytest.fixture(scope="module")
def abi():
    from chunked_weight_layers_b200 import abi
    return abi


def _message(lib):
    return lib.ttt_last_error_string().decode()


def _qk(abi, **over):
    s = lambda: abi.ttt_strides(2 * 8 * 64, 8 * 64, 64)  # noqa: E731
    d = abi.ttt_qk_desc(1, 1, 2, 2, 64, 64, 1, 0, 1e-6, 1.0, 8, 0, 0, s(), s(), s(), s(), s(), s())
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("over,status,word", [
    (dict(io_dtype=5), 2, "io_dtype"), (dict(batch=-1), 1, "batch"), (dict(q_heads=0, k_heads=0), 1, "heads"),
    (dict(width=12), 2, "width"), (dict(width=264), 2, "width"), (dict(rot=8), 2, "rot"), (dict(rot=80), 2, "rot"),
    (dict(norm=3), 1, "norm"), (dict(layout=2), 1, "layout"), (dict(eps=-1.0), 1, "eps"), (dict(eps=math.nan), 1, "eps"),
    (dict(positions_stride=3), 1, "positions_stride"),
])
def test_qk_sizes(lib, abi, over, status, word):
    d = _qk(abi, **over)
    assert lib.ttt_qk_norm_rope(ctypes.byref(d), A, A, None, None, None, A, A, A, None) == status
    assert word in _message(lib)
    assert lib.ttt_qk_norm_rope_backward(ctypes.byref(d), A, A, A, A, None, None, None, A, A, A, None, None, None, 0, None) == status


def test_qk_pointers(lib, abi):
    d = _qk(abi)
    call = lambda d, *a: lib.ttt_qk_norm_rope(ctypes.byref(d), *a, None)  # noqa: E731
    assert call(d, A + 8, A, None, None, None, A, A, A) == 1 and "q must be" in _message(lib)
    assert call(d, A, None, None, None, None, A, A, A) == 1 and "k and its output" in _message(lib)
    assert call(d, A, A, None, None, None, None, A, A) == 1 and "freqs" in _message(lib)
    assert call(_qk(abi, norm=2), A, A, A, None, None, A, A, A) == 1 and "RMS" in _message(lib)
    assert call(d, A, A, None, None, A + 4, A, A, A) == 1 and "positions" in _message(lib)
    assert call(_qk(abi, q=abi.ttt_strides(-64, 64, 64)), A, A, None, None, None, A, A, A) == 1
    assert call(_qk(abi, q_out=abi.ttt_strides(1024, 512, 32)), A, A, None, None, None, A, A, A) == 1
    assert "overlap" in _message(lib)
    assert call(_qk(abi, q_out=abi.ttt_strides(1024, 512, 68)), A, A, None, None, None, A, A, A) == 1
    assert "16-byte" in _message(lib)
    assert lib.ttt_qk_norm_rope(None, A, A, None, None, None, A, A, A, None) == 1
    # No tokens: nothing is looked at, not even the pointers.
    assert call(_qk(abi, tokens=0), None, None, None, None, None, None, None, None) == 0
    back = lib.ttt_qk_norm_rope_backward
    assert back(ctypes.byref(d), A, A, A, A, None, None, None, A, A, A, A, None, None, 0, None) == 1
    assert "not given" in _message(lib)


def _scan(abi, **over):
    s = lambda: abi.ttt_strides(2 * 8 * 64, 8 * 64, 64)  # noqa: E731
    d = abi.ttt_gated_scan_desc(1, 2, 8, 1.0, s(), s(), s(), s(), abi.ttt_strides(16, 8, 1))
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("over,status,word", [
    (dict(batch=0), 1, "batch"), (dict(heads=-1), 1, "heads"), (dict(tokens=-1), 1, "tokens"),
    (dict(batch=1 << 20, heads=1 << 10), 2, "2^24"), (dict(tokens=1 << 40), 2, "2^30"),
])
def test_scan_sizes(lib, abi, over, status, word):
    d = _scan(abi, **over)
    assert lib.ttt_gated_scan(ctypes.byref(d), A, A, A, A, None, A, None, None, 0, None, None) == status
    assert word in _message(lib)
    assert lib.ttt_gated_scan_backward(ctypes.byref(d), A, A, A, A, A, None, None, A, A, A, A, None, None, 0, None, None) == status
    assert lib.ttt_gated_scan_step(ctypes.byref(d), A, A, A, A, A, A, None) == status
    assert lib.ttt_gated_scan_workspace(ctypes.byref(d)) == 0


def test_scan_pointers(lib, abi):
    d = _scan(abi)
    call = lambda d, *a: lib.ttt_gated_scan(ctypes.byref(d), *a, None, 0, None, None)  # noqa: E731
    assert call(d, None, A, A, A, None, A, None) == 1 and "q must" in _message(lib)
    assert call(d, A, A, A + 2, A, None, A, None) == 1 and "v must" in _message(lib)
    assert call(d, A, A, A, None, None, A, None) == 1 and "g must" in _message(lib)
    assert call(d, A, A, A, A, A + 4, A, None) == 1 and "S0" in _message(lib)
    assert call(d, A, A, A, A, None, None, None) == 1 and "o must" in _message(lib)
    assert call(_scan(abi, o=abi.ttt_strides(0, 0, 64)), A, A, A, A, None, A, None) == 1 and "overlap" in _message(lib)
    assert call(_scan(abi, k=abi.ttt_strides(0, 0, 60)), A, A, A, A, None, A, None) == 1 and "k: strides" in _message(lib)
    for bad, word in ((abi.ttt_strides(0, 0, 0), "token stride 0"), (abi.ttt_strides(1 << 40, 512, 64), "2^39")):
        assert call(_scan(abi, q=bad), A, A, A, A, None, A, None) == 2 and word in _message(lib)
    assert lib.ttt_gated_scan_step(ctypes.byref(d), A, A, A, A, A, A, None) == 1 and "one token" in _message(lib)
    assert lib.ttt_gated_scan(None, A, A, A, A, None, A, None, None, 0, None, None) == 1


@pytest.mark.parametrize("args,status,word", [
    ((A, A, A, -1, 64, 64, 0), 1, "T must"), ((A, A, A, 4, 60, 64, 0), 2, "multiples of 8"),
    ((A, A, A, 4, 64, 0, 0), 2, "multiples of 8"), ((A, A, A, 4, 64, 64, 9), 1, "activation"),
    ((A, A, A, (1 << 24) + 1, 64, 64, 0), 2, "2^24"), ((None, A, A, 4, 64, 64, 0), 1, "X must"),
    ((A, A, A + 8, 4, 64, 64, 0), 1, "Wu must"),
])
def test_ffn(lib, args, status, word):
    assert lib.ttt_gated_ffn(*args, A, None, None, None, None) == status
    assert word in _message(lib)


def test_ffn_pointers(lib):
    assert lib.ttt_gated_ffn(A, A, A, 4, 64, 64, 0, A, A, None, None, None) == 1 and "together" in _message(lib)
    assert lib.ttt_gated_ffn(A, A, A, 4, 64, 64, 0, A, None, None, A + 2, None) == 1 and "status" in _message(lib)
    back = lib.ttt_gated_ffn_backward
    assert back(A, A, A, A, A, A, 4, 64, 64, 0, A, A, None, None, 0, None, None) == 1 and "together" in _message(lib)
    assert back(A, A, A, A, None, A, 4, 64, 64, 0, A, A, A, None, 0, None, None) == 1 and "G must" in _message(lib)
    assert lib.ttt_gated_ffn_backward_workspace(4, 60, 64) == 0


def test_frequencies(lib, abi):
    out, m = (ctypes.c_double * 32)(), ctypes.c_float()
    call = lambda *a: lib.ttt_rope_frequencies(*a, ctypes.addressof(out), ctypes.addressof(m))  # noqa: E731
    assert call(64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0) == 0 and m.value == 1.0
    plain = list(out)
    assert all(abs(x - 10000.0 ** (-i / 32)) <= 1e-15 for i, x in enumerate(plain))
    assert call(64, 10000.0, 1, 4.0, 0.0, 0.0, 0.0) == 0 and list(out) == [x / 4 for x in plain]
    assert call(64, 10000.0, 3, 4.0, 32768.0, 32.0, 1.0) == 0 and abs(m.value - (1 + 0.1 * math.log(4))) < 1e-6
    assert out[0] == plain[0] and abs(out[31] - plain[31] / 4) < 1e-18
    for bad in ((63, 1e4, 0, 1.0, 0, 0, 0), (0, 1e4, 0, 1.0, 0, 0, 0), (64, 1.0, 0, 1.0, 0, 0, 0), (64, 1e4, 0, 0.5, 0, 0, 0),
                (64, 1e4, 9, 1.0, 0, 0, 0), (2, 1e4, 2, 2.0, 0, 0, 0), (64, 1e4, 3, 2.0, 0.0, 32.0, 1.0),
                (64, 1e4, 3, 2.0, 100.0, 1.0, 1.0), (64, math.inf, 0, 1.0, 0, 0, 0)):
        assert call(*bad) == 1, bad
    assert lib.ttt_rope_frequencies(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None, None) == 1


def test_binding_refuses_host_tensors():
    import torch
    import chunked_weight_layers_b200 as cwl
    if not torch.cuda.is_available():
        # Without a device every call fails before it reaches the library.
        q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
        with pytest.raises(Exception):
            cwl.gated_scan(q, q, q, torch.zeros((1, 1, 2)))
        with pytest.raises(Exception):
            cwl.gated_ffn(q[0, 0], q[0, 0], q[0, 0])


def test_operator_options(lib, abi):
    call = lib.ttt_operators_set_option
    for option, bad in ((abi.TTT_OPT_WAIT_LIMIT_NS, 999_999), (abi.TTT_OPT_WAIT_LIMIT_NS, 60_000_000_001),
                        (abi.TTT_OPT_INJECT_STALL, 2), (abi.TTT_OPT_SM_PAIR, 0), (0, 0)):
        assert call(option, bad) == abi.TTT_ERR_INVALID_ARG
    assert call(abi.TTT_OPT_WAIT_LIMIT_NS, 2_000_000_000) == 0 and call(abi.TTT_OPT_INJECT_STALL, 0) == 0

"""The gated feed-forward block's form with the weights as rows, with GELU and without kept
pre-activations. Tolerances as derived in test_gpu_gated_ffn.py."""

import pytest
import torch

import tests.test_gpu_gated_ffn as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cwl():
    from chunked_weight_layers_b200 import build
    build.build()
    import chunked_weight_layers_b200 as cwl
    return cwl


@pytest.mark.parametrize("T,d,f", [(9, 1032, 9480), (17, 72, 9480), (33, 200, 9608), (128, 64, 20000), (160, 136, 9480)])
def test_weights_as_rows_with_gelu(cwl, T, d, f):
    x, wg, wu, _ = base._case(T, d, f, T + d + f)
    c = [t.cuda() for t in (x, wg, wu)]
    z, g, u = cwl.gated_ffn(*c, activation="gelu", save=True)
    base._check_forward((z, g, u), x, wg, wu, "gelu")
    assert torch.equal(z, cwl.gated_ffn(*c, activation="gelu"))

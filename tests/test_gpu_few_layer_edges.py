"""GPU checks of the few-token layer where nothing is chosen."""
import pytest
import torch

from tests.test_gpu_few_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,S", [(1, 0), (3, 0), (1, 1), (16, 0)])
def test_no_token_has_an_expert(moe, T, S, fp8):
    """NaN in every hidden row: no key is a number, no expert is chosen.  The
    output is written all the same (zeros without shared experts, NaN with
    them), the status word reports it, and the next call is as it should be."""
    L = Layer(moe, T, 256, 16, 144, 2, S, 128, fp8, seed=17)
    want = L.run()
    good = L.h.clone()
    L.h[:, 5] = float("nan")
    for _ in range(3):
        out, idx, w = L.run()                    # (run() fills the output beforehand)
        assert moe.moe_get_device_status(L.ws) == moe.MOE_ERR_NONFINITE
        assert bool(torch.isnan(out).all()) if S else bool((out == 0).all())
        assert int(moe.moe_ws_touched_experts(L.ws, L.d)) == 0
        assert not bool(moe.moe_ws_expert_counts(L.ws, L.d).any())
    L.h.copy_(good)
    assert all(torch.equal(a, b) for a, b in zip(L.run(), want))
    assert moe.moe_get_device_status(L.ws) == 0


def test_a_bias_that_is_not_a_number(moe):
    """The same from the bias, with finite hidden rows; then a single expert is left."""
    L = Layer(moe, 4, 128, 8, 64, 2, 0, 16, False, seed=18)
    L.bias[:] = float("nan")
    assert bool((L.run()[0] == 0).all())
    assert moe.moe_get_device_status(L.ws) == moe.MOE_ERR_NONFINITE
    L.bias[3] = 0.0
    out, idx, _ = L.run()
    assert moe.moe_get_device_status(L.ws) == moe.MOE_ERR_NONFINITE
    assert bool((idx[:, 0] == 3).all()) and bool(torch.isfinite(out).all()) and bool((out != 0).any())

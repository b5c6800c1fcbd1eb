"""GPU checks of the few-token layer where the hand-over of activations between
its two products is tightest: narrow gate/up tiles (16 or 32 features, so that
three or two of a CTA's four epilogue warps hold no rows and run ahead of the
others), two or more of them per CTA, and few K-blocks, so that the next tile's
sums stand ready while one is still being stored.

Inputs change from call to call, by sign and by size, so that activations left
by the call before are far from the right ones; every call is held to the
element-wise bound of the layer's own checks.
"""
import pytest
import torch

from tests.test_gpu_few_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


CASES = [  # T, D, E, F, k, S, Fs
    (1, 512, 64, 400, 8, 0, 0),        # 200 tiles of 16 features
    (1, 16, 32, 800, 8, 0, 0),         # 400 of them, a single K-block each
    (16, 128, 8, 400, 2, 0, 0),        # 200 for sixteen tokens
    (2, 256, 16, 640, 4, 1, 640),      # with a shared expert
    (1, 512, 15, 400, 15, 0, 0),       # 195 tiles of 32 features
    (3, 64, 15, 432, 5, 0, 0),         # 210 at most, a single K-block
    (5, 128, 14, 464, 9, 2, 48),
    (1, 144, 200, 992, 9, 0, 0),       # 288 tiles of 32 features
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,D,E,F,k,S,Fs", CASES)
def test_narrow_tiles_with_changing_inputs(moe, T, D, E, F, k, S, Fs, fp8):
    L = Layer(moe, T, D, E, F, k, S, Fs, fp8, seed=11)
    base = L.h.clone()
    gen = torch.Generator(device="cuda").manual_seed(D + F)
    calls = []
    for i in range(40):
        h = torch.randn(base.shape, generator=gen, device="cuda") * (1.0, -4.0, 0.25)[i % 3]
        h = h.to(torch.bfloat16)
        calls.append((h, L.run(h=h)))          # back to back: nothing waits in between
    assert moe.moe_get_device_status(L.ws) == 0
    for h, got in calls:
        L.check(*got, h=h)

"""GPU checks of one workspace that serves calls of a layer with any number of
tokens, of either kind: moe_forward and moe_forward_few (and their forms with
8-bit weights), whose scratch lies at places that move with T, while what a call
must find zero does not."""
import re

import pytest
import torch

from tests.test_gpu_few_layer import NAMES, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


LAYERS = [  # D, E, F, k, S, Fs
    (128, 8, 64, 2, 1, 64),
    (768, 40, 256, 8, 1, 512),
    (512, 24, 144, 3, 0, 0),
    (2048, 16, 512, 4, 1, 1408),       # the shared expert beside the routing, on a stream of its own
    (320, 64, 976, 8, 2, 80),          # experts wider than the hidden rows
]
SEQUENCE = [128, (1, 16), 64, (3, 7), 256, (16, 1), 300, (8, 12, 5), 16, (2, 16), 129, 32, (9, 4, 15), 31, 1, (1,),
            17, (16, 16), 256, 128, (6, 11), 100, (14, 10, 13), 8, 128]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,E,F,k,S,Fs", LAYERS)
def test_any_T_of_both_kinds(moe, D, E, F, k, S, Fs, fp8):
    """The sequence in one workspace, nothing waiting in between, gives the bits
    that every call gives in a zeroed workspace of its own."""
    L = Layer(moe, 16, D, E, F, k, S, Fs, fp8, seed=21)
    gen = torch.Generator(device="cuda").manual_seed(D)
    dims = lambda T: moe.dims(T=T, D=D, E=E, F=F, k=k, S=S, Fs=L.Fs, scale=2.5)
    size = max(moe.moe_workspace_size(dims(T)) for T in (*range(1, 17), 256, 300))
    one = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def large(h, ws):
        T = h.shape[0]
        out, w = torch.full((T, D), 777.0, device="cuda"), torch.empty((T, k), device="cuda")
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        if fp8:
            moe.moe_forward_fp8(h, L.Wr, L.bias, L.w8, dims(T), out, ws, idx, w)
        else:
            moe.moe_forward(h, L.Wr, L.bias, *[L.w[n] for n in NAMES], dims(T), out, ws, idx, w)
        return out, idx, w

    def few(h, ws):
        return L.run(h=h, d=dims(h.shape[0]), ws=ws)

    calls = []
    for item in SEQUENCE:
        for T in item if isinstance(item, tuple) else (item,):
            h = torch.randn((T, D), generator=gen, device="cuda").to(torch.bfloat16)
            f = few if isinstance(item, tuple) else large
            calls.append((f, h, f(h, one)))
    assert moe.moe_get_device_status(one) == 0
    for f, h, got in calls:
        d = dims(h.shape[0])
        own = torch.zeros(size, dtype=torch.uint8, device="cuda")
        want = f(h, own)
        assert moe.moe_get_device_status(own) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (f.__name__, h.shape[0])
        counts = torch.bincount(want[1].flatten().long(), minlength=E).int()
        again = f(h, one)                       # and what a call leaves to be asked for
        assert torch.equal(again[0], want[0])
        assert torch.equal(moe.moe_ws_expert_counts(one, d), counts)
        assert int(moe.moe_ws_touched_experts(one, d)) == int((counts > 0).sum())
    assert moe.moe_get_device_status(one) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,D,E,F,k,S,Fs", [
    (1, 16, 1, 16, 1, 0, 0),
    (1, 6144, 4, 2048, 1, 0, 0),        # the second product's K in parts
    (16, 128, 1, 2048, 1, 0, 0),        # the same for sixteen tokens
    (10, 5040, 98, 128, 3, 0, 0),       # several slots to a unit
    (16, 512, 1024, 64, 32, 2, 128),    # the most pairs
    (16, 64, 8, 1040, 8, 16, 992),      # wide experts, the most shared ones
    (13, 272, 9, 208, 4, 1, 336),
])
def test_nothing_is_written_behind_what_a_call_asks_for(moe, T, D, E, F, k, S, Fs, fp8):
    """The few-token layer in exactly the bytes its refusal names, with what
    follows them filled beforehand."""
    L = Layer(moe, T, D, E, F, k, S, Fs, fp8, seed=41)
    want = L.run()
    with pytest.raises(moe.MoeError, match="needs") as refused:
        L.run(ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    need = int(re.search(r"needs (\d+)", str(refused.value)).group(1))
    assert need <= moe.moe_workspace_size(L.d)
    room = torch.full((need + 65536,), 0xa5, dtype=torch.uint8, device="cuda")
    room[:need] = 0
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(L.run(ws=room[:need]), want))
    assert moe.moe_get_device_status(room[:need]) == 0
    assert bool((room[need:] == 0xa5).all())

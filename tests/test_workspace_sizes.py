"""Sizes of the workspace: one made for T tokens serves every call with fewer, the
few-token layer asks for scratch of its own alone, and no call of a few tokens
costs more than a call of seventeen.  What a call needs is read from its refusal
of an empty workspace; nothing is launched."""
import ctypes
import random
import re

import pytest

FAKE = 0x7F0000000000   # never dereferenced: every call below is refused

LAYERS = [  # the layer's own sizes, then odd ones
    dict(D=6144, E=256, F=2048, k=8, S=1, Fs=2048),
    dict(D=4096, E=128, F=1408, k=8, S=1, Fs=1408),
    dict(D=128, E=8, F=64, k=2, S=1, Fs=64),
    dict(D=128, E=8, F=64, k=2, S=0, Fs=64),
]


@pytest.fixture(scope="module")
def mod():
    import __graft_entry__
    __graft_entry__._build_module().build()   # no-op unless a source is newer
    import sparse_moe_layer_04_b200 as m
    return m


def needs(mod, d, few):
    lib, P = mod._lib, [FAKE] * 9
    f = lib.moe_forward_few if few else lib.moe_forward
    assert f(*P, ctypes.byref(d), FAKE, None, None, FAKE, 0, None) == mod.MOE_ERR_WORKSPACE
    return int(re.search(r"needs (\d+)", mod.moe_last_error()).group(1))


def random_layers(n):
    rng = random.Random(5)
    for _ in range(n):
        E = rng.choice([1, 3, 8, 24, 64, 200, 256, 1000, 1024])
        yield dict(D=8 * rng.randint(1, 800), E=E, F=8 * rng.randint(1, 300), k=rng.randint(1, min(E, 32)),
                   S=rng.choice([0, 1, 2, 16]), Fs=8 * rng.randint(1, 300))


@pytest.mark.parametrize("layer", [*LAYERS, *random_layers(40)], ids=str)
def test_one_size_serves_every_smaller_T(mod, layer):
    dims = lambda T: mod.dims(T=T, scale=1.0, **layer)
    steps = [*range(1, 34), *range(60, 70), *range(120, 136), *range(190, 195), *range(250, 262), *range(500, 520, 3),
             *range(576, 2050, 37), *range(2112, 19500, 1111), 18944, 18945, 30000]
    most = 0
    for T in sorted(steps):
        d = dims(T)
        size, own = mod.moe_workspace_size(d), needs(mod, d, False)
        most = max(most, own, needs(mod, d, True) if T <= 16 else 0)
        assert own <= size and size >= most, T
        if T > 16:
            assert own <= size < own + 8 * most       # (a bound, not every byte ever thought of)
    for T in (64, 128, 192, 256, 320, 448, 512, 576, 4096, 18944):   # tops of the router's cuts
        assert needs(mod, dims(T), False) <= min(mod.moe_workspace_size(dims(T + r)) for r in (0, 1, 63, 64, 65, 5000))


@pytest.mark.parametrize("layer", LAYERS, ids=str)
def test_few_tokens_cost_no_more_than_seventeen(mod, layer):
    dims = lambda T: mod.dims(T=T, scale=1.0, **layer)
    for T in range(1, 17):
        assert mod.moe_workspace_size(dims(T)) <= mod.moe_workspace_size(dims(17))
        # and the calls that are not the few-token layer's ask for none of its scratch
        k, D, F, S, Fs = (layer[n] for n in ("k", "D", "F", "S", "Fs"))
        rows = T * k * (2 * D + 2 * F + 4 * D) + S * T * (2 * Fs + 4 * D)
        sums = 64 * T * layer["E"] * 4                     # the router's, at most 64 planes
        assert needs(mod, dims(T), False) < rows + sums + 100_000


def test_host_pipelines_hold_none_of_the_few_token_scratch(mod):
    a256 = lambda n: (n + 255) // 256 * 256
    for T in (1, 16, 40):
        # experts much wider than the hidden rows: there the few-token layer needs more than the others
        d = mod.dims(T=T, D=64, E=8, F=2048, k=8, S=1, Fs=2048, scale=1.0)
        if T <= 16:
            assert needs(mod, d, True) > needs(mod, d, False)
        assert mod.moe_pipeline_device_bytes(d) == \
            2 * a256(T * 64 * 2) + 2 * a256(T * 64 * 4) + needs(mod, d, False)

"""GPU checks of a layer with shared experts through the 8-bit products (the
shared experts are groups of their own whose rows stand behind the routed ones,
as the merge expects them), with evenly spread and with one-sided routing, and
of the few-token layer with 8-bit weights whose exponents stand at any address.

Bars as in the checks of the products: each step of the tensor core is off by at
most 2^-22 of the sum of magnitudes, (K/32 + 1) steps a product; the merge adds
k + S fused terms in fp32.
"""
import pytest
import torch

import moe_inputs as mi
from tests.test_gpu_few_layer import Layer
from tests.test_gpu_fp8_products import TABLE, blocks, product64, quantize64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


@pytest.mark.parametrize("hot", [False, True])
@pytest.mark.parametrize("T,D,E,F,k,S,Fs", [
    (5, 128, 8, 64, 2, 1, 64),
    (61, 384, 12, 144, 3, 2, 272),
    (500, 256, 16, 208, 4, 1, 400),
])
def test_layer_with_shared_experts(moe, T, D, E, F, k, S, Fs, hot):
    gen = torch.Generator().manual_seed(T + S)
    d = moe.dims(T=T, D=D, E=E, F=F, k=k, S=S, Fs=Fs, scale=2.5)
    ws = moe.alloc_workspace(d)
    h = torch.randn(T, D, generator=gen).to(torch.bfloat16).cuda()
    Wr, bias = (torch.randn(E, D, generator=gen) / D ** 0.5).cuda(), torch.zeros(E, device="cuda")
    if hot:
        bias[1] = 10.0                             # one expert for every token
    shapes = dict(W1=(E, F, D), W3=(E, F, D), W2=(E, D, F), Ws1=(S, Fs, D), Ws3=(S, Fs, D), Ws2=(S, D, Fs))
    W = {n: mi.quantize_fp8_blocks((torch.randn(*s, generator=gen) / s[2] ** 0.5).bfloat16().cuda())
         for n, s in shapes.items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, inv, rw = torch.empty((T, k), **i32), torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    counts, off, perm = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    every = torch.arange(T, **i32).repeat(S)       # the shared experts' rows and their groups
    off_s = torch.arange(S + 1, **i32) * T
    logits, y, out = torch.empty((T, E), device="cuda"), torch.empty((T * k + S * T, D), device="cuda"), \
        torch.empty((T, D), device="cuda")
    buf = {}
    for n, R, width in (("r", T * k, F), ("s", S * T, Fs)):
        q = lambda K: (torch.empty((R, K), dtype=torch.uint8, device="cuda"),
                       torch.empty((R, blocks(K)), dtype=torch.int8, device="cuda"))
        buf[n] = (*q(D), torch.empty((R, width), dtype=torch.bfloat16, device="cuda"), *q(width))

    def experts(n, rows, offsets, names, to):
        x, xe, act, a, ae = buf[n]
        moe.moe_quantize_fp8(h, x, xe, idx=rows, ws=ws)
        moe.moe_gated_gemm_fp8(x, xe, *W[names[0]], *W[names[1]], act, offsets=offsets, ws=ws)
        moe.moe_quantize_fp8(act, a, ae, ws=ws)
        moe.moe_grouped_gemm_fp8(a, ae, *W[names[2]], to, offsets=offsets, ws=ws)

    def layer():
        moe.moe_router_logits(h, Wr, d, logits, ws)
        moe.moe_route(logits, bias, d, idx, rw, ws)
        moe.moe_permute(idx, d, counts, off, perm, inv, ws)
        experts("s", every, off_s, ("Ws1", "Ws3", "Ws2"), y[T * k:])
        experts("r", perm, off, ("W1", "W3", "W2"), y[:T * k])
        moe.moe_combine(y, rw, inv, d, out, ws)

    layer()
    assert moe.moe_get_device_status(ws) == 0
    if hot:
        assert int(counts[1]) == T
    ref, tol = torch.empty_like(y, dtype=torch.float64), torch.empty_like(y, dtype=torch.float64)
    for n, rows, bounds, names, part in (("r", perm, off.tolist(), ("W1", "W3", "W2"), slice(0, T * k)),
                                         ("s", every, off_s.tolist(), ("Ws1", "Ws3", "Ws2"), slice(T * k, None))):
        x, xe, act, a, ae = buf[n]
        vals, e = quantize64(h[rows.long()])
        assert torch.equal(TABLE[x.cpu().long()], vals) and torch.equal(xe.cpu().int(), e.int())
        g, gm = product64(x, xe, *W[names[0]], bounds)
        u, um = product64(x, xe, *W[names[1]], bounds)
        unit = (D / 32 + 1) * 2.0 ** -22
        silu = g * torch.sigmoid(g)
        bar = (2.0 ** -8 + 2.0 ** -16) * (silu * u).abs() + 1.1 * unit * gm * (u.abs() + unit * um) + \
            silu.abs() * unit * um + 2.0 ** -133
        assert bool(((act.double() - silu * u).abs() <= bar).all())
        vals, e = quantize64(act)
        assert torch.equal(TABLE[a.cpu().long()], vals) and torch.equal(ae.cpu().int(), e.int())
        width = act.shape[1]
        ref[part], mag = product64(a, ae, *W[names[2]], bounds)
        tol[part] = (width / 32 + 1) * 2.0 ** -22 * mag
    assert bool(((y.double() - ref).abs() <= tol).all())
    c = rw.double()[..., None]
    whole = ref[T * k:].view(S, T, D).sum(0) + (c * ref[inv.long()]).sum(1)
    size = ref[T * k:].view(S, T, D).abs().sum(0) + (c * ref[inv.long()].abs()).sum(1)
    bar = tol[T * k:].view(S, T, D).sum(0) + (c * tol[inv.long()]).sum(1) + (k + S) * 2.0 ** -23 * size
    assert bool(((out.double() - whole).abs() <= bar).all())

    # against the layer whose activations stay bf16: two roundings to E4M3 lie between
    names = ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2")
    w8 = moe.fp8_weights(*[W[n][0] for n in names], *[W[n][1] for n in names])
    other, i2 = torch.empty_like(out), torch.empty_like(idx)
    moe.moe_forward_fp8(h, Wr, bias, w8, d, other, ws, i2)
    assert torch.equal(i2, idx)
    assert float((out - other).norm() / other.norm()) < 2.0 ** -4

    graph, want = torch.cuda.CUDAGraph(), out.clone()
    with torch.cuda.graph(graph):
        layer()
    out.zero_(), y.zero_()
    graph.replay()
    assert torch.equal(out, want) and moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("T,D,E,F,k,S,Fs", [(3, 400, 9, 272, 3, 1, 144), (1, 1040, 5, 1168, 2, 0, 0),
                                            (16, 144, 4, 16, 4, 2, 16)])
def test_few_layer_with_exponents_at_any_address(moe, T, D, E, F, k, S, Fs, shift):
    """Exponent arrays that start and end off every alignment, among bytes that
    would be reported."""
    L = Layer(moe, T, D, E, F, k, S, Fs, True, seed=shift)
    want = L.run()
    names = ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2")
    kept = []

    def moved(t):
        raw = torch.full((t.numel() + 8,), 100, dtype=torch.int8, device="cuda")
        view = raw[shift:shift + t.numel()].view(t.shape)
        view.copy_(t)
        kept.append(raw)
        return view

    s = lambda n, end, f=lambda t: t: f(L.q[n + end]) if S or not n.startswith("Ws") else None
    L.w8 = moe.fp8_weights(*[s(n, "q") for n in names], *[s(n, "e", moved) for n in names])
    assert all(torch.equal(a, b) for a, b in zip(L.run(), want))
    assert moe.moe_get_device_status(L.ws) == 0

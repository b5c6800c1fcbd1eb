"""GPU checks of silu(gate) * up far from zero, where e^-gate or the sigmoid
leaves fp32 while the product does not: the fused gate of the 8-bit products and
of the few-token layer.

Every gate and every up is a single product of two short numbers, so it is exact
in fp32, and what is left is the gate's own arithmetic: fewer than eight units of
fp32 (two in each exponential and in the division, a rounding in each product),
below 2^-20 of the result, and in the 8-bit products 1.16 |gate| units more in the
exponential down to -80, below 2^-17.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

ONE = 0x38                       # the E4M3 code of 1.0


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


def codes(v):
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


GATES = [-1.0, -20.0, -40.0, -72.0, -80.0, -88.0, -96.0, -104.0, 1.0, 20.0, 40.0, 72.0, 80.0, 88.0, 96.0, 104.0]


def exact(g, u):
    """In 64 bits, from the side that does not cancel (e^-104 is a normal number there)."""
    g, u = g.double(), u.double()
    return g * u * torch.where(g < 0, torch.exp(g) / (1 + torch.exp(g)), 1 / (1 + torch.exp(-g)))


@pytest.mark.parametrize("K", [256, 4096])       # 4096: K split over a cluster
@pytest.mark.parametrize("up", [0, 60, 110])
def test_gated_product(moe, up, K):
    """x = (1, then 1 in another block), W1 = (gate, 0), W3 = (0, 1 * 2^up)."""
    R, N = 5, 16
    x = torch.zeros((R, K), dtype=torch.uint8, device="cuda")
    factor = torch.tensor([1.0, 1.125, 0.9375, 0.8125, 1.25], device="cuda")   # of the gates, row by row
    x[:, 0], x[:, 128] = codes(factor), ONE
    xe = torch.zeros((R, K // 128), dtype=torch.int8, device="cuda")
    W1, W3 = (torch.zeros((N, K), dtype=torch.uint8, device="cuda") for _ in range(2))
    gates = torch.tensor(GATES, device="cuda")
    W1[:, 0], W3[:, 128] = codes(gates), ONE
    e1, e3 = (torch.zeros((1, K // 128), dtype=torch.int8, device="cuda") for _ in range(2))
    e3[:] = up
    act = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_gated_gemm_fp8(x, xe, W1, e1, W3, e3, act)
    ref = exact(factor[:, None] * gates[None].to(torch.float8_e4m3fn).float(), torch.tensor(2.0 ** up).cuda())
    tol = (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 2.0 ** -133
    over = (act.double() - ref).abs() > tol
    assert not bool(over.any()), [(float(act[tuple(i)]), float(ref[tuple(i)])) for i in over.nonzero().tolist()]


@pytest.mark.parametrize("fp8", [False, True])
def test_few_token_layer(moe, fp8):
    """One expert whose second matrix is the identity: the layer's output is the
    activation.  The hidden row holds 1 and, in another block, 2^100."""
    D = F = 256
    d = moe.dims(T=2, D=D, E=1, F=F, k=1, S=0, Fs=16, scale=1.0)
    ws = moe.alloc_workspace(d)
    h = torch.zeros((2, D), dtype=torch.bfloat16, device="cuda")
    h[0, 0], h[1, 0], h[:, 128] = 1.0, 0.9375, 2.0 ** 100
    gates = torch.tensor(GATES, device="cuda").repeat_interleave(16)      # two kinds to a block of 32
    W1, W3 = torch.zeros((1, F, D), device="cuda"), torch.zeros((1, F, D), device="cuda")
    W1[0, :, 0], W3[0, :, 128] = gates, 1.0
    W2 = torch.eye(D, device="cuda")[None].contiguous()
    Wr, bias = torch.zeros((1, D), device="cuda"), torch.zeros(1, device="cuda")
    out = torch.full((2, D), 777.0, device="cuda")
    if fp8:
        e = lambda: torch.zeros((1, 2, 2), dtype=torch.int8, device="cuda")
        arrays = [codes(W1), codes(W3), codes(W2), None, None, None, e(), e(), e(), None, None, None]
        moe.moe_forward_few_fp8(h, Wr, bias, moe.fp8_weights(*arrays), d, out, ws)
    else:
        bf = [w.to(torch.bfloat16) for w in (W1, W3, W2)]
        moe.moe_forward_few(h, Wr, bias, *bf, None, None, None, d, out, ws)
    assert moe.moe_get_device_status(ws) == 0
    ref = exact(h[:, :1].float() * gates[None], torch.tensor(2.0 ** 100).cuda())
    # an activation's four E4M3 pieces hold it to 2^-16 of itself and 2^-29 of the
    # largest of its 32 neighbours; three bf16 pieces hold all of it
    tol = 2.0 ** -19 * ref.abs()
    if fp8:
        tol = tol + 2.0 ** -16 * ref.abs() + 2.0 ** -29 * ref.abs().amax(1, keepdim=True)
    over = (out.double() - ref).abs() > tol
    assert not bool(over.any()), [(float(out[tuple(i)]), float(ref[tuple(i)])) for i in over.nonzero().tolist()[:6]]

"""GPU checks of the few-token layer's precision against bars set near what it
reaches.

Per element: each step of the tensor core (16 or 32 products and the
running sum) is off by at most 2^-22 of the sum of magnitudes; with bf16 weights
an activation enters the second product as three bf16 pieces, of which each
leaves at most 2^-9 of what it rounds, so as itself to fp32's last bits (2^-24),
after a gate of fewer than eight units (2^-20); with E4M3 weights as four pieces
(2^-16 of itself, 2^-29 of the largest of its 32 neighbours).
As a whole: K-blocks take turns over the accumulators that tensor memory holds,
48 K-blocks at a time, so that no chain is longer than 48 K-blocks of 4 steps
over the accumulators' number; errors of single steps add up like a walk in the
first product and are averaged over F and D in the norm.  A chain of s steps that
cuts off its sum has a mean error of s / 4 units of 2^-23 and a scatter of a
third of sqrt(s): one token through D = 6144 with bf16 weights has 15
accumulators and 48 * 4 / 15 = 13 steps a chain, 3.2 units or 3.9e-7 on the mean
of its sums; gate, up and down together stay below 3 * 3.9e-7 = 1.2e-6.  One
accumulator with 384 steps would be off by 96 units, 1.1e-5, and two pieces
instead of three by 2^-18, 3.8e-6.  The bar is 2.5e-6.
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


class Close(Layer):
    """The layer's element-wise bound with the bf16 activation's own error."""

    def mlp(self, h, names, g):
        w1, w3, w2 = (self.value(n, g) for n in names)
        D, F = h.shape[1], w1.shape[0]
        x = h.double()
        step = (D / 16 + 2) * 2.0 ** -22
        eh = 2.0 ** -21 * x.abs().amax(1, keepdim=True).expand_as(x) if self.fp8 else 0 * x
        gate, up = x @ w1.t(), x @ w3.t()
        eg = step * (x.abs() @ w1.abs().t()) + eh @ w1.abs().t()
        eu = step * (x.abs() @ w3.abs().t()) + eh @ w3.abs().t()
        silu = gate * torch.sigmoid(gate)
        act = silu * up
        ea = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + (2.0 ** -16 if self.fp8 else 2.0 ** -20) * act.abs()
        if self.fp8:
            ea = ea + 2.0 ** -29 * act.abs().amax(1, keepdim=True)
        y = act @ w2.t()
        return y, ea @ w2.abs().t() + (F / 16 + 8) * 2.0 ** -22 * ((act.abs() + ea) @ w2.abs().t())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,D,E,F,k,S,Fs", [
    (1, 6144, 16, 2048, 8, 1, 2048),
    (1, 4096, 16, 1408, 8, 1, 1408),
    (1, 128, 8, 64, 2, 1, 64),
    (4, 2048, 12, 768, 3, 0, 0),
])
def test_precision(moe, T, D, E, F, k, S, Fs, fp8):
    L = Close(moe, T, D, E, F, k, S, Fs, fp8, seed=23)
    out, idx, w = L.run()
    L.check(out, idx, w)
    ref = torch.zeros((T, D), dtype=torch.float64, device="cuda")
    for g in range(S):
        ref += L.mlp(L.h, ("Ws1", "Ws3", "Ws2"), g)[0]
    for t in range(T):
        for j in range(k):
            ref[t] += w[t, j].double() * L.mlp(L.h[t:t + 1], ("W1", "W3", "W2"), int(idx[t, j]))[0][0]
    rel = float((out.double() - ref).norm() / ref.norm())
    print(f"relative error {rel:.2e}")
    assert rel < 2.5e-6, rel

"""GPU checks of the few-token layer (moe_forward_few, moe_forward_few_fp8)
against the layer's definition in 64 bits.

Bars.  A routing is right when no chosen key lies below an unchosen one by more
than NEAR_TIE, the oracle's allowance for fp32 logits summed in another order;
the output is then compared for the GPU's own choice.  Its error is bounded
element by element: each step of the tensor core (16 or 32 products and the
running sum) is off by at most 2^-22 of the sum of magnitudes; an activation
enters the second product within 2^-16 of itself (two bf16 pieces: 2^-18, four
E4M3 pieces: 2^-16) plus, for E4M3, 2^-29 of its largest neighbour; a hidden
value enters exactly (bf16) or within 2^-21 of its largest neighbour (E4M3: two
pieces end at half of 2^-13 of the block's scale, whose largest value is above
224 of it);
|silu'| <= 1.1; the merge adds at most T k + S terms in fp32.
"""
import numpy as np
import pytest
import torch

import moe_inputs as mi
from tests.gpu_helpers import NEAR_TIE
from tests.test_gpu_fp8_products import matrix64

pytestmark = pytest.mark.gpu

NAMES = ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


class Layer:
    """One layer's weights (bf16, or FP8 codes of them) and its 64-bit values."""

    def __init__(self, moe, T, D, E, F, k, S, Fs, fp8, scale=2.5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * D + E)
        self.moe, self.fp8, self.T, self.D, self.E, self.k, self.S = moe, fp8, T, D, E, k, S
        Fs = Fs or 16
        self.F, self.Fs = F, Fs
        self.d = moe.dims(T=T, D=D, E=E, F=F, k=k, S=S, Fs=Fs, scale=scale)

        def normal(shape, std, dt):
            return torch.empty(shape, dtype=dt, device="cuda").normal_(0, std, generator=g)

        self.Wr = normal((E, D), 1.6 / D ** 0.5, torch.float32)
        self.bias = normal((E,), 0.1, torch.float32)
        self.w = {n: normal((G, r, c), 1 / c ** 0.5, torch.bfloat16) for n, (G, r, c) in
                  dict(W1=(E, F, D), W3=(E, F, D), W2=(E, D, F), Ws1=(S, Fs, D), Ws3=(S, Fs, D),
                       Ws2=(S, D, Fs)).items()}
        if fp8:
            self.q = mi.fp8_layer_weights(self.w)
            s = (lambda n: self.q.get(n) if S or not n.startswith("Ws") else None)
            self.w8 = moe.fp8_weights(*[s(n + "q") for n in NAMES], *[s(n + "e") for n in NAMES])
        self.h = normal((T, D), 1.0, torch.bfloat16)
        self.ws = moe.alloc_workspace(self.d)

    def run(self, h=None, d=None, ws=None, stream=None):
        h = self.h if h is None else h
        d = d or self.d
        out = torch.full((d.T, self.D), 777.0, device="cuda")
        idx = torch.full((d.T, self.k), -7, dtype=torch.int32, device="cuda")
        w = torch.empty((d.T, self.k), device="cuda")
        ws = self.ws if ws is None else ws
        if self.fp8:
            self.moe.moe_forward_few_fp8(h, self.Wr, self.bias, self.w8, d, out, ws, idx, w, stream)
        else:
            self.moe.moe_forward_few(h, self.Wr, self.bias, *[self.w[n] for n in NAMES], d, out, ws,
                                     idx, w, stream)
        return out, idx, w

    def value(self, name, g):
        if self.fp8:
            return matrix64(self.q[name + "q"][g], self.q[name + "e"][g])
        return self.w[name][g].double()

    def mlp(self, h, names, g):
        """(value, error bound) of one expert on rows h."""
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
        ea = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + 2.0 ** -16 * act.abs()
        if self.fp8:
            ea = ea + 2.0 ** -29 * act.abs().amax(1, keepdim=True)
        y = act @ w2.t()
        ey = ea @ w2.abs().t() + (F / 16 + 8) * 2.0 ** -22 * ((act.abs() + ea) @ w2.abs().t())
        return y, ey

    def check(self, out, idx, w, h=None):
        h = self.h if h is None else h
        logits = h.double() @ self.Wr.double().t()
        s = torch.sigmoid(logits)
        key = s + self.bias.double()
        i = idx.long()
        assert bool(((i >= 0) & (i < self.E)).all())
        got = key.gather(1, i)
        assert bool((got[:, 1:] <= got[:, :-1] + NEAR_TIE).all())      # in descending order
        rest = key.scatter(1, i, -float("inf"))
        assert bool((rest.amax(1) <= got[:, -1] + NEAR_TIE).all())
        assert all(len(set(r)) == self.k for r in idx.tolist())
        ref_w = s.gather(1, i) / s.gather(1, i).sum(1, keepdim=True) * self.d.scale
        assert bool(((w.double() - ref_w).abs() <= 4e-6 * ref_w.abs()).all())
        T = h.shape[0]
        ref = torch.zeros((T, self.D), dtype=torch.float64, device="cuda")
        tol, mag = ref.clone(), ref.clone()
        for g in range(self.S):
            y, e = self.mlp(h, ("Ws1", "Ws3", "Ws2"), g)
            ref, tol, mag = ref + y, tol + e, mag + y.abs()
        for e_ in sorted(set(i.flatten().tolist())):
            t, j = (i == e_).nonzero(as_tuple=True)
            y, e = self.mlp(h[t], ("W1", "W3", "W2"), e_)
            c = w[t, j].double()[:, None]
            ref[t] += c * y
            tol[t] += c.abs() * e
            mag[t] += c.abs() * y.abs()
        tol = tol + (self.k + self.S + 8) * 2.0 ** -24 * mag
        over = (out.double() - ref).abs() > tol
        assert not bool(over.any()), (int(over.sum()), over.nonzero()[:4].tolist())
        rel = float((out.double() - ref).norm() / ref.norm())
        assert rel < 2e-5, rel


CASES = [  # T, D, E, F, k, S, Fs
    (1, 16, 1, 16, 1, 0, 0),            # the smallest layer, FP8 weights
    (2, 8, 3, 8, 2, 1, 8),              # the smallest sizes, bf16 weights
    (1, 128, 8, 64, 2, 1, 64),
    (5, 128, 8, 64, 2, 1, 64),          # the tiny layer
    (16, 256, 16, 192, 8, 1, 320),
    (7, 136, 12, 88, 3, 2, 40),         # D, F and Fs odd multiples of 8
    (3, 400, 40, 336, 5, 0, 0),         # no shared expert
    (16, 512, 1024, 64, 32, 2, 128),    # the largest E and k: up to 512 chosen experts
    (9, 1152, 64, 272, 4, 1, 2048),     # shared expert wider than the routed ones
    (2, 640, 4, 1408, 4, 1, 1408),      # every expert chosen
    (8, 2048, 32, 512, 1, 3, 64),       # three shared experts
    (16, 144, 5, 976, 1, 16, 32),       # sixteen of them
    (4, 6144, 16, 2048, 8, 1, 2048),    # full-size experts, K split over units
    (12, 4096, 12, 1408, 8, 1, 1408),
    (10, 5040, 98, 128, 3, 0, 0),       # narrow experts: several to a unit of the second product
    (7, 6144, 24, 64, 4, 16, 32),       # and shared ones
    (16, 5008, 200, 80, 13, 1, 4096),   # several choices of a token in one unit
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,D,E,F,k,S,Fs", CASES)
def test_layer(moe, T, D, E, F, k, S, Fs, fp8):
    if fp8 and (D % 16 or F % 16 or Fs % 16):
        pytest.skip("FP8 weights need multiples of 16")
    L = Layer(moe, T, D, E, F, k, S, Fs, fp8)
    out, idx, w = L.run()
    assert moe.moe_last_launch_count() == 2
    assert moe.moe_get_device_status(L.ws) == 0
    L.check(out, idx, w)
    counts = torch.bincount(idx.flatten().long(), minlength=E).int()
    assert torch.equal(moe.moe_ws_expert_counts(L.ws, L.d), counts)
    assert int(moe.moe_ws_touched_experts(L.ws, L.d)) == int((counts > 0).sum())
    for _ in range(3):                   # the same bits again: counters were left zero
        again = L.run()
        assert all(torch.equal(a, b) for a, b in zip(again, (out, idx, w)))
    assert moe.moe_get_device_status(L.ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_any_batch_in_one_workspace(moe, fp8):
    """Every T from 1 to 16 in the workspace of the largest, back to back; each
    token's row is the same bits whatever stands beside it where the tiles allow,
    and always within the bound."""
    L = Layer(moe, 16, 384, 24, 208, 4, 1, 144, fp8, seed=3)
    runs = []
    for T in [*range(1, 17), 3, 16, 1]:
        d = moe.dims(T=T, D=384, E=24, F=208, k=4, S=1, Fs=144, scale=2.5)
        runs.append((T, L.run(h=L.h[:T], d=d)))
    assert moe.moe_get_device_status(L.ws) == 0
    for T, got in runs:
        L.check(*got, h=L.h[:T])


@pytest.mark.parametrize("fp8", [False, True])
def test_matches_the_layer_for_any_batch(moe, fp8):
    """moe_forward / moe_forward_fp8 on the same tokens: the same routing, and
    outputs apart by the activation's bf16 rounding there (2^-9 of each)."""
    L = Layer(moe, 6, 512, 32, 256, 4, 1, 256, fp8, seed=5)
    out, idx, w = L.run()
    o2, i2, w2 = torch.empty_like(out), torch.empty_like(idx), torch.empty_like(w)
    if fp8:
        moe.moe_forward_fp8(L.h, L.Wr, L.bias, L.w8, L.d, o2, L.ws, i2, w2)
    else:
        moe.moe_forward(L.h, L.Wr, L.bias, *[L.w[n] for n in NAMES], L.d, o2, L.ws, i2, w2)
    assert moe.moe_get_device_status(L.ws) == 0
    assert torch.equal(idx, i2)
    assert float((out - o2).norm() / o2.norm()) < 4e-3
    again = L.run()
    assert torch.equal(again[0], out)


@pytest.mark.parametrize("fp8", [False, True])
def test_unchosen_experts_do_not_reach_a_token(moe, fp8):
    """NaN and infinite weights of experts that only some tokens choose leave
    the other tokens' rows as they were, bit for bit; so does a token that is
    not finite (which the status word reports)."""
    L = Layer(moe, 8, 256, 16, 128, 2, 1, 128, fp8, seed=9)
    out, idx, _ = L.run()
    e = int(idx[3, 0])
    hit = (idx == e).any(1)
    assert bool(hit[3]) and not bool(hit.all())
    if fp8:
        L.q["W2q"][e] = 0x7f
        L.q["W1q"][e, 5] = 0xff
    else:
        L.w["W2"][e] = float("inf")
        L.w["W1"][e, 5] = float("nan")
    z, i2, _ = L.run()
    assert torch.equal(i2, idx)
    assert torch.equal(z[~hit], out[~hit]) and not bool(torch.isfinite(z[hit]).any())
    assert moe.moe_get_device_status(L.ws) == 0
    L = Layer(moe, 8, 256, 16, 128, 2, 1, 128, fp8, seed=9)
    L.h[5, 17] = float("nan")
    z, i2, _ = L.run()
    assert moe.moe_get_device_status(L.ws) == moe.MOE_ERR_NONFINITE
    keep = torch.arange(8, device="cuda") != 5
    assert torch.equal(z[keep], out[keep]) and torch.equal(i2[keep], idx[keep])


def test_exponent_out_of_range_is_reported(moe):
    L = Layer(moe, 3, 256, 4, 128, 4, 1, 128, True, seed=2)
    for name, at in (("W1e", (2, 0, 1)), ("W3e", (1, 0, 0)), ("W2e", (3, 1, 0)), ("Ws2e", (0, 0, 0))):
        kept = L.q[name][at].item()
        for bad in (8, -118):
            L.q[name][at] = bad
            L.run()
            assert moe.moe_get_device_status(L.ws) == moe.MOE_ERR_BOUNDS, (name, bad)
        L.q[name][at] = kept
    out = L.run()
    assert moe.moe_get_device_status(L.ws) == 0
    L.check(*out)


@pytest.mark.parametrize("fp8", [False, True])
def test_streams_and_graphs(moe, fp8):
    """A captured call replayed on new inputs, and two layers at once on two
    streams with a workspace each."""
    A = Layer(moe, 4, 512, 16, 512, 4, 1, 512, fp8, seed=1)
    B = Layer(moe, 11, 640, 24, 336, 3, 1, 208, fp8, seed=2)
    want_a, want_b = A.run(), B.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            a = A.run()
        with torch.cuda.stream(s2):
            b = B.run()
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, want_a))
        assert all(torch.equal(x, y) for x, y in zip(b, want_b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = A.run()
    for k in range(4):
        A.h.normal_()
        graph.replay()
        replayed = [x.clone() for x in out]
        assert all(torch.equal(x, y) for x, y in zip(A.run(), replayed))
    assert moe.moe_get_device_status(A.ws) == 0 and moe.moe_get_device_status(B.ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_with_most_sms_held(moe, fp8):
    """All but 20 SMs are held while the layer runs: no wait may depend on a
    block that has no SM."""
    L = Layer(moe, 4, 1024, 16, 512, 4, 1, 512, fp8, seed=4)
    want = L.run()
    torch.cuda.synchronize()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    side = torch.cuda.Stream()
    moe.moe_selftest_occupy(sms - 20, 1 << 30, side)
    got = L.run()
    torch.cuda.current_stream().synchronize()
    assert moe.moe_get_device_status(L.ws) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fp8", [False, True])
def test_unchosen_experts_that_share_a_unit(moe, fp8):
    """Narrow experts, many chosen: several of them share a unit of the second
    product.  Infinite or NaN weights of some still reach only the tokens that
    chose them."""
    L = Layer(moe, 8, 2048, 64, 128, 8, 0, 128, fp8, seed=31)
    out, idx, _ = L.run()
    L.check(out, idx, _)
    bad = sorted({int(idx[0, 0]), int(idx[0, 5])})
    hit = sum((idx == e).any(1).int() for e in bad) > 0
    assert bool(hit[0]) and not bool(hit.all())
    for e in bad:
        if fp8:
            L.q["W2q"][e] = 0x7f
        else:
            L.w["W2"][e] = float("inf")
    z, i2, _ = L.run()
    assert torch.equal(i2, idx)
    assert torch.equal(z[~hit], out[~hit]) and not bool(torch.isfinite(z[hit]).any())
    assert moe.moe_get_device_status(L.ws) == 0

"""GPU checks of the 8-bit products (moe_quantize_fp8, moe_grouped_gemm_fp8,
moe_gated_gemm_fp8) against their definitions in 64 bits.

Bars.  Codes and exponents are exact.  A product of two E4M3 values is exact in
fp32; the tensor core adds 32 of them and the running sum per step, each step
off by at most two units in the last place (2^-23) of a sum no larger than
S = sum |x||w|, so |y - y64| <= (K/32 + 1) * 2^-22 * S.  A bf16 output adds half a
step, 2^-8 |y|.  The gate: |silu'| <= 1.1, and the exponential's error is at most
2 + 1.16 * 88 units, below 2^-16 relative.
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as orc

pytestmark = pytest.mark.gpu

TABLE = torch.from_numpy(orc.e4m3_value(np.arange(256, dtype=np.uint8)))


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_moe_layer_04_b200 as m
    return m


@pytest.fixture()
def status(moe):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    yield ws
    assert moe.moe_get_device_status(ws) == 0


def blocks(n):
    return -(-n // 128)


def rand_codes(gen, shape):
    """Every E4M3 code but the two NaNs."""
    c = torch.randint(0, 254, shape, generator=gen, dtype=torch.int32)
    return (c + (c >= 127).int()).to(torch.uint8).cuda()


def rand_exps(gen, shape, lo=-9, hi=5):
    return torch.randint(lo, hi + 1, shape, generator=gen, dtype=torch.int32).to(torch.int8).cuda()


def rows64(codes, exps):
    v = TABLE.cuda()[codes.long()]
    s = torch.pow(2.0, exps.double().cpu()).cuda().repeat_interleave(128, 1)[:, :codes.shape[1]]
    return v * s


def matrix64(codes, exps):
    v = TABLE.cuda()[codes.long()]
    s = torch.pow(2.0, exps.double().cpu()).cuda().repeat_interleave(128, 0)[:codes.shape[0]]
    return v * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def product64(x, xe, W, We, bounds):
    """(sum, sum of magnitudes) per row, NaN for rows of no group."""
    y = torch.full((x.shape[0], W.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    s = y.clone()
    for g, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        if b > a:
            v, m = rows64(x[a:b], xe[a:b]), matrix64(W[g], We[g])
            y[a:b] = v @ m.t()
            s[a:b] = v.abs() @ m.abs().t()
    return y, s


def operands(seed, G, R, N, K, n=1):
    gen = torch.Generator().manual_seed(seed)
    x, xe = rand_codes(gen, (R, K)), rand_exps(gen, (R, blocks(K)))
    ws = [(rand_codes(gen, (G, N, K)), rand_exps(gen, (G, blocks(N), blocks(K)))) for _ in range(n)]
    return x, xe, ws


def spread(G, R, lead=0, tail=0, seed=0):
    """Group bounds over rows [lead, R - tail) with empty groups among them."""
    gen = torch.Generator().manual_seed(seed)
    cut = torch.randint(lead, R - tail + 1, (G - 1,), generator=gen).sort().values.tolist()
    return [lead, *cut, R - tail]


CASES = [  # G, R, N, K, rows before the first group, rows behind the last
    (1, 1, 8, 16, 0, 0),           # the smallest call
    (1, 1, 256, 2048, 0, 0),       # one row: K split over a cluster
    (1, 13, 136, 1424, 0, 0),      # a K range of 12 blocks over a cluster, ragged N and K
    (1, 33, 128, 144, 0, 0),       # two row blocks of the narrow tile
    (3, 40, 200, 272, 2, 5),
    (40, 37, 72, 528, 0, 0),       # more groups than rows
    (5, 300, 392, 400, 7, 9),      # 128-row tiles
    (2, 700, 264, 656, 3, 4),      # 240-row tiles, several a group
    (1, 481, 128, 1152, 0, 0),
    (7, 2100, 640, 1024, 0, 11),   # several tiles per CTA, both accumulators
    (4, 4000, 2056, 144, 0, 0),
]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,R,N,K,lead,tail", CASES)
def test_grouped_product(moe, status, G, R, N, K, lead, tail, out):
    x, xe, [(W, We)] = operands(G * R + N, G, R, N, K)
    bounds = spread(G, R, lead, tail, K)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y = torch.full((R, N), 777.0, dtype=out, device="cuda")
    moe.moe_grouped_gemm_fp8(x, xe, W, We, y, offsets=off, ws=status)
    ref, mag = product64(x, xe, W, We, bounds)
    none = torch.isnan(ref)
    assert torch.equal(none[:, 0], torch.tensor([r < lead or r >= R - tail for r in range(R)]).cuda())
    assert bool((y[none] == 777.0).all())          # rows of no group keep what was there
    tol = (K / 32 + 1) * 2.0 ** -22 * mag + (2.0 ** -8 * ref.abs() if out == torch.bfloat16 else 0)
    over = ((y.double() - ref).abs() > tol) & ~none
    assert not bool(over.any()), (int(over.sum()), over.nonzero()[:4].tolist())
    again = torch.full_like(y, 777.0)
    moe.moe_grouped_gemm_fp8(x, xe, W, We, again, offsets=off, ws=status)
    assert torch.equal(y, again)
    if G == 1 and not lead and not tail:           # no offsets: one group of all rows
        again.fill_(0)
        moe.moe_grouped_gemm_fp8(x, xe, W[0], We[0], again)
        assert torch.equal(y, again)


@pytest.mark.parametrize("G,R,N,K,lead,tail", CASES)
def test_gated_product(moe, status, G, R, N, K, lead, tail):
    x, xe, [(W1, e1), (W3, e3)] = operands(G * R + K, G, R, N, K, 2)
    xe = xe - 10                                   # gates on both sides of zero and not all saturated
    bounds = spread(G, R, lead, tail, N)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    act = torch.full((R, N), 777.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_gated_gemm_fp8(x, xe, W1, e1, W3, e3, act, offsets=off, ws=status)
    g, gm = product64(x, xe, W1, e1, bounds)
    u, um = product64(x, xe, W3, e3, bounds)
    none = torch.isnan(g)
    assert bool((act[none] == 777.0).all())
    silu = g * torch.sigmoid(g)
    ref = silu * u
    unit = (K / 32 + 1) * 2.0 ** -22
    tol = (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 1.1 * unit * gm * (u.abs() + unit * um) + \
        silu.abs() * unit * um + 2.0 ** -133       # bf16's smallest step
    over = ((act.double() - ref).abs() > tol) & ~none
    assert not bool(over.any()), (int(over.sum()), over.nonzero()[:4].tolist())


def quantize64(x):
    """(codes' values, exponents) by the definition, in 64 bits."""
    R, K = x.shape
    x = x.double().cpu()
    vals, exps = torch.empty_like(x), torch.empty((R, blocks(K)), dtype=torch.int32)
    grid = TABLE[:127]
    for b in range(blocks(K)):
        col = x[:, b * 128:(b + 1) * 128]
        top = col.abs().amax(1)
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0)).long() - 1
        for _ in range(3):
            e = torch.where(top > 448.0 * torch.ldexp(torch.ones_like(top), e), e + 1, e)
        e = torch.where(top == 0, torch.zeros_like(e), e.clamp(-117, 120))
        v = torch.ldexp(col.abs(), -e[:, None])
        hi = torch.searchsorted(grid, v.contiguous()).clamp(1, 126)
        down, up = v - grid[hi - 1], grid[hi] - v
        take = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
        vals[:, b * 128:(b + 1) * 128] = torch.sign(col) * grid[take]
        exps[:, b] = e
    return vals, exps


@pytest.mark.parametrize("src,R,K", [(1, 1, 16), (3, 1, 128), (5, 11, 144), (64, 64, 272),
                                     (7, 300, 2048), (1000, 77, 6144), (2, 4, 4112)])
def test_quantize(moe, status, src, R, K):
    gen = torch.Generator().manual_seed(src + R + K)
    x = torch.randn(src, K, generator=gen) * torch.exp2(torch.randint(-30, 30, (src, 1), generator=gen).float())
    x[torch.rand(src, K, generator=gen) < 0.1] = 0
    x[0, :min(K, 128)] = 0                          # a block of zeros
    x[-1, 3] = 448.0                                # exactly on, and just over, the border of an exponent
    x[-1, K - 1] = 450.0
    x = x.to(torch.bfloat16).cuda()
    idx = torch.randint(0, src, (R,), generator=gen, dtype=torch.int32)
    idx[-1] = src - 1
    idx = idx.cuda()
    codes = torch.empty((R, K), dtype=torch.uint8, device="cuda")
    exps = torch.empty((R, blocks(K)), dtype=torch.int8, device="cuda")
    moe.moe_quantize_fp8(x, codes, exps, idx=idx, ws=status)
    vals, e = quantize64(x[idx.long()])
    assert torch.equal(exps.cpu().int(), e.int())
    assert torch.equal(TABLE[codes.cpu().long()], vals)
    if R <= src:
        moe.moe_quantize_fp8(x[:R].contiguous(), codes, exps, ws=status)
        vals, e = quantize64(x[:R])
        assert torch.equal(exps.cpu().int(), e.int()) and torch.equal(TABLE[codes.cpu().long()], vals)


def test_quantize_every_bf16_value(moe, status):
    """Each finite bf16 magnitude alone in its block, both signs: the exponent's
    clamp at -117, subnormals and the largest values."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    x = torch.zeros((bits.numel(), 16), dtype=torch.int16)
    x[:, 3] = bits.to(torch.int16)
    x[:, 9] = (bits | 0x8000).to(torch.int16)
    x = x.view(torch.bfloat16).cuda()
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    exps = torch.empty((x.shape[0], 1), dtype=torch.int8, device="cuda")
    moe.moe_quantize_fp8(x, codes, exps, ws=status)
    vals, e = quantize64(x)
    assert torch.equal(exps.cpu().int(), e.int())
    assert torch.equal(TABLE[codes.cpu().long()], vals)


def test_quantize_marks_nonfinite_and_bad_rows(moe):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.ones((3, 256), dtype=torch.bfloat16, device="cuda")
    x[1, 5], x[1, 6], x[1, 200] = float("nan"), -float("inf"), float("inf")
    codes = torch.full((3, 256), 9, dtype=torch.uint8, device="cuda")
    exps = torch.full((3, 2), 9, dtype=torch.int8, device="cuda")
    moe.moe_quantize_fp8(x, codes, exps, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_NONFINITE
    want = codes[0].clone()
    assert torch.equal(codes[2], want) and torch.equal(exps[1], exps[0])
    marked = (codes[1] & 0x7f) == 0x7f
    assert marked.nonzero().flatten().tolist() == [5, 6, 200]
    assert torch.equal(codes[1][~marked], want[~marked])
    idx = torch.tensor([0, 3, -1], dtype=torch.int32, device="cuda")
    codes.fill_(9), exps.fill_(9)
    moe.moe_quantize_fp8(x, codes, exps, idx=idx, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BOUNDS
    assert torch.equal(codes[0], want) and not bool(codes[1:].any()) and not bool(exps[1:].any())


def test_nan_codes_stay_in_their_row_and_column(moe):
    x, xe, [(W, We)] = operands(5, 1, 40, 256, 384)
    y = torch.empty((40, 256), dtype=torch.float32, device="cuda")
    moe.moe_grouped_gemm_fp8(x, xe, W, We, y)
    x[7, 100], W[0, 130, 383] = 0x7f, 0xff
    z = torch.empty_like(y)
    moe.moe_grouped_gemm_fp8(x, xe, W, We, z)
    assert bool(torch.isnan(z[7]).all()) and bool(torch.isnan(z[:, 130]).all())
    keep = torch.ones_like(z, dtype=torch.bool)
    keep[7], keep[:, 130] = False, False
    assert torch.equal(z[keep], y[keep])


def test_device_side_refusals(moe):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x, xe, [(W, We)] = operands(6, 3, 20, 64, 256)
    y = torch.full((20, 64), 5.0, device="cuda")
    for off in ([0, 9, 4, 20], [0, 5, 9, 21], [-1, 5, 9, 20], [0, 30, 9, 20]):
        moe.moe_grouped_gemm_fp8(x, xe, W, We, y, ws=ws,
                                 offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BOUNDS, off
        assert bool((y == 5.0).all())
    good = torch.tensor([0, 5, 9, 20], dtype=torch.int32, device="cuda")
    for which, at in ((xe, (3, 1)), (We, (2, 0, 0))):
        kept = which[at].item()
        which[at] = -128
        moe.moe_grouped_gemm_fp8(x, xe, W, We, y, offsets=good, ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_BOUNDS
        which[at] = kept
    moe.moe_grouped_gemm_fp8(x, xe, W, We, y, offsets=good, ws=ws)
    assert moe.moe_get_device_status(ws) == 0


def test_extreme_exponents(moe, status):
    """Exponents at both ends of int8 whose sums stay within fp32."""
    x, xe, [(W, We)] = operands(8, 1, 17, 64, 256)
    xe[:], We[:] = 127, -127
    xe[3], xe[4] = 60, 120
    y = torch.empty((17, 64), dtype=torch.float32, device="cuda")
    moe.moe_grouped_gemm_fp8(x, xe, W, We, y, ws=status)
    ref, mag = product64(x, xe, W, We, [0, 17])
    assert bool(((y.double() - ref).abs() <= 9 * 2.0 ** -22 * mag).all())


def test_on_another_stream_and_in_a_graph(moe, status):
    G, R, N, K = 6, 100, 256, 512
    x, xe, [(W, We)] = operands(9, G, R, N, K)
    off = torch.tensor(spread(G, R, 0, 0, 1), dtype=torch.int32, device="cuda")
    want = torch.empty((R, N), device="cuda")
    moe.moe_grouped_gemm_fp8(x, xe, W, We, want, offsets=off)
    y = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_grouped_gemm_fp8(x, xe, W, We, y, offsets=off, ws=status)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    h = torch.randn((R, K), device="cuda").to(torch.bfloat16)
    c = torch.empty((R, K), dtype=torch.uint8, device="cuda")
    e = torch.empty((R, 4), dtype=torch.int8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_quantize_fp8(h, c, e, ws=status)
        moe.moe_grouped_gemm_fp8(c, e, W, We, y, offsets=off, ws=status)
    for k in range(3):
        h.copy_(torch.randn((R, K), device="cuda"))
        graph.replay()
        moe.moe_quantize_fp8(h, x, xe)
        moe.moe_grouped_gemm_fp8(x, xe, W, We, want, offsets=off)
        assert torch.equal(y, want) and torch.equal(c, x)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_exponents_at_any_address(moe, status, shift):
    """Exponent arrays that start and end off every alignment, with the bytes
    around them holding what would be refused."""
    def moved(t):
        raw = torch.full((t.numel() + 8,), -128, dtype=torch.int8, device="cuda")
        view = raw[shift:shift + t.numel()].view(t.shape)
        view.copy_(t)
        return view

    for G, R, N, K in ((3, 50, 136, 1424), (1, 300, 72, 272), (1, 1, 256, 2048)):
        x, xe, [(W, We), (W3, We3)] = operands(shift + R, G, R, N, K, 2)
        off = torch.tensor(spread(G, R, 0, 0, 1), dtype=torch.int32, device="cuda")
        a, b = torch.empty((R, N), device="cuda"), torch.empty((R, N), device="cuda")
        moe.moe_grouped_gemm_fp8(x, xe, W, We, a, offsets=off, ws=status)
        moe.moe_grouped_gemm_fp8(x, moved(xe), W, moved(We), b, offsets=off, ws=status)
        assert torch.equal(a, b)
        a, b = a.bfloat16(), b.bfloat16()
        moe.moe_gated_gemm_fp8(x, xe - 9, W, We, W3, We3, a, offsets=off, ws=status)
        moe.moe_gated_gemm_fp8(x, moved(xe - 9), W, moved(We), W3, moved(We3), b, offsets=off, ws=status)
        assert torch.equal(a, b)


def test_wide_rows_and_every_row_tile(moe, status):
    """Average group sizes on both sides of every row-tile width, with columns
    enough that the widths are chosen by the rows."""
    for avg in (31, 33, 60, 70, 92, 100, 120, 142, 150, 170, 239, 250):
        G, N, K = 12, 1664, 144
        x, xe, [(W, We)] = operands(avg, G, avg * G, N, K)
        bounds = spread(G, avg * G, 0, 0, avg)
        off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        y = torch.empty((avg * G, N), device="cuda")
        moe.moe_grouped_gemm_fp8(x, xe, W, We, y, offsets=off, ws=status)
        ref, mag = product64(x, xe, W, We, bounds)
        assert bool(((y.double() - ref).abs() <= (K / 32 + 1) * 2.0 ** -22 * mag).all()), avg


@pytest.mark.parametrize("T,D,E,F,k", [(37, 256, 12, 144, 3), (300, 384, 8, 256, 2)])
def test_expert_ffn_from_8bit_products(moe, T, D, E, F, k):
    """Routing, grouping, the two products with their quantisations, and the
    merge, one after the other on one stream, as a layer with 8-bit activations
    runs; every step against its definition on the step before, and the whole
    against the layer with bf16 activations within what the roundings to E4M3
    (half a step, 2^-4, or half the subnormal step, 2^-10 of the block's scale)
    can make of it."""
    gen = torch.Generator().manual_seed(T)
    import moe_inputs as mi
    d = moe.dims(T=T, D=D, E=E, F=F, k=k, S=0, Fs=16, scale=2.5)
    ws = moe.alloc_workspace(d)
    h = torch.randn(T, D, generator=gen).to(torch.bfloat16).cuda()
    Wr, bias = (torch.randn(E, D, generator=gen) / D ** 0.5).cuda(), torch.zeros(E, device="cuda")
    W = {n: mi.quantize_fp8_blocks((torch.randn(E, r, c, generator=gen) / c ** 0.5).bfloat16().cuda())
         for n, (r, c) in dict(W1=(F, D), W3=(F, D), W2=(D, F)).items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, inv, rw = torch.empty((T, k), **i32), torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    counts, off, perm = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    logits, R = torch.empty((T, E), device="cuda"), T * k
    xq, aq = (torch.empty((R, n), dtype=torch.uint8, device="cuda") for n in (D, F))
    xe, ae = (torch.empty((R, blocks(n)), dtype=torch.int8, device="cuda") for n in (D, F))
    act = torch.empty((R, F), dtype=torch.bfloat16, device="cuda")
    y, out = torch.empty((R, D), device="cuda"), torch.empty((T, D), device="cuda")

    def layer():
        moe.moe_router_logits(h, Wr, d, logits, ws)
        moe.moe_route(logits, bias, d, idx, rw, ws)
        moe.moe_permute(idx, d, counts, off, perm, inv, ws)
        moe.moe_quantize_fp8(h, xq, xe, idx=perm, ws=ws)
        moe.moe_gated_gemm_fp8(xq, xe, *W["W1"], *W["W3"], act, offsets=off, ws=ws)
        moe.moe_quantize_fp8(act, aq, ae, ws=ws)
        moe.moe_grouped_gemm_fp8(aq, ae, *W["W2"], y, offsets=off, ws=ws)
        moe.moe_combine(y, rw, inv, d, out, ws)

    layer()
    assert moe.moe_get_device_status(ws) == 0
    bounds = off.tolist()
    vals, e = quantize64(h[perm.long()])
    assert torch.equal(TABLE[xq.cpu().long()], vals) and torch.equal(xe.cpu().int(), e.int())
    g, gm = product64(xq, xe, *W["W1"], bounds)
    u, um = product64(xq, xe, *W["W3"], bounds)
    unit = (D / 32 + 1) * 2.0 ** -22
    silu = g * torch.sigmoid(g)
    tol = (2.0 ** -8 + 2.0 ** -16) * (silu * u).abs() + 1.1 * unit * gm * (u.abs() + unit * um) + \
        silu.abs() * unit * um + 2.0 ** -133
    assert bool(((act.double() - silu * u).abs() <= tol).all())
    vals, e = quantize64(act)
    assert torch.equal(TABLE[aq.cpu().long()], vals) and torch.equal(ae.cpu().int(), e.int())
    ref, mag = product64(aq, ae, *W["W2"], bounds)
    assert bool(((y.double() - ref).abs() <= (F / 32 + 1) * 2.0 ** -22 * mag).all())

    # the whole, with activations that are not rounded to 8 bits
    x = h.double()[perm.long()]
    eh = 2.0 ** -4 * x.abs() + 2.0 ** -10 * torch.pow(2.0, xe.double().cpu()).cuda().repeat_interleave(128, 1)[:, :D]
    whole, err = torch.zeros_like(out, dtype=torch.float64), torch.zeros_like(out, dtype=torch.float64)
    for b in range(E):
        r = slice(bounds[b], bounds[b + 1])
        m1, m3, m2 = (matrix64(W[n][0][b], W[n][1][b]) for n in ("W1", "W3", "W2"))
        gg, uu = x[r] @ m1.t(), x[r] @ m3.t()
        eg, eu = eh[r] @ m1.abs().t(), eh[r] @ m3.abs().t()
        s = gg * torch.sigmoid(gg)
        ea = 1.1 * eg * (uu.abs() + eu) + s.abs() * eu
        step = torch.pow(2.0, ae[r].double().cpu()).cuda().repeat_interleave(128, 1)[:, :F]
        ea = ea + (2.0 ** -4 + 2.0 ** -7) * ((s * uu).abs() + ea) + 2.0 ** -10 * step
        c = rw.double().flatten()[torch.argsort(inv.flatten())][r, None]
        whole.index_add_(0, perm[r].long(), c * ((s * uu) @ m2.t()))
        err.index_add_(0, perm[r].long(), c * (ea @ m2.abs().t()))
    assert bool(((out.double() - whole).abs() <= 1.001 * err + 1e-5 * whole.abs()).all())
    rel = float((out.double() - whole).norm() / whole.norm())
    assert rel < 2.0 ** -4, rel            # no worse than one rounding of everything

    graph, want = torch.cuda.CUDAGraph(), out.clone()
    with torch.cuda.graph(graph):
        layer()
    out.zero_()
    graph.replay()
    assert torch.equal(out, want) and moe.moe_get_device_status(ws) == 0


def test_the_most_groups(moe, status):
    """1024 groups: most of them empty, one row in many, many rows in a few."""
    G, R, N, K = 1024, 900, 72, 272
    x, xe, [(W, We)] = operands(11, G, R, N, K)
    gen = torch.Generator().manual_seed(4)
    cut = torch.cat([torch.randint(0, R + 1, (500,), generator=gen),
                     torch.randint(0, 40, (523,), generator=gen)]).sort().values.tolist()
    bounds = [0, *cut, R]
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y = torch.empty((R, N), device="cuda")
    moe.moe_grouped_gemm_fp8(x, xe, W, We, y, offsets=off, ws=status)
    ref, mag = product64(x, xe, W, We, bounds)
    assert bool(((y.double() - ref).abs() <= (K / 32 + 1) * 2.0 ** -22 * mag).all())


def test_more_than_2_to_the_31_elements(moe, status):
    """Codes, exponents and outputs whose offsets pass 32 bits."""
    R, K = 360_000, 6144                        # 2.2e9 codes from five rows
    gen = torch.Generator().manual_seed(12)
    x = torch.randn(5, K, generator=gen).to(torch.bfloat16).cuda()
    idx = torch.randint(0, 5, (R,), generator=gen, dtype=torch.int32).cuda()
    codes = torch.empty((R, K), dtype=torch.uint8, device="cuda")
    exps = torch.empty((R, K // 128), dtype=torch.int8, device="cuda")
    moe.moe_quantize_fp8(x, codes, exps, idx=idx, ws=status)
    vals, e = quantize64(x)
    for r in (0, 1, 349_524, 349_526, R - 1):   # around 2^31 / 6144 too
        assert torch.equal(TABLE[codes[r].cpu().long()], vals[idx[r].item()])
        assert torch.equal(exps[r].cpu().int(), e[idx[r].item()].int())
    W, We = rand_codes(gen, (1, 8, K)), rand_exps(gen, (1, 1, K // 128))
    y = torch.empty((R, 8), device="cuda")
    moe.moe_grouped_gemm_fp8(codes, exps, W, We, y, ws=status)
    base, base_e = torch.empty((5, K), dtype=torch.uint8, device="cuda"), torch.empty((5, K // 128), dtype=torch.int8, device="cuda")
    moe.moe_quantize_fp8(x, base, base_e)
    ref, mag = product64(base, base_e, W, We, [0, 5])
    assert bool(((y.double() - ref[idx.long()]).abs() <= (K / 32 + 1) * 2.0 ** -22 * mag[idx.long()]).all())
    del codes, exps, y
    R, N, K = 270_000, 8192, 16                 # 2.2e9 outputs
    x, xe, [(W, We)] = operands(13, 1, 64, N, K)
    xs, es = x.repeat(R // 64 + 1, 1)[:R].contiguous(), xe.repeat(R // 64 + 1, 1)[:R].contiguous()
    y = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(xs, es, W, We, y, ws=status)
    small = torch.empty((64, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(x, xe, W, We, small)
    for r in (0, 131_072, 262_143, 262_144, R - 64):
        at = torch.arange(r, r + 64, device="cuda")
        assert torch.equal(y[r:r + 64], small[at % 64])


@pytest.mark.parametrize("G,R,N,K,gated", [
    (40, 5000, 3848, 144, False),      # up to 160 rows a tile; the last pair's second weight tile is behind N
    (40, 5000, 3976, 400, False),      # the last pair's second weight tile is ragged
    (40, 5000, 2056, 144, True),
    (37, 4400, 2120, 272, True),
    (1, 1001, 15496, 4112, False),     # long K: 240 rows a tile, a pair that ends behind N
    (3, 1400, 15368, 4240, False),
    (1, 700, 13000, 4112, True),
    (1, 1100, 15360, 6160, False),
])
def test_two_weight_tiles_for_the_same_rows(moe, status, G, R, N, K, gated):
    """Many tiles: a CTA takes two neighbouring weight tiles at a time."""
    x, xe, ws = operands(G + R + N + K, G, R, N, K, 2 if gated else 1)
    xe = xe - 10
    bounds = spread(G, R, 1, 2, N)
    if G > 3:                                      # like groups, an empty one, one of a single row
        bounds = [1 + (R - 3) * g // G for g in range(G)] + [R - 2]
        bounds[5] = bounds[6]
        bounds[20] = bounds[21] - 1
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y = torch.full((R, N), 777.0, dtype=torch.bfloat16, device="cuda")
    unit = (K / 32 + 1) * 2.0 ** -22
    if gated:
        call = lambda to: moe.moe_gated_gemm_fp8(x, xe, *ws[0], *ws[1], to, offsets=off, ws=status)
        g, gm = product64(x, xe, *ws[0], bounds)
        u, um = product64(x, xe, *ws[1], bounds)
        silu = g * torch.sigmoid(g)
        ref = silu * u
        tol = (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 1.1 * unit * gm * (u.abs() + unit * um) + \
            silu.abs() * unit * um + 2.0 ** -133
    else:
        call = lambda to: moe.moe_grouped_gemm_fp8(x, xe, *ws[0], to, offsets=off, ws=status)
        ref, mag = product64(x, xe, *ws[0], bounds)
        tol = unit * mag + 2.0 ** -8 * ref.abs()
    call(y)
    none = torch.isnan(ref)
    assert bool(none[0].all()) and bool((y[none] == 777.0).all())
    over = ((y.double() - ref).abs() > tol) & ~none
    assert not bool(over.any()), (int(over.sum()), over.nonzero()[:4].tolist())
    for _ in range(3):
        again = torch.full_like(y, 777.0)
        call(again)
        assert torch.equal(y, again)

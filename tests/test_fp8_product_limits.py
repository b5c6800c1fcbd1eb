"""Sizes at the end of 32 bits: refused on the host where the kernels' index
arithmetic ends (CPU), right just below (GPU)."""
import pytest
import torch

FAKE = 0x7F0000000000   # never dereferenced: every call below is refused
TOP = 2 ** 31


@pytest.fixture(scope="module")
def mod():
    import __graft_entry__
    __graft_entry__._build_module().build()   # no-op unless a source is newer
    import sparse_moe_layer_04_b200 as m
    return m


@pytest.mark.parametrize("G,R,N,K", [(1, TOP - 255, 8, 16), (1, TOP - 1, 8, 16), (1, 5, 8, TOP - 16),
                                     (1, 5, TOP - 8, 16), (1, 5, TOP - 248, 16), (1024, 5, 2 ** 21, 16),
                                     (1, TOP - 8192, 65536, 16)])
def test_products(mod, G, R, N, K):
    for call in (lambda: mod._lib.moe_grouped_gemm_fp8(FAKE, FAKE, FAKE, FAKE, FAKE, G, R, N, K, FAKE, 0, None, None),
                 lambda: mod._lib.moe_gated_gemm_fp8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, G, R, N, K, FAKE,
                                                     None, None)):
        assert call() == mod.MOE_ERR_UNSUPPORTED
        assert "at most 2^31 - 256" in mod.moe_last_error() or "too large" in mod.moe_last_error()


@pytest.mark.parametrize("K", [65535 * 1024 + 16, TOP - 16])
def test_quantize(mod, K):
    assert mod._lib.moe_quantize_fp8(FAKE, 4, FAKE, 4, K, FAKE, FAKE, None, None) == mod.MOE_ERR_UNSUPPORTED
    assert "at most" in mod.moe_last_error()


def test_binding_does_not_cut_sizes_off(mod):
    """2^32 rows would arrive as none and leave the outputs as they were."""
    rows = lambda t, n: t.expand(n, *t.shape[1:])
    x, c, e = torch.zeros(1, 16, dtype=torch.bfloat16), torch.zeros(1, 16, dtype=torch.uint8), \
        torch.zeros(1, 1, dtype=torch.int8)
    n = 2 ** 32
    with pytest.raises(ValueError, match="src = 4294967296"):
        mod.moe_quantize_fp8(rows(x, n), rows(c, n), rows(e, n))
    with pytest.raises(ValueError, match="R = 4294967296"):
        mod.moe_quantize_fp8(x, rows(c, n), rows(e, n), idx=torch.zeros(1, dtype=torch.int32).expand(n))
    W, We, y = torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int8), torch.zeros(1, 8)
    with pytest.raises(ValueError, match="R = 4294967296"):
        mod.moe_grouped_gemm_fp8(rows(c, n), rows(e, n), W, We, rows(y, n))
    with pytest.raises(ValueError, match="R = 4294967296"):
        mod.moe_gated_gemm_fp8(rows(c, n), rows(e, n), W, We, W, We, rows(y.bfloat16(), n))


@pytest.fixture()
def free_gb():
    """Free device memory once the allocator has let go of what earlier tests held."""
    torch.cuda.empty_cache()
    yield torch.cuda.mem_get_info()[0] / 1e9
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_quantize_of_2_to_the_31_minus_1_rows(mod, free_gb):
    R, K = TOP - 1, 16
    if free_gb < 60:
        pytest.skip("needs 60 GB")
    x = torch.randn(7, K, device="cuda").to(torch.bfloat16)
    want_c, want_e = torch.empty((7, K), dtype=torch.uint8, device="cuda"), torch.empty((7, 1), dtype=torch.int8, device="cuda")
    mod.moe_quantize_fp8(x, want_c, want_e)
    idx = torch.empty(R, dtype=torch.int32, device="cuda")
    for a in range(0, R, 1 << 28):
        b = min(R, a + (1 << 28))
        idx[a:b] = torch.arange(a, b, device="cuda") % 7
    codes, exps = torch.empty((R, K), dtype=torch.uint8, device="cuda"), torch.empty((R, 1), dtype=torch.int8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    mod.moe_quantize_fp8(x, codes, exps, idx=idx, ws=ws)
    assert mod.moe_get_device_status(ws) == 0
    for a in (0, 2 ** 27 - 4, 2 ** 28, 2 ** 30 - 3, R - 700):
        i = idx[a:a + 700].long()
        assert torch.equal(codes[a:a + 700], want_c[i]) and torch.equal(exps[a:a + 700], want_e[i])


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
def test_product_of_2_to_the_31_minus_256_rows(mod, gated, free_gb):
    R, N, K = TOP - 256, 8, 16
    if free_gb < 110:
        pytest.skip("needs 110 GB")
    gen = torch.Generator().manual_seed(3)
    codes = lambda *s: torch.randint(0, 0x7f, s, generator=gen, dtype=torch.int32).to(torch.uint8).cuda()
    x, xe = codes(64, K), torch.randint(-12, -8, (64, 1), generator=gen, dtype=torch.int32).to(torch.int8).cuda()
    W, We, W3 = codes(N, K), torch.zeros((1, 1), dtype=torch.int8, device="cuda"), codes(N, K)

    def call(a, ae, y):
        if gated:
            mod.moe_gated_gemm_fp8(a, ae, W, We, W3, We, y, ws=ws)
        else:
            mod.moe_grouped_gemm_fp8(a, ae, W, We, y, ws=ws)

    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = torch.empty((64, N), dtype=torch.bfloat16, device="cuda")
    call(x, xe, want)
    xs, es = torch.empty((R, K), dtype=torch.uint8, device="cuda"), torch.empty((R, 1), dtype=torch.int8, device="cuda")
    xs.view(-1, 64 * K).copy_(x.view(1, -1).expand(R // 64, -1))
    es.view(-1, 64).copy_(xe.view(1, -1).expand(R // 64, -1))
    y = torch.full((R, N), 777.0, dtype=torch.bfloat16, device="cuda")
    call(xs, es, y)
    assert mod.moe_get_device_status(ws) == 0
    for part in y.view(-1, 64 * N).split(1 << 20):
        assert bool((part == want.view(1, -1)).all())

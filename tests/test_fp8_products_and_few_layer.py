"""Host-side refusals of the 8-bit products and of the few-token layer, by the
C entry points and by the binding.  Nothing is launched and no fake pointer is
dereferenced, with or without a GPU."""
import ctypes

import pytest
import torch

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def mod():
    import __graft_entry__
    __graft_entry__._build_module().build()   # no-op unless a source is newer
    import sparse_moe_layer_04_b200 as m
    return m


def refused(mod, rc, code, text):
    assert rc == code, (rc, mod.moe_last_error())
    assert text in mod.moe_last_error(), mod.moe_last_error()


QUANTIZE = dict(x=FAKE, src=4, idx=FAKE, R=8, K=256, codes=FAKE, exps=FAKE, ws=FAKE)


@pytest.mark.parametrize("change,code,text", [
    (dict(src=-1), -1, ">= 0"), (dict(R=-1), -1, ">= 0"), (dict(K=24), -1, "multiple of 16"),
    (dict(K=0), -1, "multiple of 16"), (dict(idx=None), -1, "without an index"),
    (dict(x=None), -1, "x is NULL"), (dict(x=FAKE + 8), -1, "x is not 16-byte"),
    (dict(codes=None), -1, "codes is NULL"), (dict(codes=FAKE + 4), -1, "codes is not"),
    (dict(exps=None), -1, "exps is NULL"), (dict(idx=FAKE + 4), -1, "idx is not"),
    (dict(ws=FAKE + 16), -4, "256-byte")])
def test_quantize_refusals(mod, change, code, text):
    a = {**QUANTIZE, **change}
    refused(mod, mod._lib.moe_quantize_fp8(a["x"], a["src"], a["idx"], a["R"], a["K"], a["codes"],
                                           a["exps"], a["ws"], None), code, text)


PRODUCT = dict(x=FAKE, xe=FAKE, off=FAKE, W=FAKE, We=FAKE, W3=FAKE, W3e=FAKE, G=4, R=8, N=64, K=256,
               y=FAKE, ws=FAKE)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("change,code,text", [
    (dict(G=0), -1, "G = 0"), (dict(G=1025), -1, "G = 1025"), (dict(R=-1), -1, "R = -1"),
    (dict(N=12), -1, "N = 12"), (dict(N=0), -1, "N = 0"), (dict(K=40), -1, "K = 40"),
    (dict(G=1024, N=1 << 21), -2, "2^31"), (dict(R=(1 << 31) - 1, N=1 << 13), -2, "too large"),
    (dict(off=None), -1, "offsets is NULL"), (dict(off=FAKE + 4), -1, "offsets is not"),
    (dict(x=None), -1, "x is NULL"), (dict(x=FAKE + 1), -1, "x is not"),
    (dict(xe=None), -1, "xe is NULL"), (dict(W=None), -1, "is NULL"), (dict(W=FAKE + 8), -1, "is not"),
    (dict(We=None), -1, "e is NULL"), (dict(y=None), -1, "y is NULL"), (dict(y=FAKE + 4), -1, "y is not"),
    (dict(ws=FAKE + 64), -4, "256-byte")])
def test_product_refusals(mod, gated, change, code, text):
    a = {**PRODUCT, **change}
    if gated:
        rc = mod._lib.moe_gated_gemm_fp8(a["x"], a["xe"], a["off"], a["W"], a["We"], a["W3"], a["W3e"],
                                         a["G"], a["R"], a["N"], a["K"], a["y"], a["ws"], None)
    else:
        rc = mod._lib.moe_grouped_gemm_fp8(a["x"], a["xe"], a["off"], a["W"], a["We"], a["G"], a["R"],
                                           a["N"], a["K"], a["y"], 0, a["ws"], None)
    refused(mod, rc, code, text)


def test_gated_product_needs_both_weights(mod):
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 8, 64, 256, FAKE, None, None]
    for at, text in ((5, "W3 is NULL"), (6, "W3e is NULL")):
        bad = list(args)
        bad[at] = None
        refused(mod, mod._lib.moe_gated_gemm_fp8(*bad), -1, text)


def test_nothing_to_do_is_no_error(mod):
    lib = mod._lib
    assert lib.moe_quantize_fp8(None, 0, None, 0, 16, None, None, None, None) == 0
    assert lib.moe_grouped_gemm_fp8(None, None, None, None, None, 1, 0, 8, 16, None, 0, None, None) == 0
    assert lib.moe_gated_gemm_fp8(None, None, None, None, None, None, None, 1, 0, 8, 16, None, None,
                                  None) == 0
    d = mod.dims(T=0, D=128, E=8, F=64, k=2)
    assert lib.moe_forward_few(*([None] * 9), ctypes.byref(d), None, None, None, None, 0, None) == 0
    assert lib.moe_forward_few_fp8(None, None, None, None, ctypes.byref(d), None, None, None, None, 0,
                                   None) == 0
    assert mod.moe_last_launch_count() == 0


def few(mod, fp8, d, ptrs=(FAKE, FAKE, FAKE), out=FAKE, idx=None, w=None, ws=FAKE, n=1 << 40, w8=None):
    if fp8:
        q = mod.moe_fp8_weights_t()
        for name, _ in mod.moe_fp8_weights_t._fields_:
            setattr(q, name, (w8 or {}).get(name, FAKE))
        return mod._lib.moe_forward_few_fp8(*ptrs, ctypes.byref(q), ctypes.byref(d), out, idx, w, ws, n,
                                            None)
    return mod._lib.moe_forward_few(*ptrs, *([FAKE] * 6), ctypes.byref(d), out, idx, w, ws, n, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_few_layer_refusals(mod, fp8):
    ok = dict(T=4, D=128, E=8, F=64, k=2)
    d = mod.dims(**ok)
    need = mod.moe_workspace_size(d)
    refused(mod, few(mod, fp8, mod.dims(**{**ok, "T": 17})), -2, "at most 16 tokens")
    refused(mod, few(mod, fp8, mod.dims(**{**ok, "D": 100})), -1, "D = 100")
    refused(mod, few(mod, fp8, mod.dims(**{**ok, "k": 9})), -1, "k = 9")
    refused(mod, few(mod, fp8, d, ptrs=(None, FAKE, FAKE)), -1, "h is NULL")
    refused(mod, few(mod, fp8, d, ptrs=(FAKE, FAKE + 4, FAKE)), -1, "Wr is not")
    refused(mod, few(mod, fp8, d, ptrs=(FAKE, FAKE, None)), -1, "bias is NULL")
    refused(mod, few(mod, fp8, d, out=None), -1, "out is NULL")
    refused(mod, few(mod, fp8, d, idx=FAKE + 4), -1, "idx_out is not")
    refused(mod, few(mod, fp8, d, w=FAKE + 4), -1, "w_out is not")
    refused(mod, few(mod, fp8, d, ws=None), -4, "NULL")
    refused(mod, few(mod, fp8, d, ws=FAKE + 16), -4, "256-byte")
    refused(mod, few(mod, fp8, d, n=need - 1), -4, "needs")
    if fp8:
        refused(mod, few(mod, fp8, mod.dims(**{**ok, "D": 136})), -1, "multiple of 16")
        refused(mod, few(mod, fp8, d, w8=dict(W2=None)), -1, "W2 is NULL")
        refused(mod, few(mod, fp8, d, w8=dict(Ws1e=None)), -1, "Ws*e")


def test_few_layer_counters_stand_still_over_T(mod):
    """One workspace serves every T: it is never smaller for a larger T up to 16."""
    sizes = [mod.moe_workspace_size(mod.dims(T=t, D=256, E=16, F=128, k=4)) for t in range(1, 17)]
    assert max(sizes) == sizes[-1]


@pytest.fixture()
def on_cpu(mod, monkeypatch):
    """Lets host tensors pass for tensors of the current device, so that what is
    wrong with one argument is reached; every call below is refused before the
    library is entered."""
    monkeypatch.setattr(mod, "_device", lambda: -1)
    return mod


def test_binding_refusals_quantize(on_cpu):
    z, f = torch.zeros, on_cpu.moe_quantize_fp8
    x, c, e = z(4, 256, dtype=torch.bfloat16), z(4, 256, dtype=torch.uint8), z(4, 2, dtype=torch.int8)
    for args, kind, text in (((x, c[:3], e), ValueError, "codes"), ((x, c, e[:, :1]), ValueError, "exps"),
                             ((x.float(), c, e), TypeError, "x: expected"),
                             ((x, c.int(), e), TypeError, "codes"), ((x[0], c, e), ValueError, "x "),
                             ((x.t().contiguous().t(), c, e), ValueError, "contiguous"),
                             ((x, c, e, z(3, dtype=torch.int32)), ValueError, "codes"),
                             ((x, c, e, z(4, dtype=torch.int64)), TypeError, "idx"),
                             ((x, c, e, None, z(8)), TypeError, "ws"),
                             ((x, c, None), TypeError, "exps: expected a tensor"),
                             ((x, None, e), TypeError, "codes")):
        with pytest.raises(kind, match=text):
            f(*args)


def test_binding_refusals_products(on_cpu):
    z, u8, i8 = torch.zeros, torch.uint8, torch.int8
    c, e = z(4, 256, dtype=u8), z(4, 2, dtype=i8)
    W, We, y = z(3, 64, 256, dtype=u8), z(3, 1, 2, dtype=i8), z(4, 64)
    off = z(4, dtype=torch.int32)
    for args, kw, kind, text in (
            ((c, e, W, We, y[:, :32].contiguous()), dict(offsets=off), ValueError, "y: expected shape"),
            ((c, e, W, We, y), dict(offsets=off[:3]), ValueError, "offsets"),
            ((c, e, W, We, y), dict(offsets=off.long()), TypeError, "offsets"),
            ((c, e, W, We[:2], y), dict(offsets=off), ValueError, "We"),
            ((c, e[:, :1], W, We, y), dict(offsets=off), ValueError, "xe"),
            ((c, e, W, We, y.half()), dict(offsets=off), TypeError, "y"),
            ((c, e, W.short(), We, y), dict(offsets=off), TypeError, "W"),
            ((c, e, W, We, y), dict(offsets=off, ws=z(256)), TypeError, "ws")):
        with pytest.raises(kind, match=text):
            on_cpu.moe_grouped_gemm_fp8(*args, **kw)
    act = y.to(torch.bfloat16)
    for args, kind, text in (((c, e, W, We, W[:2], We, act), ValueError, "W3"),
                             ((c, e, W, We, W, We[:1], act), ValueError, "W3e"),
                             ((c, e, W, We, W, We, y), TypeError, "act")):
        with pytest.raises(kind, match=text):
            on_cpu.moe_gated_gemm_fp8(*args, offsets=off)


def test_binding_refusals_few_layer(on_cpu):
    z, bf = torch.zeros, torch.bfloat16
    d = on_cpu.dims(T=4, D=256, E=8, F=64, k=2)
    h, Wr, bias, out = z(4, 256, dtype=bf), z(8, 256), z(8), z(4, 256)
    W1, W2 = z(8, 64, 256, dtype=bf), z(8, 256, 64, dtype=bf)
    S1, S2, ws = W1[:1], W2[:1], z(16, dtype=torch.uint8)
    good = dict(h=h, Wr=Wr, bias=bias, W1=W1, W3=W1, W2=W2, Ws1=S1, Ws3=S1, Ws2=S2, d=d, out=out, ws=ws)
    for change, kind, text in ((dict(h=h[:3]), ValueError, "h: "), (dict(Wr=Wr.to(bf)), TypeError, "Wr"),
                               (dict(bias=bias[:4]), ValueError, "bias"), (dict(W2=W1), ValueError, "W2"),
                               (dict(W3=W1.float()), TypeError, "W3"), (dict(Ws2=S1), ValueError, "Ws2"),
                               (dict(out=out.to(bf)), TypeError, "out"),
                               (dict(idx_out=z(4, 3, dtype=torch.int32)), ValueError, "idx_out"),
                               (dict(w_out=z(4, 2, dtype=bf)), TypeError, "w_out"),
                               (dict(W1=None), TypeError, "W1: expected a tensor"),
                               (dict(ws=z(16)), TypeError, "ws")):
        with pytest.raises(kind, match=text):
            on_cpu.moe_forward_few(**{**good, **change})
    q = on_cpu.moe_fp8_weights_t()
    for change, kind, text in ((dict(h=h[:3]), ValueError, "h: "), (dict(out=out[:2]), ValueError, "out")):
        kw = {**dict(h=h, Wr=Wr, bias=bias, w8=q, d=d, out=out, ws=ws), **change}
        with pytest.raises(kind, match=text):
            on_cpu.moe_forward_few_fp8(**kw)


def test_binding_refuses_host_tensors(mod):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mod.moe_quantize_fp8(x, torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.int8))

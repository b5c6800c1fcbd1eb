"""Cases, inputs, plain forms and exact results of the 8-bit products and of the few-token layer.

Four operators:

  quantize   bf16 rows (gathered by an index) -> E4M3 codes with one power-of-two
             exponent per 128 columns of each row
  gemm       grouped product of such rows with E4M3 weights that have one exponent
             per 128 x 128 block
  gated      the same rows against two weights, silu(gate) * up, rounded to bf16
  few        the whole mixture-of-experts layer for 1..16 tokens, with bf16 or E4M3
             expert weights

An E4M3 code c with exponent e stands for e4m3(c) * 2**e everywhere.
"""
import math

import torch

own = False

B = 128          # columns (and weight rows) that share an exponent
TOP = 448.0      # the largest E4M3 value


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    """Sizes are those of the repository's own layer configurations (hidden 6144, 256 experts of width
    2048; hidden 4096, 128 experts of width 1408; the tiny layer), with top-8 routing."""
    return [
        # the rows of 13 tokens on their way to 8 experts each (a decode step)
        dict(name="quantize 104 rows", op="quantize", src=13, R=104, K=6144),
        # a prefill chunk's rows, gathered eightfold for the routed experts
        dict(name="quantize 32768 rows", op="quantize", src=4096, R=32768, K=6144),
        # one token through one down projection: launch and weight-stream latency
        dict(name="gemm 1 row", op="gemm", G=1, R=1, N=6144, K=2048, out="float32"),
        # a decode batch's down projections: about four rows for each of 256 experts
        dict(name="gemm 256 experts, 1024 rows", op="gemm", G=256, R=1024, N=6144, K=2048, out="float32"),
        # a prefill chunk through one dense projection
        dict(name="gemm dense 4099 rows", op="gemm", G=1, R=4099, N=6144, K=6144, out="bfloat16"),
        # a prefill batch's down projections of the narrower layer, K not a multiple of 256
        dict(name="gemm 128 experts, 32768 rows", op="gemm", G=128, R=32768, N=4096, K=1408, out="float32"),
        # a decode batch's gate and up projections
        dict(name="gated 128 experts, 509 rows", op="gated", G=128, R=509, N=1408, K=4096),
        # a prefill chunk's gate and up projections
        dict(name="gated 64 experts, 8192 rows", op="gated", G=64, R=8192, N=2048, K=6144),
        # one token of an interactive session through the large layer
        dict(name="few 1 token", op="few", w="bfloat16", T=1, D=6144, E=256, F=2048, k=8, S=1, Fs=2048, scale=2.5),
        # a few sessions through the narrower layer
        dict(name="few 11 tokens", op="few", w="bfloat16", T=11, D=4096, E=128, F=1408, k=8, S=1, Fs=1408, scale=1.0),
        # the tiny layer: latency alone
        dict(name="few 5 tokens tiny", op="few", w="bfloat16", T=5, D=128, E=8, F=64, k=2, S=1, Fs=64, scale=2.5),
        # a few sessions through the large layer with 8-bit experts
        dict(name="few 4 tokens 8-bit", op="few", w="float8", T=4, D=6144, E=256, F=2048, k=8, S=1, Fs=2048, scale=2.5),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number between lo and hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gated", "few", "few"])
    if op == "quantize":
        return dict(op=op, src=_log(rng, 1, 4096), R=_log(rng, 1, 32768), K=_log(rng, 16, 6144, 16))
    if op in ("gemm", "gated"):
        while True:
            c = dict(op=op, G=_log(rng, 1, 256), R=_log(rng, 1, 32768), N=_log(rng, 8, 6144, 8),
                     K=_log(rng, 64, 6144, 16))
            weights = c["G"] * c["N"] * c["K"] * (2 if op == "gated" else 1)
            if weights <= 3.2e9 and work(c)["flops"] <= 3.7e11:
                break
        if op == "gemm":
            c["out"] = rng.choice(["float32", "bfloat16"])
        return c
    while True:
        w = rng.choice(["bfloat16", "float8"])
        step = 8 if w == "bfloat16" else 16
        E = _log(rng, 4, 256)
        c = dict(op=op, w=w, T=rng.randint(1, 16), D=_log(rng, 64, 6144, step), E=E,
                 F=_log(rng, 32, 2048, step), k=rng.randint(1, min(8, E)), S=rng.choice([0, 1, 1, 2]),
                 Fs=_log(rng, 32, 2048, step), scale=rng.choice([1.0, 2.5]))
        if work(c)["bytes"] <= 1.2e9:
            return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _normal(gen, shape, std, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def _codes(gen, shape, std):
    """E4M3 codes of normal values of the given spread (in units of the codes)."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        v = _normal(gen, (n,), std, torch.bfloat16).clamp_(-TOP, TOP)
        flat[i:i + n] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _exps(gen, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").to(torch.int8)


def _weight8(gen, G, N, K):
    """G matrices as a quantiser leaves them: the block's largest value near 448, entries of about
    1 / sqrt(K) in all."""
    mid = int(round(math.log2(1.0 / (105.0 * math.sqrt(K)))))
    return (_codes(gen, (G, N, K), 105.0),
            _exps(gen, (G, -(-N // B), -(-K // B)), mid - 1, mid))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "quantize":
        # hidden rows with a few large channels, as residual streams have them
        x = _normal(gen, (case["src"], case["K"]), 1.0, torch.float32)
        x *= torch.exp(_normal(gen, (1, case["K"]), 0.7, torch.float32))
        st["x"] = x.to(torch.bfloat16)
        st["idx"] = torch.randint(0, case["src"], (case["R"],), generator=gen, device="cuda",
                                  dtype=torch.int32)
        if own:
            st["codes"] = torch.empty((case["R"], case["K"]), dtype=torch.uint8, device="cuda")
            st["exps"] = torch.empty((case["R"], -(-case["K"] // B)), dtype=torch.int8, device="cuda")
        return st
    if op in ("gemm", "gated"):
        G, R, N, K = case["G"], case["R"], case["N"], case["K"]
        st["x"] = _codes(gen, (R, K), 130.0)
        st["xe"] = _exps(gen, (R, -(-K // B)), -8, -6)
        group, _ = torch.sort(torch.randint(0, G, (R,), generator=gen, device="cuda"))
        counts = torch.bincount(group, minlength=G)
        st["offsets"] = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        st["offsets"][1:] = torch.cumsum(counts, 0)
        st["most"] = int(counts.max())
        st["W"], st["We"] = _weight8(gen, G, N, K)
        if op == "gated":
            st["W3"], st["W3e"] = _weight8(gen, G, N, K)
        st["y"] = torch.empty((R, N), device="cuda",
                              dtype=getattr(torch, case.get("out", "bfloat16")))
        return st
    T, D, E, F, S, Fs = (case[n] for n in ("T", "D", "E", "F", "S", "Fs"))
    bf = torch.bfloat16
    st["h"] = _normal(gen, (T, D), 1.0, bf)
    st["Wr"] = _normal(gen, (E, D), 1.6 / math.sqrt(D), torch.float32)
    st["bias"] = _normal(gen, (E,), 0.1, torch.float32)
    for name, n, rows, cols in (("W1", E, F, D), ("W3", E, F, D), ("W2", E, D, F),
                                ("Ws1", S, Fs, D), ("Ws3", S, Fs, D), ("Ws2", S, D, Fs)):
        if case["w"] == "bfloat16":
            st[name] = _normal(gen, (n, rows, cols), 1.0 / math.sqrt(cols), bf)
        else:
            st[name], st[name + "e"] = _weight8(gen, n, rows, cols)
    if own:
        import sparse_moe_layer_04_b200 as moe
        st["d"] = moe.dims(T=T, D=D, E=E, F=F, k=case["k"], S=S, Fs=Fs, scale=case["scale"])
        st["ws"] = moe.alloc_workspace(st["d"])
        st["out"] = torch.empty((T, D), dtype=torch.float32, device="cuda")
        st["sel"] = torch.empty((T, case["k"]), dtype=torch.int32, device="cuda")
        st["rw"] = torch.empty((T, case["k"]), dtype=torch.float32, device="cuda")
        if case["w"] == "float8":
            st["w8"] = moe.fp8_weights(*[st[n] if S or "s" not in n else None for n in
                                         ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2", "W1e", "W3e", "W2e",
                                          "Ws1e", "Ws3e", "Ws2e")])
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _run_own(st):
    import sparse_moe_layer_04_b200 as moe
    op = st["case"]["op"]
    if op == "quantize":
        moe.moe_quantize_fp8(st["x"], st["codes"], st["exps"], idx=st["idx"])
        return st["codes"].view(torch.float8_e4m3fn), st["exps"]
    if op == "gemm":
        moe.moe_grouped_gemm_fp8(st["x"], st["xe"], st["W"], st["We"], st["y"], offsets=st["offsets"])
        return st["y"]
    if op == "gated":
        moe.moe_gated_gemm_fp8(st["x"], st["xe"], st["W"], st["We"], st["W3"], st["W3e"], st["y"],
                               offsets=st["offsets"])
        return st["y"]
    if st["case"]["w"] == "bfloat16":
        moe.moe_forward_few(st["h"], st["Wr"], st["bias"], st["W1"], st["W3"], st["W2"], st["Ws1"],
                            st["Ws3"], st["Ws2"], st["d"], st["out"], st["ws"], st["sel"], st["rw"])
    else:
        moe.moe_forward_few_fp8(st["h"], st["Wr"], st["bias"], st["w8"], st["d"], st["out"], st["ws"],
                                st["sel"], st["rw"])
    return st["out"], st["sel"], st["rw"]


def _pow2(e):
    """2**e in fp32, exactly: a rounding here would move values across the borders between codes."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _decoded(codes, exps):
    """fp32 values of rows of E4M3 codes with an exponent per 128 columns."""
    K = codes.shape[-1]
    scale = _pow2(exps).repeat_interleave(B, dim=-1)[..., :K]
    return codes.view(torch.float8_e4m3fn).float() * scale


def _weights(codes, exps):
    """fp32 values of E4M3 matrices [..., rows, K] with 128 x 128 block exponents."""
    rows, K = codes.shape[-2:]
    scale = _pow2(exps).repeat_interleave(B, dim=-2)[..., :rows, :]
    scale = scale.repeat_interleave(B, dim=-1)[..., :K]
    return codes.view(torch.float8_e4m3fn).float().mul_(scale)


def _plain_quantize(x, idx):
    rows = x[idx.long()].float()
    R, K = rows.shape
    nb = -(-K // B)
    blocks = torch.nn.functional.pad(rows, (0, nb * B - K)).view(R, nb, B)
    most = blocks.abs().amax(-1)
    # the smallest e with most <= 448 * 2**e: 448 = 0.875 * 2**9
    frac, power = torch.frexp(most)
    e = torch.where(frac > 0.875, power - 8, power - 9)
    e = torch.where(most == 0, torch.zeros_like(e), e.clamp(-117, 120))
    codes = (blocks * _pow2(-e)[..., None]).view(R, nb * B)[:, :K]
    return codes.to(torch.float8_e4m3fn).contiguous(), e.to(torch.int8)


def _plain_rows(st):
    """Every group's rows side by side [G, most, K] in fp32, and where every row went."""
    x = _decoded(st["x"], st["xe"])
    off = st["offsets"].long()
    r = torch.arange(x.shape[0], device=x.device)
    g = torch.searchsorted(off[1:], r, right=True)
    at = r - off[g]
    padded = torch.zeros((off.numel() - 1, st["most"], x.shape[1]), device=x.device)
    padded[g, at] = x
    return padded, g, at


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _route(h, Wr, bias, k, scale):
    # in 64 bits up to the operator's own roundings: selection compares neighbouring keys
    logits = (h.double() @ Wr.double().t()).float()
    s = (1.0 / (1.0 + torch.exp(-logits.double()))).float()
    _, order = torch.sort(s + bias, dim=-1, descending=True, stable=True)
    idx = order[:, :k]
    chosen = s.gather(1, idx)
    return idx, chosen / chosen.sum(-1, keepdim=True) * scale


def _pick(st, name, idx):
    """fp32 weights of the experts idx names."""
    if st["case"]["w"] == "bfloat16":
        return st[name][idx].float()
    return _weights(st[name][idx], st[name + "e"][idx])


def run(state):
    st = state
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "quantize":
        return _plain_quantize(st["x"], st["idx"])
    if op == "gemm":
        rows, g, at = _plain_rows(st)
        y = torch.matmul(rows, _weights(st["W"], st["We"]).transpose(1, 2))
        return y[g, at].to(st["y"].dtype)
    if op == "gated":
        rows, g, at = _plain_rows(st)
        gate = torch.matmul(rows, _weights(st["W"], st["We"]).transpose(1, 2))
        up = torch.matmul(rows, _weights(st["W3"], st["W3e"]).transpose(1, 2))
        return (_silu(gate) * up)[g, at].to(st["y"].dtype)
    c = st["case"]
    h = st["h"].float()
    idx, w = _route(st["h"], st["Wr"], st["bias"], c["k"], c["scale"])
    x = h[:, None, :, None]                                       # [T, 1, D, 1]
    act = _silu(_pick(st, "W1", idx) @ x) * (_pick(st, "W3", idx) @ x)
    out = ((_pick(st, "W2", idx) @ act)[..., 0] * w[..., None]).sum(1)
    if c["S"]:
        every = torch.arange(c["S"], device=h.device)
        x = h.t()[None]                                           # [1, D, T]
        act = _silu(_pick(st, "Ws1", every) @ x) * (_pick(st, "Ws3", every) @ x)
        out = out + (_pick(st, "Ws2", every) @ act).sum(0).t()
    return out, idx.to(torch.int32), w


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize":
        R, K = case["R"], case["K"]
        # rows read once each (those that some index names), codes and exponents written
        src = case["src"] * (1.0 - (1.0 - 1.0 / case["src"]) ** R)
        return {"bytes": src * K * 2 + R * 4 + R * K + R * -(-K // B), "flops": 3.0 * R * K}
    if op in ("gemm", "gated"):
        G, R, N, K = case["G"], case["R"], case["N"], case["K"]
        n = 2 if op == "gated" else 1
        used = G * (1.0 - (1.0 - 1.0 / G) ** R)                   # groups with a row
        out = 4 if case.get("out") == "float32" else 2
        return {"bytes": R * K + n * used * N * K + R * N * out, "flops": 2.0 * n * R * N * K}
    T, D, E, F, k, S, Fs = (case[n] for n in ("T", "D", "E", "F", "k", "S", "Fs"))
    used = E * (1.0 - (1.0 - k / E) ** T)                         # experts that some token chose
    size = 2 if case["w"] == "bfloat16" else 1
    weights = 3.0 * D * (used * F + S * Fs)
    return {"bytes": weights * size + E * D * 4 + T * D * 6,
            "flops": 2.0 * T * D * E + 6.0 * T * D * (k * F + S * Fs)}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _e4m3_table():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    v = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        a = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v.append(math.nan if (c & 127) == 127 else -a if s else a)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_matrix(table, codes, exps, block_rows):
    """fp64 values of one matrix [rows, K], block by block of columns."""
    out = table[codes.long()]
    rows, K = out.shape
    r = torch.arange(rows, device=out.device) // block_rows
    for b in range(-(-K // B)):
        out[:, b * B:(b + 1) * B] *= torch.pow(2.0, exps[r, b].double())[:, None]
    return out


def _exact_mlp(x, a, b, c):
    g = x @ a.t()
    return (g * torch.sigmoid(g) * (x @ b.t())) @ c.t()


def exact(case, seed):
    op = case["op"]
    if work(case)["flops"] > 3.2e11 and op in ("gemm", "gated"):
        return None
    st = prepare(case, seed)
    table = _e4m3_table()
    if op == "quantize":
        x = st["x"].double()[st["idx"].long()]
        out = torch.empty_like(x)
        grid = table[:127]                                        # values of the codes 0..126, rising
        power = torch.tensor([2.0 ** i for i in range(-150, 151)], dtype=torch.float64, device="cuda")
        for b in range(-(-case["K"] // B)):
            col = x[:, b * B:(b + 1) * B]
            top = col.abs().amax(1)
            e = torch.zeros_like(top)
            for step in range(-117, 121):                         # the smallest exponent that fits
                e = torch.where((top > TOP * 2.0 ** (step - 1)) | (step == -117), float(step), e)
            e = torch.where(top == 0, 0.0, e)
            v = col.abs() / power[(e + 150).long()][:, None]
            hi = torch.searchsorted(grid, v.contiguous()).clamp(1, 126)
            lo = hi - 1
            down, up = v - grid[lo], grid[hi] - v                 # to nearest, ties to the even code
            take = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
            out[:, b * B:(b + 1) * B] = torch.sign(col) * grid[take]
        return out, None                                          # the exponents are whole numbers
    if op in ("gemm", "gated"):
        off = st["offsets"].tolist()
        out = torch.empty((case["R"], case["N"]), dtype=torch.float64, device="cuda")
        for g in range(case["G"]):
            rows = slice(off[g], off[g + 1])
            if off[g] == off[g + 1]:
                continue
            x = _exact_matrix(table, st["x"][rows], st["xe"][rows], 1)
            v = x @ _exact_matrix(table, st["W"][g], st["We"][g], B).t()
            if op == "gated":
                v = v * torch.sigmoid(v) * (x @ _exact_matrix(table, st["W3"][g], st["W3e"][g], B).t())
            out[rows] = v
        return out

    def matrix(name, e):
        m = st[name][e]
        return m.double() if case["w"] == "bfloat16" else _exact_matrix(table, m, st[name + "e"][e], B)

    h = st["h"].double()
    s = torch.sigmoid(h @ st["Wr"].double().t())
    key = s + st["bias"].double()
    out = torch.zeros((case["T"], case["D"]), dtype=torch.float64, device="cuda")
    weights = torch.empty((case["T"], case["k"]), dtype=torch.float64, device="cuda")
    chosen = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["k"]].tolist()
    for t in range(case["T"]):
        total = sum(s[t, e] for e in chosen[t])
        for j, e in enumerate(chosen[t]):
            weights[t, j] = s[t, e] / total * case["scale"]
            out[t] += weights[t, j] * _exact_mlp(h[t:t + 1], matrix("W1", e), matrix("W3", e),
                                                 matrix("W2", e))[0]
    for i in range(case["S"]):
        out += _exact_mlp(h, matrix("Ws1", i), matrix("Ws3", i), matrix("Ws2", i))
    return out, None, weights

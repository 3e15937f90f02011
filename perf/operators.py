"""The 8-bit block-scaled operators as cases to time and compare.

Three operators that belong together:

  quantize  a matrix to 8-bit floating point with one FP32 scale for each
            block of 128 (along rows, along columns, or 128 x 128),
  product   C = act(A B + bias) of two matrices held that way, in the three
            directions of a linear layer (forward, gradient of the input,
            gradient of the weights) and for a few rows,
  moe       a whole mixture-of-experts layer for a few tokens (router, chosen
            experts' gated feed-forward, weighted sum), weights in 16 bits or
            held as above.

Each case is computed either in its plain form (elementary torch operations in
FP32, rounded once at the end) or by the library's entry points.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
F16 = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}
TINY = 2.0 ** -117  # smallest block maximum that is told apart from zero
DEV = "cuda"


def ceil128(n):
    return (n + 127) // 128


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the activations of a decode batch, on their way into a product: a
        # call that is all latency
        {"name": "quant_rows_16x4096", "op": "quantize", "rows": 16, "cols": 4096, "layout": "rows", "x": "bf16", "q": "e4m3"},
        # output gradients of a training step, scaled along the tokens for the
        # gradient of the weights (odd number of tokens)
        {"name": "quant_cols_4095x11008", "op": "quantize", "rows": 4095, "cols": 11008, "layout": "cols", "x": "bf16", "q": "e4m3"},
        # a layer's FP32 master weights after an optimizer step
        {"name": "quant_blocks_11008x4096", "op": "quantize", "rows": 11008, "cols": 4096, "layout": "blocks", "x": "f32", "q": "e4m3"},
        # one token through a square projection: the smallest product
        {"name": "fwd_1x4096x4096", "op": "product", "dir": "forward", "M": 1, "N": 4096, "K": 4096, "a": "e4m3", "c": "bf16", "act": 0, "bias": False},
        # a decode batch through the up projection with bias and GELU
        {"name": "fwd_16x11008x4096_gelu", "op": "product", "dir": "forward", "M": 16, "N": 11008, "K": 4096, "a": "e4m3", "c": "bf16", "act": 1, "bias": True},
        # a prefill through the up projection: the largest product
        {"name": "fwd_4096x11008x4096", "op": "product", "dir": "forward", "M": 4096, "N": 11008, "K": 4096, "a": "e4m3", "c": "bf16", "act": 0, "bias": False},
        # gradient of the input, ragged number of tokens, gradients in e5m2
        {"name": "dgrad_1000x4096x11008", "op": "product", "dir": "dgrad", "M": 1000, "N": 4096, "K": 11008, "a": "e5m2", "c": "bf16", "act": 0, "bias": False},
        # gradient of the weights over an odd number of tokens
        {"name": "wgrad_4096x4096x4095", "op": "product", "dir": "wgrad", "M": 4096, "N": 4096, "K": 4095, "a": "e4m3", "c": "f32", "act": 0, "bias": False},
        # one token through a few large experts, 16-bit weights
        {"name": "moe_1_of_8_bf16", "op": "moe", "T": 1, "E": 8, "k": 2, "H": 4096, "I": 11008, "x": "bf16", "w": "bf16", "act": "silu", "gated": True, "renorm": True},
        # a small decode batch over many experts held in 8 bits
        {"name": "moe_16_of_32_fp8", "op": "moe", "T": 16, "E": 32, "k": 4, "H": 4096, "I": 2048, "x": "bf16", "w": "e4m3", "act": "silu", "gated": True, "renorm": True},
        # a full decode batch: nearly every expert has some tokens
        {"name": "moe_64_of_64_fp8", "op": "moe", "T": 64, "E": 64, "k": 6, "H": 2048, "I": 1024, "x": "bf16", "w": "e4m3", "act": "silu", "gated": True, "renorm": True},
        # odd sizes, no gate, plain softmax weights
        {"name": "moe_5_of_13_f16", "op": "moe", "T": 5, "E": 13, "k": 3, "H": 1008, "I": 784, "x": "f16", "w": "f16", "act": "gelu", "gated": False, "renorm": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "moe", "moe"])
    if op == "quantize":
        while True:
            rows, cols = _log(rng, 1, 12000), _log(rng, 64, 12000)
            if rows * cols <= 11008 * 4096:
                break
        return {"op": op, "rows": rows, "cols": cols, "layout": rng.choice(["rows", "cols", "blocks"]),
                "x": rng.choice(["bf16", "f16", "f32"]), "q": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "product":
        way = rng.choice(["forward", "forward", "dgrad", "wgrad"])
        while True:
            M = _log(rng, 1, 4500) if way != "wgrad" else _log(rng, 256, 11008)
            N, K = _log(rng, 256, 11008), _log(rng, 128, 11008)
            if M * N * K <= 4096 * 11008 * 4096:
                break
        act = rng.choice([0, 0, 1, 2, 3]) if way == "forward" else 0
        return {"op": op, "dir": way, "M": M, "N": N, "K": K, "a": "e4m3" if way == "forward" else rng.choice(["e4m3", "e5m2"]),
                "c": "f32" if way == "wgrad" else rng.choice(["bf16", "f16", "f32"]), "act": act, "bias": way == "forward" and rng.random() < 0.5}
    while True:
        T, E = _log(rng, 1, 64), _log(rng, 4, 64)
        k = rng.randint(1, min(8, E))
        H, I = 16 * _log(rng, 16, 256), 16 * _log(rng, 8, 688)
        if E * H * I <= 8 * 4096 * 11008:
            break
    x = rng.choice(["bf16", "f16"])
    return {"op": op, "T": T, "E": E, "k": k, "H": H, "I": I, "x": x, "w": rng.choice([x, "e4m3"]),
            "act": rng.choice(["silu", "gelu"]), "gated": rng.random() < 0.75, "renorm": rng.random() < 0.5}


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        scales = {"rows": r * ceil128(c), "cols": c * ceil128(r), "blocks": ceil128(r) * ceil128(c)}[case["layout"]]
        return {"bytes": r * c * (BYTES[case["x"]] + 1) + 4 * scales, "flops": 2 * r * c}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        scales = ceil128(K) * (M + (N if case["dir"] == "wgrad" else ceil128(N)))
        return {"bytes": M * K + N * K + 4 * scales + M * N * BYTES[case["c"]] + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    mats = 3 if case["gated"] else 2
    used = E * (1 - (1 - k / E) ** T)  # experts that get at least one token, on average
    weights = used * mats * (H * I * BYTES[case["w"]] + (4 * ceil128(H) * ceil128(I) if case["w"] == "e4m3" else 0))
    return {"bytes": weights + E * H * 2 + 2 * T * H * 2 + T * k * 8, "flops": 2 * T * k * mats * H * I + 2 * T * E * H}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _padded(rows, cols, dtype, multiple):
    """An uninitialised rows x cols matrix whose row stride is a multiple of `multiple`."""
    ld = (cols + multiple - 1) // multiple * multiple
    return torch.empty(rows, ld, dtype=dtype, device=DEV)[:, :cols]


def _activations(g, rows, cols, dtype):
    """Normal values with a few columns that are much larger, as in a trained network."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x[:, torch.randint(0, cols, (max(1, cols // 256),), generator=g, device=DEV)] *= 20.0
    return x.to(dtype)


def _quantized(x, q, layout):
    """x held in 8 bits, its row stride a multiple of 16 bytes, and the scales, theirs a multiple of 4."""
    v, s = _plain_quantize(x, q, layout)
    Q, S = _padded(*v.shape, F8[q], 16), _padded(*s.shape, torch.float32, 4)
    Q.view(torch.uint8).copy_(v.view(torch.uint8))
    S.copy_(s)
    return Q, S


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        s["X"] = _activations(g, r, c, F16[case["x"]]) if case["layout"] != "blocks" else (torch.randn(r, c, generator=g, device=DEV) / math.sqrt(c)).to(F16[case["x"]])
        qr, qc = (c, r) if case["layout"] == "cols" else (r, c)
        sr, sc = (ceil128(r), ceil128(c)) if case["layout"] == "blocks" else (ceil128(qc), qr)
        s["Q"], s["S"] = _padded(qr, qc, F8[case["q"]], 16), _padded(sr, sc, torch.float32, 4)
        return s
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        if case["dir"] == "forward":  # tokens x in, and the weights out x in
            A, B = _activations(g, M, K, torch.float32), torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
            s["A"], s["SA"] = _quantized(A, case["a"], "rows")
            s["B"], s["SB"] = _quantized(B, "e4m3", "blocks")
        elif case["dir"] == "dgrad":  # gradients tokens x out, and the same weights out x in
            A, B = torch.randn(M, K, generator=g, device=DEV) * 1e-3, torch.randn(K, N, generator=g, device=DEV) / math.sqrt(N)
            s["A"], s["SA"] = _quantized(A, case["a"], "rows")
            s["B"], s["SB"] = _quantized(B, "e4m3", "blocks")
        else:  # gradients and activations, both tokens x width, scaled along the tokens
            A, B = torch.randn(K, M, generator=g, device=DEV) * 1e-3, _activations(g, K, N, torch.float32)
            s["A"], s["SA"] = _quantized(A, case["a"], "cols")
            s["B"], s["SB"] = _quantized(B, "e4m3", "cols")
        s["bias_v"] = torch.randn(N, generator=g, device=DEV) * 0.1 if case["bias"] else None
        s["C"] = torch.empty(M, N, dtype=F16[case["c"]], device=DEV)
        return s
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    xt = F16[case["x"]]
    # Tokens in steps of 1/32 and router weights in steps of 2^-13: every
    # partial sum of a logit is exact in FP32, so the choice of experts does
    # not hang on the order of the sum, and ties between experts do occur.
    s["X"] = (torch.randn(T, H, generator=g, device=DEV).clamp_(-3.9, 3.9) * 32).round().div_(32).to(xt)
    s["router"] = (torch.randn(E, H, generator=g, device=DEV) / math.sqrt(H) * 8192).round().clamp_(-256, 256).div_(8192).to(xt)
    for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
        if name == "up" and not case["gated"]:
            s["up"] = s["up_s"] = None
            continue
        if case["w"] == "e4m3":
            w, sc = torch.empty(E, rows, cols, dtype=F8["e4m3"], device=DEV), torch.empty(E, ceil128(rows), ceil128(cols), device=DEV)
            for e in range(E):
                v, b = _plain_quantize(torch.randn(rows, cols, generator=g, device=DEV) / math.sqrt(cols), "e4m3", "blocks")
                w[e].view(torch.uint8).copy_(v.view(torch.uint8))
                sc[e] = b
            s[name], s[name + "_s"] = w, sc
        else:
            s[name] = torch.empty(E, rows, cols, dtype=xt, device=DEV)
            for e in range(E):
                s[name][e] = torch.randn(rows, cols, generator=g, device=DEV) / math.sqrt(cols)
            s[name + "_s"] = None
    s["Y"] = torch.empty(T, H, dtype=xt, device=DEV)
    s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    s["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _blocks(x, layout):
    """x in FP32, zero-padded and viewed so that dim 1 (rows) or dims 1 and 3 (blocks) run over one block."""
    r, c = x.shape
    if layout == "rows":
        return torch.nn.functional.pad(x, (0, -c % 128)).reshape(r, -1, 128)
    return torch.nn.functional.pad(x, (0, -c % 128, 0, -r % 128)).reshape(ceil128(r), 128, ceil128(c), 128)


def _plain_quantize(X, q, layout):
    x = X.float()
    if layout == "cols":
        x, layout = x.t(), "rows"
    r, c = x.shape
    b = _blocks(x, layout)
    top = b.abs().amax(dim=2 if layout == "rows" else (1, 3), keepdim=True).clamp_(min=TINY)
    limit = torch.full_like(top, F8_MAX[q])
    v = (b * (limit / top)).reshape(-1, ceil128(c) * 128)[:r, :c].to(F8[q])
    s = top / limit
    return (v, s[:, :, 0].t().contiguous()) if layout == "rows" else (v, s[:, 0, :, 0])


def _spread(S, rows, cols, kind):
    """The scales as one factor for each element of a rows x cols matrix."""
    if kind == "rows":
        return S.t().repeat_interleave(128, dim=1)[:, :cols]
    return S.repeat_interleave(128, dim=-2)[..., :rows, :].repeat_interleave(128, dim=-1)[..., :cols]


def _act(v, act):
    if act in (1, "gelu"):
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == 2:
        return torch.clamp(v, min=0.0)
    if act == 3:
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v / (1.0 + torch.exp(-v)) if act == "silu" else v


def _plain_product(s):
    a = s["A"].float() * _spread(s["SA"], *s["A"].shape, "rows")
    b = s["B"].float() * _spread(s["SB"], *s["B"].shape, "rows" if s["dir"] == "wgrad" else "blocks")
    c = a @ (b if s["dir"] == "dgrad" else b.t())
    if s["bias_v"] is not None:
        c = c + s["bias_v"]
    return _act(c, s["act"]).to(s["C"].dtype)


def _plain_moe(s):
    T, E, k, H, I = (s[n] for n in ("T", "E", "k", "H", "I"))
    x = s["X"].float()
    p = torch.softmax(x @ s["router"].float().t(), dim=1)
    ids = torch.sort(p, dim=1, descending=True, stable=True).indices[:, :k]  # ties: the lowest index first
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    # the chosen experts' matrices one by one, or all experts' where that is less
    few = T * k < E
    pick = (lambda m: m[ids.reshape(-1)]) if few else (lambda m: m)
    full = lambda n, rows, cols: pick(s[n]).float() * (_spread(pick(s[n + "_s"]), rows, cols, "blocks") if s[n + "_s"] is not None else 1.0)  # noqa: E731
    rows = x.repeat_interleave(k, dim=0).unsqueeze(1) if few else x.unsqueeze(0).expand(E, T, H)
    h = _act(rows @ full("gate", I, H).transpose(1, 2), s["act"])
    if s["gated"]:
        h = h * (rows @ full("up", I, H).transpose(1, 2))
    y = h @ full("down", H, I).transpose(1, 2)
    if few:
        y = y.reshape(T, k, H)
    else:
        y = y.transpose(0, 1).gather(1, ids.unsqueeze(2).expand(T, k, H))
    return {"y": (y * w.unsqueeze(2)).sum(dim=1).to(s["X"].dtype), "ids": ids.int(), "weights": w}


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        if s["op"] == "quantize":
            return _plain_quantize(s["X"], s["q"], s["layout"])
        return _plain_product(s) if s["op"] == "product" else _plain_moe(s)
    import dense_gemm_11_gb300 as g
    if s["op"] == "quantize":
        g.fp8_quantize(s["X"], s["Q"], s["S"], layout=s["layout"])
        return s["Q"], s["S"]
    if s["op"] == "product":
        g.gemm_fp8(s["A"], s["SA"], s["B"], s["SB"], s["C"], bias=s["bias_v"], act=s["act"], b_trans=s["dir"] != "dgrad",
                   b_scales="rows" if s["dir"] == "wgrad" else "blocks")
        return s["C"]
    scales = (s["gate_s"], s["up_s"], s["down_s"]) if s["gate_s"] is not None else None
    g.moe_few_tokens(s["X"], s["router"], s["gate"], s["up"], s["down"], s["Y"], s["k"], scales=scales,
                     act=g.GEMM_ACT_SILU if s["act"] == "silu" else g.GEMM_ACT_GELU, renormalize=s["renorm"], ids=s["ids"], weights=s["weights"])
    return {"y": s["Y"], "ids": s["ids"], "weights": s["weights"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _f64_scale(S, rows, cols, per_row):
    """Scale of element (i, j): S[j / 128, i] with one scale for 128 of a row, S[i / 128, j / 128] for a square block."""
    i, j = torch.arange(rows, device=DEV), torch.arange(cols, device=DEV) // 128
    return S.double()[j[None, :], i[:, None]] if per_row else S.double()[(i // 128)[:, None], j[None, :]]


def _f64_act(v, act):
    if act in (1, "gelu"):
        return v * torch.special.ndtr(v)
    if act == 2:
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == 3:
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v * torch.sigmoid(v) if act == "silu" else v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["X"].double()
        x = x.t() if case["layout"] == "cols" else x
        r, c = x.shape
        tall = 1 if case["layout"] != "blocks" else 128
        S = torch.zeros((r + tall - 1) // tall, ceil128(c), dtype=torch.float64, device=DEV)
        for j in range(ceil128(c)):
            m = x[:, 128 * j:128 * (j + 1)].abs().amax(dim=1)
            for_rows = torch.zeros(S.shape[0] * tall, dtype=torch.float64, device=DEV)
            for_rows[:r] = m
            S[:, j] = for_rows.reshape(-1, tall).amax(dim=1)
        S = S.clamp(min=TINY) / F8_MAX[case["q"]]
        each = S[(torch.arange(r, device=DEV) // tall)[:, None], (torch.arange(c, device=DEV) // 128)[None, :]]
        v = x / each
        # nearest value with 3 (e4m3) or 2 (e5m2) bits after the point, ties to even
        bits, low = (3, -6) if case["q"] == "e4m3" else (2, -14)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))) - bits)
        v = (torch.round(v / step) * step).clamp(-F8_MAX[case["q"]], F8_MAX[case["q"]])
        return v, (S if case["layout"] == "blocks" else S.t().contiguous())
    if case["op"] == "product":
        a = s["A"].double() * _f64_scale(s["SA"], *s["A"].shape, True)
        b = s["B"].double() * _f64_scale(s["SB"], *s["B"].shape, case["dir"] == "wgrad")
        c = torch.mm(a, b if case["dir"] == "dgrad" else b.t())
        if s["bias_v"] is not None:
            c += s["bias_v"].double()
        return _f64_act(c, case["act"])
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    x = s["X"].double()
    logits = x @ s["router"].double().t()
    p = torch.exp(logits - logits.logsumexp(dim=1, keepdim=True))
    chosen = torch.zeros(T, k, dtype=torch.int64, device=DEV)
    left = logits.clone()
    for j in range(k):
        best = left.amax(dim=1, keepdim=True)
        chosen[:, j] = torch.where(left == best, torch.arange(E, device=DEV), E).amin(dim=1)
        left.scatter_(1, chosen[:, j:j + 1], -math.inf)
    w = p.gather(1, chosen)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    y = torch.zeros(T, H, dtype=torch.float64, device=DEV)

    def matrix(name, e, rows, cols):
        m = s[name][e].double()
        return m if s[name + "_s"] is None else m * _f64_scale(s[name + "_s"][e], rows, cols, False)

    for e in chosen.unique().tolist():
        t, j = (chosen == e).nonzero(as_tuple=True)
        h = _f64_act(x[t] @ matrix("gate", e, I, H).t(), case["act"])
        if case["gated"]:
            h = h * (x[t] @ matrix("up", e, I, H).t())
        y.index_add_(0, t, (h @ matrix("down", e, H, I).t()) * w[t, j][:, None])
    return {"y": y, "ids": None, "weights": w}

"""The operators of a mixture-of-experts layer for many tokens, as cases to time and compare.

Four operators that belong together, each in the directions a training step
needs:

  dispatch  a router's choice sorted by expert, and the tokens' rows copied
            into that order,
  combine   the experts' rows back to their tokens, with the router's weights
            (forward), the gradient of that (rows and weights), and the
            gradient of the copy (the same sum without weights),
  product   the experts' products over the sorted rows: forward, gradient of
            the rows, gradient of every expert's weights,
  gated     the gated activation h = act(g) u whose inputs are kept for the
            backward pass in 8 bits (one FP32 scale for 128 of a row), and
            that backward pass.

Each case is computed either in its plain form (elementary torch operations in
FP32, rounded once at the end) or by the library's entry points.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8_FLOOR = {"e4m3": 2.0 ** -117, "e5m2": 2.0 ** -110}  # smallest block maximum that is told apart from zero
ACT = {"gelu": 1, "relu": 2, "gelu_tanh": 3, "silu": 4}
DEV = "cuda"


def ceil128(n):
    return (n + 127) // 128


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a decode batch on its way to the experts: a call that is all latency
        {"name": "dispatch_16x2_of_8", "op": "dispatch", "T": 16, "E": 8, "k": 2, "H": 4096, "t": "bf16", "drop": 0.0},
        # a training step's tokens over many experts
        {"name": "dispatch_8192x6_of_64", "op": "dispatch", "T": 8192, "E": 64, "k": 6, "H": 2048, "t": "bf16", "drop": 0.0},
        # the experts' rows back to an odd number of tokens, some of which lost a slot to a full expert
        {"name": "combine_4095x2_of_8", "op": "combine", "dir": "forward", "T": 4095, "E": 8, "k": 2, "H": 4096, "t": "bf16", "drop": 0.02},
        # its gradient over many experts: rows and weights
        {"name": "combine_grad_8192x6_of_64", "op": "combine", "dir": "grad", "T": 8192, "E": 64, "k": 6, "H": 2048, "t": "bf16", "drop": 0.0},
        # the gradient of the copy for a small odd model in FP16
        {"name": "dispatch_grad_1000x3_of_13", "op": "combine", "dir": "copy_grad", "T": 1000, "E": 13, "k": 3, "H": 1008, "t": "f16", "drop": 0.0},
        # a decode batch over many experts, a few rows each: the weights' bytes
        {"name": "product_64x6_of_64", "op": "product", "dir": "forward", "T": 64, "E": 64, "k": 6, "N": 1024, "K": 2048, "t": "bf16", "c": "bf16", "drop": 0.0},
        # a prefill through the up projection of a few large experts: the largest product
        {"name": "product_4096x2_of_8", "op": "product", "dir": "forward", "T": 4096, "E": 8, "k": 2, "N": 11008, "K": 4096, "t": "bf16", "c": "bf16", "drop": 0.0},
        # gradient of the rows over many experts, ragged everywhere
        {"name": "product_dgrad_4095x6_of_64", "op": "product", "dir": "dgrad", "T": 4095, "E": 64, "k": 6, "N": 2048, "K": 1024, "t": "bf16", "c": "bf16", "drop": 0.0},
        # gradient of the weights of a few large experts, kept in FP32 for the optimizer
        {"name": "product_wgrad_4096x2_of_8", "op": "product", "dir": "wgrad", "T": 4096, "E": 8, "k": 2, "M": 11008, "N": 4096, "t": "bf16", "c": "f32", "drop": 0.0},
        # the activation of a decode batch's rows: latency
        {"name": "gated_32x11008", "op": "gated", "dir": "forward", "R": 32, "I": 11008, "t": "bf16", "q": "e4m3", "act": "silu", "gated": True, "h": True},
        # the activation of a training step's rows and their 8-bit copies
        {"name": "gated_8192x11008", "op": "gated", "dir": "forward", "R": 8192, "I": 11008, "t": "bf16", "q": "e4m3", "act": "silu", "gated": True, "h": True},
        # the backward pass from the 8-bit copies, an odd number of rows, h formed again for the gradient of the next weights
        {"name": "gated_grad_8191x11008", "op": "gated", "dir": "grad", "R": 8191, "I": 11008, "t": "bf16", "q": "e4m3", "act": "silu", "gated": True, "h": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine", "product", "product", "product", "gated", "gated"])
    t = rng.choice(["bf16", "bf16", "f16"])
    if op == "gated":
        while True:
            R, I = _log(rng, 1, 20000), _log(rng, 64, 12000)
            if R * I <= 8192 * 11008:
                break
        return {"op": op, "dir": rng.choice(["forward", "grad"]), "R": R, "I": I, "t": rng.choice([t, t, "f32"]), "q": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]), "gated": rng.random() < 0.75, "h": rng.random() < 0.5}
    T, E = _log(rng, 1, 9000), _log(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    drop = rng.choice([0.0, 0.0, 0.05])
    if op == "dispatch" or op == "combine":
        while True:
            H = _log(rng, 64, 8192)
            if T * k * H * (2 if t != "f32" else 4) <= 8192 * 6 * 2048 * 2:
                break
        case = {"op": op, "T": T, "E": E, "k": k, "H": H, "t": t, "drop": drop}
        if op == "combine":
            case["dir"] = rng.choice(["forward", "grad", "grad", "copy_grad"])
        return case
    way = rng.choice(["forward", "forward", "dgrad", "wgrad"])
    while True:
        a, b = _log(rng, 64, 11008), _log(rng, 64, 11008)
        if T * k * a * b <= 4096 * 2 * 11008 * 4096 and E * a * b <= 8 * 11008 * 4096:
            break
    case = {"op": op, "dir": way, "T": T, "E": E, "k": k, "t": t, "c": rng.choice([t, t, "f32"]), "drop": drop}
    case.update({"M": a, "N": b} if way == "wgrad" else {"N": a, "K": b})
    return case


def work(case):
    if case["op"] == "gated":
        R, I, b = case["R"], case["I"], BYTES[case["t"]]
        mats = 2 if case["gated"] else 1
        kept = mats * (R * I + 4 * R * ceil128(I))
        wide = mats + 1 + (1 if case["dir"] == "grad" and case["h"] else 0)  # forward: g, u, h; backward: dh, dg, du, h
        return {"bytes": kept + wide * R * I * b, "flops": (8 if case["dir"] == "forward" else 12) * R * I}
    T, E, k, b = case["T"], case["E"], case["k"], BYTES[case["t"]]
    n = T * k * (1 - case["drop"])
    if case["op"] == "dispatch":
        return {"bytes": 8 * T * k + 4 * (E + 1) + (T + n) * case["H"] * b, "flops": 0}
    if case["op"] == "combine":
        H = case["H"]
        if case["dir"] == "grad":
            return {"bytes": 12 * T * k + (T + 2 * n) * H * b, "flops": 3 * n * H}
        return {"bytes": (8 if case["dir"] == "forward" else 4) * T * k + (T + n) * H * b, "flops": 2 * n * H}
    used = E * (1 - (1 - k * (1 - case["drop"]) / E) ** T)  # experts that get at least one row, on average
    if case["dir"] == "wgrad":
        M, N = case["M"], case["N"]
        return {"bytes": n * (M + N) * b + E * M * N * BYTES[case["c"]] + 4 * (E + 1), "flops": 2 * n * M * N}
    N, K = case["N"], case["K"]
    return {"bytes": n * K * b + used * N * K * b + n * N * BYTES[case["c"]] + 4 * (E + 1), "flops": 2 * n * N * K}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _padded(shape, dtype, multiple, fill=None):
    """A tensor whose rows are a multiple of `multiple` elements apart."""
    cols = shape[-1]
    ld = (cols + multiple - 1) // multiple * multiple
    full = list(shape[:-1]) + [ld]
    x = torch.empty(full, dtype=dtype, device=DEV) if fill is None else torch.full(full, fill, dtype=dtype, device=DEV)
    return x[..., :cols]


def _normal(g, shape, dtype, scale=1.0):
    """Normal values, rows padded to 16 bytes; a 3-D tensor is made one matrix at a time."""
    x = _padded(shape, dtype, 16 // dtype.itemsize)
    for part in (x if len(shape) == 3 else [x]):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * scale)
    return x


def _route(g, case):
    """Experts and weights of every token, as an uneven router chooses them; -1 where a full expert refused."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    top, ids = logits.topk(k, dim=1)
    ids = ids.int()
    if case["drop"] > 0.0:
        ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < case["drop"], torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(top, dim=1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    t = TYPES[case["t"]]
    if case["op"] == "gated":
        R, I, q = case["R"], case["I"], case["q"]
        if case["dir"] == "forward":
            s["G"], s["U"] = _normal(g, (R, I), t, 2.0), _normal(g, (R, I), t) if case["gated"] else None
            s["H"] = _padded((R, I), t, 16 // t.itemsize)
            s["kept"] = [(_padded((R, I), F8[q], 16), _padded((ceil128(I), R), torch.float32, 4)) for _ in range(2 if case["gated"] else 1)]
        else:
            s["dH"] = _normal(g, (R, I), t, 1e-2)
            s["kept"] = []
            for scale in (2.0, 1.0)[:2 if case["gated"] else 1]:
                v, b = _plain_keep(_normal(g, (R, I), t, scale), q)
                Q, S = _padded((R, I), F8[q], 16), _padded((ceil128(I), R), torch.float32, 4)
                Q.view(torch.uint8).copy_(v.view(torch.uint8))
                S.copy_(b)
                s["kept"].append((Q, S))
            s["dG"] = _padded((R, I), t, 16 // t.itemsize)
            s["dU"] = _padded((R, I), t, 16 // t.itemsize) if case["gated"] else None
            s["H"] = _padded((R, I), t, 16 // t.itemsize) if case["h"] else None
        return s
    T, E, k = case["T"], case["E"], case["k"]
    s["ids"], s["weights"] = _route(g, case)
    step = 16 // t.itemsize
    if case["op"] == "dispatch":
        s["X"] = _normal(g, (T, case["H"]), t)
        s["Xs"] = _padded((T * k, case["H"]), t, step, 0.0)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["rows"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        return s
    offsets, s["rows"] = _plain_sort(s["ids"], E)
    s["offsets"] = offsets
    if case["op"] == "combine":
        H = case["H"]
        if case["dir"] == "grad":
            s["dY"], s["Ys"] = _normal(g, (T, H), t, 1e-2), _normal(g, (T * k, H), t)
            s["dYs"], s["dweights"] = _padded((T * k, H), t, step, 0.0), torch.empty(T, k, device=DEV)
        else:
            s["Ys"], s["Y"] = _normal(g, (T * k, H), t), _padded((T, H), t, step)
        return s
    s["bounds"] = offsets.tolist()
    R, c = T * k, TYPES[case["c"]]
    if case["dir"] == "wgrad":
        s["A"], s["B"] = _normal(g, (R, case["M"]), t, 1e-2), _normal(g, (R, case["N"]), t)
        s["C"] = _padded((E, case["M"], case["N"]), c, 16 // c.itemsize)
        return s
    N, K = case["N"], case["K"]
    s["A"] = _normal(g, (R, K), t)
    s["B"] = _normal(g, (E, N, K) if case["dir"] == "forward" else (E, K, N), t, 1.0 / math.sqrt(K))
    s["C"] = _padded((R, N), c, 16 // c.itemsize, 0.0)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_sort(ids, E):
    """(offsets, rows): where each expert's rows start, and the row of each slot in the order of the experts."""
    flat = ids.reshape(-1).long()
    known = (flat >= 0) & (flat < E)
    key = torch.where(known, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=DEV)
    rows = torch.where(known, rows, torch.full_like(rows, -1))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets.int(), rows.reshape(ids.shape).int()


def _plain_dispatch(s):
    offsets, rows = _plain_sort(s["ids"], s["E"])
    flat, k = rows.reshape(-1).long(), s["k"]
    Xs = torch.zeros(flat.numel() + 1, s["H"], dtype=s["X"].dtype, device=DEV)  # the last row takes what has no expert
    Xs[torch.where(flat < 0, torch.full_like(flat, flat.numel()), flat)] = s["X"].repeat_interleave(k, dim=0)
    return {"offsets": offsets, "rows": rows, "Xs": Xs[:-1]}


def _taken(s, name):
    """FP32 rows of the slots, (T, k, H), zeros for slots without one."""
    idx = s["rows"].long()
    return torch.where((idx >= 0).unsqueeze(2), s[name][idx.clamp(min=0)].float(), torch.zeros((), device=DEV))


def _plain_combine(s):
    if s["dir"] == "copy_grad":
        return _taken(s, "Ys").sum(dim=1).to(s["Ys"].dtype)
    if s["dir"] == "forward":
        return (_taken(s, "Ys") * s["weights"].unsqueeze(2)).sum(dim=1).to(s["Ys"].dtype)
    dy = s["dY"].float().unsqueeze(1)
    dweights = (_taken(s, "Ys") * dy).sum(dim=2)
    flat, n = s["rows"].reshape(-1).long(), s["rows"].numel()
    dYs = torch.zeros(n + 1, s["H"], dtype=s["Ys"].dtype, device=DEV)
    dYs[torch.where(flat < 0, torch.full_like(flat, n), flat)] = (dy * s["weights"].unsqueeze(2)).to(dYs.dtype).reshape(n, -1)
    return {"dYs": dYs[:-1], "dweights": dweights}


def _plain_product(s):
    b = s["bounds"]
    if s["dir"] == "wgrad":
        C = torch.zeros(s["C"].shape, dtype=s["C"].dtype, device=DEV)
        for e in range(s["E"]):
            if b[e + 1] > b[e]:
                C[e] = (s["A"][b[e]:b[e + 1]].float().t() @ s["B"][b[e]:b[e + 1]].float()).to(C.dtype)
        return C
    C = torch.zeros(s["C"].shape, dtype=s["C"].dtype, device=DEV)
    for e in range(s["E"]):
        if b[e + 1] > b[e]:
            w = s["B"][e].float()
            C[b[e]:b[e + 1]] = (s["A"][b[e]:b[e + 1]].float() @ (w.t() if s["dir"] == "forward" else w)).to(C.dtype)
    return C


def _act(v, act):
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "relu":
        return torch.clamp(v, min=0.0)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v / (1.0 + torch.exp(-v))


def _act_slope(v, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if act == "relu":
        return (v > 0.0).float()
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + th) + 0.5 * v * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * v * v)
    p = 1.0 / (1.0 + torch.exp(-v))
    return p * (1.0 + v * (1.0 - p))


def _plain_keep(X, q):
    """X in 8 bits and the scales, one for each 128 of a row, as (blocks, rows)."""
    r, c = X.shape
    b = torch.nn.functional.pad(X.float(), (0, -c % 128)).reshape(r, -1, 128)
    top = b.abs().amax(dim=2, keepdim=True).clamp_(min=F8_FLOOR[q])
    limit = torch.full_like(top, F8_MAX[q])
    v = (b * (limit / top)).reshape(r, -1)[:, :c].to(F8[q])
    return v, (top / limit)[:, :, 0].t().contiguous()


def _plain_gated(s):
    if s["dir"] == "forward":
        h = _act(s["G"].float(), s["act"])
        if s["gated"]:
            h = h * s["U"].float()
        return {"h": h.to(s["G"].dtype), "kept": [_plain_keep(s[n], s["q"]) for n in ("G", "U")[:len(s["kept"])]]}
    back = [Q.float() * S.t().repeat_interleave(128, dim=1)[:, :Q.shape[1]] for Q, S in s["kept"]]
    dh, g = s["dH"].float(), back[0]
    t = s["dH"].dtype
    a = _act(g, s["act"])
    dg = dh * _act_slope(g, s["act"])
    out = {"dg": ((dg * back[1]) if s["gated"] else dg).to(t)}
    if s["gated"]:
        out["du"] = (dh * a).to(t)
    if s["h"]:
        out["h"] = ((a * back[1]) if s["gated"] else a).to(t)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"dispatch": _plain_dispatch, "combine": _plain_combine, "product": _plain_product, "gated": _plain_gated}[s["op"]](s)
    import dense_gemm_11_gb300 as g
    if s["op"] == "dispatch":
        g.moe_dispatch(s["ids"], s["X"], s["Xs"], s["offsets"], s["rows"])
        return {"offsets": s["offsets"], "rows": s["rows"], "Xs": s["Xs"]}
    if s["op"] == "combine":
        if s["dir"] == "grad":
            g.moe_combine_grad(s["dY"], s["Ys"], s["rows"], s["weights"], s["dYs"], s["dweights"])
            return {"dYs": s["dYs"], "dweights": s["dweights"]}
        g.moe_combine(s["Ys"], s["rows"], s["Y"], weights=s["weights"] if s["dir"] == "forward" else None)
        return s["Y"]
    if s["op"] == "product":
        if s["dir"] == "wgrad":
            g.gemm_grouped_wgrad(s["A"], s["B"], s["C"], s["offsets"])
        else:
            g.gemm_grouped(s["A"], s["B"], s["C"], s["offsets"], b_trans=s["dir"] == "forward")
        return s["C"]
    kept = s["kept"] if s["gated"] else [s["kept"][0], (None, None)]
    if s["dir"] == "forward":
        g.fp8_gated_act(s["G"], s["U"], s["H"], *kept[0], *kept[1], act=ACT[s["act"]])
        return {"h": s["H"], "kept": s["kept"]}
    g.fp8_gated_act_grad(s["dH"], *kept[0], *kept[1], s["dG"], s["dU"], s["H"], act=ACT[s["act"]])
    out = {"dg": s["dG"]}
    if s["gated"]:
        out["du"] = s["dU"]
    if s["h"]:
        out["h"] = s["H"]
    return out


# ---------------------------------------------------------------- the definitions in 64 bits
def _f64_act(v, act):
    """(act(v), its slope)."""
    if act == "relu":
        on = (v > 0).double()
        return v * on, on
    if act == "gelu":
        cdf = torch.special.ndtr(v)
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":  # (1 + tanh z) / 2 = sigmoid(2 z)
        z2 = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        p = torch.sigmoid(z2)
        return v * p, p + v * p * torch.sigmoid(-z2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * v ** 2)
    p = torch.sigmoid(v)
    return v * p, p + v * p * torch.sigmoid(-v)


def _f64_keep(x, q):
    """The nearest 8-bit values of x over its scale, ties to even, and the scales."""
    r, c = x.shape
    S = torch.zeros(ceil128(c), r, dtype=torch.float64, device=DEV)
    v = torch.empty_like(x)
    bits, low = (3, -6) if q == "e4m3" else (2, -14)
    for j in range(ceil128(c)):
        part = x[:, 128 * j:128 * (j + 1)]
        S[j] = part.abs().amax(dim=1).clamp(min=F8_FLOOR[q]) / F8_MAX[q]
        w = part / S[j][:, None]
        step = torch.exp2(torch.floor(torch.log2(w.abs().clamp(min=2.0 ** low))) - bits)
        v[:, 128 * j:128 * (j + 1)] = (torch.round(w / step) * step).clamp(-F8_MAX[q], F8_MAX[q])
    return v, S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gated":
        if case["dir"] == "forward":
            g = s["G"].double()
            h = _f64_act(g, case["act"])[0]
            if case["gated"]:
                h = h * s["U"].double()
            return {"h": h, "kept": [_f64_keep(s[n].double(), case["q"]) for n in ("G", "U")[:len(s["kept"])]]}
        block = torch.arange(case["I"], device=DEV) // 128
        values = [Q.double() * S.double()[block, :].t() for Q, S in s["kept"]]
        a, slope = _f64_act(values[0], case["act"])
        u = values[1] if case["gated"] else torch.ones((), dtype=torch.float64, device=DEV)
        out = {"dg": s["dH"].double() * slope * u}
        if case["gated"]:
            out["du"] = s["dH"].double() * a
        if case["h"]:
            out["h"] = a * u
        return out
    T, E, k = case["T"], case["E"], case["k"]
    ids = s["ids"].cpu().reshape(-1).tolist()
    members = [[] for _ in range(E)]  # the slots of each expert, in the order of the tokens
    for slot, e in enumerate(ids):
        if 0 <= e < E:
            members[e].append(slot)
    starts = [0]
    for m in members:
        starts.append(starts[-1] + len(m))
    slots = torch.tensor([i for m in members for i in m], dtype=torch.int64, device=DEV)  # of each sorted row
    if case["op"] == "dispatch":
        rows = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
        rows[slots] = torch.arange(slots.numel(), device=DEV)
        Xs = torch.zeros(T * k, case["H"], dtype=torch.float64, device=DEV)
        Xs[:slots.numel()] = s["X"].double()[slots // k]
        return {"offsets": torch.tensor(starts, device=DEV).int(), "rows": rows.reshape(T, k).int(), "Xs": Xs}
    token, w = slots // k, s["weights"].double().reshape(-1)[slots][:, None]
    if case["op"] == "combine":
        ys = s["Ys"].double()[:slots.numel()]
        if case["dir"] != "grad":
            return torch.zeros(T, case["H"], dtype=torch.float64, device=DEV).index_add_(0, token, ys * w if case["dir"] == "forward" else ys)
        dy = s["dY"].double()[token]
        dYs = torch.zeros(T * k, case["H"], dtype=torch.float64, device=DEV)
        dYs[:slots.numel()] = w * dy
        dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        dw[slots] = torch.einsum("rh,rh->r", ys, dy)
        return {"dYs": dYs, "dweights": dw.reshape(T, k)}
    C = torch.zeros(s["C"].shape, dtype=torch.float64, device=DEV)
    for e in range(E):
        lo, hi = starts[e], starts[e + 1]
        if lo == hi:
            continue
        a, b = s["A"][lo:hi].double(), s["B"]
        if case["dir"] == "wgrad":
            torch.mm(a.t(), b[lo:hi].double(), out=C[e])
        else:
            C[lo:hi] = torch.einsum("rk,nk->rn" if case["dir"] == "forward" else "rk,kn->rn", a, b[e].double())
    return C

"""Plain implementations, in 64 bits, of the block-scaled 8-bit operators the tests compare against."""
import numpy as np
import torch

TINY = np.float32(2.0 ** -117)
LIMIT = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
GRID = {torch.float8_e4m3fn: (3, -6), torch.float8_e5m2: (2, -14)}  # mantissa bits, smallest normal exponent


def round8(v, dtype):
    """float64 -> the nearest 8-bit value, ties to even, clamped to the largest; NaN stays."""
    bits, low = GRID[dtype]
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(v), v, 0.0))
        step = np.ldexp(1.0, np.maximum(e - 1, low) - bits)
        return np.clip(np.rint(v / step) * step, -LIMIT[dtype], LIMIT[dtype])


def quantize(x, dtype, layout):
    """(values of q, scales) of a 2-D float array, both float64 holding the exact results of the FP32 formula."""
    x = np.asarray(x, dtype=np.float32)
    if layout == "cols":
        x = x.T
    r, c = x.shape
    tall = 128 if layout == "blocks" else 1
    rb, cb = -(-r // tall), -(-c // 128)
    S = np.zeros((rb, cb), dtype=np.float32)
    q = np.zeros((r, c))
    F = np.float32(LIMIT[dtype])
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        for i in range(rb):
            for j in range(cb):
                blk = x[i * tall:(i + 1) * tall, j * 128:(j + 1) * 128]
                known = np.abs(blk[~np.isnan(blk)])
                a = max(TINY, known.max()) if known.size else TINY
                S[i, j] = a / F
                q[i * tall:(i + 1) * tall, j * 128:(j + 1) * 128] = round8((blk * np.float32(F / a)).astype(np.float64), dtype)
    return q, (S if layout == "blocks" else S.T).astype(np.float64)


def dequantize(Q, S, layout):
    """float64 values of a quantized matrix as Q stores it."""
    q, s = Q.double(), S.double()
    if layout == "blocks":
        return q * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q * s.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def act64(v, act):
    if act == 1:
        return 0.5 * v * torch.erfc(-v * 0.5 ** 0.5)
    if act == 2:
        return v.clamp(min=0)
    if act == 3:
        return 0.5 * v * (1 + torch.tanh((2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
    if act == 4:
        return v / (1 + torch.exp(-v))
    return v


def product(A, SA, B, SB, b_trans, b_scales, alpha=1.0, beta=0.0, C=None, bias=None, act=0):
    """(float64 result, per-element error scale |alpha| sum |a||b| + |beta||c|)."""
    a = dequantize(A, SA, "rows")
    b = dequantize(B, SB, b_scales)
    b = b.t() if b_trans else b
    v, S = alpha * (a @ b), abs(alpha) * (a.abs() @ b.abs())
    if beta != 0.0:
        v, S = v + beta * C.double(), S + abs(beta) * C.double().abs()
    if bias is not None:
        v = v + bias.double()
    return act64(v, act), S


def moe(X, router, gate, up, down, top_k, scales=None, act=4, renormalize=True):
    """(y, ids, weights, per-element error scale of y) in float64."""
    x = X.double().cpu()
    E = router.shape[0]
    logits = x @ router.double().cpu().t()
    T = x.shape[0]
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -logits.numpy()), axis=1)[:, :top_k]
    ids = torch.from_numpy(np.ascontiguousarray(order))
    p = torch.softmax(logits, dim=1)
    w = p.gather(1, ids)
    if renormalize:
        w = w / w.sum(dim=1, keepdim=True)

    def matrix(m, i, e):
        return m[e].double().cpu() if scales is None else dequantize(m[e], scales[i][e], "blocks").cpu()

    y, S = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        h = act64(x[t] @ matrix(gate, 0, e).t(), act)
        if up is not None:
            h = h * (x[t] @ matrix(up, 1, e).t())
        d = matrix(down, 2, e)
        y.index_add_(0, t, (h @ d.t()) * w[t, j][:, None])
        S.index_add_(0, t, (h.abs() @ d.abs().t()) * w[t, j][:, None])
    return y, ids, w, S

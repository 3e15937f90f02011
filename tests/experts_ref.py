"""Plain implementations, in 64 bits, of the mixture-of-experts operators for many tokens, and the bounds on their errors."""
import math

import torch

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
SMALLEST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half of the smallest step


def rounded(bound, want, dtype):
    """A bound on an FP32 value widened by its rounding to dtype."""
    return bound + UNIT[dtype] * (want.abs() + bound) + SMALLEST[dtype]


def close(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[:4].tolist()}, worst excess {float((err - bound)[bad].max()):.3e}, largest {float(err[bad].max()):.3e}"


def sort(ids, E):
    """(offsets, rows) by the definition, slot by slot."""
    flat = ids.reshape(-1).tolist()
    members = [[i for i, e in enumerate(flat) if e == x] for x in range(E)]
    offsets, rows = [0], [-1] * len(flat)
    for m in members:
        for i, slot in enumerate(m):
            rows[slot] = offsets[-1] + i
        offsets.append(offsets[-1] + len(m))
    return torch.tensor(offsets), torch.tensor(rows, dtype=torch.int64).reshape(ids.shape)


def combine(Ys, rows, weights=None):
    """(sum, sum of magnitudes)."""
    r = rows.long().cpu()
    y = Ys.double().cpu()
    out, mag = torch.zeros(r.shape[0], y.shape[1], dtype=torch.float64), torch.zeros(r.shape[0], y.shape[1], dtype=torch.float64)
    for j in range(r.shape[1]):
        on = (r[:, j] >= 0) & (r[:, j] < y.shape[0])
        w = torch.ones(int(on.sum()), 1, dtype=torch.float64) if weights is None else weights.double().cpu()[on, j][:, None]
        out[on] += w * y[r[on, j]]
        mag[on] += (w * y[r[on, j]]).abs()
    return out, mag


def grouped(A, B, offsets, b_trans, alpha=1.0, beta=0.0, C=None):
    """(result over all rows, error scale); rows that no expert has are NaN."""
    a, o = A.double(), offsets.tolist()
    N = B.shape[1] if b_trans else B.shape[2]
    out = torch.full((A.shape[0], N), math.nan, dtype=torch.float64, device=A.device)
    mag = torch.zeros_like(out)
    for e in range(B.shape[0]):
        w = B[e].double().t() if b_trans else B[e].double()
        s = slice(o[e], o[e + 1])
        out[s] = alpha * (a[s] @ w)
        mag[s] = abs(alpha) * (a[s].abs() @ w.abs())
        if beta:
            out[s] += beta * C[s].double()
            mag[s] += abs(beta) * C[s].double().abs()
    return out, mag


def wgrad(A, B, offsets, alpha=1.0, beta=0.0, C=None):
    o = offsets.tolist()
    E = len(o) - 1
    out = torch.zeros(E, A.shape[1], B.shape[1], dtype=torch.float64, device=A.device)
    mag = torch.zeros_like(out)
    for e in range(E):
        s = slice(o[e], o[e + 1])
        a, b = A[s].double(), B[s].double()
        out[e], mag[e] = alpha * (a.t() @ b), abs(alpha) * (a.abs().t() @ b.abs())
    if beta:
        out, mag = out + beta * C.double(), mag + abs(beta) * C.double().abs()
    return out, mag


# The tensor core multiplies exactly and adds 16 products to the sum at a time,
# each time cutting off less than 2^-22 of the magnitudes: 32 times in a chunk of
# 512, 7.6e-6 of S.  Adding K / 512 chunks, scaling and beta are 2^-24 each: 1.4e-6
# for K = 11008.
PRODUCT = 1e-5


def act(v, code):
    """(act, slope, bound on act, bound on the slope), FP32 evaluation with exp and reciprocal to 2 ulp.

    The exponent's rounding, |z| 2^-24, is the exponential's relative error beside
    its own 2^-22; an error of (1 - p) where p is near 1 is absolute, 2^-23.
    """
    u = 2.0 ** -23
    if code == 0:
        return v, torch.ones_like(v), 0 * v, 0 * v
    if code == 1:
        cdf = 0.5 * torch.erfc(-v * 0.5 ** 0.5)
        slope = cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        # the tail's polynomial is good to 0.75e-7, its evaluation to
        # (x^2 / 2 + 8) 2^-23 Q(x), at most 4.8e-7; |x| phi(x) (x^2 / 2 + 8) 2^-23 is at most 2.5e-7
        return v * cdf, slope, 6e-7 * v.abs() + u * (v * cdf).abs(), 1e-6 + 0 * v
    if code == 2:
        return v.clamp(min=0), (v > 0).double(), 0 * v, 0 * v
    z = v if code == 4 else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    dz = torch.ones_like(v) if code == 4 else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v ** 2)
    p = torch.sigmoid(z)
    slope = p + v * p * torch.sigmoid(-z) * dz
    rel = (4 * z.abs() + 12) * u  # of p; z itself has three roundings with code 3
    tiny = 2.0 ** -126  # the reciprocal is 0 where p is below the smallest normal number, so p is off by less than that
    return v * p, slope, rel * (v * p).abs() + tiny * v.abs(), tiny * (1 + (v * dz).abs()) + rel * p * (1 + 3 * (v * dz).abs() * torch.sigmoid(-z)) + (v * dz).abs().clamp(max=60) * p * u


def kept(Q, S):
    return Q.double() * S.double().t().repeat_interleave(128, 1)[:, :Q.shape[1]]

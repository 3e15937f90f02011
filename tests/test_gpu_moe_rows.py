"""Rows of the tokens sorted by expert, and back: against plain implementations in 64 bits (GB300)."""
import pytest
import torch

import dense_gemm_11_gb300 as g
from experts_ref import UNIT, close, combine, rounded, sort

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def strided(rows, cols, dtype, pad, shift=0, fill=0.0):
    """rows x cols with rows cols + pad apart, starting `shift` elements into its memory."""
    full = torch.full(((rows + 1) * (cols + pad) + shift,), fill, device="cuda").to(dtype)
    return full[shift:].as_strided((rows, cols), (cols + pad, 1))


def choice(T, k, E, seed, drop=0.0):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(max(E, k), generator=gen)[:k] % E for _ in range(T)]) if T else torch.zeros(0, k, dtype=torch.int64)
    ids[torch.rand(T, k, generator=gen) < drop] = -1
    return ids.int().cuda()


# T, k, E, H, type, padding of the rows, first element
SHAPES = [
    (1, 1, 1, 1, F32, 0, 0), (1, 2, 8, 64, BF16, 0, 0), (3, 3, 5, 7, F16, 0, 0), (16, 2, 8, 4096, BF16, 0, 0), (257, 6, 64, 129, BF16, 7, 0),
    (1000, 3, 13, 1008, F16, 0, 0), (100, 8, 256, 2056, F32, 0, 0), (33, 1, 4096, 40, BF16, 8, 0), (130, 4, 7, 200, BF16, 0, 3), (5, 128, 129, 24, F32, 1, 1),
    (2048, 2, 3, 264, BF16, 0, 0),
]


@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("T,k,E,H,dtype,pad,shift", SHAPES)
def test_dispatch(T, k, E, H, dtype, pad, shift, drop):
    ids = choice(T, k, E, seed=T + E, drop=drop)
    if drop == 0.3:
        ids[ids == E - 1] = E + 5  # past the last expert: chooses none either
    X = strided(T, H, dtype, pad, shift)
    X.copy_(torch.randn(T, H, device="cuda"))
    Xs = strided(T * k + 2, H, dtype, pad, shift, fill=-7.0)
    offsets, rows = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    g.moe_dispatch(ids, X, Xs, offsets, rows)
    assert g.check() == g.GEMM_OK
    want_offsets, want_rows = sort(ids.cpu(), E)
    assert torch.equal(offsets.cpu().long(), want_offsets) and torch.equal(rows.cpu().long(), want_rows)
    want = torch.full((T * k + 2, H), -7.0).to(dtype)
    on = want_rows >= 0
    want[want_rows[on]] = X.cpu().repeat_interleave(k, 0)[on.reshape(-1)]
    assert torch.equal(Xs.cpu(), want)  # rows behind the last expert's too
    if pad:
        gap = Xs.as_strided((T * k + 2, pad), (H + pad, 1), storage_offset=Xs.storage_offset() + H)
        assert (gap == -7.0).all()  # and what is between the rows


def test_dispatch_keeps_nan_and_infinity():
    X = torch.tensor([[float("nan"), float("inf")], [-float("inf"), -0.0]], device="cuda")
    ids = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    Xs, offsets, rows = torch.zeros(2, 2, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    g.moe_dispatch(ids, X, Xs, offsets, rows)
    assert torch.equal(Xs.view(torch.int32), X.flip(0).view(torch.int32))


def test_order_alone_and_no_tokens():
    ids = choice(77, 3, 9, 1, drop=0.1)
    offsets, rows = torch.empty(10, dtype=torch.int32, device="cuda"), torch.empty(77, 3, dtype=torch.int32, device="cuda")
    g.moe_dispatch(ids, None, None, offsets, rows)
    want = sort(ids.cpu(), 9)
    assert torch.equal(offsets.cpu().long(), want[0]) and torch.equal(rows.cpu().long(), want[1])
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    g.moe_dispatch(none, torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda"), offsets, none)
    assert (offsets == 0).all()
    empty = torch.full((1,), 5, dtype=torch.int32, device="cuda")  # no experts
    g.moe_dispatch(ids, None, None, empty, rows)
    assert (empty == 0).all() and (rows == -1).all()


def test_dispatch_many_slots_and_one_expert():
    """More slots than a CTA ranks at a time, all of one expert, and the same expert twice in a token."""
    ids = torch.full((40000, 4), 2, dtype=torch.int32, device="cuda")
    ids[::3, 1] = 0
    X = torch.arange(40000, device="cuda", dtype=F32)[:, None].repeat(1, 4)
    Xs, offsets, rows = torch.empty(160000, 4, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(40000, 4, dtype=torch.int32, device="cuda")
    g.moe_dispatch(ids, X, Xs, offsets, rows)
    key = ids.reshape(-1).cpu()
    order = torch.sort(key, stable=True).indices
    want = torch.empty_like(order)
    want[order] = torch.arange(160000)
    assert torch.equal(rows.reshape(-1).cpu().long(), want)
    assert offsets.tolist() == [0, 13334, 13334, 160000, 160000]
    assert torch.equal(Xs[rows.reshape(-1).long(), 0], X[:, 0].repeat_interleave(4))


# Rows of 4 KB and more go through shared memory: all of a CTA's at once, more of them than it holds, several batches of 1024 slots,
# more slots of a token than lanes, sizes that are not multiples of 128 bytes, rows of which few or none fit.
@pytest.mark.parametrize("T,k,E,H,dtype,pad", [
    (2100, 3, 9, 2048, BF16, 0), (9001, 2, 4, 2048, F32, 8), (1201, 2, 5, 8192, F32, 0), (1500, 1, 5, 16384, BF16, 0), (700, 2, 3, 30000, F16, 8), (400, 2, 3, 60000, F16, 0),
    (3100, 40, 64, 2056, BF16, 16), (30001, 6, 64, 2048, BF16, 0), (153, 2, 8, 2048, F16, 0), (151, 6, 300, 12296, F32, 4),
])
def test_dispatch_long_rows(T, k, E, H, dtype, pad):
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    X = strided(T, H, dtype, pad)
    X.copy_(torch.randn(T, H, generator=gen, device="cuda"))
    Xs = strided(T * k, H, dtype, pad, fill=-7.0)
    offsets, rows = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    want_offsets, want_rows = sort(ids.cpu(), E)
    for _ in range(2):
        g.moe_dispatch(ids, X, Xs, offsets, rows)
        assert g.check() == g.GEMM_OK
        assert torch.equal(offsets.cpu().long(), want_offsets) and torch.equal(rows.cpu().long(), want_rows)
        flat = rows.reshape(-1).long()
        taken = (flat >= 0).nonzero()[:, 0]
        for part in taken.split(4096):
            assert torch.equal(Xs[flat[part]], X[part // k])
        assert (Xs[int(offsets[-1]):] == -7.0).all()
        if pad:
            assert (Xs.as_strided((T * k, pad), (H + pad, 1), storage_offset=H) == -7.0).all()
        X.neg_()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,E,H,dtype,pad,shift", SHAPES)
def test_combine(T, k, E, H, dtype, pad, shift, weighted):
    _, rows = sort(choice(T, k, E, seed=T, drop=0.2).cpu(), E)
    rows = rows.int().cuda()
    R = T * k
    rows[rows == R - 1] = R + 3  # outside: adds nothing
    Ys = strided(R, H, dtype, pad, shift)
    Ys.copy_(torch.randn(R, H, device="cuda"))
    w = torch.rand(T, k, device="cuda") if weighted else None
    Y = strided(T, H, dtype, pad, shift, fill=-7.0)
    g.moe_combine(Ys, rows, Y, w)
    assert g.check() == g.GEMM_OK
    want, mag = combine(Ys, rows, w)
    close(Y.cpu(), want, rounded((k + 1) * 2.0 ** -24 * mag, want, dtype))


@pytest.mark.parametrize("T,k,E,H,dtype,pad,shift", SHAPES)
def test_combine_grad(T, k, E, H, dtype, pad, shift):
    _, rows = sort(choice(T, k, E, seed=T, drop=0.2).cpu(), E)
    R = T * k
    dY, Ys, dYs = strided(T, H, dtype, pad, shift), strided(R, H, dtype, pad, shift), strided(R, H, dtype, pad, shift, fill=-7.0)
    dY.copy_(torch.randn(T, H, device="cuda"))
    Ys.copy_(torch.randn(R, H, device="cuda"))
    w, dw = torch.rand(T, k, device="cuda"), torch.full((T, k), -7.0, device="cuda")
    g.moe_combine_grad(dY, Ys, rows.int().cuda(), w, dYs, dw)
    assert g.check() == g.GEMM_OK
    on = rows >= 0
    t = torch.arange(T)[:, None].expand(T, k)[on]
    dy, ys, wt = dY.double().cpu()[t], Ys.double().cpu()[rows[on]], w.double().cpu()[on]
    want = torch.full((R, H), -7.0, dtype=torch.float64)
    want[rows[on]] = dy * wt[:, None]
    bound = rounded(2.0 ** -24 * want.abs(), want, dtype)
    bound[(want == -7.0).all(1)] = 0  # rows of no slot stay as they are
    close(dYs.cpu(), want, bound, "dYs")
    want_w, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    want_w[on], mag[on] = (dy * ys).sum(1), (dy * ys).abs().sum(1)
    # additions that one product passes through: a thread's, the shuffles' and the warps'
    close(dw.cpu(), want_w, (8 * -(-H // 2048) + 5 + 8) * 2.0 ** -24 * mag, "dweights")


def test_combine_gradient_against_differences():
    T, k, H = 6, 3, 40
    rows = torch.randperm(T * k, device="cuda").int().reshape(T, k)
    Ys, w, dY = torch.randn(T * k, H, device="cuda"), torch.rand(T, k, device="cuda"), torch.randn(T, H, device="cuda")
    dYs, dw, Y = torch.empty_like(Ys), torch.empty_like(w), torch.empty(T, H, device="cuda")
    g.moe_combine_grad(dY, Ys, rows, w, dYs, dw)

    def loss(y, v):
        g.moe_combine(y, rows, Y, v)
        return float((Y.double() * dY.double()).sum())

    step = 0.5  # the function is linear in each: a large step loses nothing but roundings, 2^-24 of about 100
    for i in (0, 7, 17):
        d = torch.zeros_like(Ys)
        d[i, i] = step
        assert abs((loss(Ys + d, w) - loss(Ys - d, w)) / (2 * step) - float(dYs[i, i])) <= 1e-4
    for t, j in ((0, 0), (5, 2)):
        d = torch.zeros_like(w)
        d[t, j] = step
        assert abs((loss(Ys, w + d) - loss(Ys, w - d)) / (2 * step) - float(dw[t, j])) <= 1e-4


def test_tokens_without_a_row():
    Ys, Y = torch.full((4, 24), float("nan"), device="cuda").bfloat16(), torch.full((3, 24), 5.0, device="cuda").bfloat16()
    rows = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    g.moe_combine(Ys, rows, Y)
    assert (Y == 0).all()
    dYs, dw = torch.full_like(Ys, 2.0), torch.full((3, 2), 9.0, device="cuda")
    g.moe_combine_grad(Y, Ys, rows, torch.ones(3, 2, device="cuda"), dYs, dw)
    assert (dYs == 2.0).all() and (dw == 0).all()
    g.moe_combine(Ys[:0], rows, Y)
    assert (Y == 0).all()


def test_unit_roundoffs():
    for t, u in UNIT.items():
        assert u == torch.finfo(t).eps / 2


@pytest.mark.parametrize("T,k,E,H,dtype,pad", [(900, 3, 13, 2056, BF16, 0), (1300, 2, 7, 3001, F16, 5), (1250, 2, 9, 4104, F32, 0), (40, 2, 8, 9000, F32, 0), (6, 5, 8, 8200, BF16, 0)])
def test_combine_grad_in_several_steps(T, k, E, H, dtype, pad):
    """Slots with more columns than their threads take at once: 32 threads where there are 16 slots an SM and more, else 128."""
    lanes = 1
    while lanes < 128 and lanes * 32 < H:
        lanes *= 2
    if T * k >= 16 * torch.cuda.get_device_properties(0).multi_processor_count:
        lanes = min(lanes, 32)
    assert H > 32 * lanes
    torch.manual_seed(H)
    _, rows = sort(choice(T, k, E, seed=T, drop=0.2).cpu(), E)
    R = T * k
    dY, Ys, dYs = strided(T, H, dtype, pad), strided(R, H, dtype, pad), strided(R, H, dtype, pad, fill=-7.0)
    dY.copy_(torch.randn(T, H, device="cuda"))
    Ys.copy_(torch.randn(R, H, device="cuda"))
    w, dw = torch.rand(T, k, device="cuda"), torch.full((T, k), -7.0, device="cuda")
    g.moe_combine_grad(dY, Ys, rows.int().cuda(), w, dYs, dw)
    assert g.check() == g.GEMM_OK
    on = rows >= 0
    t = torch.arange(T)[:, None].expand(T, k)[on]
    dy, ys, wt = dY.double().cpu()[t], Ys.double().cpu()[rows[on]], w.double().cpu()[on]
    want = torch.full((R, H), -7.0, dtype=torch.float64)
    want[rows[on]] = dy * wt[:, None]
    bound = rounded(2.0 ** -24 * want.abs(), want, dtype)
    bound[(want == -7.0).all(1)] = 0
    close(dYs.cpu(), want, bound, "dYs")
    want_w, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    want_w[on], mag[on] = (dy * ys).sum(1), (dy * ys).abs().sum(1)
    # roundings that one product passes through: a thread's fused additions, eight for each 8 x lanes columns, five of the
    # shuffles and four of the warps'; (1 + 2^-24)^n - 1 is below 1.001 n 2^-24 for these n
    n = 8 * -(-H // (8 * lanes)) + 5 + 4
    close(dw.cpu(), want_w, 1.001 * n * 2.0 ** -24 * mag, "dweights")


@pytest.mark.parametrize("T,k,E,H,dtype,pad", [(3000, 2, 4096, 2048, BF16, 0), (700, 3, 4000, 16384, BF16, 8)])
def test_dispatch_long_rows_many_experts(T, k, E, H, dtype, pad):
    """The experts' counters take 32 KB of the shared memory that the rows go through."""
    test_dispatch_long_rows(T, k, E, H, dtype, pad)


def test_as_many_slots_as_there_may_be():
    """2^31 - 32,768 slots, one a token: every one gets its row (the order alone; 17 GB)."""
    n, E, part = 2 ** 31 - 32768, 8, 1 << 27

    def pieces():
        for i in range(0, n, part):
            j = torch.arange(i, min(i + part, n), device="cuda")
            yield i, j, j * 5 % E  # of eight neighbouring slots one for each expert

    ids, rows = torch.empty(n, 1, dtype=torch.int32, device="cuda"), torch.full((n, 1), -9, dtype=torch.int32, device="cuda")
    for i, j, e in pieces():
        ids[i:i + len(j), 0] = e.int()
    offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    g.moe_dispatch(ids, None, None, offsets, rows)
    assert g.check() == g.GEMM_OK
    assert offsets.tolist() == [e * (n // E) for e in range(E + 1)]
    for i, j, e in pieces():
        assert torch.equal(rows[i:i + len(j), 0].long(), e * (n // E) + j // E)

"""Products over rows sorted by expert, against FP64 (GB300)."""
import pytest
import torch

import dense_gemm_11_gb300 as g
from experts_ref import PRODUCT, close, grouped, rounded, wgrad

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def padded(*shape, dtype, fill=None, scale=1.0, pad=None):
    """A tensor whose rows start on 16-byte boundaries (or have `pad` elements between them)."""
    cols = shape[-1]
    ld = -(-cols // 8) * 8 if pad is None else cols + pad
    full = torch.randn(*shape[:-1], ld, device="cuda") * scale if fill is None else torch.full((*shape[:-1], ld), fill, device="cuda")
    return full.to(dtype)[..., :cols]


def offsets_of(sizes):
    return torch.tensor([0] + list(sizes), device="cuda").cumsum(0).int()


# rows of each expert, N, K
SIZES = [
    ([1], 1, 1), ([1, 0, 2], 8, 16), ([0, 0, 5, 0], 24, 72), ([3, 130, 257, 1, 0, 64], 264, 200), ([128, 128], 256, 64), ([300], 520, 1100),
    ([0, 700, 33], 129, 65), ([5] * 40, 136, 128), ([31, 32, 33, 255, 256], 40, 513), ([2, 1, 0, 4], 1000, 1024),
]


@pytest.mark.parametrize("c", [F32, BF16])
@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("sizes,N,K", SIZES)
def test_rows(sizes, N, K, b_trans, c):
    t = F16 if N % 16 == 8 else BF16
    torch.manual_seed(N + K)
    R, E = sum(sizes) + 3, len(sizes)
    A, B = padded(R, K, dtype=t), padded(E, *((N, K) if b_trans else (K, N)), dtype=t)
    C = padded(R, N, dtype=c, fill=-7.0)
    g.gemm_grouped(A, B, C, offsets_of(sizes), b_trans=b_trans)
    assert g.check() == g.GEMM_OK
    want, mag = grouped(A, B, offsets_of(sizes), b_trans)
    n = sum(sizes)
    close(C[:n], want[:n], rounded(PRODUCT * mag[:n], want[:n], c))
    assert (C[n:] == -7.0).all()  # rows behind the last expert's


@pytest.mark.parametrize("c", [F32, F16, BF16])
@pytest.mark.parametrize("sizes,M,N", [(s, n, k) for s, n, k in SIZES] + [([65, 63, 0, 1], 264, 264), ([64, 128, 192], 256, 8), ([513, 511], 136, 300)])
def test_weights(sizes, M, N, c):
    t = F16 if M % 16 == 8 else BF16
    torch.manual_seed(M + N)
    R, E = sum(sizes) + 5, len(sizes)
    A, B = padded(R, M, dtype=t), padded(R, N, dtype=t)
    C = padded(E, M, N, dtype=c, fill=-7.0)
    g.gemm_grouped_wgrad(A, B, C, offsets_of(sizes))
    assert g.check() == g.GEMM_OK
    want, mag = wgrad(A, B, offsets_of(sizes))
    close(C, want, rounded(PRODUCT * mag, want, c))


@pytest.mark.parametrize("t", [F16, BF16])
def test_many_rows(t):
    """More than one tile an expert and a CTA pair, ragged in every direction, empty experts among them."""
    torch.manual_seed(7)
    for sizes, N, K in (([400, 0, 513, 96, 1, 300], 777, 520), ([256] * 3, 512, 64), ([1000, 24], 260, 8), ([200] * 20, 2300, 136), ([999], 1024, 4160)):
        off, R = offsets_of(sizes), sum(sizes) + 2
        A = padded(R, K, dtype=t)
        for bt in (True, False):
            B, C = padded(len(sizes), *((N, K) if bt else (K, N)), dtype=t), padded(R, N, dtype=t, fill=-7.0)
            g.gemm_grouped(A, B, C, off, 0.5, b_trans=bt)
            assert g.check() == g.GEMM_OK
            want, mag = grouped(A, B, off, bt, 0.5)
            n = sum(sizes)
            close(C[:n], want[:n], rounded(PRODUCT * mag[:n], want[:n], t))
            assert (C[n:] == -7.0).all()
        X, dW = padded(R, N, dtype=t), padded(len(sizes), max(K, 136), N, dtype=t, fill=-7.0)
        A = padded(R, max(K, 136), dtype=t)
        g.gemm_grouped_wgrad(A, X, dW, off, 0.5)
        assert g.check() == g.GEMM_OK
        want, mag = wgrad(A, X, off, 0.5)
        close(dW, want, rounded(PRODUCT * mag, want, t))


@pytest.mark.parametrize("t", [F16, BF16])
def test_neighbours_do_not_leak(t):
    """NaN and infinity in another expert's rows, in its weights and behind the last row reach nobody else."""
    sizes, N, K = [70, 1, 100, 0, 29], 72, 136
    off = offsets_of(sizes)
    A, X = padded(240, K, dtype=t), padded(240, N, dtype=t)
    for m in (A, X):
        m[70] = float("nan")
        m[200:] = float("inf")
    B = padded(5, N, K, dtype=t)
    B[1], B[3] = float("nan"), float("inf")
    for bt in (True, False):
        b = B if bt else B.transpose(1, 2).contiguous()
        C = padded(240, N, dtype=F32, fill=0.0)
        g.gemm_grouped(A, b, C, off, b_trans=bt)
        assert C[70].isnan().all() and not C[:70].isnan().any() and torch.isfinite(C[71:200]).all() and (C[200:] == 0).all()
    dW = padded(5, K, N, dtype=F32, fill=float("nan"))
    g.gemm_grouped_wgrad(A, X, dW, off)
    assert g.check() == g.GEMM_OK
    assert dW[1].isnan().all() and torch.isfinite(dW[[0, 2, 3, 4]]).all() and (dW[3] == 0).all()


@pytest.mark.parametrize("alpha,beta", [(0.5, 2.0), (0.0, 0.5), (-1.0, 0.0), (0.0, 0.0)])
def test_alpha_beta(alpha, beta):
    sizes, N, K = [40, 0, 200], 80, 600
    off = offsets_of(sizes)
    A, B, C0 = padded(243, K, dtype=BF16), padded(3, N, K, dtype=BF16), padded(243, N, dtype=F16)
    C = padded(243, N, dtype=F16)
    C.copy_(C0)
    if beta == 0.0:
        C[:240] = float("nan")
    g.gemm_grouped(A, B, C, off, alpha, beta)
    want, mag = grouped(A, B, off, True, alpha, beta, C0)
    close(C[:240], want[:240], rounded(PRODUCT * mag[:240], want[:240], F16))
    assert torch.equal(C[240:], C0[240:])
    A2, D0 = padded(243, N, dtype=BF16), padded(3, N, K, dtype=F32)
    D = D0.clone()
    if beta == 0.0:
        D[:] = float("nan")
    g.gemm_grouped_wgrad(A2, A, D, off, alpha, beta)
    want, mag = wgrad(A2, A, off, alpha, beta, D0)
    close(D, want, rounded(PRODUCT * mag, want, F32))


def test_alpha_zero_reads_nothing():
    off = offsets_of([10, 6])
    A, B, C = padded(16, 32, dtype=F16, fill=float("nan")), padded(2, 8, 32, dtype=F16, fill=float("nan")), padded(16, 8, dtype=F32, fill=3.0)
    g.gemm_grouped(A, B, C, off, 0.0, 2.0)
    assert (C == 6.0).all()


@pytest.mark.parametrize("pad", [0, 1, 3])
@pytest.mark.parametrize("c", [F32, BF16])
def test_any_rows_of_c(c, pad):
    """C whose rows are not aligned for wide stores, and what lies between its rows."""
    sizes, N, K = [150, 300], 129, 96
    off = offsets_of(sizes)
    A, B = padded(450, K, dtype=BF16), padded(2, N, K, dtype=BF16)
    full = torch.full((450 * (N + pad) + 1,), -7.0, device="cuda", dtype=c)
    C = full[1:].as_strided((450, N), (N + pad, 1))
    g.gemm_grouped(A, B, C, off)
    want, mag = grouped(A, B, off, True)
    close(C, want, rounded(PRODUCT * mag, want, c))
    if pad:
        assert (full[1:].as_strided((450, pad), (N + pad, 1), storage_offset=1 + N) == -7.0).all()
    D = torch.full((2 * (K * (N + pad) + 5),), -7.0, device="cuda", dtype=c)
    dW = D.as_strided((2, K, N), (K * (N + pad) + 5, N + pad, 1))
    X = padded(450, N, dtype=BF16)
    g.gemm_grouped_wgrad(A, X, dW, off)
    want, mag = wgrad(A, X, off)
    close(dW, want, rounded(PRODUCT * mag, want, c))
    assert (D[-5:] == -7.0).all()


def test_offsets_outside_are_taken_as_the_nearer_end():
    A, B, C = padded(20, 16, dtype=F16), padded(3, 8, 16, dtype=F16), padded(20, 8, dtype=F32, fill=-7.0)
    g.gemm_grouped(A, B, C, torch.tensor([-5, 4, 12, 1000], dtype=torch.int32, device="cuda"))
    want, mag = grouped(A, B, torch.tensor([0, 4, 12, 20]), True)
    close(C, want, rounded(PRODUCT * mag, want, F32))
    C.fill_(-7.0)
    g.gemm_grouped(A, B, C, torch.tensor([3, 4, 4, 9], dtype=torch.int32, device="cuda"))
    want, mag = grouped(A, B, torch.tensor([3, 4, 4, 9]), True)
    close(C[3:9], want[3:9], rounded(PRODUCT * mag[3:9], want[3:9], F32))
    assert (C[:3] == -7.0).all() and (C[9:] == -7.0).all()


def test_many_experts_and_tiles():
    """More experts than a warp has lanes, most without rows; more tiles than CTA pairs."""
    torch.manual_seed(1)
    sizes = [(i * 37) % 11 if i % 3 == 0 else 0 for i in range(300)] + [900]
    off = offsets_of(sizes)
    R = sum(sizes)
    A, B, C = padded(R, 64, dtype=BF16), padded(301, 520, 64, dtype=BF16), padded(R, 520, dtype=F32, fill=-7.0)
    g.gemm_grouped(A, B, C, off)
    want, mag = grouped(A, B, off, True)
    close(C, want, rounded(PRODUCT * mag, want, F32))
    X, dW = padded(R, 264, dtype=BF16), padded(301, 264, 64, dtype=F32, fill=-7.0)
    g.gemm_grouped_wgrad(X, A, dW, off)
    assert g.check() == g.GEMM_OK
    want, mag = wgrad(X, A, off)
    close(dW, want, rounded(PRODUCT * mag, want, F32))


def test_sums_to_nearest():
    """Equal signs: the tensor core's truncation would show over a long contraction without the chunks."""
    K = 8192
    A, B = padded(256, K, dtype=BF16).abs(), padded(1, 256, K, dtype=BF16).abs()
    C = padded(256, 256, dtype=F32)
    g.gemm_grouped(A, B, C, offsets_of([256]))
    want, mag = grouped(A, B, offsets_of([256]), True)
    err = ((C.double() - want) / mag).abs()
    assert float(err.max()) <= 3e-6 and float(((C.double() - want) / mag).mean().abs()) <= 3e-6


SPLIT = [([3, 0, 16, 1], 200, 4100), ([64, 60], 256, 8192), ([1, 1], 1000, 4096), ([130, 0, 5], 24, 2056), ([256], 300, 11008)]


@pytest.mark.parametrize("t,c", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("sizes,N,K", SPLIT)
def test_units_share_a_contraction(sizes, N, K, t, c):
    """Few tiles, a long contraction: its parts' sums are added in one order, whichever CTA comes last."""
    torch.manual_seed(K)
    off, R = offsets_of(sizes), sum(sizes) + 1
    A, C0 = padded(R, K, dtype=t), padded(R, N, dtype=c)
    for bt in (True, False):
        B = padded(len(sizes), *((N, K) if bt else (K, N)), dtype=t)
        results = []
        for beta in (0.0, 0.0, 0.5):
            C = padded(R, N, dtype=c)
            C.copy_(C0)
            g.gemm_grouped(A, B, C, off, 1.0, beta, b_trans=bt)
            assert "splitk" in g.last_plan() and g.check() == g.GEMM_OK
            want, mag = grouped(A, B, off, bt, 1.0, beta, C0)
            close(C[:R - 1], want[:R - 1], rounded(PRODUCT * mag[:R - 1], want[:R - 1], c))
            assert torch.equal(C[R - 1], C0[R - 1])
            results.append(C)
        assert torch.equal(results[0], results[1])


@pytest.mark.parametrize("sizes,M,N", [([2000, 0, 777], 100, 130), ([8000], 256, 512), ([3, 900, 64, 1300], 16, 40), ([20000, 0, 9001], 100, 130), ([7, 33000], 264, 256)])
def test_units_share_rows(sizes, M, N):
    off, R = offsets_of(sizes), sum(sizes) + 9
    A, B = padded(R, M, dtype=BF16), padded(R, N, dtype=BF16)
    A[R - 9:] = float("nan")
    for beta in (0.0, 2.0):
        C0 = padded(len(sizes), M, N, dtype=F32)
        C, D = C0.clone(), C0.clone()
        g.gemm_grouped_wgrad(A, B, C, off, 0.25, beta)
        assert ("splitk" in g.last_plan() or R < 20000) and g.check() == g.GEMM_OK
        g.gemm_grouped_wgrad(A, B, D, off, 0.25, beta)
        assert torch.equal(C, D)
        want, mag = wgrad(A, B, off, 0.25, beta, C0)
        close(C, want, rounded(PRODUCT * mag, want, F32))


def test_descending_offsets_stay_inside():
    """What they give is not defined, but nothing is written outside C, and the next call is right."""
    full = torch.full((130, 64), -7.0, device="cuda")
    C, A, B = full[1:129], padded(128, 4096, dtype=BF16), padded(6, 64, 4096, dtype=BF16)
    g.gemm_grouped(A, B, C, torch.tensor([0, 128, 0, 128, 0, 128, 0], dtype=torch.int32, device="cuda"))
    assert g.check() == g.GEMM_OK and (full[0] == -7.0).all() and (full[129] == -7.0).all()
    off = offsets_of([20, 0, 30, 40, 8, 30])
    g.gemm_grouped(A, B, C, off)
    want, mag = grouped(A, B, off, True)
    close(C, want, rounded(PRODUCT * mag, want, F32))


@pytest.mark.parametrize("c", [F16, BF16])
@pytest.mark.parametrize("N", [1, 7, 31, 33, 250, 513, 1021])
def test_short_contractions_into_16_bits(N, c):
    """Rows of C on 16 bytes and not, any last column, more tiles than CTA pairs: what lies between the rows stays."""
    torch.manual_seed(N)
    sizes = [1, 8, 9, 0, 127, 129, 250, 255, 257, 300, 64] * 8
    off, n, K = offsets_of(sizes), sum(sizes), 40
    A, B = padded(n, K, dtype=c), padded(len(sizes), N, K, dtype=c)
    want, mag = grouped(A, B, off, True)
    for pad, start in ((-N % 8 + 8, 0), (-N % 8, 8), (-N % 8 + 8, 4), (-N % 2 + 2, 0)):
        full = torch.full((n + 2, N + pad), -7.0, device="cuda", dtype=c).reshape(-1)
        C = full[start:start + n * (N + pad)].reshape(n, N + pad)[:, :N]
        g.gemm_grouped(A, B, C, off, b_trans=True)
        assert g.check() == g.GEMM_OK
        close(C, want, rounded(PRODUCT * mag, want, c))
        C.fill_(-7.0)
        assert (full == -7.0).all()
    for M, few in ((130, [3, 64, 0, 65, 200]), (515, [3, 64, 0, 65, 20] * 9), (77, [300, 350])):
        R = sum(few) + 8
        X, Y = padded(R, M, dtype=c), padded(R, N, dtype=c)
        want, mag = wgrad(X, Y, offsets_of(few))
        for pad, start in ((-N % 8 + 8, 0), (-N % 8, 8), (-N % 8 + 8, 4), (-N % 2 + 2, 0)):
            full = torch.full((len(few) + 1, M + 3, N + pad), -7.0, device="cuda", dtype=c).reshape(-1)
            C = full[start:start + len(few) * (M + 3) * (N + pad)].reshape(len(few), M + 3, N + pad)[:, :M, :N]
            g.gemm_grouped_wgrad(X, Y, C, offsets_of(few))
            assert g.check() == g.GEMM_OK
            close(C, want, rounded(PRODUCT * mag, want, c))
            C.fill_(-7.0)
            assert (full == -7.0).all()


def test_weights_into_16_bits_streams_and_graphs():
    """Twice, on two streams at once and from a graph: the same bits; NaN of one expert stays there; no rows at all give zeros."""
    torch.manual_seed(5)
    sizes, M, N = [3, 70, 0, 129, 64] * 6, 300, 520
    off, R = offsets_of(sizes), sum(sizes)
    X, Y = padded(R, M, dtype=BF16), padded(R, N, dtype=BF16)
    X[73 + 64] = float("nan")  # of expert 3
    outs = [padded(len(sizes), M, N, dtype=BF16, fill=-7.0) for _ in range(4)]
    g.gemm_grouped_wgrad(X, Y, outs[0], off)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, C in zip(side, outs[1:3]):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.gemm_grouped_wgrad(X, Y, C, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemm_grouped_wgrad(X, Y, outs[3], off)
    outs[3].fill_(-7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert g.check() == g.GEMM_OK
    for C in outs[1:]:
        assert torch.equal(C.view(torch.int16), outs[0].view(torch.int16))
    others = [e for e in range(len(sizes)) if e != 3]
    assert outs[0][3].isnan().all() and torch.isfinite(outs[0][others]).all() and (outs[0][2] == 0).all()
    want, mag = wgrad(X, Y, off)
    close(outs[0][others], want[others], rounded(PRODUCT * mag[others], want[others], BF16))
    g.gemm_grouped_wgrad(X, Y, outs[0], torch.zeros_like(off))
    g.gemm_grouped_wgrad(X, Y, outs[1], off, 0.0)
    g.gemm_grouped_wgrad(X[:0], Y[:0], outs[2], torch.zeros_like(off))
    assert all((C == 0).all() for C in outs[:3])


def test_many_experts_without_rows():
    """The walk of their offsets to the last one, which has rows, outlasts the two seconds that a wait has otherwise."""
    E = 2 ** 28
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 3
    A, B, C = padded(5, 8, dtype=BF16), torch.zeros(E, 1, 8, dtype=BF16, device="cuda"), torch.full((5, 1), -7.0, device="cuda")
    B[E - 1] = torch.randn(1, 8)
    g.gemm_grouped(A, B, C, off)
    assert g.check() == g.GEMM_OK
    want, mag = grouped(A[:3], B[E - 1:], torch.tensor([0, 3]), True)
    close(C[:3], want, rounded(PRODUCT * mag, want, F32))
    assert (C[3:] == -7.0).all()


def test_all_rows_of_one_expert():
    """A contraction of 3 * 2^28 rows, which one CTA pair walks alone: so does that."""
    E, e, R = 5000, 3211, 3 * 2 ** 28
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[e + 1:] = R
    gen = torch.Generator(device="cuda").manual_seed(3)
    A, B = (torch.randint(-1, 2, (R, 8), generator=gen, device="cuda", dtype=torch.int8).to(BF16) for _ in range(2))
    C = torch.full((E, 8, 8), -7.0, device="cuda")
    g.gemm_grouped_wgrad(A, B, C, off)
    assert g.check() == g.GEMM_OK and g.last_plan() == "grouped_wgrad_pair"
    want = sum(a.double().t() @ b.double() for a, b in zip(A.split(2 ** 24), B.split(2 ** 24)))
    assert float(want.abs().max()) < 2 ** 22  # of -1, 0 and 1: every partial sum is far from 2^24, so exact
    assert torch.equal(C[e].double(), want) and int((C != 0).sum()) == int((want != 0).sum())


LARGEST = 2 ** 31 - 512


def parts(n, size=2 ** 27):
    return [slice(i, min(i + size, n)) for i in range(0, n, size)]


def test_as_many_rows_as_there_may_be():
    """2^31 - 512 rows of one expert (39 GB)."""
    A, C = torch.empty(LARGEST, 8, dtype=BF16, device="cuda"), torch.full((LARGEST, 1), -7.0, dtype=BF16, device="cuda")
    for s in parts(LARGEST):
        A[s] = (torch.arange(s.start, s.stop, device="cuda") % 5 - 2).to(BF16)[:, None]
    B = torch.tensor([1.0, 2, 3, -4, 5, 6, 7, 8], device="cuda").to(BF16).reshape(1, 1, 8)  # 28 together
    g.gemm_grouped(A, B, C, torch.tensor([0, LARGEST], dtype=torch.int32, device="cuda"))
    assert g.check() == g.GEMM_OK
    for s in parts(LARGEST):
        assert torch.equal(C[s, 0], A[s, 0] * 28)


def test_as_many_columns_as_there_may_be():
    """A matrix gradient of 2^31 - 512 rows (9 GB)."""
    A, B, C = torch.empty(1, LARGEST, dtype=BF16, device="cuda"), torch.full((1, 1), 2.0, dtype=BF16, device="cuda"), torch.full((1, LARGEST, 1), -7.0, dtype=BF16, device="cuda")
    for s in parts(LARGEST):
        A[0, s] = (torch.arange(s.start, s.stop, device="cuda") % 5 - 2).to(BF16)
    g.gemm_grouped_wgrad(A, B, C, torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert g.check() == g.GEMM_OK
    for s in parts(LARGEST):
        assert torch.equal(C[0, s, 0], A[0, s] * 2)

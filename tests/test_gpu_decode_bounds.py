"""The few-row linears where a result is far smaller than its terms, against 64 bits: what is held on the way shows
there, and not in results that are rounded to bf16 next to a large value.

Every product of a piece of an activation (8 bits) and a code (4 bits) is exact in fp32.  A window of 128 codes is summed in
fp32, then windows, waves and the bias: at most 128 * 3 pieces + K / 128 + 16 additions, each off by 2 u of the sum of
absolute terms at the most (the matrix cores may cut instead of rounding), u = 2^-24."""
import math

import pytest

torch = pytest.importorskip("torch")

from guard import check_guard, guarded_output  # noqa: E402
from test_gpu_decode import BF, DT, U, dev, gen, hadamard64, qv, random_weights  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def pack(q):
    return (q[:, 0::2] & 15 | q[:, 1::2] << 4).view(torch.uint8).contiguous()


def linear(qv, dev, X, q, ws, group, rotate, yt, epi=0):
    M, K = X.shape
    Y = torch.empty((M, q.shape[0]), dtype=DT[yt], device=dev)
    if rotate:
        work = torch.empty(max(1, qv.qv_w4a16_linear_workspace_size(M, K)), dtype=torch.uint8, device=dev)
        qv.qv_w4a16_linear(X.to(dev), None, pack(q).to(dev), ws.to(dev), group, None, Y, work, epi)
    else:
        qv.qv_w4a16_gemv(X.to(dev), pack(q).to(dev), ws.to(dev), group, None, Y, epi)
    return Y.double().cpu()


@pytest.mark.parametrize("size", [1e5, 1e6, 1e7, 1e37])
@pytest.mark.parametrize("M,K,N,group,xt", [
    (1, 1024, 64, 128, "bf16"), (5, 2048, 700, 256, "bf16"), (16, 4096, 900, 4096, "bf16"), (3, 4096, 2500, 512, "bf16"),
    (20, 1024, 4100, 128, "bf16"), (4, 1024, 9000, 128, "bf16"), (16, 1024, 17000, 1024, "bf16"), (2, 1024, 100, 128, "fp32"),
])
def test_outlier_against_zero_codes(qv, dev, M, K, N, group, xt, size):
    """A large activation whose codes are zero adds exactly nothing to a bf16 result."""
    g = gen(K + N)
    q, _, ws = random_weights(N, K, group, g)
    X = torch.randn((M, K), generator=g)
    at = torch.randint(K, (3,), generator=g)
    q[:, at] = 0
    X[:, at] = size * torch.tensor([1.0, -1.0, 0.77])
    X = X.to(DT[xt])
    Y = linear(qv, dev, X, q, ws, group, False, "bf16")
    w = q.double() * ws.double().repeat_interleave(group, 1)
    y, terms = X.double() @ w.t(), X.double().abs() @ w.abs().t()
    tol = BF * 1.01 * y.abs() + 2 * (3 * 128 + K / 128 + 16) * U * terms
    worst = ((Y - y).abs() / tol).max().item()
    assert worst <= 1.0, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("xt,K,rotate", [("fp32", 128, False), ("fp32", 2048, False), ("fp32", 1024, True), ("fp32", 4096, True),
                                         ("bf16", 1024, True), ("bf16", 4096, True)])
@pytest.mark.parametrize("M", [1, 5, 17])
def test_last_bits_of_an_activation(qv, dev, xt, K, rotate, M):
    """Two activations that agree in their first bits cancel: a bf16 result shows the bits behind them, exactly.

    Unrotated 1 + 2^-8 + 2^-17 and 1 + 2^-8; rotated, a row of three values a, b, c, whose elements are (+-a +- b +- c) /
    sqrt K: those of the same signs for a and b and either sign for c differ by 2 c / sqrt K.  Every sum on the way is exact."""
    N = 40
    X = torch.zeros((M, K))
    q = torch.zeros((N, K), dtype=torch.int8)
    if rotate:
        a, b, c = 1 + 2.0 ** -7, 2.0 ** -8 + 2.0 ** -15, 2.0 ** -17
        at = (3, 5 + 8, K // 2 + 1)
        X[:, at[0]], X[:, at[1]], X[:, at[2]] = a, b, c
        h = hadamard64(K)[list(at)]
        plus = ((h[0] > 0) & (h[1] > 0) & (h[2] > 0)).nonzero()[:, 0]
        minus = ((h[0] > 0) & (h[1] > 0) & (h[2] < 0)).nonzero()[:, 0]
        value = 2 * c / math.sqrt(K)
    else:
        plus, minus = torch.arange(0, 64, 2), torch.arange(1, 64, 2)
        X[:, plus], X[:, minus] = 1 + 2.0 ** -8 + 2.0 ** -17, -(1 + 2.0 ** -8)
        value = 2.0 ** -17
    for n in range(N):
        q[n, plus[n % len(plus)]] = 7
        q[n, minus[(3 * n) % len(minus)]] = -7 if rotate else 7
    ws = torch.full((N, K // 128), 0.5)
    Y = linear(qv, dev, X.to(DT[xt]), q, ws, 128, rotate, "bf16")
    assert bool((Y == 3.5 * value).all()), (Y / (3.5 * value)).unique()


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
def test_single_row_of_any_stride(qv, dev, xt):
    """One row of a tensor whose row stride is odd: the stride of a single row counts for nothing."""
    g = gen(7)
    q, packed, ws = random_weights(24, 256, 128, g)
    wide = torch.randn((3, 259), generator=g).to(DT[xt]).to(dev)
    Y = torch.empty((3, 31), device=dev)
    qv.qv_w4a16_gemv(wide[:1, :256], packed.to(dev), ws.to(dev), 128, None, Y[:1, :24])
    y = wide[:1, :256].double().cpu() @ (q.double() * ws.double().repeat_interleave(128, 1)).t()
    assert bool(((Y[:1, :24].double().cpu() - y).abs() <= 1e-4).all())
    with pytest.raises(qv.QVError, match="ALIGN"):  # the next row is not aligned
        qv.qv_w4a16_gemv(wide[:2, :256], packed.to(dev), ws.to(dev), 128, None, Y[:2, :24])


def test_rows_in_several_launches(qv, dev):
    """More rows than one launch takes, against a call of the last of them alone."""
    M, K, N, last = (1 << 20) + 45, 1024, 8, 61
    g = gen(11)
    q, packed, ws = random_weights(N, K, 128, g)
    X = torch.randn((M, K), device=dev, dtype=torch.bfloat16)
    Y = torch.full((M, N), float("nan"), device=dev)
    work = torch.empty(qv.qv_w4a16_linear_workspace_size(M, K), dtype=torch.uint8, device=dev)
    args = (None, packed.to(dev), ws.to(dev), 128, None)
    qv.qv_w4a16_linear(X, *args, Y, work)
    assert not bool(torch.isnan(Y).any())
    for at in (0, (1 << 20) - 30, M - last):
        few = torch.empty((last, N), device=dev)
        qv.qv_w4a16_linear(X[at:at + last], *args, few, work)
        assert torch.equal(few, Y[at:at + last])


@pytest.mark.parametrize("M,K,N,group,xt,yt", [
    (2, 4096, 1500, 128, "bf16", "bf16"), (2, 4096, 3000, 256, "bf16", "bf16"), (4, 4096, 2000, 512, "fp32", "fp32"),
    (3, 4096, 4000, 128, "fp32", "fp32"), (5, 4096, 8300, 128, "bf16", "bf16"), (5, 4096, 9001, 512, "fp32", "fp32"),
    (2, 4096, 17000, 4096, "bf16", "fp32"), (1, 4096, 6000, 128, "fp32", "bf16"), (12, 1024, 9000, 128, "bf16", "bf16"),
    (11, 1024, 8201, 1024, "fp32", "fp32"), (7, 1024, 5000, 256, "fp32", "bf16"), (1, 1024, 17000, 128, "bf16", "fp32"),
    (13, 1024, 9000, 128, "bf16", "bf16"), (6, 4096, 9000, 128, "bf16", "fp32"), (2, 4096, 9000, 128, "bf16", "bf16"),
    (3, 4096, 1000, 256, "fp32", "bf16"),
])
def test_wide_rotated_layers(qv, dev, M, K, N, group, xt, yt):
    """Rotated rows with every number of channels to a block.  The rotation adds log2 K roundings to an activation, each of u of
    the row's norm over sqrt K at the most in the root of their squares: 12 u |x| / sqrt K |s q| in the whole."""
    check_wide(qv, dev, M, K, N, group, xt, yt, True)


@pytest.mark.parametrize("M,K,N,group,xt,yt", [
    (3, 1152, 9001, 128, "fp32", "fp32"), (16, 2048, 9000, 512, "fp32", "fp32"), (1, 4096, 8300, 128, "fp32", "bf16"),
    (31, 2048, 2000, 128, "bf16", "fp32"), (40, 1024, 3000, 256, "bf16", "bf16"), (100, 512, 12000, 128, "bf16", "bf16"),
    (20, 4096, 9000, 4096, "fp32", "fp32"), (2, 2176, 1030, 128, "bf16", "bf16"), (2, 4224, 1000, 128, "fp32", "bf16"),
])
def test_wide_layers(qv, dev, M, K, N, group, xt, yt):
    """Rows out of memory with every number of channels and row tiles to a block."""
    check_wide(qv, dev, M, K, N, group, xt, yt, False)


def check_wide(qv, dev, M, K, N, group, xt, yt, rotate):
    """An fp32 sum of K exact products errs like a random walk of them: 8 deviations of sqrt(K) u |s x q| in an element."""
    g = gen(M + K + N)
    q, packed, ws = random_weights(N, K, group, g)
    X = torch.randn((M, K), generator=g).to(DT[xt])
    work = torch.empty(qv.qv_w4a16_linear_workspace_size(M, K), dtype=torch.uint8, device=dev)
    full, Y = guarded_output(M, N, DT[yt], dev, 5)
    if rotate:
        qv.qv_w4a16_linear(X.to(dev), None, packed.to(dev), ws.to(dev), group, None, Y, work)
    else:
        qv.qv_w4a16_gemv(X.to(dev), packed.to(dev), ws.to(dev), group, None, Y)
    check_guard(full, M, N)
    x = X.double() @ hadamard64(K) / math.sqrt(K) if rotate else X.double()
    w = q.double() * ws.double().repeat_interleave(group, 1)
    y, norm = x @ w.t(), ((x ** 2) @ (w.t() ** 2)).sqrt()
    extra = 12 * U * (x.norm(dim=1, keepdim=True) / math.sqrt(K)) * w.norm(dim=1) if rotate else 0.0
    tol = 8 * (math.sqrt(K) * U * norm + extra) + (BF * 1.01 * y.abs() if yt == "bf16" else U * y.abs())
    worst = ((Y.double().cpu() - y).abs() / tol).max().item()
    assert worst <= 1.0, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("M,K,N,group,xt,rotate", [
    (4, 1024, 1000, 128, "bf16", False), (16, 4096, 3000, 512, "fp32", False), (3, 4096, 1024, 128, "bf16", True),
    (40, 2048, 4100, 128, "bf16", False), (12, 1024, 2000, 1024, "fp32", True), (1, 8192, 700, 256, "bf16", False),
])
def test_whole_fp32_results(qv, dev, M, K, N, group, xt, rotate):
    """The 2-norm of all errors over that of |s x q|.  Up to 384 additions of a window's exact products at partial sums that
    grow to its norm: the root of 384 / 2 times u / sqrt 3, 8 u; then K / 128 + 8 sums of windows and waves (72 / 2: 3.5 u); the
    rotation's log2 K roundings of an activation (2 u).  The root of their squares is below 10 u."""
    g = gen(M * 31 + N)
    q, _, ws = random_weights(N, K, group, g)
    X = torch.randn((M, K), generator=g).to(DT[xt])
    Y = linear(qv, dev, X, q, ws, group, rotate, "fp32")
    x = X.double() @ hadamard64(K) / math.sqrt(K) if rotate else X.double()
    w = q.double() * ws.double().repeat_interleave(group, 1)
    off = ((Y - x @ w.t()).norm() / ((x ** 2) @ (w.t() ** 2)).sqrt().norm()).item()
    assert off <= 10 * U, f"{off / U:.1f} u"


@pytest.mark.parametrize("M,K,N,xt,yt", [(1, 1024, 16450, "bf16", "bf16"), (12, 1024, 16385, "fp32", "bf16"), (3, 4096, 16391, "bf16", "bf16"),
                                         (4, 4096, 16390, "bf16", "fp32"), (2, 4096, 33000, "fp32", "fp32")])
def test_rotated_layers_of_several_rounds(qv, dev, M, K, N, xt, yt):
    """More channels than one round of blocks takes, where rows are rotated by a kernel before from fewer rows on."""
    check_wide(qv, dev, M, K, N, 128, xt, yt, True)

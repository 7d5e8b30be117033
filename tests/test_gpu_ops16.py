"""GPU checks of the 16-bit operators against plain 64-bit forms.

Every tolerance is a bound, not a fit.  With h = finfo(dtype).eps / 2, the
half step of the output's rounding, an output may be off by h |y| plus what
fp32 arithmetic loses before it:
  products    n 2^-24 sum |terms| for a sum of n products (any order), times
              the activation's steepest slope (1.13 for GELU, 1.1 for SiLU),
              2^-20 |p| for the activation itself, 2^-23 (|y| + |r|) for the
              last additions;
  layer norm  a row's sums go through at most 80 additions in a row (48 per
              thread at most, then the tree), so they are off by 80 2^-24 of
              the sum of magnitudes;
  rotations   2^-22 (|a| + |b|): the angle's 2^-25 half turns (9.4e-8) and the
              sine's and cosine's own 2^-23, then two products and a sum.
"""
import ctypes

import pytest
import torch

import w4a4_quantized_gemm_smooth_b200 as S

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SLOPE = {S.EPI_NONE: 1.0, S.EPI_GELU: 1.13, S.EPI_SILU: 1.1}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "gpu tests need a CUDA device"
    S.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, m, k, dtype, scale=1.0, ld=None, guard=None):
    """[m, k] values in rows of ld elements; the padding holds `guard`."""
    ld = ld or -(-k // 8) * 8
    x = torch.full((m, ld), float("nan") if guard is None else guard, dtype=dtype, device="cuda")
    x[:, :k] = (torch.randn((m, k), generator=g, device="cuda") * scale).to(dtype)
    return x[:, :k]


def out(m, k, dtype, ld=None):
    """[m, k] to be written, in rows whose padding holds 77."""
    return torch.full((m, ld or -(-k // 8) * 8 + 8), 77.0, dtype=dtype, device="cuda")[:, :k]


def padding_kept(y):
    base = y._base
    return bool((base[:, y.shape[1]:] == 77.0).all())


def half(dtype):
    return torch.finfo(dtype).eps / 2


def close(y, ref, tol, what=""):
    d = (y.double() - ref).abs()
    tiny = 2.0 ** -25 if y.dtype == F16 else 1e-37
    bad = ~(d <= tol + tiny)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / (tol + tiny)).nan_to_num(1e9).max()):.3g} x the bound"


def act64(p, epi):
    if epi == S.EPI_GELU:
        return p * torch.special.ndtr(p)
    return p * torch.sigmoid(p) if epi == S.EPI_SILU else p


def act_grad64(p, epi):
    if epi == S.EPI_GELU:
        return torch.special.ndtr(p) + p * torch.exp(-p * p / 2) / (2 * torch.pi) ** 0.5
    if epi == S.EPI_SILU:
        q = torch.sigmoid(p)
        return q * (1 + p * (1 - q))
    return torch.ones_like(p)


# ------------------------------------------------------------------- linear
def check_linear(M, K, N, dtype, epi, bias=True, res=True, pre=True, seed=0, inplace=False):
    g = gen(seed)
    X, W = rows(g, M, K, dtype), rows(g, N, K, dtype, K ** -0.5)
    b = torch.randn((N,), generator=g, device="cuda").to(dtype) if bias else None
    Y, P = out(M, N, dtype), out(M, N, dtype) if pre else None
    R = rows(g, M, N, dtype) if res else None
    r64 = R.double() if res else 0.0
    if inplace:
        Y.copy_(R)
        R = Y
    S.svdq_linear16(X, W, Y, b, R, epi, P)
    S.svdq_get_op_error()
    x, w = X.double(), W.double()
    p = x @ w.T + (b.double() if bias else 0.0)
    e_p = (K + 1) * 2.0 ** -24 * (x.abs() @ w.abs().T + (b.double().abs() if bias else 0.0))
    a = act64(p, epi)
    y = a + r64
    e = SLOPE[epi] * e_p + (2.0 ** -20 * p.abs() if epi else 0.0) + 2.0 ** -23 * (a.abs() + (r64.abs() if res else 0.0))
    h = half(dtype)
    close(Y, y, h * (y.abs() + e) + e, "Y")
    assert padding_kept(Y)
    if pre:
        close(P, p, h * (p.abs() + e_p) + e_p, "P")
        assert padding_kept(P)


@pytest.mark.parametrize("M,K,N", [
    (1, 1, 1), (1, 8, 8), (1, 64, 128), (2, 65, 7), (3, 1152, 6912), (8, 1153, 130), (16, 200, 96),
    (17, 4608, 1152), (64, 256, 512), (127, 333, 257), (128, 128, 128), (129, 129, 129),
    (200, 64, 1000), (256, 1152, 1152), (300, 100, 2307), (1000, 520, 72), (777, 1153, 385),
])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_sizes(M, K, N, dtype):
    check_linear(M, K, N, dtype, S.EPI_GELU, seed=M + K + N)


@pytest.mark.parametrize("M,K,N", [
    (20, 2696, 1599), (133, 2640, 2583), (92, 2866, 5), (137, 1606, 1297), (132, 2764, 1236), (424, 5, 2475),
    (128, 12288, 1152), (60, 9000, 300), (700, 1000, 4000)])
def test_linear_forms(M, K, N):
    """Sizes for which the other tile widths and splits are chosen."""
    check_linear(M, K, N, BF16, S.EPI_GELU, seed=K)
    check_linear(M, K, N, F16, S.EPI_NONE, bias=False, pre=False, seed=K)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17])
@pytest.mark.parametrize("K,N", [(1, 1), (31, 9), (32, 8), (250, 4737), (4097, 33), (1153, 5000), (12287, 129)])
def test_linear_few_rows(M, K, N):
    for dtype in (BF16, F16):
        check_linear(M, K, N, dtype, S.EPI_SILU, seed=M + K)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("epi", [S.EPI_NONE, S.EPI_GELU, S.EPI_SILU])
@pytest.mark.parametrize("bias,res,pre", [(False, False, False), (True, False, False), (False, True, False),
                                          (False, False, True), (True, True, True)])
@pytest.mark.parametrize("M", [1, 150])
def test_linear_epilogues(dtype, epi, bias, res, pre, M):
    check_linear(M, 328, 301, dtype, epi, bias, res, pre, seed=5)


@pytest.mark.parametrize("M,K,N", [(1, 1152, 640), (40, 300, 200), (500, 700, 1200)])
def test_linear_residual_in_place(M, K, N):
    check_linear(M, K, N, BF16, S.EPI_NONE, inplace=True, pre=False, seed=9)


@pytest.mark.parametrize("M,K,N,dtype", [(4096, 1152, 4608, BF16), (2500, 4608, 1160, F16), (5000, 72, 9216, BF16),
                                         (20000, 128, 264, BF16)])
def test_linear_many_tiles(M, K, N, dtype):
    check_linear(M, K, N, dtype, S.EPI_SILU, seed=3)


def test_linear_strides_and_column_views():
    """Operands and output as column slices of wider arrays."""
    g = gen(1)
    wide = rows(g, 100, 512, BF16)
    X, W = wide[:, 64:64 + 128], rows(g, 48, 128, BF16, 0.1, ld=200)
    buf = torch.full((100, 256), 77.0, dtype=BF16, device="cuda")
    S.svdq_linear16(X, W, buf[:, 96:144])
    ref = X.double() @ W.double().T
    e = 128 * 2.0 ** -24 * (X.double().abs() @ W.double().abs().T)
    close(buf[:, 96:144], ref, half(BF16) * (ref.abs() + e) + e)
    assert bool((buf[:, :96] == 77).all()) and bool((buf[:, 144:] == 77).all())


@pytest.mark.parametrize("M", [1, 5, 70, 300])
def test_linear_rows_are_independent(M):
    """A row with NaN or infinities spoils its own output row only."""
    g = gen(2)
    X, W = rows(g, M, 200, BF16), rows(g, 136, 200, BF16, 0.1)
    Y0, Y1 = out(M, 136, BF16), out(M, 136, BF16)
    S.svdq_linear16(X, W, Y0)
    bad = X.clone()
    bad[M // 2, 3] = float("nan")
    if M > 1:
        bad[0, 5] = float("inf")
    S.svdq_linear16(bad, W, Y1)
    touched = torch.zeros(M, dtype=torch.bool, device="cuda")
    touched[M // 2] = True
    touched[0] |= M > 1
    assert torch.equal(Y0[~touched], Y1[~touched])
    assert bool(Y1[M // 2].isnan().all())
    if M > 1:
        assert not bool(Y1[0].isfinite().any())


def test_linear_extreme_activations():
    """Pre-activations far outside, infinite and NaN through both activations."""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 12.0, -12.0, 90.0, -90.0, 3e4, -3e4,
                      float("inf"), float("-inf"), float("nan"), -1e38], device="cuda").to(BF16)
    X = torch.zeros((16, 8), dtype=BF16, device="cuda")
    X[:, 0] = v
    W = torch.zeros((8, 8), dtype=BF16, device="cuda")
    W[0, 0] = 1.0
    for epi, at_minus_inf in ((S.EPI_GELU, float("nan")), (S.EPI_SILU, float("nan"))):
        Y = out(16, 8, BF16)
        S.svdq_linear16(X, W, Y, epilogue=epi)
        y, ref = Y[:, 0].double(), act64(v.double(), epi)
        fin = v.isfinite()
        assert bool((y[fin] - ref[fin]).abs().le(half(BF16) * ref[fin].abs() + 2.0 ** -20 * v[fin].double().abs()).all())
        assert bool(y[12].isposinf()) and bool(y[14].isnan())
        # -inf times a zero factor: no finite value can be right, and 0 is the limit
        assert bool(y[13].isnan()) or float(y[13]) == 0.0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [8, 40, 3000])
def test_linear_activation_tails(dtype, M):
    """Activations and slopes far on the negative side, where they are tiny,
    keep their relative accuracy: the products here are exact, so a value may
    be off by its rounding, by 2^-15 of itself (the Gaussian tail's form and
    its exponential's argument, up to 90, in fp32) and by what fp32 cannot hold.
    Phi is taken from erfc: 1 + erf, which ndtr computes, cancels here (at -7 it
    keeps three digits of 64 bits)."""
    Phi = lambda p: torch.special.erfc(-p * 0.5 ** 0.5) / 2
    phi = lambda p: torch.exp(-p * p / 2) / (2 * torch.pi) ** 0.5
    g = gen(M)
    v = (-14.0 * torch.rand((M, 1), generator=g, device="cuda")).to(dtype)
    X = torch.zeros((M, 8), dtype=dtype, device="cuda")
    X[:, :1] = v
    W = torch.zeros((8, 8), dtype=dtype, device="cuda")
    W[:, 0] = 1.0
    h, tiny = half(dtype), 16 * 2.0 ** -126 + (2.0 ** -25 if dtype == F16 else 0.0)
    for epi in (S.EPI_GELU, S.EPI_SILU):
        Y = out(M, 8, dtype)
        S.svdq_linear16(X, W, Y, epilogue=epi)
        ref = v.double() * Phi(v.double()) if epi == S.EPI_GELU else act64(v.double(), epi)
        assert bool(((Y.double() - ref).abs() <= (h + 2.0 ** -15) * ref.abs() + tiny).all())
        # one row's db is its dP: the slopes along 8 M columns
        P = v.reshape(1, -1).contiguous()
        db = torch.empty((M,), dtype=dtype, device="cuda")
        ws = torch.empty((S.svdq_linear16_backward_workspace(1, 8, M, epi),), dtype=torch.uint8, device="cuda")
        S.svdq_linear16_backward(torch.ones_like(P), None, None, P, None, None, db, ws, epi)
        p = P[0].double()
        ref = Phi(p) + p * phi(p) if epi == S.EPI_GELU else act_grad64(p, epi)
        # the slope's two terms cancel in part: the errors are theirs
        parts = Phi(p) + p.abs() * phi(p) if epi == S.EPI_GELU else torch.sigmoid(p) * (1 + p.abs())
        assert bool(((db.double() - ref).abs() <= h * ref.abs() + 2.0 ** -15 * parts + tiny).all())


@pytest.mark.parametrize("M", [16, 200])
def test_linear_silu_to_the_least_numbers(M):
    """SiLU and its slope where exp(-x) leaves fp32 but the result is still a
    bf16 number, down to its least ones (steps of 2^-133), and at infinity,
    where the slope is 1 and 0."""
    v = torch.linspace(-104.0, -70.0, M, device="cuda").to(BF16)
    X = torch.zeros((M, 8), dtype=BF16, device="cuda")
    X[:, 0] = v
    W = torch.zeros((8, 8), dtype=BF16, device="cuda")
    W[:, 0] = 1.0
    Y = out(M, 8, BF16)
    S.svdq_linear16(X, W, Y, epilogue=S.EPI_SILU)
    p = v.double()[:, None]
    ref = act64(p, S.EPI_SILU)
    # half a step, 2^-15 of itself for the exponential's argument, 128 roundings at fp32's least number
    bound = lambda r, parts: half(BF16) * r.abs() + 2.0 ** -15 * parts.abs() + 2.0 ** -134 + 2.0 ** -142
    assert bool(((Y.double() - ref).abs() <= bound(ref, ref)).all()) and bool((Y[p[:, 0] > -90] != 0).all())
    ends = torch.tensor([float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 200.0, -200.0, 0.0], device="cuda").to(BF16)
    P = torch.cat([v, ends])[None].contiguous()
    n = P.shape[1]
    db = torch.empty((n,), dtype=BF16, device="cuda")
    ws = torch.empty((S.svdq_linear16_backward_workspace(1, 8, n, S.EPI_SILU),), dtype=torch.uint8, device="cuda")
    S.svdq_linear16_backward(torch.ones_like(P), None, None, P, None, None, db, ws, S.EPI_SILU)
    q = torch.sigmoid(p[:, 0])
    ref = q * (1 + p[:, 0] * (1 - q))
    assert bool(((db[:M].double() - ref).abs() <= bound(ref, ref)).all())
    assert db[M:M + 2].tolist() == [1.0, 0.0] and bool(db[M + 2].isnan())
    assert db[M + 3:].tolist() == [1.0, 0.0, 1.0, 0.0, 0.5]


def check_linear_bwd(M, K, N, dtype, epi, bias=True, seed=0, want=(True, True, True)):
    g = gen(seed)
    X, W = rows(g, M, K, dtype), rows(g, N, K, dtype, K ** -0.5)
    dY, P = rows(g, M, N, dtype), rows(g, M, N, dtype, 1.5)
    dX, dW = out(M, K, dtype) if want[0] else None, out(N, K, dtype) if want[1] else None
    db = torch.full((N,), 77.0, dtype=dtype, device="cuda") if want[2] else None
    ws = torch.empty((max(S.svdq_linear16_backward_workspace(M, K, N, epi), 1),), dtype=torch.uint8, device="cuda")
    S.svdq_linear16_backward(dY, X, W, P if epi else None, dX, dW, db, ws, epi)
    S.svdq_get_op_error()
    x, w, d = X.double(), W.double(), dY.double()
    h = half(dtype)
    dp = d * act_grad64(P.double(), epi) if epi else d
    # the fp32 slope is good to 2^-20 of its largest value, 1.13; dP is then an operand of 16 bits
    e32 = 2.0 ** -20 * d.abs() if epi else torch.zeros_like(d)
    tiny = 2.0 ** -25 if dtype == F16 else 0.0
    e16 = e32 + h * (dp.abs() + e32) + tiny if epi else e32
    m = dp.abs() + e16
    if want[0]:
        ref = dp @ w
        e = e16 @ w.abs() + N * 2.0 ** -24 * (m @ w.abs())
        close(dX, ref, h * (ref.abs() + e) + e, "dX")
        assert padding_kept(dX)
    if want[1]:
        ref = dp.T @ x
        e = e16.T @ x.abs() + M * 2.0 ** -24 * (m.T @ x.abs())
        close(dW, ref, h * (ref.abs() + e) + e, "dW")
        assert padding_kept(dW)
    if want[2]:
        ref = dp.sum(0)
        e = e32.sum(0) + M * 2.0 ** -24 * m.sum(0)
        close(db, ref, h * (ref.abs() + e) + e, "db")


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17])
@pytest.mark.parametrize("K,N", [(1, 1), (7, 300), (64, 4737), (131, 33), (1153, 700), (4097, 65), (9000, 20)])
def test_linear_backward_few_rows(M, K, N):
    for dtype, epi in ((BF16, S.EPI_SILU), (F16, S.EPI_GELU), (BF16, S.EPI_NONE)):
        check_linear_bwd(M, K, N, dtype, epi, seed=M + N)


@pytest.mark.parametrize("M", [1, 8, 16])
def test_linear_backward_few_rows_replayed(M):
    """Captured and replayed on other contents, on another stream: the same bits as a plain call."""
    g = gen(M)
    K, N = 1153, 2001
    X, W, dY, P = rows(g, M, K, BF16), rows(g, N, K, BF16), rows(g, M, N, BF16), rows(g, M, N, BF16)
    dX, dW, db = out(M, K, BF16), out(N, K, BF16), torch.empty((N,), dtype=BF16, device="cuda")
    ws = torch.empty((S.svdq_linear16_backward_workspace(M, K, N, S.EPI_GELU),), dtype=torch.uint8, device="cuda")
    call = lambda: S.svdq_linear16_backward(dY, X, W, P, dX, dW, db, ws, S.EPI_GELU)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    X.copy_(rows(g, M, K, BF16))
    dY.copy_(rows(g, M, N, BF16))
    call()
    want = [t.clone() for t in (dX, dW, db)]
    for _ in range(3):
        for t in (dX, dW, db, ws):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dX, dW, db), want))


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (True, False, True),
                                  (False, True, True)])
@pytest.mark.parametrize("M", [1, 7, 16])
def test_linear_backward_few_rows_parts(M, want):
    for epi in (S.EPI_NONE, S.EPI_GELU):
        check_linear_bwd(M, 650, 1001, BF16, epi, seed=4, want=want)


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 200, 136), (2, 65, 7), (33, 72, 300), (64, 64, 64), (129, 130, 131),
                                   (333, 1153, 77), (777, 200, 1001), (1000, 1152, 320)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("epi", [S.EPI_NONE, S.EPI_GELU, S.EPI_SILU])
def test_linear_backward(M, K, N, dtype, epi):
    check_linear_bwd(M, K, N, dtype, epi, seed=M)


@pytest.mark.parametrize("M,K,N", [(5, 2712, 668), (535, 5, 469), (100, 198, 2980), (198, 5, 693), (203, 68, 2488),
                                   (65, 40, 300), (64, 40, 300)])
def test_linear_backward_forms(M, K, N):
    check_linear_bwd(M, K, N, BF16, S.EPI_SILU, seed=K)


@pytest.mark.parametrize("M,K,N,dtype", [(4096, 1152, 1160, BF16), (9000, 136, 400, F16)])
def test_linear_backward_long(M, K, N, dtype):
    check_linear_bwd(M, K, N, dtype, S.EPI_GELU, seed=8)


# Sizes for which between them every form of a product is chosen (which the CPU
# tests check): forward, dX alone, dW alone, both in one launch or in two.
FORM_SIZES = {
    0: [(20, 42, 41), (285, 967, 386), (29, 1159, 41), (17, 42, 4939), (531, 1643, 501), (261, 1205, 398), (47, 3950, 42),
        (19, 42, 9476), (539, 2300, 972), (404, 2225, 580), (313, 4357, 393), (9877, 41, 131), (2074, 194, 1046),
        (1621, 650, 2037)],
    1: [(9, 46, 41), (391, 580, 919), (294, 329, 586), (13, 42, 834), (9, 9569, 44), (541, 897, 2276), (526, 524, 2209),
        (284, 349, 4524), (129, 9585, 50), (1690, 1286, 658)],
    2: [(9, 46, 41), (877, 605, 397), (611, 342, 273), (463, 42, 44), (9, 9569, 44), (2377, 947, 531), (2340, 479, 515),
        (4581, 321, 292), (12, 131, 9510), (645, 1258, 1813)],
    3: [(9, 46, 41), (65, 45, 1094), (196, 46, 605), (482, 41, 476), (11, 4817, 41), (87, 137, 2958), (205, 65, 2198),
        (9, 9569, 44), (654, 2757, 43),
        # two launches
        (16, 64, 12288), (67, 74, 5182), (40, 1103, 8924), (60, 2692, 8797), (687, 245, 5347), (7711, 3470, 194),
        (12, 4881, 4461), (260, 333, 2913), (2199, 45, 7330), (266, 340, 3670), (12, 2449, 3359), (587, 946, 9051),
        (539, 452, 4116), (158, 513, 4380), (649, 131, 9811), (4562, 1022, 290), (9449, 461, 92), (8879, 974, 586),
        (13833, 964, 78)],
}


@pytest.mark.parametrize("gradients,M,K,N", [(w, *size) for w, sizes in FORM_SIZES.items() for size in sizes])
def test_linear_every_form(gradients, M, K, N):
    for dtype in (BF16, F16):
        if gradients == 0:
            check_linear(M, K, N, dtype, S.EPI_GELU, seed=M)
        else:
            check_linear_bwd(M, K, N, dtype, S.EPI_NONE, seed=M, want=(bool(gradients & 1), bool(gradients & 2), False))
            check_linear_bwd(M, K, N, dtype, S.EPI_GELU, seed=K, want=(bool(gradients & 1), bool(gradients & 2), True))


@pytest.mark.parametrize("M,K,N", [(16, 64, 12288), (260, 333, 2913), (587, 946, 9051)])
def test_linear_backward_two_launches_replayed(M, K, N):
    """Two products behind one another, eager, captured and replayed: the same bits."""
    assert len(S.svdq_debug_linear16_forms(M, K, N, 3)) == 2
    g = gen(M)
    X, W, dY = rows(g, M, K, F16), rows(g, N, K, F16, 0.1), rows(g, M, N, F16)
    dX, dW, db = out(M, K, F16), out(N, K, F16), torch.empty((N,), dtype=F16, device="cuda")
    ws = torch.empty((S.svdq_linear16_backward_workspace(M, K, N, S.EPI_NONE),), dtype=torch.uint8, device="cuda")
    call = lambda: S.svdq_linear16_backward(dY, X, W, None, dX, dW, db, ws)
    call()
    want = [t.clone() for t in (dX, dW, db)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for again in (graph.replay, call, graph.replay):
        for t in (dX, dW, db, ws):
            t.fill_(7)
        again()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dX, dW, db), want))
    S.svdq_get_op_error()


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("epi", [S.EPI_NONE, S.EPI_SILU])
def test_linear_backward_parts(want, epi):
    check_linear_bwd(100, 136, 72, BF16, epi, want=want)


@pytest.mark.parametrize("M,K,N,epi", [(8, 28672, 8192, S.EPI_NONE), (8, 28672, 8192, S.EPI_GELU), (4, 40000, 600, S.EPI_SILU),
                                       (1, 64, 300, S.EPI_NONE), (40, 64, 300, S.EPI_NONE)])
def test_linear_backward_of_the_bias_alone(M, K, N, epi):
    """Without X and W the call does not know K; the workspace that the query
    gives for the layer is enough."""
    g = gen(M)
    dY, P = rows(g, M, N, BF16), rows(g, M, N, BF16)
    db, want = (torch.empty((N,), dtype=BF16, device="cuda") for _ in range(2))
    ws = torch.full((S.svdq_linear16_backward_workspace(M, K, N, epi),), 255, dtype=torch.uint8, device="cuda")
    S.svdq_linear16_backward(dY, None, None, P if epi else None, None, None, db, ws, epi)
    d = dY.double() * act_grad64(P.double(), epi)
    e = (2.0 ** -20 * dY.double().abs()).sum(0) * bool(epi) + (M + 3) * 2.0 ** -24 * d.abs().sum(0)
    close(db, d.sum(0), half(BF16) * (d.sum(0).abs() + e) + e, "db")
    if M <= 8 and not epi:                              # no partial sums: none is needed
        S.svdq_linear16_backward(dY, None, None, None, None, None, want, None)
        assert torch.equal(db, want)


def test_linear_backward_of_an_empty_batch_is_zero():
    dW, db = out(24, 40, BF16), torch.full((24,), 77.0, dtype=BF16, device="cuda")
    e = lambda k: torch.empty((0, k), dtype=BF16, device="cuda")
    W = torch.ones((24, 40), dtype=BF16, device="cuda")
    S.svdq_linear16_backward(e(24), e(40), W, None, e(40), dW, db, None)
    assert bool((dW == 0).all()) and bool((db == 0).all()) and padding_kept(dW)


def test_linear_layer_with_another_weight():
    """A layer whose weight, type, bias or epilogue has been exchanged since the
    last call of as many rows: its buffers follow."""
    g = gen(12)
    layer = S.Linear16(rows(g, 48, 64, BF16, 0.1), None)
    for N, K, dtype, epi, bias in ((48, 64, BF16, S.EPI_NONE, False), (48, 64, F16, S.EPI_NONE, True), (80, 64, F16, S.EPI_GELU, True),
                                   (80, 40, F16, S.EPI_NONE, True), (48, 40, BF16, S.EPI_SILU, False), (48, 40, BF16, S.EPI_SILU, True)):
        layer.weight, layer.epilogue = rows(g, N, K, dtype, 0.1), epi
        layer.bias = torch.randn((N,), generator=g, device="cuda").to(dtype) if bias else None
        X, dY = rows(g, 20, K, dtype), rows(g, 20, N, dtype)
        Y = layer(X, save=True)
        want = torch.empty((20, N), dtype=dtype, device="cuda")
        S.svdq_linear16(X, layer.weight, want, layer.bias, epilogue=epi)
        assert torch.equal(Y, want)
        dX, dW, db = layer.backward(dY)
        assert dX.shape == X.shape and dW.shape == layer.weight.shape and dX.dtype == dW.dtype == dtype
        assert (db is not None) == bias and (db is None or (db.shape == (N,) and db.dtype == dtype))
        ref = (dY.double() * act_grad64(layer.P.double() if epi else dY.double(), epi)).T @ X.double()
        assert float((dW.double() - ref).norm() / ref.norm()) <= 2 * half(dtype)


def test_linear_gradients_against_differences():
    """Central differences of the 64-bit loss sum(Y dY) through the GPU's own
    forward pass would drown in 16-bit steps, so the differences are of the
    64-bit formula at the GPU's pre-activation."""
    g = gen(11)
    M, K, N = 40, 72, 56
    X, W = rows(g, M, K, F16), rows(g, N, K, F16, 0.1)
    b = torch.randn((N,), generator=g, device="cuda").to(F16)
    dY = rows(g, M, N, F16)
    layer = S.Linear16(W, b, S.EPI_GELU)
    layer.forward(X, save=True)
    dX, dW, db = layer.backward(dY)
    loss = lambda x, w, c: (act64(x @ w.T + c, S.EPI_GELU) * dY.double()).sum()
    x, w, c, t = X.double(), W.double(), b.double(), 1e-5
    for grad, k in ((dX, 0), (dW, 1), (db, 2)):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        at = lambda s: loss(*[v + s * t * d if i == k else v for i, v in enumerate((x, w, c))])
        num = float((at(1) - at(-1)) / (2 * t))
        # P is rounded to fp16 (slope changes by at most 0.8 2^-11 |p|), dP and the result once each
        scale = float((grad.double().abs() * d.abs()).sum())
        assert abs(float((grad.double() * d).sum()) - num) <= 4 * 2.0 ** -11 * scale


# --------------------------------------------------------------- layer norm
def norm64(X, w, b, eps, off, rpg):
    x = X.double()
    mu = x.mean(1, keepdim=True)
    d = x - mu
    rstd = ((d * d).mean(1, keepdim=True) + eps).rsqrt()
    y = d * rstd
    grp = torch.arange(X.shape[0], device="cuda") // (rpg or max(X.shape[0], 1))
    ww = (w.double()[grp] if w.dim() == 2 else w.double()[None]) + off if w is not None else torch.ones_like(x[:1])
    bb = (b.double()[grp] if b.dim() == 2 else b.double()[None]) if b is not None else torch.zeros_like(x[:1])
    return x, mu, d, rstd, y, ww, bb, grp


def check_norm(M, K, dtype, pt, groups=1, off=0.0, affine=True, offset=0.0, seed=0, eps=1e-6, inplace=False):
    g = gen(seed)
    X = rows(g, M, K, dtype)
    X += torch.tensor(offset, dtype=dtype, device="cuda")
    rpg = -(-M // groups) if groups > 1 else 0
    used = -(-M // rpg) if rpg else 1
    w = rows(g, used, K, pt, 0.3, guard=5.0) if affine else None
    b = rows(g, used, K, pt, 0.3, guard=5.0) if affine else None
    if affine and groups == 1:
        w, b = w[0], b[0]
    x, mu, d, rstd, y0, ww, bb, _ = norm64(X, w, b, eps, off, rpg)
    Y = out(M, K, dtype)
    if inplace:
        Y.copy_(X)
    mean, rs = torch.empty((M,), device="cuda"), torch.empty((M,), device="cuda")
    S.svdq_layer_norm(Y if inplace else X, Y, w, b, eps, off, rpg, mean, rs)
    u = 2.0 ** -24
    e_d = 80 * u * x.abs().mean(1, keepdim=True) + u * d.abs()
    sd = (d * d).mean(1, keepdim=True) + eps
    e_r = 0.5 * (84 * u + (e_d * e_d).mean(1, keepdim=True) / sd + 2 * (e_d * d.abs() * u).mean(1, keepdim=True) / sd
                 + 2 * 80 * u * x.abs().mean(1, keepdim=True) * 80 * u * d.abs().mean(1, keepdim=True) / sd) + 3 * u
    y = y0 * ww + bb
    e = rstd * ww.abs() * e_d * 1.001 + (y0 * ww).abs() * (e_r + 4 * u) + 2 * u * (y.abs() + bb.abs())
    h = half(dtype)
    close(Y, y, h * (y.abs() + e) + e, "Y")
    assert padding_kept(Y)
    close(mean, mu[:, 0], 81 * u * x.abs().mean(1), "mean")
    close(rs, rstd[:, 0], (rstd * (e_r + u))[:, 0], "rstd")


SHORT = [(1001, 68), (777, 119), (4099, 40), (515, 16), (2050, 128), (333, 130), (1500, 256)]
SIZES = SHORT + [(1, 1), (1, 2), (3, 7), (5, 8), (2, 63), (4, 64), (7, 255), (129, 256), (130, 257), (33, 768), (6, 1152),
         (1000, 1152), (9, 1281), (40, 2049), (20, 3073), (17, 4608), (5, 5121), (3, 8193), (2, 12288), (2, 16384)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dtype,pt", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_norm_sizes(M, K, dtype, pt):
    check_norm(M, K, dtype, pt, seed=M + K)


# the longest row of each way to hold one (threads to a row, 16-byte vectors to
# a thread), and one a little shorter
@pytest.mark.parametrize("team,vectors", [(8, 1), (16, 1), (32, 1), (32, 2), (32, 3), (32, 4), (32, 5), (128, 2), (128, 3),
                                          (128, 4), (128, 5), (256, 3), (256, 4), (256, 5), (512, 3), (512, 4), (512, 5),
                                          (512, 6), (512, 7), (512, 8)])
def test_norm_every_row_form(team, vectors):
    for dtype, pt in ((BF16, BF16), (F16, F32), (F32, F32)):
        v = 128 // torch.finfo(dtype).bits * team * vectors
        for K in (v, v - 3):
            if K <= 16384:
                check_norm(37, K, dtype, pt, 2, 1.0, seed=K)
                check_norm_bwd(37, K, dtype, pt, 2, 1.0, seed=K)
                check_norm_bwd(37, K, dtype, pt, want=(True, False, False), seed=K)


@pytest.mark.parametrize("M,K,groups", [(8, 72, 8), (10, 1152, 3), (1000, 136, 4), (7, 4608, 7), (5, 520, 2),
                                        (103, 24, 13), (1001, 60, 3), (999, 125, 2)])
@pytest.mark.parametrize("off", [0.0, 1.0])
def test_norm_groups(M, K, groups, off):
    check_norm(M, K, BF16, BF16, groups, off, seed=K)
    check_norm(M, K, F32, F32, groups, off, seed=K)


@pytest.mark.parametrize("M,K,groups", [(1500, 5130, 1), (900, 2601, 3), (700, 7562, 2), (500, 10241, 1), (310, 14001, 3),
                                        (300, 16384, 1)])
@pytest.mark.parametrize("dtype,pt", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_norm_many_long_rows(M, K, groups, dtype, pt):
    """More rows than blocks, of the lengths at which whole blocks work."""
    check_norm(M, K, dtype, pt, groups, 1.0, seed=K)
    check_norm_bwd(M, K, dtype, pt, groups, 1.0, seed=K)


@pytest.mark.parametrize("offset", [100.0, -3000.0])
@pytest.mark.parametrize("K", [64, 1153, 9000])
def test_norm_large_mean(offset, K):
    """A mean far above the spread: the variance must not cancel."""
    check_norm(12, K, F32, F32, offset=offset, affine=False)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_norm_plain_and_in_place(inplace, affine):
    check_norm(100, 1152, BF16, BF16, affine=affine, inplace=inplace)
    check_norm(9, 2500, F16, F32, affine=affine, inplace=inplace)


def test_norm_constant_and_bad_rows():
    """Constant rows give the shift exactly; NaN and infinity stay in their row."""
    X = torch.randn((6, 200), device="cuda")
    X[1] = 3.0
    X[2] = 0.0
    X[3, 7] = float("nan")
    X[4, 9] = float("inf")
    w, b = torch.randn((200,), device="cuda"), torch.randn((200,), device="cuda")
    Y, Z = torch.empty_like(X), torch.empty_like(X)
    S.svdq_layer_norm(X, Y, w, b)
    assert torch.equal(Y[1], b) and torch.equal(Y[2], b)
    assert bool(Y[3].isnan().all()) and bool(Y[4].isnan().all())
    X[3], X[4] = 1.0, 2.0
    S.svdq_layer_norm(X, Z, w, b)
    assert torch.equal(Y[[0, 1, 2, 5]], Z[[0, 1, 2, 5]])


@pytest.mark.parametrize("K", [64, 119, 120, 125, 200, 1000, 1153, 2601, 4608, 5121, 8191, 14001])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_of_constant_rows(K, dtype):
    """Rows of one value each, whose sums are exact in fp32 (at most 11 bits
    times K, 22 to 24 bits): the mean is the value itself and the output the
    shift, at any length."""
    bits = 11 if K <= 8192 else 8
    v = torch.tensor([3.0, 100.0, 1000.0, -7.3125, 0.1015625, 255.0, 1e4, 2.0 ** -20, 0.0, -1.0, 1.0], device="cuda")
    m, e = torch.frexp(v)
    v = torch.ldexp((m * 2 ** bits).round(), e - bits).to(dtype)
    X = out(len(v), K, dtype)
    X.copy_(v[:, None].expand(-1, K))
    w, b = torch.randn((K,), device="cuda"), torch.randn((K,), device="cuda")
    Y, mean, rs = out(len(v), K, dtype), torch.empty((len(v),), device="cuda"), torch.empty((len(v),), device="cuda")
    S.svdq_layer_norm(X, Y, w, b, 1e-6, mean=mean, rstd=rs)
    assert torch.equal(mean, v.float())
    assert torch.equal(Y, b.to(dtype).expand(len(v), K))
    assert bool(((rs.double() * 1e-3 - 1).abs() <= 2.0 ** -22).all())        # 1 / sqrt(eps), of eps in fp32


def test_norm_keeps_an_infinite_mean():
    X = torch.randn((4, 256), device="cuda")[:, :250]
    X[1, 3], X[2, 5], X[3, 7] = float("inf"), float("-inf"), float("nan")
    Y, mean = torch.empty((4, 256), device="cuda")[:, :250], torch.empty((4,), device="cuda")
    S.svdq_layer_norm(X, Y, mean=mean)
    assert bool(mean[0].isfinite()) and bool(mean[1] == float("inf")) and bool(mean[2] == float("-inf"))
    assert bool(mean[3].isnan()) and bool(Y[1:].isnan().all())


def test_norm_of_no_rows():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    S.svdq_layer_norm(e, e)
    dw = torch.full((64,), 7.0, dtype=BF16, device="cuda")
    z = torch.empty((0,), device="cuda")
    S.svdq_layer_norm_backward(e, e, z, z, e, dweight=dw)
    assert bool((dw == 0).all())


def check_norm_bwd(M, K, dtype, pt, groups=1, off=0.0, affine=True, seed=0, want=(True, True, True), alias=None):
    g = gen(seed)
    X, dY = rows(g, M, K, dtype), rows(g, M, K, dtype)
    X += 0.5
    rpg = -(-M // groups) if groups > 1 else 0
    used = -(-M // rpg) if rpg else 1
    w = rows(g, used, K, pt, 0.3, guard=5.0) if affine else None
    x, mu, d, rstd, _, ww, _, grp = norm64(X, w, None, 1e-6, off, rpg)
    mean, rs = mu[:, 0].float(), rstd[:, 0].float()
    dX = out(M, K, dtype) if want[0] else None
    if alias:
        dX.copy_(X if alias == "X" else dY)
    dw, db = (out(used, K, pt) if f else None for f in want[1:])
    n = S.svdq_layer_norm_backward_workspace(M, K, rpg)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    S.svdq_layer_norm_backward(dX if alias == "dY" else dY, dX if alias == "X" else X, mean, rs, dX, w, off, rpg,
                               dw, db, ws)
    u = 2.0 ** -24
    r = rs.double()[:, None]
    h = (x - mean.double()[:, None]) * r
    dy = dY.double()
    t = dy * ww
    th = t * h
    m1, m2 = t.mean(1, keepdim=True), th.mean(1, keepdim=True)
    eps_h = half(dtype)
    if want[0]:
        ref = r * (t - m1 - h * m2)
        e = r * (4 * u * t.abs() + 84 * u * t.abs().mean(1, keepdim=True)
                 + h.abs() * 90 * u * th.abs().mean(1, keepdim=True) + 6 * u * ((h * m2).abs() + m1.abs()))
        close(dX, ref, eps_h * (ref.abs() + e) + e, "dX")
        assert padding_kept(dX)
    hp = half(pt)
    zero = torch.zeros((used, K), dtype=torch.float64, device="cuda")
    count = torch.bincount(grp, minlength=used)[:, None]
    for got, terms, name in ((dw, dy * h, "dweight"), (db, dy, "dbias")):
        if got is not None:
            ref = zero.index_add(0, grp, terms)
            e = (count + 3) * u * zero.index_add(0, grp, terms.abs())
            close(got, ref, hp * (ref.abs() + e) + e, name)
            assert padding_kept(got)


@pytest.mark.parametrize("M,K", SIZES + [(5000, 64), (3000, 1152), (1500, 4608), (700, 9216)])
@pytest.mark.parametrize("dtype,pt", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_norm_backward_sizes(M, K, dtype, pt):
    check_norm_bwd(M, K, dtype, pt, seed=M + K)


@pytest.mark.parametrize("M,K,groups", [(8, 72, 8), (10, 1152, 3), (1000, 136, 4), (7, 4608, 7), (2000, 520, 2),
                                        (1100, 1153, 5), (103, 24, 13), (1001, 60, 3), (999, 125, 2)])
@pytest.mark.parametrize("off", [0.0, 1.0])
def test_norm_backward_groups(M, K, groups, off):
    check_norm_bwd(M, K, BF16, BF16, groups, off, seed=K)
    check_norm_bwd(M, K, F32, F32, groups, off, seed=K)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
@pytest.mark.parametrize("K", [200, 2000, 9000])
def test_norm_backward_parts(want, K):
    check_norm_bwd(300, K, BF16, F32, want=want)


@pytest.mark.parametrize("alias", ["X", "dY"])
@pytest.mark.parametrize("K", [200, 2000, 9000])
def test_norm_backward_in_place(alias, K):
    check_norm_bwd(50, K, BF16, F32, alias=alias)


def test_norm_backward_without_weight():
    check_norm_bwd(300, 1152, BF16, BF16, affine=False, want=(True, False, False))
    # the sums do not need the weight
    check_norm_bwd(300, 1152, BF16, BF16, affine=False)


@pytest.mark.parametrize("wshape,bshape", [("shared", "group"), ("group", "shared"), ("shared", "shared"),
                                           ("row", "group"), ("group", "row"), ("shared", None), (None, "row")])
@pytest.mark.parametrize("M,K,rpg", [(300, 1152, 77), (40, 136, 1), (2000, 4608, 500), (9, 64, 9), (9, 64, 20)])
def test_norm_layer_sums_the_gradient_of_a_shared_parameter(M, K, rpg, wshape, bshape):
    """A scale or a shift that all groups share has one gradient, over all rows."""
    g = gen(M + K)
    groups = -(-M // rpg)
    shape = {"shared": (K,), "row": (1, K), "group": (groups, K)}
    w, b = (None if s is None else torch.randn(shape[s], generator=g, device="cuda") for s in (wshape, bshape))
    X, dY = rows(g, M, K, BF16), rows(g, M, K, BF16)
    layer = S.LayerNorm(w, b, weight_offset=1.0)
    layer.forward(X, rows_per_group=rpg, save=True)
    dX, dw, db = layer.backward(dY)
    u = 2.0 ** -24
    x, dy, r = X.double(), dY.double(), layer.rstd.double()[:, None]
    h = (x - layer.mean.double()[:, None]) * r
    grp = torch.arange(M, device="cuda") // rpg
    ww = 1.0 if w is None else (w.double().expand(groups, K)[grp] + 1.0)
    t = dy * ww
    th = t * h
    ref = r * (t - t.mean(1, keepdim=True) - h * th.mean(1, keepdim=True))
    e = r * (4 * u * t.abs() + 84 * u * t.abs().mean(1, keepdim=True)
             + h.abs() * 90 * u * th.abs().mean(1, keepdim=True)
             + 6 * u * ((h * th.mean(1, keepdim=True)).abs() + t.mean(1, keepdim=True).abs()))
    close(dX, ref, half(BF16) * (ref.abs() + e) + e, "dX")
    for p, got, terms in ((w, dw, dy * h), (b, db, dy)):
        if p is None:
            assert got is None
            continue
        assert got.shape == p.shape and got.dtype == p.dtype
        n = p.shape[0] if p.dim() == 2 else 1
        at = grp if n == groups else torch.zeros_like(grp)
        zero = torch.zeros((n, K), dtype=torch.float64, device="cuda")
        count = torch.bincount(at, minlength=n)[:, None]
        ref = zero.index_add(0, at, terms)
        e = (count + 3) * u * zero.index_add(0, at, terms.abs())
        close(got.reshape(n, K), ref, half(F32) * (ref.abs() + e) + e, "parameter")


def test_norm_layer_in_place_keeps_nothing():
    g = gen(3)
    X = rows(g, 50, 72, BF16)
    layer, Y = S.LayerNorm(), out(50, 72, BF16)
    layer.forward(X, out=Y)
    with pytest.raises(ValueError):
        layer.forward(X, out=X, save=True)
    assert layer.forward(X, out=X) is X and torch.equal(X, Y)
    with pytest.raises(RuntimeError):
        layer.backward(X)
    e = torch.empty((0, 72), dtype=BF16, device="cuda")
    layer.forward(e, out=e, save=True)                  # nothing is overwritten


def test_norm_layer_without_rows_has_zero_gradients():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    layer = S.LayerNorm(torch.ones((64,), device="cuda"), torch.ones((1, 64), device="cuda"))
    layer.forward(e, rows_per_group=4, save=True)
    dX, dw, db = layer.backward(e)
    assert dX.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("scale", [1e-18, 1e15])
@pytest.mark.parametrize("K", [96, 1300])
def test_norm_of_very_small_and_large_rows(scale, K):
    """eps = 0 and rows whose spread is far from 1 (its square is in fp32's
    range): nothing else on the way leaves that range."""
    g = gen(31)
    X, dY = rows(g, 20, K, F32), rows(g, 20, K, F32)
    X *= scale
    x = X.double()
    mu = x.mean(1, keepdim=True)
    rstd = ((x - mu) ** 2).mean(1, keepdim=True).rsqrt()
    Y, mean, rs = out(20, K, F32), torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    S.svdq_layer_norm(X, Y, eps=0.0, mean=mean, rstd=rs)
    ref = (x - mu) * rstd
    assert float((Y.double() - ref).abs().max()) <= 2.0 ** -15        # 80 roundings of values up to 5
    dX, dw = out(20, K, F32), torch.empty((K,), device="cuda")
    ws = torch.empty((max(S.svdq_layer_norm_backward_workspace(20, K), 1),), dtype=torch.uint8, device="cuda")
    S.svdq_layer_norm_backward(dY, X, mean, rs, dX, dweight=dw, workspace=ws)
    t, h = dY.double(), (x - mean.double()[:, None]) * rs.double()[:, None]
    refd = rs.double()[:, None] * (t - t.mean(1, keepdim=True) - h * (t * h).mean(1, keepdim=True))
    assert bool(((dX.double() - refd).abs() <= 2.0 ** -15 * rs.double()[:, None]).all())
    assert bool(((dw.double() - (t * h).sum(0)).abs() <= 2.0 ** -18 * (t * h).abs().sum(0)).all())


def test_norm_gradients_against_differences():
    g = gen(4)
    M, K, rpg = 12, 96, 5
    X, dY = rows(g, M, K, F32), rows(g, M, K, F32)
    w, b = rows(g, 3, K, F32), rows(g, 3, K, F32)
    layer = S.LayerNorm(w, b, 1e-5, 1.0)
    layer.forward(X, rows_per_group=rpg, save=True)
    dX, dw, db = layer.backward(dY)

    def loss(x, ww, bb):
        grp = torch.arange(M, device="cuda") // rpg
        d = x - x.mean(1, keepdim=True)
        y = d * ((d * d).mean(1, keepdim=True) + 1e-5).rsqrt() * (ww[grp] + 1.0) + bb[grp]
        return (y * dY.double()).sum()

    at0, t = (X.double(), w.double(), b.double()), 1e-5
    for grad, k in ((dX, 0), (dw, 1), (db, 2)):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        at = lambda s: loss(*[v + s * t * d if i == k else v for i, v in enumerate(at0)])
        num = float((at(1) - at(-1)) / (2 * t))
        scale = float((grad.double().abs() * d.abs()).sum())
        assert abs(float((grad.double() * d).sum()) - num) <= 2.0 ** -17 * scale


# --------------------------------------------------------------------- rope
def rope64(X, pos, pairs, freq, pairing, inverse):
    n = len(freq)
    axis = torch.tensor([a for a, p in enumerate(pairs) for _ in range(p)], device="cuda")
    f = torch.tensor(freq, dtype=torch.float64, device="cuda")
    rowi = torch.arange(X.shape[0], device="cuda") % pos.shape[0]
    ang = pos[rowi].double()[:, axis] * f * (-1.0 if inverse else 1.0)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x, y = X.double(), X.double().clone()
    ia, ib = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairing == S.ROPE_INTERLEAVED
              else (slice(0, n), slice(n, 2 * n)))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag = torch.zeros_like(y)
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def check_rope(T, H, D, pairs, pairing, dtype, inverse=False, far=1000, pad=0, head_pad=0, shift=0, prows=None,
               inplace=False, seed=0, freq=None):
    g = gen(seed)
    xt = H * (D + head_pad) + pad
    buf = torch.randn((T * xt + shift,), generator=g, device="cuda").to(dtype)
    view = lambda v: v[shift:].view(T, xt)[:, :H * (D + head_pad)].unflatten(1, (H, D + head_pad))[..., :D]
    X = view(buf)
    obuf = buf.clone() if inplace else torch.full_like(buf, 77.0)
    O = view(obuf)
    pos = torch.randint(-far, far, (prows or T, len(pairs)), generator=g, device="cuda", dtype=torch.int32)
    freq = freq or S.rope_frequencies(pairs)
    plan = S.svdq_rope_create(pairs, freq, pairing)
    S.svdq_rope(plan, pos, O if inplace else X, O, inverse)
    ref, mag = rope64(X, pos, pairs, freq, pairing, inverse)
    e = 2.0 ** -22 * mag
    n = 2 * len(freq)
    # the 64-bit reference's own angle is good to 2^-53 of its size
    e = e + 2.0 ** -52 * far * max(abs(f) for f in freq) * mag
    close(O, ref, half(dtype) * (ref.abs() + e) + e, "rope")
    assert torch.equal(O[..., n:], X[..., n:])
    kept = torch.ones_like(obuf, dtype=torch.bool)
    view(kept).fill_(False)
    assert torch.equal(obuf[kept], (buf if inplace else torch.full_like(buf, 77.0))[kept])


@pytest.mark.parametrize("pairing", [S.ROPE_INTERLEAVED, S.ROPE_HALVES])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,H,D,pairs", [
    (1, 1, 2, (1,)), (1, 48, 128, (8, 28, 28)), (5, 3, 8, (2, 2)), (7, 2, 72, (12, 12, 12)), (9, 5, 64, (10, 10, 8)),
    (33, 4, 38, (3, 8, 8)), (100, 9, 42, (15, 2)), (20, 2, 256, (32, 48, 48)), (3, 1, 1024, (128,)), (50, 1, 6, (1, 0, 1)),
])
def test_rope_sizes(T, H, D, pairs, pairing, dtype):
    check_rope(T, H, D, pairs, pairing, dtype, seed=T + D)
    check_rope(T, H, D, pairs, pairing, dtype, inverse=True, pad=24, seed=T)


@pytest.mark.parametrize("pairing", [S.ROPE_INTERLEAVED, S.ROPE_HALVES])
@pytest.mark.parametrize("shift,pad,head_pad", [(1, 0, 0), (2, 3, 0), (4, 4, 4), (0, 1, 0), (0, 0, 1), (3, 5, 7)])
def test_rope_any_alignment(shift, pad, head_pad, pairing):
    for dtype in (BF16, F32):
        check_rope(11, 3, 48, (8, 8, 4), pairing, dtype, shift=shift, pad=pad, head_pad=head_pad)


@pytest.mark.parametrize("pairing", [S.ROPE_INTERLEAVED, S.ROPE_HALVES])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rope_far_positions(pairing, dtype):
    check_rope(64, 3, 128, (8, 28, 28), pairing, dtype, far=2 ** 31 - 1)
    check_rope(64, 2, 16, (4, 4), pairing, dtype, far=2 ** 20, freq=[1.0, -2.5, 3e-9, 0.0, 100.0, 7.5, 1e-3, 6.0])


def exact_angles(pos, freq):
    """pos freq modulo 2 pi as fp64, [positions, pairs], from integers: 2 pi to
    400 bits by Machin's formula."""
    from fractions import Fraction
    one = 1 << 420

    def arctan_inverse(x):
        total = term = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            sign, n = -sign, n + 2
        return total

    two_pi = Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)
    return torch.tensor([[float(Fraction(f) * p % two_pi) for f in freq] for p in pos], dtype=torch.float64)


@pytest.mark.parametrize("pairing", [S.ROPE_INTERLEAVED, S.ROPE_HALVES])
def test_rope_large_frequencies_at_far_positions(pairing):
    """The angle of any position is exact modulo a turn for any frequency that
    a plan takes, not only for those up to 1."""
    freq = [1.0, -1.0, 3.7e3, -65535.9, 1048575.9, 523456.789, 1e-9, 2.0 ** 19 / 3]
    pos = [0, 1, -1, 7, 12345, -99999, 2 ** 24 + 1, 2 ** 30 + 12347, 2 ** 31 - 1, -2 ** 31]
    g = gen(71)
    X = torch.randn((len(pos), 2, 2 * len(freq)), generator=g, device="cuda")
    Y = torch.empty_like(X)
    plan = S.svdq_rope_create([len(freq)], freq, pairing)
    S.svdq_rope(plan, torch.tensor(pos, device="cuda").to(torch.int32)[:, None], X, Y)
    ang = exact_angles(pos, freq).cuda()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    n = len(freq)
    ia, ib = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairing == S.ROPE_INTERLEAVED
              else (slice(0, n), slice(n, 2 * n)))
    a, b = X[..., ia].double(), X[..., ib].double()
    mag = 2.0 ** -22 * (a.abs() + b.abs())
    close(Y[..., ia], a * c - b * s, half(F32) * mag + mag, "first")
    close(Y[..., ib], a * s + b * c, half(F32) * mag + mag, "second")


@pytest.mark.parametrize("inplace", [False, True])
def test_rope_shared_positions_and_in_place(inplace):
    check_rope(60, 6, 72, (12, 12, 12), S.ROPE_HALVES, BF16, prows=15, inplace=inplace, pad=216)
    check_rope(60, 6, 96, (12, 12, 12), S.ROPE_INTERLEAVED, BF16, prows=60, inplace=inplace, pad=288)


def test_rope_many_heads_and_tokens():
    check_rope(4608, 64, 128, (8, 28, 28), S.ROPE_INTERLEAVED, BF16, far=64)
    check_rope(2, 1000, 8, (4,), S.ROPE_HALVES, F16)
    check_rope(70000, 1, 8, (1, 1), S.ROPE_INTERLEAVED, F16)


def test_rope_of_no_tokens():
    plan = S.svdq_rope_create([2, 2], S.rope_frequencies([2, 2]))
    X = torch.empty((0, 3, 8), dtype=BF16, device="cuda")
    S.svdq_rope(plan, torch.empty((0, 2), dtype=torch.int32, device="cuda"), X, X)
    S.svdq_rope(plan, torch.zeros((4, 2), dtype=torch.int32, device="cuda"), X, torch.empty_like(X))


def test_rope_copies_what_it_does_not_turn():
    """NaN and infinity past the pairs pass through; inside a pair they stay in it."""
    X = torch.randn((4, 2, 24), device="cuda").to(BF16)
    X[:, :, 10:] = float("inf")
    X[1, 1, 12] = float("nan")
    X[2, 0, 0] = float("nan")
    for pairing, mates in ((S.ROPE_INTERLEAVED, [0, 1]), (S.ROPE_HALVES, [0, 5])):
        plan = S.svdq_rope_create([5], S.rope_frequencies([5]), pairing)
        Y = torch.empty_like(X)
        S.svdq_rope(plan, torch.arange(4, dtype=torch.int32, device="cuda")[:, None], X, Y)
        assert torch.equal(Y[..., 10:].view(torch.int16), X[..., 10:].view(torch.int16))
        bad = Y[..., :10].isnan().nonzero().tolist()
        assert bad == [[2, 0, m] for m in mates]


def test_rope_inverse_undoes_it_and_is_the_gradient():
    g = gen(6)
    X, G = torch.randn((30, 4, 40), generator=g, device="cuda"), torch.randn((30, 4, 40), generator=g, device="cuda")
    pos = torch.randint(0, 10 ** 6, (30, 2), generator=g, device="cuda", dtype=torch.int32)
    plan = S.svdq_rope_create([8, 8], S.rope_frequencies([8, 8]))
    Y, B, GX = torch.empty_like(X), torch.empty_like(X), torch.empty_like(X)
    S.svdq_rope(plan, pos, X, Y)
    S.svdq_rope(plan, pos, Y, B, inverse=True)
    assert float((B - X).abs().max()) <= 2 * 2.0 ** -21 * float(X.abs().max())
    S.svdq_rope(plan, pos, G, GX, inverse=True)       # <R x, g> = <x, R^T g>
    lhs, rhs = float((Y.double() * G.double()).sum()), float((X.double() * GX.double()).sum())
    assert abs(lhs - rhs) <= 2.0 ** -20 * float((Y.double() * G.double()).abs().sum())


# ------------------------------------------------- streams, graphs, together
def test_calls_on_a_side_stream_and_in_a_graph():
    """Captured and replayed calls on new inputs give the eager bits."""
    g = gen(21)
    M, K, N = 130, 200, 264
    X, W, dY = rows(g, M, K, BF16), rows(g, N, K, BF16, 0.1), rows(g, M, N, BF16)
    lin, norm = S.Linear16(W, torch.zeros((N,), dtype=BF16, device="cuda"), S.EPI_SILU), \
        S.LayerNorm(torch.ones((K,), device="cuda"), torch.zeros((K,), device="cuda"))
    plan = S.svdq_rope_create([2, 2], S.rope_frequencies([2, 2]))
    pos = torch.arange(M, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2)
    R = torch.empty((M, 33, 8), dtype=BF16, device="cuda")

    def step():
        n = norm(X, save=True)
        y = lin(n, save=True)
        dn, dW, db = lin.backward(dY)
        dx, dw, dbn = norm.backward(dn)
        S.svdq_rope(plan, pos, y.unflatten(1, (33, 8)), R)
        return [y, dn, dW, db, dx, dw, dbn, R]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in step():
            pass
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    X.copy_(torch.randn((M, K), generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in captured]
    eager = step()
    torch.cuda.synchronize()
    for a, b in zip(got, eager):
        assert torch.equal(a, b)
    S.svdq_get_op_error()


def test_results_repeat_bit_for_bit():
    g = gen(22)
    X, W, dY, P = rows(g, 3000, 200, F16), rows(g, 136, 200, F16, 0.1), rows(g, 3000, 136, F16), rows(g, 3000, 136, F16)
    ws = torch.empty((S.svdq_linear16_backward_workspace(3000, 200, 136, S.EPI_GELU),), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(5):
        Y, dX, dW, db = out(3000, 136, F16), out(3000, 200, F16), out(136, 200, F16), torch.empty((136,), dtype=F16, device="cuda")
        S.svdq_linear16(X, W, Y, epilogue=S.EPI_GELU)
        S.svdq_linear16_backward(dY, X, W, P, dX, dW, db, ws, S.EPI_GELU)
        now = [Y, dX, dW, db]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_calls_from_other_threads_and_streams():
    """Concurrent calls with their own buffers do not disturb one another."""
    import threading
    g = gen(23)
    jobs = [(rows(g, 70 + 40 * i, 264, BF16), rows(g, 200, 264, BF16, 0.1)) for i in range(4)]
    want = []
    for X, W in jobs:
        Y = out(X.shape[0], 200, BF16)
        S.svdq_linear16(X, W, Y)
        want.append(Y)
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    Y = out(jobs[i][0].shape[0], 200, BF16)
                    S.svdq_linear16(jobs[i][0], jobs[i][1], Y)
                torch.cuda.current_stream().synchronize()
            got[i] = Y
        except Exception as e:      # handed to the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_epilogue_past_32_bits_is_refused():
    X, W = torch.zeros((4, 64), dtype=BF16, device="cuda"), torch.zeros((8, 64), dtype=BF16, device="cuda")
    Y, db = torch.zeros((4, 8), dtype=BF16, device="cuda"), torch.zeros((8,), dtype=BF16, device="cuda")
    for epi in (1 << 32, (1 << 32) + 1, -(1 << 32)):
        with pytest.raises(S.SVDQError) as e:
            S.svdq_linear16(X, W, Y, epilogue=epi)
        assert e.value.status == 1
        with pytest.raises(S.SVDQError) as e:
            S.svdq_linear16_backward(Y, None, None, None, None, None, db, None, epi)
        assert e.value.status == 1
    with pytest.raises(OverflowError):
        S.svdq_linear16(X, W, Y, epilogue=1 << 64)


def test_offsets_past_32_bits():
    """More than 2^31 elements in an operand: the last rows are what they are
    by themselves (norm, rotation), or what 64 bits give (products)."""
    g = gen(81)
    M, K = 140000, 16384
    X = torch.randn((M, K), generator=g, device="cuda", dtype=BF16)
    Y = torch.empty_like(X)
    mean, rs = torch.empty((M,), device="cuda"), torch.empty((M,), device="cuda")
    S.svdq_layer_norm(X, Y, mean=mean, rstd=rs)
    last = torch.empty((50, K), dtype=BF16, device="cuda")
    S.svdq_layer_norm(X[-50:], last)
    assert torch.equal(Y[-50:], last)
    S.svdq_layer_norm_backward(X, X, mean, rs, Y)
    S.svdq_layer_norm_backward(X[-50:], X[-50:], mean[-50:], rs[-50:], last)
    assert torch.equal(Y[-50:], last)
    plan = S.svdq_rope_create([64], S.rope_frequencies([64]))
    heads = lambda t: t.unflatten(1, (128, 128))
    pos = torch.arange(M, dtype=torch.int32, device="cuda")[:, None]
    S.svdq_rope(plan, pos, heads(X), heads(Y))
    S.svdq_rope(plan, pos[-50:], heads(X[-50:]), heads(last))
    assert torch.equal(Y[-50:], last)
    # products: rows of X and dX, then rows of W and dW, past that limit
    h = half(BF16)
    W, dY = rows(g, 24, K, BF16, K ** -0.5), rows(g, M, 24, BF16)
    Z, dW, db = out(M, 24, BF16), out(24, K, BF16), torch.empty((24,), dtype=BF16, device="cuda")
    ws = torch.empty((S.svdq_linear16_backward_workspace(M, K, 24),), dtype=torch.uint8, device="cuda")
    S.svdq_linear16(X, W, Z)
    S.svdq_linear16_backward(dY, X, W, None, Y, dW, db, ws)
    x, w, d = X[-50:].double(), W.double(), dY[-50:].double()
    e = K * 2.0 ** -24 * (x.abs() @ w.abs().T)
    close(Z[-50:], x @ w.T, h * ((x @ w.T).abs() + e) + e, "Y")
    e = 24 * 2.0 ** -24 * (d.abs() @ w.abs())
    close(Y[-50:], d @ w, h * ((d @ w).abs() + e) + e, "dX")
    dw, mag = torch.zeros((24, K), dtype=torch.float64, device="cuda"), torch.zeros((24, K), dtype=torch.float64, device="cuda")
    for i in range(0, M, 10000):
        p, q = dY[i:i + 10000].double().T, X[i:i + 10000].double()
        dw += p @ q
        mag += p.abs() @ q.abs()
    e = M * 2.0 ** -24 * mag
    close(dW, dw, h * (dw.abs() + e) + e, "dW")
    for rows_ in (3, 20):
        A = rows(g, rows_, K, BF16)
        V = torch.empty((rows_, M), dtype=BF16, device="cuda")
        S.svdq_linear16(A, X, V)                                    # X as the weight
        e = K * 2.0 ** -24 * (A.double().abs() @ x.abs().T)
        ref = A.double() @ x.T
        close(V[:, -50:], ref, h * (ref.abs() + e) + e, "Y")
        G = torch.randn((rows_, M), generator=g, device="cuda").to(BF16)
        S.svdq_linear16_backward(G, A, X, None, None, Y, None, None)
        ref = G[:, -50:].double().T @ A.double()
        e = rows_ * 2.0 ** -24 * (G[:, -50:].double().abs().T @ A.double().abs())
        close(Y[-50:], ref, h * (ref.abs() + e) + e, "dW")
    S.svdq_get_op_error()


def test_binding_through_torchs_public_functions():
    """The calls find the device and the current stream through what stands in
    for the private functions where a torch lacks them."""
    g = gen(24)
    X, W = rows(g, 5, 64, BF16), rows(g, 48, 64, BF16)
    Y, Z = out(5, 48, BF16), out(5, 48, BF16)
    S.svdq_linear16(X, W, Y)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    S._fastcall().init((BF16, F16, F32), torch.int32, torch.cuda.current_device,
                       lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    try:
        with torch.cuda.graph(graph, stream=side):          # lands in the capture: the current stream is the one
            S.svdq_linear16(X, W, Z)
        assert bool((Z == 77).all())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)
    finally:
        S._fast = None                                      # the module's functions are set anew
        S._fastcall()


def test_status_codes_reach_python():
    X = torch.zeros((4, 64), dtype=BF16, device="cuda")
    W = torch.zeros((8, 64), dtype=BF16, device="cuda")
    Y = torch.zeros((4, 8), dtype=BF16, device="cuda")
    with pytest.raises(S.SVDQError) as e:
        S.svdq_linear16(X, W, Y, epilogue=7)
    assert e.value.status == 1
    with pytest.raises(S.SVDQError) as e:
        S.svdq_linear16(torch.zeros((4, 70), dtype=BF16, device="cuda")[:, 3:67], W, Y)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        S.svdq_linear16(X, W.to(F16), Y)
    with pytest.raises(ValueError):
        S.svdq_linear16(X, W, Y.T)
    with pytest.raises(ValueError):
        S.svdq_linear16(X, W, Y, bias=torch.zeros((7,), dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        S.svdq_layer_norm(X, X, torch.zeros((3, 64), dtype=BF16, device="cuda"), rows_per_group=1)


def test_chains_keep_their_order():
    """Operators that follow one another on a stream start early but read what
    the one before wrote; a torch kernel in between sees and changes it too."""
    g = gen(41)
    X0 = torch.randn((300, 1152), generator=g, device="cuda").to(BF16)
    W = (torch.randn((1152, 1152), generator=g, device="cuda") * 1152 ** -0.5).to(BF16)
    plan = S.svdq_rope_create([6, 6], S.rope_frequencies([6, 6]))
    pos = torch.randint(0, 99, (300, 2), generator=g, device="cuda", dtype=torch.int32)

    def chain(sync):
        X, Y = X0.clone(), torch.empty_like(X0)
        wait = torch.cuda.synchronize if sync else (lambda: None)
        for i in range(12):
            S.svdq_layer_norm(X, X)
            wait()
            S.svdq_linear16(X, W, Y, residual=X, epilogue=S.EPI_SILU)
            wait()
            X.mul_(0.5)
            wait()
            h = Y.unflatten(1, (48, 24))
            S.svdq_rope(plan, pos, h, h, inverse=bool(i % 2))
            wait()
            S.svdq_linear16(Y[:2], W, X[1:3], residual=X[1:3])
            wait()
            X.add_(Y)
            wait()
        torch.cuda.synchronize()
        return X

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)


@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("captured", [False, True])
def test_few_row_products_in_a_row(M, captured):
    """Products of few rows that follow one another with nothing in between:
    each reads the rows and the bias that the one before has just written, and
    adds in place."""
    g = gen(M)
    K = 264
    X0, W0 = rows(g, M, K, BF16), rows(g, K, K, BF16, K ** -0.5)

    def chain(sync):
        X, Y, W = X0.clone(), torch.zeros((M, K), dtype=BF16, device="cuda"), W0.clone()
        b = torch.zeros((1, K), dtype=BF16, device="cuda")
        wait = torch.cuda.synchronize if sync else (lambda: None)

        def run():
            for _ in range(6):
                S.svdq_linear16(X, W, Y, residual=Y)                      # Y += X W^T
                wait()
                S.svdq_linear16(Y, W, X, bias=b[0], residual=X, epilogue=S.EPI_SILU)
                wait()
                S.svdq_linear16(X[:1], W, b, epilogue=S.EPI_SILU)         # the next bias
                wait()
        if captured and not sync:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            graph.replay()
        else:
            run()
        torch.cuda.synchronize()
        return X, Y, b

    want = chain(True)
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


FIRST_CAPTURED = """
import sys, torch
sys.path.insert(0, {root!r})
import w4a4_quantized_gemm_smooth_b200 as S
dev = dict(device="cuda", dtype=torch.bfloat16)
X, W, dY = torch.randn((200, 128), **dev), torch.randn((264, 128), **dev), torch.randn((200, 264), **dev)
outs = lambda: [torch.empty((200, 264), **dev), torch.empty((200, 128), **dev), torch.empty((264, 128), **dev),
                torch.empty((264,), **dev), torch.empty((200, 128), **dev), torch.empty((200, 33, 8), **dev)]
mean, rstd = torch.empty((200,), device="cuda"), torch.empty((200,), device="cuda")
ws = torch.empty((S.svdq_linear16_backward_workspace(200, 128, 264),), dtype=torch.uint8, device="cuda")
pos = torch.zeros((200, 1), dtype=torch.int32, device="cuda")
def run(o):
    S.svdq_linear16(X, W, o[0])
    S.svdq_linear16_backward(dY, X, W, None, o[1], o[2], o[3], ws)
    S.svdq_layer_norm(X, o[4], mean=mean, rstd=rstd)
    S.svdq_rope(S.svdq_rope_create([2], [1.0, 0.5]), pos, o[0].unflatten(1, (33, 8)), o[5])
a, b = outs(), outs()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run(a)
graph.replay()
run(b)
torch.cuda.synchronize()
S.svdq_get_op_error()
assert all(torch.equal(x, y) for x, y in zip(a, b))
print("captured first")
"""


def test_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURED.format(root=root)], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_two_graphs_on_forked_streams():
    """A captured fork and join: two branches with their own buffers."""
    g = gen(42)
    X, W = rows(g, 260, 264, BF16), rows(g, 200, 264, BF16, 0.1)
    Y, Z, N = out(260, 200, BF16), out(260, 200, BF16), out(260, 264, BF16)
    S.svdq_linear16(X, W, Y)
    want = Y.clone()
    S.svdq_layer_norm(X, N)
    wantn = N.clone()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            S.svdq_linear16(X, W, Z)
            S.svdq_layer_norm(X, N)
        S.svdq_linear16(X, W, Y)
        cur.wait_stream(side)
        Y.add_(Z)
    for _ in range(3):
        Y.zero_(), Z.zero_(), N.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Z, want) and torch.equal(N, wantn) and torch.equal(Y, want + want)


def test_a_failed_call_leaves_no_error_behind():
    """The runtime remembers the last error until it is read: a call that
    answers with a status must not leave it to the next check of a launch.  A
    capture into which a synchronisation came takes no more launches."""
    g = gen(62)
    X, W, P = rows(g, 40, 64, BF16), rows(g, 48, 64, BF16), rows(g, 40, 48, BF16)
    Y, dX, dW, N, db = (torch.empty(s, dtype=BF16, device="cuda") for s in ((40, 48), (40, 64), (48, 64), (40, 64), (48,)))
    need = max(S.svdq_linear16_backward_workspace(m, 64, 48, S.EPI_GELU) for m in (4, 40))
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    mean, rs = torch.zeros((40,), device="cuda"), torch.ones((40,), device="cuda")
    plan, pos = S.svdq_rope_create([4], [1.0] * 4), torch.zeros((40, 1), dtype=torch.int32, device="cuda")
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line)
    rt = ctypes.CDLL(path)
    side = torch.cuda.Stream()
    calls = [
        lambda st: S.svdq_linear16(X, W, Y, stream=st),
        lambda st: S.svdq_linear16(X[:4], W, Y[:4], stream=st),
        lambda st: S.svdq_linear16_backward(P, X, W, P, dX, dW, db, ws, S.EPI_GELU, stream=st),
        lambda st: S.svdq_linear16_backward(P[:4], X[:4], W, P[:4], dX[:4], dW, db, ws, S.EPI_GELU, stream=st),
        lambda st: S.svdq_layer_norm(X, N, stream=st),
        lambda st: S.svdq_layer_norm_backward(X, X, mean, rs, N, stream=st),
        lambda st: S.svdq_rope(plan, pos, X.unflatten(1, (4, 16)), N.unflatten(1, (4, 16)), stream=st),
    ]
    for call in calls:
        call(None)
    torch.cuda.synchronize()
    assert rt.cudaPeekAtLastError() == 0
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(handle, 2) == 0            # relaxed
    try:
        with pytest.raises(S.SVDQError) as e:
            S.svdq_get_op_error(side)                           # synchronises
        left = [("svdq_get_op_error", e.value.status, rt.cudaPeekAtLastError())]
        for i, call in enumerate(calls):
            with pytest.raises(S.SVDQError) as e:
                call(side)
            left.append((i, e.value.status, rt.cudaPeekAtLastError()))
    finally:
        rt.cudaStreamEndCapture(handle, ctypes.byref(graph))
        rt.cudaGetLastError()
    assert [(s, p) for _, s, p in left] == [(6, 0)] * len(left), left
    S.svdq_linear16(X, W, Y)
    ref = X.double() @ W.double().T
    err = 65 * 2.0 ** -24 * (X.double().abs() @ W.double().abs().T)
    close(Y, ref, half(BF16) * (ref.abs() + err) + err)
    S.svdq_get_op_error()


def test_slices_of_one_buffer_are_no_overlap():
    """Inputs and outputs that interleave in one buffer are taken, and give
    what separate arrays give; an output over an input is refused."""
    g = gen(61)
    M, K, N = 70, 64, 48
    W = rows(g, N, K, BF16, 0.1)
    buf = torch.full((M, 512), 77.0, dtype=BF16, device="cuda")
    X, Y, P, R, dY, dX, Nm = buf[:, :64], buf[:, 64:112], buf[:, 112:160], buf[:, 160:208], buf[:, 208:256], \
        buf[:, 256:320], buf[:, 320:384]
    for t in (X, R, dY):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    y, p, dx, nm = (torch.empty((M, n), dtype=BF16, device="cuda") for n in (N, N, K, K))
    S.svdq_linear16(X, W, Y, residual=R, epilogue=S.EPI_GELU, preact=P)
    S.svdq_linear16(X.contiguous(), W, y, residual=R.contiguous(), epilogue=S.EPI_GELU, preact=p)
    ws = torch.empty((S.svdq_linear16_backward_workspace(M, K, N, S.EPI_GELU),), dtype=torch.uint8, device="cuda")
    S.svdq_linear16_backward(dY, X, W, P, dX, None, None, ws, S.EPI_GELU)
    S.svdq_linear16_backward(dY.contiguous(), X, W, p, dx, None, None, ws, S.EPI_GELU)
    S.svdq_layer_norm(X, Nm)
    S.svdq_layer_norm(X.contiguous(), nm)
    plan = S.svdq_rope_create([4], S.rope_frequencies([4]))
    pos = torch.arange(M, dtype=torch.int32, device="cuda")[:, None]
    qk = torch.empty((M, 4, 16), dtype=BF16, device="cuda")
    S.svdq_rope(plan, pos, X.unflatten(1, (4, 16)), buf[:, 384:448].unflatten(1, (4, 16)))
    S.svdq_rope(plan, pos, X.unflatten(1, (4, 16)).contiguous(), qk)
    # the input's heads are shared (a stride of 0), its rows interleave with the output's
    S.svdq_rope(plan, pos, buf[:, None, :16].expand(M, 4, 16), buf[:, 448:512].unflatten(1, (4, 16)))
    assert torch.equal(Y, y) and torch.equal(P, p) and torch.equal(dX, dx) and torch.equal(Nm, nm)
    assert torch.equal(buf[:, 384:448], qk.flatten(1)) and torch.equal(buf[:, 448:512].unflatten(1, (4, 16))[:, 3], qk[:, 0])
    for call in (lambda: S.svdq_linear16(X, W, buf[:, 32:80]), lambda: S.svdq_linear16(X, W, X[:, :N]),
                 lambda: S.svdq_layer_norm(X, buf[:, 56:120]), lambda: S.svdq_layer_norm(X[1:], X[:-1]),
                 lambda: S.svdq_linear16(W, W, W[:, :48])):
        with pytest.raises(S.SVDQError) as e:
            call()
        assert e.value.status == 1


# ------------------------------------------- the paths of the quantised layers
def _packed(K, N, rank, seed):
    import synth
    L = synth.make_layer(synth.layer_spec(f"ops16_{K}_{N}", 64, K, N, rank, seed, tiny=True))
    return S.svdq_pack_weights(L.W, S.svdq_calib_absmax(L.X), rank, bias_bits=L.b)


def test_qkv_path():
    """Modulated norm, W4A4 QKV product, rotation of its queries and keys:
    the same bits as the calls one by one; the values are not touched."""
    g = gen(51)
    M, K, heads, kv, D = 150, 256, 4, 2, 32
    w = _packed(K, (heads + 2 * kv) * D, 16, 7)
    scale, shift = (rows(g, 3, K, BF16, 0.3) for _ in range(2))
    X = rows(g, M, K, BF16)
    pos = torch.randint(0, 60, (50, 3), generator=g, device="cuda", dtype=torch.int32)
    plan = S.svdq_rope_create([4, 6, 6], S.rope_frequencies([4, 6, 6]))
    path = S.SVDQQKV(w, heads, D, plan, S.LayerNorm(scale, shift, weight_offset=1.0), kv_heads=kv)
    Y = path.forward(X, pos, rows_per_group=50).clone()
    N = torch.empty((M, K), dtype=BF16, device="cuda")
    S.svdq_layer_norm(X, N, scale, shift, weight_offset=1.0, rows_per_group=50)
    P = S.SVDQLinear(w)(N)
    qk = P[:, :(heads + kv) * D].unflatten(1, (-1, D))
    R = torch.empty_like(qk)
    S.svdq_rope(plan, pos, qk, R)
    torch.cuda.synchronize()
    S.svdq_get_device_error(w)
    assert torch.equal(Y[:, :(heads + kv) * D], R.flatten(1))
    assert torch.equal(Y[:, (heads + kv) * D:], P[:, (heads + kv) * D:])
    with pytest.raises(ValueError):
        S.SVDQQKV(w, heads, D + 8, plan)
    w.free()


@pytest.mark.parametrize("fused", [False, True])
def test_mlp_path_with_norm(fused):
    g = gen(52)
    fc1, fc2 = _packed(256, 512, 16, 8), _packed(512, 256, 16, 9)
    X = rows(g, 100, 256, BF16)
    norm = S.LayerNorm(torch.rand((256,), generator=g, device="cuda") + 0.5)
    Y = S.SVDQMLP(fc1, fc2, norm).forward(X, fused=fused).clone()
    N = torch.empty((100, 256), dtype=BF16, device="cuda")
    S.svdq_layer_norm(X, N, norm.weight)
    Z = S.SVDQMLP(fc1, fc2).forward(N, fused=fused)
    torch.cuda.synchronize()
    assert torch.equal(Y, Z)
    fc1.free()
    fc2.free()


def test_a_block_of_them_eager_and_captured():
    """norm, QKV and rotation, a 16-bit projection of the values added to the
    residual stream, norm, MLP: each step against the 64-bit form of its own
    input, then the whole as a graph, bit for bit."""
    g = gen(53)
    M, C, heads, D = 200, 256, 8, 32
    qkv, fc1, fc2 = _packed(C, 3 * C, 16, 1), _packed(C, 512, 16, 2), _packed(512, C, 16, 3)
    plan = S.svdq_rope_create([4, 12], S.rope_frequencies([4, 12]), S.ROPE_HALVES)
    pos = torch.randint(0, 64, (M, 2), generator=g, device="cuda", dtype=torch.int32)
    X = rows(g, M, C, BF16)
    Wo, bo = rows(g, C, C, BF16, C ** -0.5), torch.randn((C,), generator=g, device="cuda").to(BF16)
    attn = S.SVDQQKV(qkv, heads, D, plan, S.LayerNorm())
    proj, mlp = S.Linear16(Wo, bo), S.SVDQMLP(fc1, fc2, S.LayerNorm())
    H, Yo = torch.empty_like(X.contiguous()), torch.empty((M, C), dtype=BF16, device="cuda")

    def block():
        Q = attn(X, pos)
        proj(Q[:, 2 * C:], residual=X, out=H)
        return Q, mlp(H, out=Yo)

    Q, Y = (t.clone() for t in block())
    h = half(BF16)
    # the normed input and the product's rows before the rotation
    N = torch.empty((M, C), dtype=BF16, device="cuda")
    S.svdq_layer_norm(X, N)
    x, _, _, _, y0, _, _, _ = norm64(X, None, None, 1e-6, 0.0, 0)
    close(N, y0, (h + 2.0 ** -14) * (y0.abs() + 2.0 ** -14), "norm")
    P = S.SVDQLinear(qkv)(N)
    ref, mag = rope64(P[:, :2 * C].unflatten(1, (2 * heads, D)), pos, [4, 12], S.rope_frequencies([4, 12]),
                      S.ROPE_HALVES, False)
    close(Q[:, :2 * C].unflatten(1, (2 * heads, D)), ref, h * (ref.abs() + 2.0 ** -21 * mag) + 2.0 ** -21 * mag, "rope")
    v, wo = P[:, 2 * C:].double(), Wo.double()
    ref = v @ wo.T + bo.double() + X.double()
    e = (C + 2) * 2.0 ** -24 * (v.abs() @ wo.abs().T + bo.double().abs() + X.double().abs())
    close(H, ref, h * (ref.abs() + e) + e, "projection")
    N2 = torch.empty((M, C), dtype=BF16, device="cuda")
    S.svdq_layer_norm(H, N2)
    assert torch.equal(Y, S.SVDQMLP(fc1, fc2)(N2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        Qc, Yc = block()
    Qc.zero_(), Yc.zero_(), H.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Qc, Q) and torch.equal(Yc, Y)
    for w in (qkv, fc1, fc2):
        w.free()

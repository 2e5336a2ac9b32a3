"""The 8-bit activation path against plain 64-bit implementations of the definitions: MXFP8 quantize (bit-exact), RMS
norm with the residual's addition and its backward pass, the W4A8 product and rotary positions with several axes.

Tolerances, u = 2^-24 (fp32), v = 2^-8 (twice bf16's half unit in the last place):
  norm       s rounds once; a sum of squares of K terms runs through chains of at most 32 + 64 additions, so the mean is
             off by at most 100 u and inv_rms by half of it; three more products: 60 u of |y|, + v |y| in bf16.
  backward   c = mean(g n) is off by at most 100 u mean|g n|: dx by 120 u inv_rms (|g| + |n| mean|g n|) + 4 u |dh|;
             dweight by (chain length) u sum|dy n|, chain <= rows per workgroup + 64.
  product    1e-5 sum|a b| per element, as for the library's other products, + v |y| in bf16.
  rotation   1e-6 for sine and cosine and two roundings: 1.3e-6 (|x1| + |x2|), + v |y| in bf16.
"""
import numpy as np
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, V = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)


def rnd(*shape, seed=0, dtype=F32, wide=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g, dtype=F32)
    if wide and x.numel():
        x[..., :: 37] *= 20
    return x.to(dtype)


def pitched(t, ld):
    """A device copy of the matrix t inside rows of ld elements, the rest NaN."""
    big = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=DEV)
    big[:, : t.shape[1]] = t.to(DEV)
    return big[:, : t.shape[1]]


# ---- MXFP8 by the definition, in 64 bits ----------------------------------------------------------

def e4m3_round(q):
    """The E4M3 value nearest to q (numpy float64), ties to even, saturating."""
    mag = np.abs(q)
    with np.errstate(divide="ignore"):
        e = np.where(mag > 0, np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6)
    e = np.where(2.0 ** (e + 1) <= mag, e + 1, e)
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.sign(q) * np.minimum(np.rint(mag / step) * step, 448.0)


def mx8_ref(x):
    """(scale bytes, values of the codes) of float64 x [M, K]; finite inputs."""
    v = x.reshape(x.shape[0], -1, 32)
    amax = np.abs(v).max(2)
    e = np.frexp(amax)[1] - 1
    b = np.where(amax > 0, np.maximum(e + 127 - 8, 0), 0)
    q = v * 2.0 ** (127.0 - b)[:, :, None]
    return b.astype(np.uint8), e4m3_round(q).reshape(x.shape)


def code_values(codes):
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()


def dequantized(codes, scales):
    M, K = codes.shape
    X = 2.0 ** (scales.cpu().numpy().astype(np.float64) - 127)
    return (code_values(codes).reshape(M, -1, 32) * X[:, :, None]).reshape(M, K)


@pytest.mark.parametrize("M,K,ld,dtype", [(1, 32, 32, F32), (1, 32, 40, BF), (3, 96, 104, F32), (65, 1152, 1152, BF),
                                          (257, 2592, 2600, F32), (1000, 4608, 4608, BF), (7, 12288, 12288, F32)])
def test_quantize_bit_exact(M, K, ld, dtype):
    say("[mx8 quantize]", M, K, ld, dtype)
    x = rnd(M, K, seed=M + K, dtype=dtype)
    x[:, 0::64] *= 2.0 ** -20
    if K >= 96:
        x[0, 32:64] = 0
        x[-1, 64:96] = -0.0
        x[0, 64:96] = torch.tensor([460.0, 452.0, 448.0, 500.0, 17.0, 18.0, 19.0, -18.0] * 4)  # saturation and ties
        x[0, 64] = 256.0
    xd = pitched(x, ld)
    codes, scales = nv.nvfp4_mx8_quantize(xd)
    torch.cuda.synchronize()
    b, q = mx8_ref(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), b)
    assert np.array_equal(code_values(codes), q)
    neg = (codes.cpu().numpy() & 0x80) != 0
    assert np.array_equal(neg, np.signbit(x.double().numpy()))


@pytest.mark.parametrize("mag", [-149, -140, -127, -100, 100, 127])
def test_quantize_extreme_magnitudes(mag):
    x = torch.zeros(4, 64, dtype=torch.float64)
    x[:, ::3] = 2.0 ** mag
    x[1, ::5] = -1.5 * 2.0 ** max(mag, -148)
    x = x.float()
    codes, scales = nv.nvfp4_mx8_quantize(x.to(DEV))
    b, q = mx8_ref(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), b) and np.array_equal(code_values(codes), q)


def test_quantize_non_finite_blocks_stay_apart():
    x = rnd(5, 128, seed=3)
    clean_codes, clean_scales = nv.nvfp4_mx8_quantize(x.to(DEV))
    for i, bad in enumerate((float("inf"), float("-inf"), float("nan"))):
        x[i, 40 + i] = bad
    codes, scales = nv.nvfp4_mx8_quantize(x.to(DEV))
    s = scales.cpu().numpy()
    assert (s[:3, 1] == 255).all() and (codes.cpu()[:3, 32:64] == 0x7F).all()
    keep = np.ones((5, 4), bool)
    keep[:3, 1] = False
    assert np.array_equal(s[keep], clean_scales.cpu().numpy()[keep])
    k = torch.from_numpy(keep.repeat(32, 1))
    assert torch.equal(codes.cpu()[k], clean_codes.cpu()[k])


# ---- RMS norm -------------------------------------------------------------------------------------

def check_mx8_of(codes, scales, y64, rel):
    """codes and scales are MXFP8 of some y within rel |y64| of y64."""
    M, K = y64.shape
    v = y64.reshape(M, -1, 32)
    lo, hi = np.abs(v).max(2) * (1 - rel), np.abs(v).max(2) * (1 + rel)
    byte = lambda a: np.where(a > 0, np.maximum(np.frexp(a)[1] - 1 + 119, 0), 0)  # noqa: E731
    s = scales.cpu().numpy().astype(np.int64)
    assert ((s >= byte(lo)) & (s <= byte(hi))).all()
    X = (2.0 ** (s - 127.0))[:, :, None]
    q = dequantized(codes, scales).reshape(v.shape) / X
    t = np.minimum(np.abs(v / X), 448.0)
    half = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(t, 2.0 ** -6))) - 4), 2.0 ** -10)
    assert (np.abs(q - np.sign(v) * t) <= half * (1 + 1e-5) + rel * t + 1e-12).all()


NORM_SIZES = [(1, 32), (1, 4608), (2, 64), (3, 96), (5, 2048), (6, 2080), (9, 2592), (4, 8192), (3, 8224), (2, 32768),
              (1003, 1152), (130, 6176)]


@pytest.mark.parametrize("M,K", NORM_SIZES)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(M, K, dtype, residual):
    say("[rmsnorm]", M, K, dtype, residual)
    x, w = rnd(M, K, seed=M * K, dtype=dtype), (1 + 0.2 * rnd(K, seed=7, wide=False)).to(BF if M % 2 else F32)
    r = rnd(M, K, seed=M * K + 1, dtype=dtype) if residual else None
    out = nv.nvfp4_rmsnorm(pitched(x, K + 8), None if r is None else pitched(r, K + 16), w.to(DEV), 1e-5, mx8=True,
                           y_dtype=F32, save_inv_rms=True)
    torch.cuda.synchronize()
    s = x.double() + (r.double() if residual else 0)
    inv = 1 / (s.square().mean(1) + 1e-5).sqrt()
    y = (s * inv[:, None] * w.double()).numpy()
    assert (out.h is None) == (not residual)
    if residual:
        assert torch.equal(out.h.cpu(), (x.float() + r.float()).to(dtype))
    assert (np.abs(out.inv_rms.cpu().double().numpy() - inv.numpy()) <= 55 * U * inv.numpy()).all()
    assert (np.abs(out.y.cpu().double().numpy() - y) <= 60 * U * np.abs(y)).all()
    check_mx8_of(out.codes, out.scales, y, 60 * U)
    # the codes are the MXFP8 of the very y that is written
    c2, s2 = nv.nvfp4_mx8_quantize(out.y)
    assert torch.equal(c2, out.codes) and torch.equal(s2, out.scales)


@pytest.mark.parametrize("K", [64, 2304, 9216])
def test_rmsnorm_outputs_agree(K):
    """Every selection of outputs gives the same values; bf16 y is the rounded y; the fake-quantized y is what the
    codes stand for; no weight is a weight of ones; h in place of x or residual."""
    x, r = rnd(6, K, seed=1, dtype=BF).to(DEV), rnd(6, K, seed=2, dtype=BF).to(DEV)
    full = nv.nvfp4_rmsnorm(x, r, None, y_dtype=F32)
    assert torch.equal(nv.nvfp4_rmsnorm(x, r, torch.ones(K, device=DEV), y_dtype=F32, mx8=False).y, full.y)
    only = nv.nvfp4_rmsnorm(x, r)
    assert torch.equal(only.codes, full.codes) and torch.equal(only.scales, full.scales) and only.y is None
    assert torch.equal(nv.nvfp4_rmsnorm(x, r, y_dtype=BF, mx8=False).y, full.y.to(BF))
    for dt in (F32, BF):
        fq = nv.nvfp4_rmsnorm(x, r, mx8=False, y_dtype=dt, fake_quantize=True).y
        assert np.array_equal(fq.double().cpu().numpy(), dequantized(full.codes, full.scales))
    for k in range(2):
        a, b = x.clone(), r.clone()
        out = nv.nvfp4_rmsnorm(a, b, h=(a, b)[k], y_dtype=F32)
        assert out.h is (a, b)[k] and torch.equal(out.h, full.h) and torch.equal(out.y, full.y)
        assert torch.equal((b, a)[k], (r, x)[k])


def test_rmsnorm_zero_rows_and_tiny_and_bad_rows():
    x = rnd(7, 2304, seed=5)
    x[1] = 0
    x[3] *= 1e-25
    x[4, 100], x[5, 7] = float("nan"), float("inf")
    out = nv.nvfp4_rmsnorm(x.to(DEV), None, None, y_dtype=F32)
    y = out.y.cpu()
    assert (y[1] == 0).all() and (out.codes.cpu()[1] & 0x7F == 0).all() and (out.scales.cpu()[1] == 0).all()
    assert torch.isnan(y[4]).all() and (out.scales.cpu()[4] == 255).all()
    assert (out.scales.cpu()[5, 0] == 255) and torch.isfinite(y[[0, 1, 2, 3, 6]]).all()
    good = nv.nvfp4_rmsnorm(x[[0, 2, 3, 6]].to(DEV), None, None, y_dtype=F32)
    assert torch.equal(good.codes.cpu(), out.codes.cpu()[[0, 2, 3, 6]])


def grad_ref(dy, h, inv, w, dh):
    dy, h, w = dy.double(), h.double(), w.double()
    n = h * inv.double()[:, None]
    g = dy * w
    c = (g * n).mean(1, keepdim=True)
    dx = inv.double()[:, None] * (g - n * c) + (0 if dh is None else dh.double())
    tol = 120 * U * inv.double()[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    tol = tol + (0 if dh is None else 4 * U * dh.double().abs())
    return dx, tol, (dy * n).sum(0), (dy * n).abs().sum(0)


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (5, 2048), (6, 2080), (3, 8224), (2, 32768), (1003, 1152),
                                 (2500, 2592), (700, 5120)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("with_dh", [False, True])
def test_rmsnorm_backward(M, K, dtype, with_dh):
    say("[rmsnorm backward]", M, K, dtype, with_dh)
    h, dy = rnd(M, K, seed=M + K, dtype=dtype), rnd(M, K, seed=M + K + 1, dtype=dtype)
    dh = rnd(M, K, seed=M + K + 2, dtype=dtype) if with_dh else None
    w = (1 + 0.2 * rnd(K, seed=9, wide=False)).to(dtype)
    inv = 1 / (h.double().square().mean(1) + 1e-6).sqrt().float()
    args = (pitched(dy, K + 8), pitched(h, K + 24), inv.to(DEV), w.to(DEV), None if dh is None else pitched(dh, K + 8))
    dx, dw = nv.nvfp4_rmsnorm_backward(*args)
    torch.cuda.synchronize()
    rx, tol, rw, aw = grad_ref(dy, h, inv, w, dh)
    if dtype == BF:
        tol = tol + V * rx.abs()
    assert ((dx.cpu().double() - rx).abs() <= tol + 1e-30).all()
    assert ((dw.cpu().double() - rw).abs() <= (M / 256 + 80) * U * aw + 1e-30).all()
    dx2, dw2 = nv.nvfp4_rmsnorm_backward(*args)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    dx3, none = nv.nvfp4_rmsnorm_backward(*args, dweight=False)
    assert none is None and torch.equal(dx, dx3)
    into = args[0].contiguous().clone()  # dx in dy's place
    nv.nvfp4_rmsnorm_backward(into, *args[1:], dx=into)
    assert torch.equal(into, dx)


def test_rmsnorm_autograd_against_formula_and_differences():
    M, K = 3, 64
    x, r, w = (rnd(M, K, seed=i, wide=False).to(DEV).requires_grad_() for i in (1, 2, 3))
    w = (1 + 0.1 * w[0]).detach().requires_grad_()
    u, p = rnd(M, K, seed=4, wide=False).to(DEV), rnd(M, K, seed=5, wide=False).to(DEV)

    def loss(a, b, c):
        y, h = nv.rmsnorm(a, b, c, 1e-6)
        return (y.double() * u.double()).sum() + (h.double() * p.double()).sum()

    loss(x, r, w).backward()
    xs, rs, ws = (t.detach().double().requires_grad_() for t in (x, r, w))
    s = xs + rs
    ref = (s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * ws * u.double()).sum() + (s * p.double()).sum()
    ref.backward()
    for got, want in ((x.grad, xs.grad), (r.grad, rs.grad), (w.grad, ws.grad)):
        assert (got.double() - want).abs().max() <= 300 * U * want.abs().max()
    # central differences of the kernel's own forward: truncation e^2, rounding 60 u sum|u y| / e
    e = 1e-2
    size = float((u.double() * s).abs().sum().detach() + (p.double() * s).abs().sum().detach())
    for k, t in enumerate((x, r, w)):
        d = rnd(*t.shape, seed=10 + k, wide=False).to(DEV)
        hi, lo = ([v.detach() + (sgn * e * d if i == k else 0) for i, v in enumerate((x, r, w))] for sgn in (1, -1))
        diff = float(loss(*hi) - loss(*lo)) / (2 * e)
        assert abs(diff - float((t.grad.double() * d.double()).sum())) <= 60 * U * size / e + 10 * e * e * d.numel() ** 0.5


def test_rmsnorm_autograd_shapes_and_straight_through():
    x = rnd(2, 3, 5, 96, seed=1, dtype=BF).to(DEV).requires_grad_()
    w = torch.ones(96, device=DEV, dtype=BF, requires_grad=True)
    y, h = nv.rmsnorm(x, None, w)
    assert h is None and y.shape == x.shape
    y.float().square().sum().backward()
    g = x.grad.clone()
    x.grad = None
    yq, _ = nv.rmsnorm(x, None, w, fake_quantize=True)
    yq.backward((2 * y.float()).to(BF).detach())  # the same incoming gradient goes straight through
    assert torch.equal(x.grad, g)
    x.grad = None
    r = x.detach().clone().requires_grad_()
    _, h = nv.rmsnorm(x, r, w)
    h.sum().backward()  # y unused
    assert (x.grad == 1).all() and (r.grad == 1).all()


# ---- W4A8 product ---------------------------------------------------------------------------------

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def mx_operands(M, N, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(0, 256, (M, K), generator=g, dtype=torch.uint8)
    a[(a & 0x7F) == 0x7F] = 0x70  # no NaN codes
    sa = torch.randint(117, 137, (M, K // 32), generator=g, dtype=torch.uint8)
    b = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    sb = torch.randint(117, 137, (N, K // 32), generator=g, dtype=torch.uint8)
    return a, sa, b, sb


def mx_values(a, sa, b, sb):
    X = lambda s: torch.exp2(s.double() - 127).repeat_interleave(32, 1)  # noqa: E731
    A = a.view(torch.float8_e4m3fn).double() * X(sa)
    n = torch.stack([b & 15, b >> 4], 2).reshape(b.shape[0], -1)
    return A, E2M1[n.long()] * X(sb)


def check_product(y, A, B):
    Y, R = A @ B.t(), A.abs() @ B.abs().t()
    tol = 1e-5 * R + (V * Y.abs() if y.dtype == BF else 0)
    err = (y.cpu().double() - Y).abs()
    assert (err <= tol + 1e-30).all(), f"max err / tol {float((err / (tol + 1e-30)).max()):.3g}"


GEMM_SIZES = [(1, 1, 32), (1, 16, 64), (1, 33, 96), (1, 1152, 1152), (2, 130, 160), (3, 4608, 1152), (7, 17, 4064),
              (15, 100, 512), (16, 256, 8192), (17, 64, 128), (31, 999, 1184), (33, 520, 640), (48, 96, 2080),
              (64, 128, 384), (65, 129, 416), (100, 300, 1024), (128, 128, 128), (129, 257, 1152), (255, 511, 4096),
              (300, 1000, 96), (513, 130, 544), (777, 1001, 2080), (1024, 1152, 4608), (2049, 2304, 1152)]


@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_w4a8(M, N, K, dtype):
    say("[w4a8]", M, N, K, dtype)
    ops = mx_operands(M, N, K, seed=M + N + K)
    y = nv.nvfp4_mx_gemm_w4a8(*[t.to(DEV) for t in ops], dtype)
    torch.cuda.synchronize()
    check_product(y, *mx_values(*ops))


@pytest.mark.parametrize("M,N,K", [(1, 50, 96), (40, 70, 256), (200, 300, 1152), (600, 1003, 608)])
@pytest.mark.parametrize("dtype,ldc", [(F32, 1), (F32, 4), (BF, 1), (BF, 8)])
def test_w4a8_output_pitch_and_untouched_columns(M, N, K, dtype, ldc):
    say("[w4a8 pitch]", M, N, K, dtype, ldc)
    ops = mx_operands(M, N, K, seed=5)
    ld = (N + 9) // 8 * 8 + (1 if ldc == 1 else 0)
    big = torch.full((M + 1, ld), 7.0, dtype=dtype, device=DEV)
    y = nv.nvfp4_mx_gemm_w4a8(*[t.to(DEV) for t in ops], out=big[:M, :N])
    torch.cuda.synchronize()
    check_product(y, *mx_values(*ops))
    assert (big[:M, N:] == 7).all() and (big[M] == 7).all()


def test_w4a8_scale_blocks_and_positions():
    """One value and one scale at a time: every k meets its own weight and its own block's scales."""
    M, N, K = 3, 5, 256
    for k in (0, 15, 16, 31, 32, 63, 64, 100, 127, 128, 200, 255):
        a, sa = torch.zeros(M, K, dtype=torch.uint8), torch.full((M, K // 32), 127, dtype=torch.uint8)
        b, sb = torch.zeros(N, K // 2, dtype=torch.uint8), torch.full((N, K // 32), 127, dtype=torch.uint8)
        a[1, k] = 0x3C  # 1.5
        b[:, k // 2] = 0x5 << (4 * (k & 1))  # 3
        sa[1, k // 32], sb[3, k // 32] = 129, 126
        y = nv.nvfp4_mx_gemm_w4a8(*[t.to(DEV) for t in (a, sa, b, sb)], F32).cpu()
        want = torch.zeros(M, N)
        want[1] = 18.0
        want[1, 3] = 9.0
        assert torch.equal(y, want), k
        big = nv.nvfp4_mx_gemm_w4a8(*[t.repeat(100, 1).to(DEV) for t in (a, sa)], b.to(DEV), sb.to(DEV), F32).cpu()
        assert torch.equal(big, want.repeat(100, 1)), k


@pytest.mark.parametrize("M", [3, 40, 200, 700])
def test_w4a8_non_finite_rows_stay_apart(M):
    """A row of the norm with a NaN or an infinity gives NaN in its own outputs only."""
    N, K = 300, 1152
    x = rnd(M, K, seed=M)
    clean = nv.nvfp4_mx8_quantize(x.to(DEV))
    _, _, b, sb = (t.to(DEV) for t in mx_operands(1, N, K, seed=4))
    want = nv.nvfp4_mx_gemm_w4a8(*clean, b, sb, F32)
    x[1, 1151], x[M - 1, 5] = float("nan"), float("-inf")
    got = nv.nvfp4_mx_gemm_w4a8(*nv.nvfp4_mx8_quantize(x.to(DEV)), b, sb, F32)
    bad = torch.zeros(M, dtype=torch.bool)
    bad[1] = bad[M - 1] = True
    assert torch.isnan(got.cpu()[bad]).all() and torch.equal(got.cpu()[~bad], want.cpu()[~bad])


@pytest.mark.parametrize("M", [1, 24, 150, 600])
@pytest.mark.parametrize("sa,sb", [(10, 200), (3, 240), (246, 12), (240, 100), (60, 60)])
def test_w4a8_extreme_scales(M, sa, sb):
    """Scales far from 1 on either side: widened operands down to bf16's subnormals and up to its largest exponents."""
    N, K = 70, 160
    a, _, b, _ = mx_operands(M, N, K, seed=6)
    ops = (a, torch.full((M, K // 32), sa, dtype=torch.uint8), b, torch.full((N, K // 32), sb, dtype=torch.uint8))
    y = nv.nvfp4_mx_gemm_w4a8(*[t.to(DEV) for t in ops], F32)
    A, B = mx_values(*ops)
    Y, R = A @ B.t(), A.abs() @ B.abs().t()
    fits = R < 3e38
    err = (y.cpu().double() - Y).abs()
    assert (err <= 1e-5 * R + K * 2.0 ** -149)[fits].all()


def test_w4a8_short_rows_of_scales():
    """K below one scale word, many tiles."""
    for M, N, K in ((1, 20000, 96), (5000, 300, 32), (3000, 3000, 64), (40000, 9000, 96)):
        say("[w4a8 short K]", M, N, K)
        ops = mx_operands(M, N, K, seed=7)
        y = nv.nvfp4_mx_gemm_w4a8(*[t.to(DEV) for t in ops], F32)
        for r in (slice(0, 70), slice(M - 70 if M > 70 else 0, M)):
            check_product(y[r], *mx_values(ops[0][r], ops[1][r], *ops[2:]))


def test_w4a8_rows_past_32_bits():
    """An activation of more than 4 GiB: its last rows and its first."""
    M, N, K = 140001, 40, 32768
    g = torch.Generator(device=DEV).manual_seed(1)
    a = torch.randint(0, 120, (M, K), generator=g, device=DEV, dtype=torch.uint8)
    sa = torch.randint(120, 130, (M, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    _, _, b, sb = mx_operands(1, N, K, seed=2)
    y = nv.nvfp4_mx_gemm_w4a8(a, sa, b.to(DEV), sb.to(DEV), F32)
    for rows in (slice(0, 70), slice(65530, 65600), slice(M - 70, M)):
        check_product(y[rows], *mx_values(a[rows].cpu(), sa[rows].cpu(), b, sb))


# ---- rotary positions -----------------------------------------------------------------------------

def rope_ref(x, pos, dims, f, halves, inverse):
    out, bound = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    p = at = 0
    for a, d in enumerate(dims):
        ang = (pos[:, a, None] * f[p: p + d // 2]).double()[:, None]  # rounded to fp32 first
        c, s = ang.cos(), -ang.sin() if inverse else ang.sin()
        i = torch.arange(d // 2)
        i1, i2 = (at + i, at + i + d // 2) if halves else (at + 2 * i, at + 2 * i + 1)
        x1, x2 = x.double()[..., i1], x.double()[..., i2]
        out[..., i1], out[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
        bound[..., i1] = bound[..., i2] = 1.3e-6 * (x1.abs() + x2.abs())
        p, at = p + d // 2, at + d
    return out, bound


ROPE = [(1, 1, 8, (8,)), (1, 32, 72, (24, 24, 24)), (2, 3, 64, (64,)), (5, 7, 72, (36, 36)), (67, 5, 128, (44, 42, 42)),
        (33, 12, 128, (16, 56, 56)), (9, 2, 96, (30, 20)), (3, 1, 1024, (512, 256, 128, 100)), (130, 40, 80, (80,)),
        (17, 3, 104, (2, 0, 50)), (4, 2, 16, (0,)), (6, 140, 64, (32, 16, 16)),
        # heads in chunks, the last one shorter; many tokens of few heads; sections of one and two pairs
        (3, 57, 200, (66, 66, 66)), (2, 17, 1024, (20, 2, 1000)), (9000, 1, 40, (20, 20)), (5003, 2, 24, (4, 6, 14)),
        (2, 40007, 8, (8,)), (700, 32, 72, (24, 24, 24)), (8201, 3, 16, (2, 4, 6, 2))]


@pytest.mark.parametrize("T,H,D,dims", ROPE)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", [nv.ROPE_PAIRS, nv.ROPE_HALVES])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(T, H, D, dims, dtype, layout, inverse):
    say("[rope]", T, H, D, dims, dtype, layout, inverse)
    x = rnd(T, H, D, seed=T + H + D, dtype=dtype)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(-50, 70000, (T, len(dims)), generator=g).float() + 0.25
    f = nv.rope_inv_freq(dims, device="cpu")
    big = torch.full((T, H + 2, D + 8), 3.0, dtype=dtype)  # a view with gaps
    big[:, 1: H + 1, :D] = x
    xd = big.to(DEV)[:, 1: H + 1, :D]
    args = (pos.to(DEV), dims, f.to(DEV))
    y = nv.nvfp4_rope_axes(xd, *args, layout=layout, inverse=inverse)
    torch.cuda.synchronize()
    want, tol = rope_ref(x, pos, dims, f, layout == nv.ROPE_HALVES, inverse)
    if dtype == BF:
        tol = tol + V * want.abs()
    assert ((y.cpu().double() - want).abs() <= tol).all()
    rest = sum(dims)
    assert torch.equal(y.cpu()[..., rest:], x[..., rest:])
    # in place, and into a heads-first tensor; nothing outside is written
    whole = big.to(DEV)
    here = whole[:, 1: H + 1, :D]
    nv.nvfp4_rope_axes(here, *args, layout=layout, inverse=inverse, out=here)
    assert torch.equal(here, y)
    whole[:, 1: H + 1, :D] = 3.0
    assert (whole == 3).all()
    first = torch.empty(H, T, D, dtype=dtype, device=DEV)
    nv.nvfp4_rope_axes(xd, *args, layout=layout, inverse=inverse, out=first.transpose(0, 1))
    assert torch.equal(first.transpose(0, 1), y)


def test_rope_passes_non_finite_tails_and_keeps_them_apart():
    x = rnd(3, 2, 32, seed=1)
    x[0, 0, 30], x[1, 1, 31] = float("inf"), float("nan")
    for layout in (nv.ROPE_PAIRS, nv.ROPE_HALVES):
        y = nv.nvfp4_rope_axes(x.to(DEV), torch.ones(3, 1, device=DEV), (20,), nv.rope_inv_freq((20,)), layout=layout)
        assert torch.equal(y.cpu()[..., 20:].nan_to_num(5, 6), x[..., 20:].nan_to_num(5, 6))
        assert torch.isfinite(y[..., :20]).all()


def test_rope_strides_past_32_bits():
    big = torch.empty((1 << 32) + 4096, dtype=BF, device=DEV)
    x = big.as_strided((3, 2, 64), (1 << 31, 128, 1))
    src = rnd(3, 2, 64, seed=8, dtype=BF)
    x.copy_(src)
    pos = torch.tensor([[1.0], [2.0], [500.0]])
    for layout in (nv.ROPE_PAIRS, nv.ROPE_HALVES):
        y = nv.nvfp4_rope_axes(x, pos.to(DEV), (64,), nv.rope_inv_freq((64,)), layout=layout)
        want, tol = rope_ref(src, pos, (64,), nv.rope_inv_freq((64,), device="cpu"), layout == nv.ROPE_HALVES, False)
        assert ((y.cpu().double() - want).abs() <= tol + V * want.abs()).all()


@pytest.mark.parametrize("layout", [nv.ROPE_PAIRS, nv.ROPE_HALVES])
def test_rope_more_tokens_than_one_launch_takes(layout):
    T = (16 << 22) + 37
    x = torch.zeros(T, 1, 8, dtype=BF, device=DEV)
    pos = torch.zeros(T, 1, device=DEV)
    at = [0, 1, (16 << 22) - 1, 16 << 22, (16 << 22) + 20, T - 1]
    src, p = rnd(len(at), 1, 8, seed=2, dtype=BF), torch.tensor([[1.0], [7.0], [30.0], [11.0], [5.0], [500.0]])
    x[at], pos[at] = src.to(DEV), p.to(DEV)
    y = nv.nvfp4_rope_axes(x, pos, (8,), nv.rope_inv_freq((8,)), layout=layout)
    want, tol = rope_ref(src, p, (8,), nv.rope_inv_freq((8,), device="cpu"), layout == nv.ROPE_HALVES, False)
    assert ((y[at].cpu().double() - want).abs() <= tol + V * want.abs()).all()
    assert int((y != 0).any(2).sum()) == len(at)


@pytest.mark.parametrize("layout", [nv.ROPE_PAIRS, nv.ROPE_HALVES])
def test_rope_gradient_against_formula_and_differences(layout):
    T, H, D, dims = 5, 3, 72, (24, 20, 16)
    x = rnd(T, H, D, seed=1, wide=False).to(DEV).requires_grad_()
    pos = torch.rand(T, 3, generator=torch.Generator().manual_seed(2)).to(DEV) * 40
    f, u = nv.rope_inv_freq(dims), rnd(T, H, D, seed=3, wide=False).to(DEV)
    loss = lambda t: (nv.rope_axes(t, pos, dims, f, layout).double() * u.double()).sum()  # noqa: E731
    loss(x).backward()
    want, tol = rope_ref(u.cpu(), pos.cpu(), dims, f.cpu(), layout == nv.ROPE_HALVES, True)
    assert ((x.grad.cpu().double() - want).abs() <= tol).all()
    d = rnd(T, H, D, seed=4, wide=False).to(DEV)
    with torch.no_grad():
        diff = float(loss(x + d) - loss(x - d)) / 2  # linear in x: no truncation
        size = float((x.abs() + d.abs()).double().sum() * u.abs().max())
    assert abs(diff - float((x.grad.double() * d.double()).sum())) <= 4e-6 * size
    # a head that several outputs share: its gradient is the sum of theirs
    shared = x.detach()[:, :1].clone().requires_grad_()
    (nv.rope_axes(shared.expand(T, H, D), pos, dims, f, layout).double() * u.double()).sum().backward()
    assert ((shared.grad.cpu().double() - want.sum(1, keepdim=True)).abs() <= 4 * tol.sum(1, keepdim=True) + 1e-6).all()


# ---- streams, graphs, empty calls -----------------------------------------------------------------

def everything(x, r, w, b, sb, pos, dims, f, **kw):
    n = nv.nvfp4_rmsnorm(x, r, w, save_inv_rms=True, **kw)
    q = nv.nvfp4_mx_gemm_w4a8(n.codes, n.scales, b, sb, **kw)
    y = nv.nvfp4_rope_axes(q.view(q.shape[0], -1, 64), pos, dims, f, **kw)
    c, s = nv.nvfp4_mx8_quantize(y.view(y.shape[0], -1), **kw)
    dx, dw = nv.nvfp4_rmsnorm_backward(r, n.h, n.inv_rms, w, x, **kw)
    return n.h, n.codes, n.scales, q, y, c, s, dx, dw


def chain_inputs(M=130, K=576, N=384):
    _, _, b, sb = mx_operands(1, N, K, seed=3)
    dims = (20, 22, 22)
    return ([rnd(M, K, seed=i, dtype=BF).to(DEV) for i in (1, 2)] + [torch.ones(K, device=DEV), b.to(DEV), sb.to(DEV),
            torch.arange(3 * M, device=DEV).view(M, 3).float(), dims, nv.rope_inv_freq(dims)])


@pytest.mark.parametrize("M", [1, 130])
def test_side_stream_and_graph_replays(M):
    args = chain_inputs(M)
    want = everything(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything(*args)
    for i in range(4):
        args[0].mul_(-0.5)
        want = everything(*args)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_empty_calls():
    z = torch.empty(0, 96, device=DEV, dtype=BF)
    w = torch.ones(96, device=DEV)
    c, s = nv.nvfp4_mx8_quantize(z)
    assert c.shape == (0, 96) and s.shape == (0, 3)
    assert nv.nvfp4_rmsnorm(z, z, w, y_dtype=BF).y.shape == (0, 96)
    dx, dw = nv.nvfp4_rmsnorm_backward(z, z, torch.empty(0, device=DEV), w)
    assert dx.shape == (0, 96) and (dw == 0).all()
    _, _, b, sb = (t.to(DEV) for t in mx_operands(1, 8, 96))
    assert nv.nvfp4_mx_gemm_w4a8(c, s, b, sb).shape == (0, 8)
    one = nv.nvfp4_mx8_quantize(torch.ones(2, 96, device=DEV))
    assert nv.nvfp4_mx_gemm_w4a8(*one, b[:0], sb[:0]).shape == (2, 0)
    for shape in ((0, 3, 16), (3, 0, 16)):
        x = torch.empty(shape, device=DEV)
        assert nv.nvfp4_rope_axes(x, torch.zeros(shape[0], 1, device=DEV), (16,), nv.rope_inv_freq((16,))).shape == shape


def test_debug_checks_refuse_what_the_header_names():
    args = chain_inputs(4)
    x, r, w, b, sb, pos, dims, f = args
    bad = x.clone()
    bad[2, 5] = float("nan")
    c, s = nv.nvfp4_mx8_quantize(x)
    nan_code, nan_scale = c.clone(), s.clone()
    nan_code[1, 3], nan_scale[3, 1] = 0xFF, 0xFF
    bad_pos = pos.clone()
    bad_pos[0, 1] = float("inf")
    inv = torch.ones(4, device=DEV)
    calls = [lambda: nv.nvfp4_mx8_quantize(bad), lambda: nv.nvfp4_rmsnorm(x, bad, w),
             lambda: nv.nvfp4_rmsnorm_backward(x, r, inv, w, bad), lambda: nv.nvfp4_mx_gemm_w4a8(nan_code, s, b, sb),
             lambda: nv.nvfp4_mx_gemm_w4a8(c, nan_scale, b, sb),
             lambda: nv.nvfp4_rope_axes(x.view(4, 9, 64), bad_pos, dims, f)]
    prev = nv.nvfp4_set_debug_checks(True)
    try:
        everything(*args)
        for i, call in enumerate(calls):
            with pytest.raises(nv.NVFP4Error) as e:
                call()
            assert e.value.status == nv.Status.ERR_PRECONDITION, i
    finally:
        nv.nvfp4_set_debug_checks(prev)

"""Every kernel that the W4A8 product's launcher can choose, in both output types, against 64-bit products of all operands;
and the ends of the scales' range.

Tolerances: 1e-5 sum|a b| per element, as for the library's other products, + bf16's rounding (2^-8 |y|).  Under activation
scale bytes 0 to 2 the operands' steps of 2^-136 to 2^-134 round to bf16's 2^-133: at most that times sum|b| more."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

DEV, V, BF, F32 = "cuda", 2.0 ** -8, torch.bfloat16, torch.float32

# the launcher's tiles: rows, columns, waves along rows and columns, K groups
TILES = {"32x32": (32, 32, 1, 1, 4), "64x32": (64, 32, 2, 1, 4), "64x64 long": (64, 64, 1, 1, 4), "64x64": (64, 64, 2, 2, 2),
         "128x64 long": (128, 64, 2, 1, 2), "128x64": (128, 64, 2, 2, 1), "128x128": (128, 128, 2, 2, 1),
         "256x256": (256, 256, 2, 4, 1)}


def plan(M, N, K):
    """The launcher's rule (csrc/w4a8.hip): kernel, and how a tile's scales are loaded (16, 4 or 1 bytes)."""
    t = lambda r, c: -(-M // r) * -(-N // c)  # noqa: E731
    nk = -(-K // 128)
    if 256 * K >= 1 << 31 or (K < 128 and (M > 32 * 65535 or t(32, 16) > 1 << 22)):
        return "generic", 0
    if M <= 16 and N <= 6144:
        return "16 waves, 16 rows" if nk > 16 else "8 waves, 16 rows", 0
    if (M <= 32 and N <= 2048 and nk <= 18) or K < 128:
        return "8 waves, 32 rows", 0
    if t(32, 32) <= 300:
        tile = "32x32"
    elif t(64, 32) <= 256:
        tile = "64x32"
    elif t(64, 64) <= 256:
        tile = "64x64 long" if nk >= 48 else "64x64"
    elif t(128, 64) <= 256:
        tile = "128x64 long" if nk >= 24 else "128x64"
    else:
        tile = "128x128" if 0.29 / 256 * t(128, 128) <= -(-t(256, 256) // 256) else "256x256"
    groups = TILES[tile][4]
    run = -(-nk // groups)
    return tile, 1 if K % 128 else 16 if K % 512 == 0 and (groups == 1 or run % 4 == 0) else 4


SIZES = [(64, 1150, 2048), (60, 1152, 1152), (64, 1152, 1184), (16, 8192, 640), (60, 8190, 2048), (64, 8192, 1152),
         (61, 8187, 1184), (250, 4090, 8192), (256, 4096, 6272), (255, 4093, 6176), (256, 4096, 6656), (250, 4090, 1024),
         (256, 4096, 1152), (255, 4093, 1184), (33, 9000, 160), (500, 4090, 4096), (512, 4096, 3200), (505, 4093, 3104),
         (500, 4090, 512), (512, 4096, 1152), (505, 4093, 608), (1000, 4600, 1024), (1024, 4608, 1152), (1001, 4603, 1184),
         (2001, 8101, 512), (2048, 8192, 640), (1990, 8187, 608), (2001, 8104, 4096), (2048, 8192, 2176),
         (2001, 8101, 2080), (16, 4090, 2176), (16, 4090, 2048), (30, 2041, 2304),
         # few rows of wide weights
         (1, 12289, 1152), (16, 17000, 640), (1, 33000, 1056), (32, 28672, 512), (20, 70000, 160)]
GENERIC = [(2097200, 16, 32), (3, 5, (1 << 23) + 32)]


def test_sizes_reach_every_kernel():
    plans = {plan(*s) for s in SIZES} | {plan(*s) for s in GENERIC}
    assert plans == {(t, s) for t in TILES for s in (1, 4, 16)} | {
        ("16 waves, 16 rows", 0), ("8 waves, 16 rows", 0), ("8 waves, 32 rows", 0), ("generic", 0)}


def operands(M, N, K, seed, sa=(117, 137), sb=(117, 137)):
    g = torch.Generator(device=DEV).manual_seed(seed)
    draw = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    a = draw(0, 256, M, K)
    a[(a & 0x7F) == 0x7F] = 0x70  # no NaN codes
    return a, draw(*sa, M, K // 32), draw(0, 256, N, K // 2), draw(*sb, N, K // 32)


def values(a, sa, b, sb):
    """Both operands in 64 bits, on the GPU."""
    X = lambda s: torch.exp2(s.double() - 127).repeat_interleave(32, 1)  # noqa: E731
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
    n = torch.stack([b & 15, b >> 4], 2).reshape(b.shape[0], -1)
    return a.view(torch.float8_e4m3fn).double() * X(sa), grid[n.long()] * X(sb)


def worst(y, A, B, more=0.0):
    """The largest error over its tolerance."""
    Bt = B.t().contiguous()
    Y, R = A @ Bt, A.abs() @ Bt.abs()
    tol = 1e-5 * R + (V * Y.abs() if y.dtype == BF else 0) + more + 1e-30
    return float(((y.double() - Y).abs() / tol).nan_to_num(float("inf")).max())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_product(M, N, K, dtype):
    print("[w4a8 plan]", M, N, K, dtype, plan(M, N, K), flush=True)
    ops = operands(M, N, K, seed=M + N + K)
    ld = (N + 7) // 8 * 8 + (0 if N % 2 else 8)
    big = torch.full((M + 1, ld), 7.0, dtype=dtype, device=DEV)
    y = nv.nvfp4_mx_gemm_w4a8(*ops, out=big[:M, :N])
    assert worst(y, *values(*ops)) <= 1
    assert (big[:M, N:] == 7).all() and (big[M] == 7).all()
    assert torch.equal(nv.nvfp4_mx_gemm_w4a8(*ops, dtype), y)  # a dense result, where rows may not be 16-byte aligned


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_short_rows_under_any_scales(dtype):
    """More rows of K = 32 than the few-row kernel's grid takes.  Scales whose product alone leaves fp32, both ways."""
    M, N, K = GENERIC[0]
    print("[w4a8 plan]", M, N, K, dtype, plan(M, N, K), flush=True)
    a, sa, b, sb = operands(M, N, K, seed=1)
    sa.copy_(torch.tensor([127, 5, 245, 246, 100], dtype=torch.uint8, device=DEV)[torch.arange(M, device=DEV) % 5, None])
    sb.copy_(torch.tensor([127, 240, 3, 250], dtype=torch.uint8, device=DEV)[torch.arange(N, device=DEV) % 4, None])
    a[7::11] = 0
    a[8::11, 1:] = 0  # one small value: 2^-9
    a[8::11, 0] = 1
    y = nv.nvfp4_mx_gemm_w4a8(a, sa, b, sb, dtype)
    A, B = values(a, torch.full_like(sa, 127), b, torch.full_like(sb, 127))
    X = torch.exp2(sa.double() + sb.double().t() - 254)  # [M, N]
    Bt = B.t().contiguous()
    Y, R = (A @ Bt) * X, (A.abs() @ Bt.abs()) * X
    fits = R < 3.3e38
    tol = 1e-5 * R + (V * Y.abs() if dtype == BF else 0) + 2.0 ** -133
    assert ((y.double() - Y).abs() <= tol)[fits].all()
    over = Y.abs() > 3.5e38
    assert over.any() and (y.double() == torch.where(Y > 0, torch.inf, -torch.inf))[over].all()
    assert (y[7::11] == 0).all()


@pytest.mark.gpu
def test_one_row_of_eight_million():
    M, N, K = GENERIC[1]
    print("[w4a8 plan]", M, N, K, plan(M, N, K), flush=True)
    ops = operands(M, N, K, seed=2)
    y = nv.nvfp4_mx_gemm_w4a8(*ops, F32)
    A, B = values(*ops)
    Bt = B.t().contiguous()
    # one chain of K / 32 fp32 additions of blocks of 32
    assert ((y.double() - A @ Bt).abs() <= (K / 32 + 32) * 2.0 ** -24 * (A.abs() @ Bt.abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 150, 600])
@pytest.mark.parametrize("K", [96, 160, 1152])
@pytest.mark.parametrize("sa", [0, 1, 2, 3])
@pytest.mark.parametrize("sb", [127, 235, 250])
def test_smallest_activation_scales(M, K, sa, sb):
    N = 70
    ops = operands(M, N, K, seed=3, sa=(sa, sa + 1), sb=(sb, sb + 1))
    A, B = values(*ops)
    # a product of numbers below 2^-126 may itself be lost under fp32's least subnormal
    more = (2.0 ** -133 if sa < 3 else 0) * B.abs().sum(1) + K * 2.0 ** -149
    assert worst(nv.nvfp4_mx_gemm_w4a8(*ops, F32), A, B, more) <= 1

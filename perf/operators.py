"""Workloads of the 8-bit activation path: residual + RMS norm with MXFP8 output (and its backward pass), the product of
MXFP8 activations with MXFP4 weights, and rotary positions with several axes.

MXFP8 is E4M3 codes with one power-of-two E8M0 scale byte per 32 values; MXFP4 is packed E2M1 codes, the even element in
the low nibble, with the same scales.  ``run`` computes each operator in plain torch operations (32 bits), or, where
``own`` is true, through the package's calls.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's norm before a linear of hidden size 4608: one token, latency
        {"name": "norm_token", "op": "norm", "M": 1, "K": 4608, "dtype": "bf16", "residual": True, "train": False},
        # a long prompt or a batch of images: bandwidth
        {"name": "norm_prompt", "op": "norm", "M": 16384, "K": 8192, "dtype": "bf16", "residual": True, "train": False},
        # a training forward in fp32 of a ragged batch, hidden size no power of two
        {"name": "norm_train_odd", "op": "norm", "M": 1003, "K": 2592, "dtype": "f32", "residual": True, "train": True},
        # the norm's backward pass in an image block: 4096 tokens, hidden 1152
        {"name": "norm_back", "op": "norm_back", "M": 4096, "K": 1152, "dtype": "bf16", "residual": True},
        # one token through fc1 of the image block: latency
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 4608, "K": 1152, "out": "bf16", "quantize": False},
        # a decode batch through a large linear: the weight's bandwidth
        {"name": "gemm_few", "op": "gemm", "M": 16, "N": 8192, "K": 8192, "out": "bf16", "quantize": False},
        # the image block's fc1 on a bf16 activation: quantise, then multiply
        {"name": "linear_block", "op": "gemm", "M": 4096, "N": 4608, "K": 1152, "out": "bf16", "quantize": True},
        # ragged tokens, sizes that no tile divides, fp32 out
        {"name": "gemm_odd", "op": "gemm", "M": 777, "N": 1001, "K": 2080, "out": "f32", "quantize": False},
        # a prompt through a large linear: the matrix units' rate
        {"name": "gemm_large", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "out": "bf16", "quantize": False},
        # one token's q and k: latency
        {"name": "rope_token", "op": "rope", "T": 1, "H": 32, "D": 72, "axes": "24,24,24", "layout": "pairs",
         "inverse": False, "dtype": "bf16", "gap": 16},
        # q and k of a video: 16 frames of 32 x 20 tokens, read from the QKV linear's rows
        {"name": "rope_video", "op": "rope", "T": 10240, "H": 64, "D": 128, "axes": "44,42,42", "layout": "pairs",
         "inverse": False, "dtype": "bf16", "gap": 32},
        # the gradient of an image's q and k with a class token (4097), halves layout, 72 dims a head
        {"name": "rope_back_odd", "op": "rope", "T": 4097, "H": 32, "D": 72, "axes": "36,36", "layout": "halves",
         "inverse": True, "dtype": "bf16", "gap": 0},
    ]


def _size(rng, lo, hi, step=1):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    n = max(step, n // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "gemm", "gemm", "rope"])
    if op == "gemm":
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 256, 8192), "K": _size(rng, 256, 8192, 32),
                "out": rng.choice(["bf16", "f32"]), "quantize": rng.random() < 0.3}
    if op == "rope":
        D = rng.choice([64, 72, 80, 96, 104, 128])
        parts = rng.choice([1, 2, 3])
        first = 2 * rng.randint(2, D // (2 * parts))
        dims = {1: [first], 2: [first, D // 2 // 2 * 2], 3: [first, D // 3 // 2 * 2, D // 3 // 2 * 2]}[parts]
        return {"op": op, "T": _size(rng, 1, 10240), "H": _size(rng, 1, 64), "D": D, "axes": ",".join(map(str, dims)),
                "layout": rng.choice(["pairs", "halves"]), "inverse": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "gap": rng.choice([0, 8, 32])}
    f32 = rng.random() < 0.3
    case = {"op": op, "M": _size(rng, 1, 16384 if not f32 else 4096), "K": _size(rng, 256, 8192, 32),
            "dtype": "f32" if f32 else "bf16", "residual": rng.random() < 0.7}
    return dict(case, train=rng.random() < 0.4) if op == "norm" else case


def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a = 2 * M * K if case["quantize"] else M * K * 33 / 32
        return {"bytes": a + N * K * 17 / 32 + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": 2 * n * es + 4 * case["T"] * (case["axes"].count(",") + 1), "flops": 3 * n}
    n, r = case["M"] * case["K"], case["residual"]
    if case["op"] == "norm_back":
        return {"bytes": n * es * (3 + r) + 4 * case["M"] + case["K"] * (es + 4), "flops": 10 * n}
    y = n * es + 4 * case["M"] if case["train"] else n * 33 / 32
    return {"bytes": n * es * (1 + 2 * r) + y + case["K"] * es, "flops": 8 * n}


# ---- inputs -----------------------------------------------------------------------------------------

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activation(g, rows, cols, dtype):
    """N(0, 1) with one channel in a hundred twenty times as large."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    wide = torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 100)]
    x[:, wide] *= 20
    return x.to(dtype)


def _mx4(w):
    """MXFP4 codes and scale bytes of a weight."""
    v = w.view(w.shape[0], -1, 32)
    b = ((v.abs().amax(2).view(torch.int32) >> 23) - 2).clamp(min=0)
    q = v * ((254 - b) << 23).view(torch.float32).unsqueeze(2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    codes = (torch.bucketize(q.abs(), edges) + 8 * (q < 0)).view(w.shape).to(torch.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), b.to(torch.uint8)


def _sections(axes, layout, device):
    """(axis, first element, second element) of every rotated pair."""
    axis, first, second, at = [], [], [], 0
    for a, d in enumerate(axes):
        for i in range(d // 2):
            axis.append(a)
            first.append(at + (2 * i if layout == "pairs" else i))
            second.append(at + (2 * i + 1 if layout == "pairs" else i + d // 2))
        at += d
    return [torch.tensor(v, device=device) for v in (axis, first, second)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activation(g, M, K, torch.bfloat16)
        s["b"], s["bs"] = _mx4(0.02 * torch.randn(N, K, generator=g, device="cuda"))
        if case["quantize"]:
            s["x"] = x
        else:
            s["a"], s["as"] = _plain_mx8(x.float())
        return s
    dtype = _dt(case["dtype"])
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        axes = [int(d) for d in case["axes"].split(",")]
        rows = torch.randn(T, (H + case["gap"]) * D, generator=g, device="cuda").to(dtype)
        s["x"] = rows[:, : H * D].view(T, H, D) if case["gap"] == 0 else rows.view(T, -1, D)[:, :H]
        # the last axis runs fastest, twenty tokens wide, the one before it 32; the first takes the rest.  The first
        # token is not at the origin: a later frame, or a token that follows a prompt
        t = torch.arange(T, device="cuda") + torch.randint(1, 4096, (1,), generator=g, device="cuda")
        grid = [t] if len(axes) == 1 else [t // 20, t % 20] if len(axes) == 2 else [t // 640, t // 20 % 32, t % 20]
        s["positions"] = torch.stack(grid, 1).float().contiguous()
        s["axes"] = axes
        s["inv_freq"] = torch.cat([10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
                                   for d in axes]).float()
        s["pairs"] = _sections(axes, case["layout"], "cuda")
        return s
    M, K = case["M"], case["K"]
    s["weight"] = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(dtype)
    x = _activation(g, M, K, dtype)
    r = _activation(g, M, K, dtype) if case["residual"] else None
    if case["op"] == "norm":
        s["x"], s["r"] = x, r
    else:
        s["h"], s["dh"] = x, r
        s["inv_rms"] = torch.rsqrt(x.float().square().mean(1) + EPS)
        s["dy"] = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    return s


# ---- one pass ---------------------------------------------------------------------------------------

def _plain_mx8(y):
    """MXFP8 codes (E4M3) and scale bytes of y, fp32."""
    v = y.view(y.shape[0], -1, 32)
    b = ((v.abs().amax(2).view(torch.int32) >> 23) - 8).clamp(min=0)
    q = (v * ((254 - b) << 23).view(torch.float32).unsqueeze(2)).clamp(-448, 448)
    return q.view(y.shape).to(torch.float8_e4m3fn).view(torch.uint8), b.to(torch.uint8)


def _spread(scales):
    """2^(b - 127) of every value of a row."""
    return torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127).repeat_interleave(32, 1)


def _as_numbers(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import nvfp4_quantized_gemm_amd as nv
    case = s["case"]
    if case["op"] == "gemm":
        a, sa = nv.nvfp4_mx8_quantize(s["x"]) if case["quantize"] else (s["a"], s["as"])
        return nv.nvfp4_mx_gemm_w4a8(a, sa, s["b"], s["bs"], _dt(case["out"]))
    if case["op"] == "rope":
        layout = nv.ROPE_PAIRS if case["layout"] == "pairs" else nv.ROPE_HALVES
        return nv.nvfp4_rope_axes(s["x"], s["positions"], s["axes"], s["inv_freq"], layout=layout,
                                  inverse=case["inverse"])
    if case["op"] == "norm_back":
        return nv.nvfp4_rmsnorm_backward(s["dy"], s["h"], s["inv_rms"], s["weight"], s["dh"])
    if case["train"]:
        out = nv.nvfp4_rmsnorm(s["x"], s["r"], s["weight"], EPS, mx8=False, y_dtype=s["x"].dtype, save_inv_rms=True)
        return {"h": out.h, "y": out.y, "inv_rms": out.inv_rms}
    out = nv.nvfp4_rmsnorm(s["x"], s["r"], s["weight"], EPS)
    codes, scales = _as_numbers(out.codes, out.scales)
    return {"h": out.h, "codes": codes, "scales": scales}


def _plain(s):
    case = s["case"]
    if case["op"] == "gemm":
        a, sa = _plain_mx8(s["x"].float()) if case["quantize"] else (s["a"], s["as"])
        A = a.view(torch.float8_e4m3fn).float() * _spread(sa)
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=a.device)
        nibbles = torch.stack([s["b"] & 15, s["b"] >> 4], 2).view(s["b"].shape[0], -1)
        B = table[nibbles.int()] * _spread(s["bs"])
        return (A @ B.t()).to(_dt(case["out"]))
    if case["op"] == "rope":
        axis, first, second = s["pairs"]
        angle = s["positions"][:, axis] * s["inv_freq"]
        c, sn = angle.cos().unsqueeze(1), angle.sin().unsqueeze(1) * (-1 if case["inverse"] else 1)
        x = s["x"].float()
        out, x1, x2 = x.clone(), x[..., first], x[..., second]
        out[..., first] = x1 * c - x2 * sn
        out[..., second] = x2 * c + x1 * sn
        return out.to(s["x"].dtype)
    w = s["weight"].float()
    if case["op"] == "norm_back":
        h, dy = s["h"].float(), s["dy"].float()
        rstd = s["inv_rms"].unsqueeze(1)
        n, g = h * rstd, dy * w
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return dx.to(s["h"].dtype), (dy * n).sum(0)
    t = s["x"].float()
    if s["r"] is not None:
        t = t + s["r"].float()
    h = t.to(s["x"].dtype) if s["r"] is not None else None
    inv_rms = torch.rsqrt(t.square().mean(1) + EPS)
    y = t * inv_rms.unsqueeze(1) * w
    if case["train"]:
        return {"h": h, "y": y.to(s["x"].dtype), "inv_rms": inv_rms}
    codes, scales = _as_numbers(*_plain_mx8(y))
    return {"h": h, "codes": codes, "scales": scales}


# ---- the definitions in 64 bits ---------------------------------------------------------------------

def _exact_mx8(y):
    """(values of the E4M3 codes, scales) of y in 64 bits; rounding is to the nearest, ties to even."""
    v = y.reshape(y.shape[0], -1, 32)
    top = v.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top)[1].double() - 1, torch.full_like(top, -1000.0))
    X = torch.exp2((e - 8).clamp(min=-127))
    q = v / X.unsqueeze(2)
    step = torch.exp2((torch.frexp(q)[1].double() - 1).clamp(min=-6) - 3)
    return (torch.round(q / step) * step).clamp(-448, 448).reshape(y.shape), X


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        if case["quantize"]:
            q, X = _exact_mx8(s["x"].double())
        else:
            q, X = s["a"].view(torch.float8_e4m3fn).double(), torch.exp2(s["as"].double() - 127)
        A = q.reshape(q.shape[0], -1, 32) * X.unsqueeze(2)
        grid = torch.tensor(E2M1, device="cuda", dtype=torch.float64)
        b = torch.empty(s["b"].shape[0], 2 * s["b"].shape[1], device="cuda", dtype=torch.float64)
        for j, nib in enumerate((s["b"] % 16, s["b"] // 16)):
            b[:, j::2] = torch.where(nib >= 8, -1.0, 1.0) * grid[(nib % 8).long()]
        B = b.reshape(b.shape[0], -1, 32) * torch.exp2(s["bs"].double() - 127).unsqueeze(2)
        return A.reshape(A.shape[0], -1) @ B.reshape(B.shape[0], -1).t().contiguous()
    if case["op"] == "rope":
        out, p, at = s["x"].double().clone(), 0, 0
        for a, d in enumerate(s["axes"]):
            angle = s["positions"][:, a].double()[:, None] * s["inv_freq"][p: p + d // 2].double()
            turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, None]
            part = s["x"].double()[..., at: at + d]
            if case["layout"] == "pairs":
                z = torch.complex(part[..., 0::2].contiguous(), part[..., 1::2].contiguous()) * turn
                out[..., at: at + d] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(part[..., : d // 2].contiguous(), part[..., d // 2:].contiguous()) * turn
                out[..., at: at + d] = torch.cat([z.real, z.imag], -1)
            p, at = p + d // 2, at + d
        return out
    w = s["weight"].double()
    if case["op"] == "norm_back":
        h, dy, rstd = s["h"].double(), s["dy"].double(), s["inv_rms"].double()[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = rstd * dy * w - h * rstd ** 3 * dot / case["K"]
        return (dx if s["dh"] is None else dx + s["dh"].double()), (dy * h * rstd).sum(0)
    t = s["x"].double() + (0 if s["r"] is None else s["r"].double())
    rms = (t.square().sum(1) / case["K"] + EPS).sqrt()
    y, h = t / rms[:, None] * w, t if s["r"] is not None else None
    if case["train"]:
        return {"h": h, "y": y, "inv_rms": 1 / rms}
    codes, scales = _exact_mx8(y)
    return {"h": h, "codes": codes, "scales": scales}

"""Workloads of attention: whole prompts and images with packed sequences and grouped heads, its gradients, writing new
keys and values into a paged cache, and one new token per sequence over that cache.

Queries, keys and values are bf16 [tokens, heads, D], read where the QKV product left them.  A causal query i of n_q
attends the keys up to i + n_k - n_q of its sequence; a query that attends none gives zeros (and a log sum of -inf).
The cache is [pages, heads, page size, D] in bf16 or in MXFP8 (E4M3 codes, one E8M0 scale byte per 32 values of a head;
the last block of a head may be shorter).  ``run`` computes each operator in plain torch operations (32 bits), or, where
``own`` is true, through the package's calls.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # an image block's self-attention: 4096 tokens, hidden 1152 = 16 heads of 72
        {"name": "attn_image", "op": "attn", "nq": "4096", "nk": "", "Hq": 16, "Hkv": 16, "D": 72, "causal": False,
         "tail": 0, "train": False},
        # its cross-attention to a text of 77 tokens: little work, latency
        {"name": "attn_cross", "op": "attn", "nq": "1024", "nk": "77", "Hq": 16, "Hkv": 16, "D": 72, "causal": False,
         "tail": 0, "train": False},
        # a long prompt with grouped heads: the matrix units' rate
        {"name": "attn_prompt", "op": "attn", "nq": "8192", "nk": "", "Hq": 32, "Hkv": 8, "D": 128, "causal": True,
         "tail": 0, "train": False},
        # packed prompts of a training batch, one of them empty, with padding behind the last
        {"name": "attn_packed", "op": "attn", "nq": "1,17,1003,0,2049,777", "nk": "", "Hq": 24, "Hkv": 8, "D": 80,
         "causal": True, "tail": 5, "train": True},
        # the image block's gradients
        {"name": "back_image", "op": "back", "nq": "4096", "nk": "", "Hq": 16, "Hkv": 16, "D": 72, "causal": False,
         "tail": 0},
        # gradients of a prompt with grouped heads
        {"name": "back_prompt", "op": "back", "nq": "4096", "nk": "", "Hq": 32, "Hkv": 8, "D": 128, "causal": True,
         "tail": 0},
        # gradients of packed sequences whose keys are more than their queries (a prefix that is attended, not trained)
        {"name": "back_packed", "op": "back", "nq": "129,64,1,500", "nk": "200,64,333,1003", "Hq": 12, "Hkv": 4, "D": 64,
         "causal": True, "tail": 3},
        # a decode step's keys and values of 64 sequences into a bf16 cache: latency
        {"name": "append_token", "op": "append", "B": 64, "n": 1, "max": 4097, "Hkv": 8, "D": 128, "page": 16,
         "kind": "bf16"},
        # two prompts into an MXFP8 cache: bandwidth
        {"name": "append_prompt", "op": "append", "B": 2, "n": 8192, "max": 8192, "Hkv": 8, "D": 128, "page": 64,
         "kind": "mx8"},
        # one sequence's next token: latency
        {"name": "decode_token", "op": "decode", "B": 1, "max": 4097, "Hq": 32, "Hkv": 8, "D": 128, "page": 16,
         "kind": "bf16"},
        # a batch of sequences of all lengths over an MXFP8 cache: bandwidth
        {"name": "decode_batch", "op": "decode", "B": 64, "max": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 64,
         "kind": "mx8"},
        # two very long sequences, split over their length
        {"name": "decode_long", "op": "decode", "B": 2, "max": 131072, "Hq": 32, "Hkv": 8, "D": 128, "page": 256,
         "kind": "bf16"},
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    return max(kv, rng.choice([1, 2, 3, 4, 8]) * kv if kv * 8 <= most else most // kv * kv), kv


def draw(rng):
    op = rng.choice(["attn", "attn", "back", "append", "decode", "decode"])
    D = rng.choice([64, 72, 80, 96, 104, 128])
    if op in ("attn", "back"):
        Hq, Hkv = _heads(rng, 32)
        nq = [_size(rng, 1, 4096) for _ in range(rng.choice([1, 1, 2, 5]))]
        total = 8192 if op == "attn" else 4096
        while sum(nq) > total:
            nq = [max(1, n // 2) for n in nq]
        nk = [n if rng.random() < 0.5 else _size(rng, 1, 4096) for n in nq] if rng.random() < 0.3 else []
        while sum(nk) > total:
            nk = [max(1, n // 2) for n in nk]
        if op == "back":  # over a single key the gradients of queries and keys are 0, and their computed values rounding
            nq[0], nk[:1] = max(nq[0], 32), [max(n, 32) for n in nk[:1]]
        case = {"op": op, "nq": ",".join(map(str, nq)), "nk": ",".join(map(str, nk)), "Hq": Hq, "Hkv": Hkv, "D": D,
                "causal": rng.random() < 0.6, "tail": rng.choice([0, 0, 7])}
        if op == "attn":
            case["train"] = rng.random() < 0.4
        most = max(work(c)["flops"] for c in listed() if c["op"] == op)
        while work(case)["flops"] > most:
            case["Hq"] = case["Hkv"] = max(1, case["Hkv"] // 2)
        return case
    kind, page = rng.choice(["bf16", "mx8"]), rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        n = rng.choice([1, _size(rng, 1, 4096)])
        B = min(_size(rng, 1, 64), max(1, 16384 // n))
        return {"op": op, "B": B, "n": n, "max": n + rng.randint(0, 2000), "Hkv": rng.choice([1, 2, 4, 8]), "D": D,
                "page": page, "kind": kind}
    Hq, Hkv = _heads(rng, 32)
    B = _size(rng, 1, 64)
    return {"op": op, "B": B, "max": _size(rng, 1, min(131072, 262144 // B)), "Hq": Hq, "Hkv": min(Hkv, 8) if Hq % 8 == 0 else Hkv,
            "D": D, "page": page, "kind": kind}


def _numbers(text):
    return [int(n) for n in text.split(",") if n]


def _lengths(case):
    """Tokens of each sequence in the cache, the call's own among them: spread evenly, the first one the longest."""
    least = case.get("n", 1)
    return [max(least, int(case["max"] * (1 - b * 0.6180339887 % 1))) for b in range(case["B"])]


def _pairs(case):
    """Attended (query, key) pairs of one head."""
    nq = _numbers(case["nq"])
    nk = _numbers(case["nk"]) or nq
    if not case["causal"]:
        return sum(a * b for a, b in zip(nq, nk))
    total = 0
    for a, b in zip(nq, nk):
        seen = min(a, b)  # the last `seen` queries attend b - seen + 1 .. b keys, the others none
        total += seen * (b - seen) + seen * (seen + 1) // 2
    return total


def work(case):
    op, D = case["op"], case["D"]
    if op in ("attn", "back"):
        Tq = sum(_numbers(case["nq"]))
        Tk = sum(_numbers(case["nk"])) or Tq
        q, kv, p = Tq * case["Hq"] * D, 2 * Tk * case["Hkv"] * D, _pairs(case) * case["Hq"]
        if op == "attn":
            return {"bytes": 2 * (2 * q + kv) + (4 * Tq * case["Hq"] if case["train"] else 0), "flops": 4 * D * p}
        return {"bytes": 2 * (4 * q + 2 * kv) + 4 * Tq * case["Hq"], "flops": 10 * D * p}
    per_row = 2 * D if case["kind"] == "bf16" else D + (D + 31) // 32
    if op == "append":
        rows = 2 * case["B"] * case["n"] * case["Hkv"]
        return {"bytes": rows * (2 * D + per_row), "flops": 4 * rows * D}
    n = sum(_lengths(case))
    return {"bytes": 2 * n * case["Hkv"] * per_row + 4 * case["B"] * case["Hq"] * D, "flops": 4 * n * case["Hq"] * D}


# ---- inputs -----------------------------------------------------------------------------------------

BF = torch.bfloat16


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _offsets(n):
    return torch.tensor([0] + n, device="cuda").cumsum(0).int()


def _pages(g, case, lengths):
    """(pages of the cache, page table [B, pages a sequence]): scattered pages, -1 where a sequence has none."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    return pages, table


def _to_mx8(x):
    """MXFP8 codes (E4M3) and scale bytes of x [..., D] fp32, blocks of 32 along D, the last one maybe shorter."""
    D = x.shape[-1]
    blocks = -(-D // 32)
    v = torch.nn.functional.pad(x, (0, 32 * blocks - D)).unflatten(-1, (blocks, 32))
    b = ((v.abs().amax(-1).view(torch.int32) >> 23) - 8).clamp(min=0)
    q = (v * ((254 - b) << 23).view(torch.float32).unsqueeze(-1)).clamp(-448, 448)
    codes = q.flatten(-2)[..., :D].to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), b.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    if op in ("attn", "back"):
        nq = _numbers(case["nq"])
        nk = _numbers(case["nk"]) or nq
        Hq = case["Hq"]
        Tq, Tk = sum(nq) + case["tail"], sum(nk) + case["tail"]
        packed = len(nq) > 1 or case["tail"] > 0
        s["cu_q"] = _offsets(nq) if packed else None
        s["cu_k"] = (s["cu_q"] if nk == nq else _offsets(nk)) if packed else None
        if nk == nq:  # views of one QKV output
            rows = _randn(g, Tq, Hq + 2 * Hkv, D).to(BF)
            s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq: Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            rows = _randn(g, Tk, 2 * Hkv, D).to(BF)
            s["q"], s["k"], s["v"] = _randn(g, Tq, Hq, D).to(BF), rows[:, :Hkv], rows[:, Hkv:]
        if op == "back":
            out, lse = _attend(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], case["causal"])
            s["out"], s["lse"] = out.to(BF), lse
            s["dout"] = _randn(g, Tq, Hq, D).to(BF)
        return s
    lengths = _lengths(case)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pages, s["table"] = _pages(g, case, lengths)
    cache = [_randn(g, pages, Hkv, case["page"], D).to(BF) for _ in range(2)]
    if case["kind"] == "mx8":
        (k, ks), (v, vs) = (_to_mx8(t.float()) for t in cache)
        s["cache"] = [k, v, ks, vs]
    else:
        s["cache"] = cache + [None, None]
    if op == "decode":
        s["q"] = _randn(g, case["B"], case["Hq"], D).to(BF)
        return s
    T = case["B"] * case["n"]
    rows = _randn(g, T, 2 * Hkv, D).to(BF)
    s["k"], s["v"] = rows[:, :Hkv], rows[:, Hkv:]
    s["cu"] = _offsets([case["n"]] * case["B"]) if case["n"] > 1 else None
    return s


# ---- one pass ---------------------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import nvfp4_quantized_gemm_amd as nv
    case = s["case"]
    if case["op"] == "attn":
        out, lse = nv.nvfp4_attention(s["q"], s["k"], s["v"], causal=case["causal"], cu_q=s["cu_q"], cu_k=s["cu_k"],
                                      save_lse=case["train"])
        return {"out": out, "lse": lse} if case["train"] else out
    if case["op"] == "back":
        return nv.nvfp4_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], causal=case["causal"],
                                           cu_q=s["cu_q"], cu_k=s["cu_k"])
    cache = nv.PagedCache(*s["cache"])
    if case["op"] == "decode":
        return nv.nvfp4_paged_attention(s["q"], cache, s["table"], s["lengths"])
    nv.nvfp4_cache_append(s["k"], s["v"], cache, s["table"], s["lengths"], s["cu"])
    return _as_numbers(s["cache"])


def _as_numbers(cache):
    k, v, ks, vs = cache
    if ks is None:
        return [k, v]
    return [k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks.view(torch.float8_e8m0fnu),
            vs.view(torch.float8_e8m0fnu)]


def _attended(Tq, Tk, cu_q, cu_k, causal, device):
    """Truth values [Tq, Tk]: which keys a query attends."""
    if cu_q is None:
        cu_q, cu_k = (torch.tensor([0, T], device=device) for T in (Tq, Tk))
    i, j = torch.arange(Tq, device=device), torch.arange(Tk, device=device)
    bq = torch.searchsorted(cu_q[1:].contiguous(), i, right=True)
    bk = torch.searchsorted(cu_k[1:].contiguous(), j, right=True)
    last = len(cu_q) - 1
    mask = (bq[:, None] == bk[None, :]) & (bq < last)[:, None]
    if causal:  # counted from the ends of the sequences
        behind_q = cu_q[(bq + 1).clamp(max=last)] - i
        behind_k = cu_k[(bk + 1).clamp(max=last)] - j
        mask &= behind_k[None, :] >= behind_q[:, None]
    return mask


def _by_head(t, heads):
    """[T, H, D] -> fp32 [heads, T, D], each head as often as the queries' heads share it."""
    t = t.float().transpose(0, 1)
    return t.repeat_interleave(heads // t.shape[0], 0).contiguous()


def _attend(q, k, v, cu_q, cu_k, causal):
    """(out fp32 [Tq, Hq, D], log sums [Hq, Tq])."""
    H, D = q.shape[1:]
    mask = _attended(q.shape[0], k.shape[0], cu_q, cu_k, causal, q.device)
    Q, K, V = (_by_head(t, H) for t in (q, k, v))
    scores = torch.bmm(Q, K.transpose(1, 2).contiguous()) * D ** -0.5
    scores.masked_fill_(~mask, -math.inf)
    top = scores.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (scores - top).exp_()
    total = p.sum(2, keepdim=True)
    out = torch.bmm(p, V) / torch.where(total == 0, 1.0, total)
    return out.transpose(0, 1), (total.log() + top).squeeze(2)


def _plain(s):
    case = s["case"]
    D = case["D"]
    if case["op"] == "attn":
        out, lse = _attend(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], case["causal"])
        out = out.to(BF).contiguous()
        return {"out": out, "lse": lse} if case["train"] else out
    if case["op"] == "back":
        q, k, v, H, Hkv = s["q"], s["k"], s["v"], case["Hq"], case["Hkv"]
        mask = _attended(q.shape[0], k.shape[0], s["cu_q"], s["cu_k"], case["causal"], q.device)
        Q, K, V, O, dO = (_by_head(t, H) for t in (q, k, v, s["out"], s["dout"]))
        lse = s["lse"].unsqueeze(2)
        p = (torch.bmm(Q, K.transpose(1, 2).contiguous()) * D ** -0.5 - torch.where(lse == -math.inf, 0.0, lse)).exp_()
        p.masked_fill_(~mask, 0.0)
        dV = torch.bmm(p.transpose(1, 2).contiguous(), dO)
        ds = p * (torch.bmm(dO, V.transpose(1, 2).contiguous()) - (dO * O).sum(2, keepdim=True)) * D ** -0.5
        dQ = torch.bmm(ds, K)
        dK = torch.bmm(ds.transpose(1, 2).contiguous(), Q)
        dK, dV = (t.unflatten(0, (Hkv, H // Hkv)).sum(1) for t in (dK, dV))
        return [t.transpose(0, 1).to(BF).contiguous() for t in (dQ, dK, dV)]
    page, lengths, table = case["page"], s["lengths"].long(), s["table"]
    if case["op"] == "append":
        T = s["k"].shape[0]
        cu = torch.arange(T + 1, device="cuda") if s["cu"] is None else s["cu"].long()
        t = torch.arange(T, device="cuda")
        b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        at = lengths[b] - (cu[b + 1] - t)
        where = table[b, at // page].long()
        for i, x in ((0, s["k"]), (1, s["v"])):
            if case["kind"] == "bf16":
                s["cache"][i][where, :, at % page] = x
            else:
                codes, scales = _to_mx8(x.float())
                s["cache"][i][where, :, at % page] = codes
                s["cache"][2 + i][where, :, at % page] = scales
        return _as_numbers(s["cache"])
    B, H, Hkv = case["B"], case["Hq"], case["Hkv"]

    def rows(i):  # fp32 [B, Hkv, tokens, D]
        pages = table.clamp(min=0).long()
        x = s["cache"][i][pages]
        if case["kind"] == "mx8":
            scale = torch.ldexp(torch.ones((), device="cuda"), s["cache"][2 + i][pages].int() - 127)
            x = x.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(32, -1)[..., :D]
        return x.float().transpose(1, 2).flatten(2, 3)

    K, V = rows(0), rows(1)
    Q = s["q"].float().view(B, Hkv, H // Hkv, D)
    scores = torch.matmul(Q, K.transpose(2, 3).contiguous()) * D ** -0.5
    past = torch.arange(K.shape[2], device="cuda") >= lengths[:, None]
    scores.masked_fill_(past[:, None, None], -math.inf)
    p = (scores - scores.amax(3, keepdim=True)).exp_()
    return (torch.matmul(p, V) / p.sum(3, keepdim=True)).view(B, H, D).to(BF)


# ---- the definitions in 64 bits ---------------------------------------------------------------------

def _exact_attention(q, k, v, nq, nk, causal, group):
    """Softmax attention in 64 bits, sequence by sequence and head by head, differentiable: (out, log sums [Tq, Hq])."""
    scale = 1 / math.sqrt(q.shape[2])
    outs, sums, a, b = [], [], 0, 0
    for m, n in zip(nq, nk):
        heads = []
        for h in range(q.shape[1]):
            if m == 0 or n == 0:
                heads.append((q[a: a + m, h] * 0, q[a: a + m, h, 0] * 0 - math.inf))
                continue
            sc = q[a: a + m, h] @ k[b: b + n, h // group].t() * scale
            rows = torch.arange(m, device=q.device)[:, None]
            seen = torch.arange(n, device=q.device)[None] - rows <= n - m if causal else torch.ones_like(sc, dtype=torch.bool)
            some = seen.any(1, keepdim=True)
            sc = torch.where(seen, sc, torch.where(some, -math.inf, 0.0).double())
            o = torch.where(some, torch.softmax(sc, 1) @ v[b: b + n, h // group], 0.0)
            heads.append((o, torch.where(some[:, 0], torch.logsumexp(sc, 1), -math.inf)))
        outs.append(torch.stack([o for o, _ in heads], 1))
        sums.append(torch.stack([x for _, x in heads], 1))
        a, b = a + m, b + n
    left = q.shape[0] - a
    outs.append(torch.zeros_like(q[a:]))
    sums.append(torch.full((left, q.shape[1]), -math.inf, dtype=torch.float64, device=q.device))
    return torch.cat(outs), torch.cat(sums)


def _exact_mx8(x):
    """(values of the E4M3 codes, scales) of x [..., D] in 64 bits; rounding is to the nearest, ties to even."""
    codes, scales = [], []
    for at in range(0, x.shape[-1], 32):
        v = x[..., at: at + 32]
        top = v.abs().amax(-1, keepdim=True)
        e = torch.where(top > 0, torch.frexp(top)[1].double() - 1, torch.full_like(top, -1000.0))
        X = torch.exp2((e - 8).clamp(min=-127))
        q = v / X
        step = torch.exp2((torch.frexp(q)[1].double() - 1).clamp(min=-6) - 3)
        codes.append((torch.round(q / step) * step).clamp(-448, 448))
        scales.append(X)
    return torch.cat(codes, -1), torch.cat(scales, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("attn", "back"):
        nq = _numbers(case["nq"])
        nk = _numbers(case["nk"]) or nq
        q, k, v = (s[n].double().requires_grad_(case["op"] == "back") for n in "qkv")
        out, sums = _exact_attention(q, k, v, nq, nk, case["causal"], case["Hq"] // case["Hkv"])
        if case["op"] == "back":
            return list(torch.autograd.grad(out, (q, k, v), s["dout"].double()))
        return {"out": out, "lse": sums.t().contiguous()} if case["train"] else out
    page, D = case["page"], case["D"]
    lengths, table = s["lengths"].tolist(), s["table"].tolist()
    numbers = [t.double() for t in _as_numbers(s["cache"])]
    if case["op"] == "append":
        n = case["n"]
        for b in range(case["B"]):
            at = lengths[b] - n
            while at < lengths[b]:  # page by page
                end = min(lengths[b], (at // page + 1) * page)
                p, token = table[b][at // page], b * n + at - (lengths[b] - n)
                for i, x in ((0, s["k"]), (1, s["v"])):
                    x = x[token: token + end - at].double().transpose(0, 1)
                    place = (p, slice(None), slice(at % page, at % page + end - at))
                    if case["kind"] == "bf16":
                        numbers[i][place] = x
                    else:
                        numbers[i][place], numbers[2 + i][place] = _exact_mx8(x)
                at = end
        return numbers
    outs = []
    for b in range(case["B"]):
        n = lengths[b]
        rows = []
        for i in range(2):
            t = numbers[i][table[b][: -(-n // page)]]
            if case["kind"] == "mx8":
                x = numbers[2 + i][table[b][: -(-n // page)]]
                t = torch.cat([t[..., 32 * j: 32 * j + 32] * x[..., j: j + 1] for j in range(x.shape[-1])], -1)
            rows.append(t.permute(1, 0, 2, 3).reshape(case["Hkv"], -1, D)[:, :n])
        group = case["Hq"] // case["Hkv"]
        for h in range(case["Hq"]):
            w = torch.softmax(rows[0][h // group] @ s["q"][b, h].double() / math.sqrt(D), 0)
            outs.append(w @ rows[1][h // group])
    return torch.stack(outs).view(case["B"], case["Hq"], D)

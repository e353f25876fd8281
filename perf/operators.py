"""Measured cases of the 8-bit decode step and of beam search.

Four operators of ``lm_head_gemm_amd.flashsample``:

* ``norm``: ``rms_norm_i8`` (root-mean-square norm of x + residual, with the
  result in 8 bits and one scale per token) and ``quantize_i8``, the same
  rounding without the norm (LM-head rows, activations that are normed already);
* ``product``: ``matmul_i8`` (8-bit integer product with a scale per token and
  per channel);
* ``select``: ``beam_select`` (the best continuations over beams and vocabulary);
* ``reorder``: ``beam_reorder`` (each beam's cache rows follow its parent, in place).

``run`` computes a case in plain torch operations, or, where ``own`` is true,
with the calls a user makes. The 8-bit codes are signed whole numbers, returned
as such beside their scales: the rounding rule leaves no code open, so both
sides have to give the same ones.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}


def listed():
    return [
        # one token of a 4096-wide model before its LM head: latency
        {"name": "norm-1x4096", "op": "norm", "M": 1, "D": 4096, "dtype": "bf16", "gain": "bf16", "residual": True},
        # a decode batch of a 7168-wide model whose norm weights are kept in 32 bits
        {"name": "norm-64x7168", "op": "norm", "M": 64, "D": 7168, "dtype": "bf16", "gain": "f32", "residual": True},
        # a prompt of a few thousand tokens, 8192 wide
        {"name": "norm-4099x8192", "op": "norm", "M": 4099, "D": 8192, "dtype": "bf16", "gain": "bf16", "residual": True},
        # an LM head brought to 8 bits when it is loaded
        {"name": "quantize-128256x4096", "op": "norm", "M": 128256, "D": 4096, "dtype": "bf16", "gain": "none",
         "residual": False},
        # one token against a whole LM head: the weights' read is all
        {"name": "product-1x128256x4096", "op": "product", "M": 1, "N": 128256, "K": 4096, "out": "f32"},
        # a small layer with sizes that no tile divides
        {"name": "product-45x5003x2320", "op": "product", "M": 45, "N": 5003, "K": 2320, "out": "f32"},
        # a decode batch, logits in 16 bits
        {"name": "product-64x152064x3584", "op": "product", "M": 64, "N": 152064, "K": 3584, "out": "bf16"},
        # the largest batch of the widest vocabulary product: bound by the matrix cores
        {"name": "product-1024x129280x7168", "op": "product", "M": 1024, "N": 129280, "K": 7168, "out": "bf16"},
        # one user's beam search: latency
        {"name": "select-1x4x128256", "op": "select", "B": 1, "beams": 4, "V": 128256, "n": 8, "dtype": "f32"},
        # many users, twice as many candidates as beams (some will end with the end token)
        {"name": "select-64x8x152064", "op": "select", "B": 64, "beams": 8, "V": 152064, "n": 16, "dtype": "bf16"},
        # a small model's cache after a few tokens: latency
        {"name": "reorder-1x4-len33", "op": "reorder", "layers": 8, "B": 1, "beams": 4, "heads": 8, "T": 64, "len": 33,
         "d": 64, "dtype": "bf16"},
        # keys and values of 16 layers of a 128-wide head model, 1000 tokens of room for 1024
        {"name": "reorder-8x4-len1000", "op": "reorder", "layers": 32, "B": 8, "beams": 4, "heads": 8, "T": 1024,
         "len": 1000, "d": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "product", "select", "reorder"])
    if op == "norm":
        D = 8 * _log(rng, 8, 2048)
        M = min(_log(rng, 1, 16384), max(1, (4099 * 8192) // D))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        gain = rng.choice(["none", "f32", "bf16" if dtype == "bf16" else "f32"])
        return {"op": op, "M": M, "D": D, "dtype": dtype, "gain": gain,
                "residual": gain != "none" and rng.random() < 0.7}
    if op == "product":
        K = 16 * _log(rng, 4, 512)
        N = _log(rng, 64, 152064)
        M = min(_log(rng, 1, 1024), max(1, 1024 * 129280 * 7168 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "f32"])}
    if op == "select":
        beams = rng.randint(1, 12)
        V = _log(rng, 1000, 152064)
        B = min(_log(rng, 1, 64), max(1, (64 * 8 * 152064) // (beams * V)))
        return {"op": op, "B": B, "beams": beams, "V": V, "n": beams * rng.choice([1, 2]),
                "dtype": rng.choice(["bf16", "f32"])}
    T = _log(rng, 1, 1024)
    B = _log(rng, 1, 8)
    return {"op": op, "layers": rng.randint(2, 32), "B": B, "beams": rng.randint(2, 4 if B > 4 else 8),
            "heads": rng.choice([1, 2, 4, 8]), "T": T, "len": rng.randint(1, T),
            "d": rng.choice([20, 64, 72, 80, 128]), "dtype": rng.choice(["bf16", "bf16", "i8"])}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "norm":
        M, D, t = case["M"], case["D"], DTYPES[case["dtype"]]
        if case["gain"] == "none":
            # rows of a head: near-Gaussian weights, some rows larger
            s["x"] = (normal(M, D) * 0.02).mul_(1 + 3 * (uniform(M, 1) < 0.01)).to(t)
        else:
            s["x"] = normal(M, D).to(t)
            # gains near one; a few channels carry activations tens of times the others'
            s["gain"] = (1 + 0.2 * normal(D)).to(DTYPES[case["gain"]])
            if case["residual"]:
                s["residual"] = (normal(M, D) * 2 * (1 + 30 * (uniform(D) < 0.002))).to(t)
    elif case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        # codes of Gaussian rows whose largest magnitude is near 4.2 deviations
        s["q"] = (normal(M, K) * 30).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = (normal(N, K) * 30).round_().clamp_(-127, 127).to(torch.int8)
        s["q_scales"] = (0.02 + 0.02 * uniform(M)).float()
        s["w_scales"] = (3e-4 + 6e-4 * uniform(N)).float()
    elif case["op"] == "select":
        B, K, V = case["B"], case["beams"], case["V"]
        logits = normal(B * K, V) * 2
        logits[:, V - V // 500:] = torch.finfo(DTYPES[case["dtype"]]).min  # entries that pad the vocabulary
        logits.masked_fill_(uniform(V) < 0.01, -math.inf)                  # entries that may not follow
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        scores = -5 - 3 * uniform(B, K)
        scores[:, 1:][uniform(B, K - 1) < 0.03] = -math.inf                # beams not in use
        s["scores"] = scores.float()
        s["finished"] = uniform(B, K) < 0.05
        s["pad"] = 2
    else:
        L, R, t = case["layers"], case["B"] * case["beams"], DTYPES[case["dtype"]]
        shape = (L, R, case["heads"], case["T"], case["d"])
        if t == torch.int8:
            s["cache"] = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        else:
            s["cache"] = torch.empty(shape, device="cuda", dtype=t)
            for layer in s["cache"]:
                layer.copy_(normal(*shape[1:]))
        s["parents"] = torch.randint(0, case["beams"], (case["B"], case["beams"]), generator=g, device="cuda",
                                     dtype=torch.int32)
        s["valid"] = s["cache"][:, :, :, : case["len"]]
    return s


def _norm(s):
    """h = x + residual in the inputs' type; codes round(127 u / max|u|) of u = h * gain; scale
    max|u| rstd / 127. In 64 bits: codes next to a border."""
    x = s["x"]
    out = {}
    h = x
    if "residual" in s:
        h = (x.float() + s["residual"].float()).to(x.dtype)
        out["sum"] = h
    h = h.double()
    u, rstd = h, 1.0
    if "gain" in s:
        u = h * s["gain"].double()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS)
    top = u.abs().amax(-1, keepdim=True)
    out["q"] = torch.where(top > 0, 127 * u / top, 0.0).round().to(torch.int8)
    out["scales"] = (top[:, 0] * rstd / 127).float()
    return out


def _product(s):
    """The sums are whole numbers far below 2^24: exact in 32 bits."""
    y = s["q"].float() @ s["w"].float().t()
    return {"out": (y * s["q_scales"][:, None] * s["w_scales"]).to(DTYPES[s["case"]["out"]])}


def _order_keys(x, V):
    """Whole numbers that sort like (value, lowest index first)."""
    bits = (x + 0.0).view(torch.int32)
    ordered = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return (ordered << 32) + (V - 1 - torch.arange(V, device=x.device))


def _select(s):
    c = s["case"]
    B, K, V, n = c["B"], c["beams"], c["V"], c["n"]
    x = s["logits"].float()
    m = min(n, V)
    tokens = V - 1 - (_order_keys(x, V).topk(m, dim=-1).values & 0xFFFFFFFF)
    x = x.double()
    best = x.gather(1, tokens) - x.logsumexp(-1, keepdim=True)
    total = s["scores"].double().view(B * K, 1) + best
    # a finished beam stands for itself, once
    done = s["finished"].view(B * K, 1)
    first = torch.arange(m, device=x.device) == 0
    total = torch.where(done, torch.where(first, s["scores"].double().view(B * K, 1), -math.inf), total)
    tokens = torch.where(done, s["pad"], tokens)
    flat = tokens + V * torch.arange(K, device=x.device).repeat(B)[:, None]
    total, flat = total.view(B, K * m), flat.view(B, K * m)
    flat, at = flat.sort(dim=-1)                       # ties go to the lowest (beam, token)
    total, at = total.gather(1, at).sort(dim=-1, descending=True, stable=True)
    total, flat = total[:, :n], flat.gather(1, at)[:, :n]
    none = total == -math.inf
    return {"scores": total.float(), "parents": torch.where(none, -1, flat // V).int(),
            "tokens": torch.where(none, -1, flat % V).int()}


def _reorder(s):
    B, K = s["parents"].shape
    src = (s["parents"].long() + K * torch.arange(B, device="cuda")[:, None]).view(-1)
    s["valid"].copy_(s["valid"].index_select(1, src))
    return {"cache": s["cache"]}


def _own(s):
    from lm_head_gemm_amd import flashsample as fs
    c = s["case"]
    if c["op"] == "norm":
        if "gain" not in s:
            q, scales = fs.quantize_i8(s["x"])
            return {"q": q, "scales": scales}
        if "residual" not in s:
            q, scales = fs.rms_norm_i8(s["x"], s["gain"], EPS)
            return {"q": q, "scales": scales}
        q, scales, total = fs.rms_norm_i8(s["x"], s["gain"], EPS, residual=s["residual"])
        return {"sum": total, "q": q, "scales": scales}
    if c["op"] == "product":
        return {"out": fs.matmul_i8(s["q"], s["q_scales"], s["w"], s["w_scales"], out_dtype=DTYPES[c["out"]])}
    if c["op"] == "select":
        scores, parents, tokens = fs.beam_select(s["logits"], s["scores"], c["n"], finished=s["finished"],
                                                 pad_token=s["pad"])
        return {"scores": scores, "parents": parents, "tokens": tokens}
    fs.beam_reorder(s["valid"], s["parents"], dim=1)
    return {"cache": s["cache"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "product": _product, "select": _select, "reorder": _reorder}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        e = 2 if case["dtype"] == "bf16" else 4
        moved = M * D * (e + 1) + 4 * M          # x read, codes and scales written
        if case["residual"]:
            moved += 2 * M * D * e               # residual read, sum written
        if case["gain"] != "none":
            moved += D * (2 if case["gain"] == "bf16" else 4)
        return {"bytes": moved, "flops": 6 * M * D}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K + M * K + 4 * (M + N) + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    if case["op"] == "select":
        B, K, V, n = case["B"], case["beams"], case["V"], case["n"]
        return {"bytes": B * K * V * (2 if case["dtype"] == "bf16" else 4) + 5 * B * K + 12 * B * n,
                "flops": 4 * B * K * V}
    K = case["beams"]
    row = case["heads"] * case["len"] * case["d"] * {"bf16": 2, "f32": 4, "i8": 1}[case["dtype"]]
    # random parents: a row keeps its place with chance 1/K and need not move; a row that some
    # other beam takes (chance 1 - (1 - 1/K)^(K-1)) is read once
    rows = (1 - 1 / K) + (1 - (1 - 1 / K) ** (K - 1))
    return {"bytes": case["layers"] * case["B"] * K * (row * rows) + 4 * case["B"] * K, "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        total = s["x"].double()
        out = {}
        if "residual" in s:
            # a sum of two 16-bit values is rounded to 32 bits on its way to 16
            total = (total + s["residual"].double()).float().to(s["x"].dtype).double()
            out["sum"] = total
        y = total
        if "gain" in s:
            y = total / torch.sqrt((total * total).sum(1, keepdim=True) / case["D"] + EPS) * s["gain"].double()
        scales = torch.maximum(y.max(1).values, -y.min(1).values) / 127
        out["q"] = None
        out["scales"] = scales
        return out
    if case["op"] == "product":
        q = s["q"].double()
        parts = []
        for i in range(0, case["N"], 16384):
            w = s["w"][i:i + 16384].double() * s["w_scales"][i:i + 16384, None].double()
            parts.append(torch.mm(q, w.t()) * s["q_scales"].double().unsqueeze(1))
        return {"out": torch.cat(parts, 1)}
    if case["op"] == "select":
        # every (beam, token) of a group in one list, 64 bits
        B, K, V, n = case["B"], case["beams"], case["V"], case["n"]
        scores = []
        for b in range(B):
            p = torch.log_softmax(s["logits"][b * K:(b + 1) * K].double(), dim=1) + s["scores"][b].double()[:, None]
            p[s["finished"][b]] = -math.inf
            p[s["finished"][b], s["pad"]] = s["scores"][b][s["finished"][b]].double()
            best = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
            k = min(n, K * V)
            best[:k] = p.flatten().topk(k).values
            scores.append(best)
        return {"scores": torch.stack(scores), "parents": None, "tokens": None}
    moved = s["cache"].clone()
    for b in range(case["B"]):
        for k, p in enumerate(s["parents"][b].tolist()):
            moved[:, b * case["beams"] + k, :, : case["len"]] = s["cache"][:, b * case["beams"] + p, :, : case["len"]]
    return {"cache": moved.double()}

"""The operators that train an 8-bit mixture-of-experts layer, as cases that can be run and timed.

Operators: the root-mean-square norm with the residual's addition and 8-bit output (serving and training) and
its gradient, the gradient of sorting tokens by expert and of summing them back with their weights, the
gradient of the SwiGLU with 8-bit output, and the gradient of the experts' weights.

Each case runs in two forms.  The plain form is elementary torch arithmetic in float32, rounded once at the
end.  The other one (``own``) makes the calls of the package's public entry points.  ``exact`` evaluates the
definitions in float64.

8-bit matrices are E4M3 codes with a power-of-two scale per 128 elements of a row: s = 2^k, the smallest with
absmax / s <= 448; scales are stored as [K / 128][rows].  What is quantised is the BF16 value that the unfused
operator would store.  Codes come back as E4M3 numbers and scales as powers of two in 8 bits (2^-127 for the
zero scale of a group of zeros).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token's hidden state, residual added, on its way into an 8-bit Linear: latency counts
        {"name": "norm 1x7168", "op": "norm", "M": 1, "K": 7168, "residual": True, "gamma": "bf16", "train": False},
        # the benchmark's activation, a training batch: bandwidth counts
        {"name": "norm 16384x7168", "op": "norm", "M": 16384, "K": 7168, "residual": True, "gamma": "bf16", "train": True},
        # a small fine-tuning batch on a narrow layer, the gain kept in float32, an odd number of rows
        {"name": "norm-grad 509x1984", "op": "norm-grad", "M": 509, "K": 1984, "gamma": "f32", "dres": False},
        # the benchmark's activation, the residual stream's gradient added
        {"name": "norm-grad 16384x7168", "op": "norm-grad", "M": 16384, "K": 7168, "gamma": "bf16", "dres": True},
        # a small fine-tuning batch, an odd number of experts
        {"name": "sort-grad 509 tokens", "op": "sort-grad", "T": 509, "E": 63, "k": 6, "N": 2048, "add": False},
        # the benchmark's layer: 8192 tokens, 8 of 32 experts, hidden size 7168
        {"name": "sort-grad 8192 tokens", "op": "sort-grad", "T": 8192, "E": 32, "k": 8, "N": 7168, "add": True},
        # a ragged batch on a narrow expert
        {"name": "swiglu-grad 333x1408", "op": "swiglu-grad", "M": 333, "I": 1408},
        # the benchmark's experts: the rows of 8192 tokens' choices, inner size 2048
        {"name": "swiglu-grad 67712x2048", "op": "swiglu-grad", "M": 67712, "I": 2048},
        # a small fine-tuning batch: few rows an expert, the outputs' bytes count
        {"name": "experts-grad 509 tokens", "op": "experts-grad", "T": 509, "E": 12, "k": 4, "N": 1024, "K": 1408, "f32": True},
        # the benchmark's gate/up projection: the tensor cores count
        {"name": "experts-grad 8192 gate/up", "op": "experts-grad", "T": 8192, "E": 32, "k": 8, "N": 4096, "K": 7168, "f32": True},
        # the benchmark's down projection, gradients stored in BF16
        {"name": "experts-grad 8192 down", "op": "experts-grad", "T": 8192, "E": 32, "k": 8, "N": 7168, "K": 2048, "f32": False},
    ]


def _odd(rng, lo, hi, powers=(1, 1, 2, 16)):
    """An odd number times a small power of two, over the logarithm of [lo, hi]."""
    p = rng.choice([q for q in powers if q <= max(1, hi // max(1, lo))])
    v = math.exp(rng.uniform(math.log(lo), math.log(hi))) / p
    return min(int(hi), max(1, 2 * int(v / 2) + 1) * p)


def _width(rng, hi, units=(128, 128, 256, 512)):
    """An odd multiple of 128, 256 or 512, at most hi."""
    unit = rng.choice([u for u in units if u <= hi])
    return unit * (2 * rng.randint(0, max(0, (hi // unit - 1) // 2)) + 1)


def draw(rng):
    op = rng.choice(("norm", "norm-grad", "sort-grad", "swiglu-grad", "experts-grad"))
    if op == "norm":
        return {"op": op, "M": _odd(rng, 1, 16384), "K": _width(rng, 7168), "residual": rng.random() < 0.6,
                "gamma": rng.choice(("bf16", "f32")), "train": rng.random() < 0.5}
    if op == "norm-grad":
        return {"op": op, "M": _odd(rng, 1, 16384), "K": 8 * _odd(rng, 16, 896, powers=(1, 1, 16)),
                "gamma": rng.choice(("bf16", "f32")), "dres": rng.random() < 0.5}
    if op == "swiglu-grad":
        return {"op": op, "M": _odd(rng, 1, 65536), "I": _width(rng, 2048)}
    E = _odd(rng, 2, 32)
    k = rng.randint(1, min(8, E))
    if op == "sort-grad":
        return {"op": op, "T": _odd(rng, 1, 8192), "E": E, "k": k, "N": _width(rng, 7168), "add": rng.random() < 0.5}
    return {"op": op, "T": _odd(rng, 1, 4096), "E": E, "k": k, "N": _width(rng, 4096), "K": _width(rng, 7168),
            "f32": rng.random() < 0.6}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * sigma


def _activation(g, shape):
    """N(0, 1) with one value in a thousand fifty times as large, as the benchmark's activations."""
    x = _normal(g, shape, 1.0)
    hit = torch.rand(shape, generator=g, device=DEV) < 1e-3
    return torch.where(hit, x * 50.0, x).to(torch.bfloat16)


def _routing(g, T, E, k):
    """Distinct choices of k experts a token, expert e drawn in proportion to (e + 1)^-1.1."""
    logw = -1.1 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-30, 1 - 1e-7)
    return torch.topk(logw - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)


def _layout(idx, E):
    """(offsets [E + 1], row_token [rows], row_of [T, k]): the chosen pairs by expert, then by token, each
    expert's segment padded to a multiple of 128 rows; -1 for choices and rows without one another."""
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, order.values, torch.ones_like(flat))
    first = torch.cumsum(counts, 0) - counts
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum((counts[:E] + 127) // 128 * 128, 0)])
    here = order.values < E
    at = offsets[order.values] + torch.arange(T * k, device=DEV) - first[order.values]
    rows = (T * k + min(E, T * k) * 127 + 127) // 128 * 128
    row_token = torch.full((rows + 1,), -1, dtype=torch.int32, device=DEV)
    row_token.scatter_(0, torch.where(here, at, rows), torch.where(here, order.indices // k, -1).to(torch.int32))
    row_of = torch.empty(T * k, dtype=torch.int64, device=DEV).scatter_(0, order.indices, torch.where(here, at, -1))
    return offsets.to(torch.int32), row_token[:rows].clone(), row_of.view(T, k).to(torch.int32)


def _gain(g, K, kind):
    v = 1.0 + _normal(g, (K,), 0.2)
    return v.to(torch.bfloat16) if kind == "bf16" else v


def _codes_out(M, K):
    return (torch.empty((M, K), dtype=torch.uint8, device=DEV), torch.empty((K // 128, M), dtype=torch.float32, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        s["x"] = _activation(g, (M, K))
        s["res"] = _activation(g, (M, K)) if case["residual"] else None
        s["gain"] = _gain(g, K, case["gamma"])
        s["r"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV) if case["residual"] else None
        s["q"], s["s"] = _codes_out(M, K)
        s["rstd"] = torch.empty(M, dtype=torch.float32, device=DEV) if case["train"] else None
    elif op == "norm-grad":
        M, K = case["M"], case["K"]
        s["r"] = _activation(g, (M, K))
        s["dy"] = _normal(g, (M, K), 1e-3).to(torch.bfloat16)
        s["gain"] = _gain(g, K, case["gamma"])
        s["rstd"] = torch.cat([torch.rsqrt(p.to(torch.float64).square().mean(1) + EPS) for p in s["r"].split(2048)]).to(torch.float32)
        s["dres"] = _normal(g, (M, K), 1e-3).to(torch.bfloat16) if case["dres"] else None
        s["dx"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
        s["dgain"] = torch.empty(K, dtype=torch.float32, device=DEV)
        # scratch memory, more than the call asks for
        s["ws"] = torch.empty(4 * min(M, 4096) * K + 4096, dtype=torch.uint8, device=DEV)
    elif op == "sort-grad":
        T, E, k, N = (case[n] for n in ("T", "E", "k", "N"))
        idx = _routing(g, T, E, k)
        idx[torch.rand(T, generator=g, device=DEV) < 0.02] = -1       # masked tokens have no expert
        _, s["row_token"], s["row_of"] = _layout(idx, E)
        rows = s["row_token"].numel()
        s["dout"] = _normal(g, (T, N), 1e-3).to(torch.bfloat16)
        s["y"] = _normal(g, (rows, N), 1.0).to(torch.bfloat16)
        s["w"] = torch.softmax(_normal(g, (T, k), 1.0), dim=1)
        s["d"] = _normal(g, (rows, N), 1e-3).to(torch.bfloat16)
        s["add"] = _normal(g, (T, N), 1e-3).to(torch.bfloat16) if case["add"] else None
        s["q"], s["s"] = _codes_out(rows, N)
        s["dw"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        s["dx"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    elif op == "swiglu-grad":
        M, I = case["M"], case["I"]
        s["h"] = _normal(g, (M, 2 * I), 2.0).to(torch.bfloat16)
        s["dv"] = _normal(g, (M, I), 1e-3).to(torch.bfloat16)
        pad = torch.rand(M, generator=g, device=DEV) < 0.03
        s["live"] = torch.where(pad, -1, 0).to(torch.int32)
        s["q"], s["s"] = _codes_out(M, 2 * I)
    else:
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        s["offsets"], row_token, _ = _layout(_routing(g, T, E, k), E)
        s["bounds"] = s["offsets"].tolist()
        for name, width, sigma in (("a", N, 1e-3), ("b", K, 1.0)):
            v = _normal(g, (width, row_token.numel()), sigma).to(torch.bfloat16)
            v = torch.where((row_token >= 0)[None, :], v, torch.zeros((), dtype=v.dtype, device=DEV))
            s[name], _, s["s" + name] = _plain_quantise(v)
        s["out"] = torch.empty((E, N, K), dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _plain_quantise(v):
    """(codes [M, K], scales as bytes of an exponent and as float32, [K / 128, M]) of BF16 v [M, K]."""
    M, K = v.shape
    v = v.to(torch.float32).view(M, K // 128, 128)
    m, e = torch.frexp(v.abs().amax(dim=2))
    k = torch.where(m > 0, e - 9 + (m > 0.875).to(torch.int32), -127).clamp(min=-126)
    byte = torch.where(m > 0, k + 127, 0)
    q = (v * torch.exp2(-k.to(torch.float32))[:, :, None]).view(M, K).to(torch.float8_e4m3fn)
    byte = byte.t().contiguous()
    scale = torch.where(byte > 0, (byte << 23).to(torch.int32).view(torch.float32), torch.zeros((), device=v.device))
    return q.view(torch.uint8), byte.to(torch.uint8), scale


def _numbers(q, byte):
    """Codes and scale exponents as the numbers that they stand for."""
    return q.view(torch.float8_e4m3fn), byte.view(torch.float8_e8m0fnu)


def _plain_norm(s):
    r = s["x"].to(torch.float32)
    if s["res"] is not None:
        r = (r + s["res"].to(torch.float32)).to(torch.bfloat16).to(torch.float32)
    rstd = 1.0 / torch.sqrt((r * r).mean(dim=1) + EPS)
    y = (r * rstd[:, None] * s["gain"].to(torch.float32)).to(torch.bfloat16)
    q, byte, _ = _plain_quantise(y)
    q, byte = _numbers(q, byte)
    return {"r": None if s["res"] is None else r.to(torch.bfloat16), "q": q, "s": byte, "rstd": rstd if s["train"] else None}


def _plain_norm_grad(s):
    dy, xhat = s["dy"].to(torch.float32), s["r"].to(torch.float32) * s["rstd"][:, None]
    t = dy * s["gain"].to(torch.float32)
    dx = s["rstd"][:, None] * (t - xhat * (t * xhat).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].to(torch.float32)
    return {"dx": dx.to(torch.bfloat16), "dgain": (dy * xhat).sum(dim=0)}


def _plain_sort_grad(s):
    row_of, token = s["row_of"].long(), s["row_token"]
    has = row_of >= 0
    at = torch.where(has, row_of, 0)
    w_row = torch.zeros(token.numel() + 1, dtype=torch.float32, device=DEV)
    w_row[torch.where(has, row_of, token.numel()).reshape(-1)] = s["w"].reshape(-1)
    dout = s["dout"].to(torch.float32)
    dy = torch.where((token >= 0)[:, None], dout[token.clamp(min=0)] * w_row[:-1, None], torch.zeros((), device=DEV))
    q, byte, _ = _plain_quantise(dy.to(torch.bfloat16))
    q, byte = _numbers(q, byte)
    zero = torch.zeros((), device=DEV)
    dw = torch.where(has, (dout[:, None, :] * s["y"][at].to(torch.float32)).sum(dim=2), zero)
    dx = torch.where(has[:, :, None], s["d"][at].to(torch.float32), zero).sum(dim=1)
    if s["add"] is not None:
        dx = dx + s["add"].to(torch.float32)
    return {"q": q, "s": byte, "dw": dw, "dx": dx.to(torch.bfloat16)}


def _plain_swiglu_grad(s):
    gate, up = s["h"].to(torch.float32).chunk(2, dim=1)
    dv = s["dv"].to(torch.float32)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dup = dv * (gate * sig)
    dgate = dv * up * (sig * (1.0 + gate * (1.0 - sig)))
    dh = torch.cat([dgate, dup], dim=1)
    dh = torch.where((s["live"] >= 0)[:, None], dh, torch.zeros((), device=DEV))
    q, byte, _ = _plain_quantise(dh.to(torch.bfloat16))
    q, byte = _numbers(q, byte)
    return {"q": q, "s": byte}


def _plain_experts_grad(s):
    a, b = (s[n].view(torch.float8_e4m3fn).to(torch.float32) * s["s" + n].t().repeat_interleave(128, dim=1) for n in ("a", "b"))
    at = s["bounds"]
    for e in range(s["E"]):          # segments differ in length: one product each
        s["out"][e] = (a[:, at[e]:at[e + 1]] @ b[:, at[e]:at[e + 1]].t()).to(s["out"].dtype)
    return {"d": s["out"]}


PLAIN = {"norm": _plain_norm, "norm-grad": _plain_norm_grad, "sort-grad": _plain_sort_grad,
         "swiglu-grad": _plain_swiglu_grad, "experts-grad": _plain_experts_grad}


# ------------------------------------------------------------------------------------ the package's calls

def _run_own(s):
    import fp8_fine_grained_fp8bs_gb300 as fp8bs
    op = s["op"]
    if op in ("norm", "norm-grad"):
        kind = fp8bs.IN_BF16 if s["gamma"] == "bf16" else fp8bs.IN_F32
        M, K = s["M"], s["K"]
    if op == "norm":
        fp8bs.fp8bs_rmsnorm_quantize(s["x"], M, K, K, s["res"], K, s["gain"], kind, EPS, s["r"], None, s["q"], s["s"],
                                     fp8bs.SCALE_POW2, s["rstd"])
        return {"r": s["r"], "q": s["q"].view(torch.float8_e4m3fn), "s": s["s"].to(torch.float8_e8m0fnu), "rstd": s["rstd"]}
    if op == "norm-grad":
        fp8bs.fp8bs_rmsnorm_backward(s["dy"], M, K, K, s["r"], K, s["gain"], kind, s["rstd"], s["dres"], K, s["dx"],
                                     s["dgain"], 0, s["ws"], s["ws"].numel())
        return {"dx": s["dx"], "dgain": s["dgain"]}
    if op == "sort-grad":
        T, N, k, rows = s["T"], s["N"], s["k"], s["row_token"].numel()
        fp8bs.fp8bs_moe_combine_backward(s["dout"], T, N, N, s["y"], rows, s["row_of"], s["row_token"], s["w"], k, None,
                                         s["q"], s["s"], fp8bs.SCALE_POW2, s["dw"])
        fp8bs.fp8bs_moe_dispatch_backward(s["d"], rows, N, s["row_of"], T, k, s["add"], s["dx"])
        return {"q": s["q"].view(torch.float8_e4m3fn), "s": s["s"].to(torch.float8_e8m0fnu), "dw": s["dw"], "dx": s["dx"]}
    if op == "swiglu-grad":
        M, I = s["M"], s["I"]
        fp8bs.fp8bs_swiglu_backward_quantize(s["h"], M, I, 2 * I, s["dv"], I, s["live"], None, s["q"], s["s"],
                                             fp8bs.SCALE_POW2)
        return {"q": s["q"].view(torch.float8_e4m3fn), "s": s["s"].to(torch.float8_e8m0fnu)}
    fp8bs.fp8bs_grouped_wgrad_pow2(s["a"], s["sa"], s["b"], s["sb"], s["a"].shape[1], s["offsets"], s["E"], s["out"],
                                   fp8bs.OUT_F32 if s["f32"] else fp8bs.OUT_BF16, s["N"], s["K"], 0)
    return {"d": s["out"]}


def run(state):
    return _run_own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "norm":
        n = case["M"] * case["K"]
        gain = case["K"] * (2 if case["gamma"] == "bf16" else 4)
        return {"bytes": n * (2 + (4 if case["residual"] else 0) + 1) + n // 32 + gain + (4 * case["M"] if case["train"] else 0),
                "flops": 8 * n}
    if op == "norm-grad":
        n = case["M"] * case["K"]
        gain = case["K"] * (2 if case["gamma"] == "bf16" else 4)
        return {"bytes": n * (6 + (2 if case["dres"] else 0)) + 4 * case["M"] + gain + 4 * case["K"], "flops": 12 * n}
    if op == "sort-grad":
        T, k, N = case["T"], case["k"], case["N"]
        pairs = T * k
        # tokens read and written once, the chosen rows of y and d read, their codes and scales written
        return {"bytes": T * N * (4 + (2 if case["add"] else 0)) + pairs * N * 5 + pairs * (N // 32 + 16), "flops": 6 * pairs * N}
    if op == "swiglu-grad":
        n = case["M"] * case["I"]
        return {"bytes": n * 8 + n // 16 + 4 * case["M"], "flops": 20 * n}
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    pairs = T * k
    return {"bytes": pairs * (N + K) + pairs * (N + K) // 32 + E * N * K * (4 if case["f32"] else 2), "flops": 2 * pairs * N * K}


# ------------------------------------------------------------------------------------------- in 64 bits

def _nearest_64(v, bits, low):
    """v on the grid of `bits` mantissa bits, exponents from `low`; ties to even."""
    a = v.abs()
    _, e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))
    step = torch.exp2((e.to(torch.float64) - 1).clamp(min=low) - bits)
    return torch.sign(v) * torch.round(a / step) * step


def _quantise_64(v):
    """Codes and scales of v [M, K] rounded to BF16, group by group of 128."""
    M, K = v.shape
    groups = _nearest_64(v, 7, -126).view(M, K // 128, 128)
    top = groups.abs().amax(dim=2)
    # BF16 values lie 2^-8 apart: what is taken off keeps a rounded logarithm of a power of two from the next one
    s = torch.exp2(torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448) - 1e-6))
    s = torch.where(top > 0, s, torch.full_like(s, 2.0 ** -127))
    return {"q": _nearest_64(groups / s[:, :, None], 3, -6).view(M, K), "s": s.t().contiguous()}


def _placed(s):
    """(row, token, slot) of every choice that has a row."""
    t, j = torch.nonzero(s["row_of"] >= 0, as_tuple=True)
    return s["row_of"][t, j].long(), t, j


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "norm":
        r = s["x"].to(f64)
        if case["residual"]:
            r = _nearest_64(r + s["res"].to(f64), 7, -126)
        rstd = torch.rsqrt(r.square().mean(1) + EPS)
        out = _quantise_64(r * rstd[:, None] * s["gain"].to(f64)[None, :])
        return {"r": r if case["residual"] else None, **out, "rstd": rstd if case["train"] else None}
    if op == "norm-grad":
        K = case["K"]
        dy, r, gain = s["dy"].to(f64), s["r"].to(f64), s["gain"].to(f64)
        rstd = s["rstd"].to(f64)[:, None]
        # y = gain r rstd with rstd = (mean r^2 + eps)^-1/2: d rstd / d r = -rstd^3 r / K
        through = (dy * gain * r).sum(1, keepdim=True)
        dx = dy * gain * rstd - through * rstd ** 3 * r / K
        if case["dres"]:
            dx = dx + s["dres"].to(f64)
        return {"dx": dx, "dgain": torch.einsum("mk,mk->k", dy, r * rstd)}
    if op == "sort-grad":
        T, k, N, rows = case["T"], case["k"], case["N"], s["row_token"].numel()
        row, t, j = _placed(s)
        w = s["w"].to(f64)
        dy = torch.zeros((rows, N), dtype=f64, device=DEV)
        # the product of the float32 weight is rounded to float32 on its way to BF16
        dy[row] = (w[t, j, None] * s["dout"].to(f64)[t]).to(torch.float32).to(f64)
        out = _quantise_64(dy)
        del dy
        dw = torch.zeros((T, k), dtype=f64, device=DEV)
        dx = s["add"].to(f64) if case["add"] else torch.zeros((T, N), dtype=f64, device=DEV)
        for slot in range(k):
            here = j == slot
            dw[t[here], slot] = (s["dout"].to(f64)[t[here]] * s["y"][row[here]].to(f64)).sum(1)
            dx[t[here]] += s["d"][row[here]].to(f64)
        return {**out, "dw": dw, "dx": dx}
    if op == "swiglu-grad":
        I = case["I"]
        q, scale = [], []
        for h, dv, live in zip(s["h"].split(8192), s["dv"].split(8192), s["live"].split(8192)):
            gate, up, dv = h[:, :I].to(f64), h[:, I:].to(f64), dv.to(f64) * (live >= 0).to(f64)[:, None]
            p = torch.sigmoid(gate)
            part = _quantise_64(torch.cat([dv * up * (p + gate * p * torch.sigmoid(-gate)), dv * gate * p], dim=1))
            q.append(part["q"].to(torch.float32))        # E4M3 numbers are exact in float32
            scale.append(part["s"])
        return {"q": torch.cat(q), "s": torch.cat(scale, dim=1)}
    a, b = (s[n].view(torch.float8_e4m3fn) for n in ("a", "b"))
    d = torch.zeros(s["out"].shape, dtype=f64, device=DEV)
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if hi > lo:
            x, y = (m[:, lo:hi].to(f64).view(m.shape[0], -1, 128) * c[lo // 128:hi // 128].t().to(f64)[:, :, None]
                    for m, c in ((a, s["sa"]), (b, s["sb"])))
            torch.matmul(x.flatten(1), y.flatten(1).t(), out=d[e])
    return {"d": d}

"""The operators of a 4-bit mixture-of-experts layer, as cases that can be run and timed.

Operators: the 4-bit quantisers (BF16 rows, gathered rows, SwiGLU of the gate/up projection) with the
dequantiser that reads their codes back, the 4-bit product, its grouped form over experts, the router with
the row layout of its choices (serving), and the router with the balance loss and its gradient (training).

Each case runs in two forms.  The plain form is elementary torch arithmetic in float32, rounded once at the
end.  The other one (``own``) makes the calls of the package's public entry points.  ``exact`` evaluates the
definitions in float64.

Formats (``fmt``), along K of a row-major matrix, two E2M1 codes a byte (the even element in the low half):
  0  one E4M3 scale per 16 elements and one float32 scale per row:  value = code * s * g
  1  one UE8M0 scale (a power of two) per 32 elements:              value = code * s
Scales are stored in 512-byte blocks of 128 rows x 4 scales: the scale of row r and group j is byte
((r/128) * ceil(J/4) + j/4) * 512 + (r%32) * 16 + (r%128)/32 * 4 + j%4, J the groups of a row.
"""
import math

import torch

own = False

DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # the magnitudes of E2M1
TINY = 1e-20                                       # guards the sums that scores are divided by


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token's hidden state on its way into a 4-bit Linear: latency counts
        {"name": "quantise 1x7168", "op": "quantise", "source": "rows", "fmt": 0, "M": 1, "K": 7168},
        # the benchmark's activation, a training or prefill batch: bandwidth counts
        {"name": "quantise 16384x7168", "op": "quantise", "source": "rows", "fmt": 0, "M": 16384, "K": 7168},
        # the input of the down projection, an odd number of rows
        {"name": "swiglu-quantise 8191x2048", "op": "quantise", "source": "swiglu", "fmt": 0, "M": 8191, "K": 2048},
        # one decoded token through a Linear: the weight's bytes count
        {"name": "product 1x7168x7168", "op": "product", "fmt": 0, "M": 1, "N": 7168, "K": 7168, "f32": False},
        # a ragged batch on a narrow layer, float32 out
        {"name": "product 333x2056x1984", "op": "product", "fmt": 1, "M": 333, "N": 2056, "K": 1984, "f32": True},
        # the benchmark's dense Linear: the tensor cores count
        {"name": "product 4096x7168x7168", "op": "product", "fmt": 0, "M": 4096, "N": 7168, "K": 7168, "f32": False},
        # decoding: 16 tokens' gate/up projection, every expert's weight read for a few rows each
        {"name": "experts 16 tokens", "op": "experts", "fmt": 0, "T": 16, "E": 32, "k": 8, "N": 4096, "K": 7168},
        # the benchmark's gate/up projection: 8192 tokens, skewed routing
        {"name": "experts 8192 tokens", "op": "experts", "fmt": 0, "T": 8192, "E": 32, "k": 8, "N": 4096, "K": 7168},
        # one decoded token picks its experts, and the rows of the expert segments are laid out
        {"name": "route 1 token", "op": "route", "T": 1, "E": 256, "k": 8, "score": 1, "bias": True, "dtype": "f32"},
        # a prefill batch of 32749 tokens (odd), softmax scores
        {"name": "route 32749 tokens", "op": "route", "T": 32749, "E": 256, "k": 8, "score": 0, "bias": False,
         "dtype": "f32"},
        # a training batch of packed sequences (an empty one among them, padding masked): forward and backward
        {"name": "route-train 131072 tokens", "op": "train", "T": 131072, "E": 256, "k": 8, "score": 1, "bias": True,
         "dtype": "f32", "S": 32},
        # a small fine-tuning batch of one sequence, an odd number of experts, softmax of BF16 logits
        {"name": "route-train 509 tokens", "op": "train", "T": 509, "E": 63, "k": 6, "score": 0, "bias": False,
         "dtype": "bf16", "S": 1},
    ]


def _odd(rng, lo, hi, powers=(1, 1, 2, 16)):
    """An odd number times a small power of two, over the logarithm of [lo, hi]."""
    p = rng.choice([q for q in powers if q <= max(1, hi // max(1, lo))])
    v = math.exp(rng.uniform(math.log(lo), math.log(hi))) / p
    return min(int(hi), max(1, 2 * int(v / 2) + 1) * p)


def _k(rng, lo, hi):
    """A length of K: an odd multiple of 64, 256 or 512."""
    unit = rng.choice((64, 64, 256, 512))
    top = max(0, (hi // unit - 1) // 2)
    low = min(top, max(0, (lo // unit - 1) // 2))
    return unit * (2 * rng.randint(low, top) + 1)


def draw(rng):
    op = rng.choice(("quantise", "product", "experts", "route", "train"))
    if op == "quantise":
        K = _k(rng, 64, 7168)
        return {"op": op, "source": rng.choice(("rows", "gather", "swiglu")), "fmt": rng.randint(0, 1),
                "M": _odd(rng, 1, 16384), "K": K}
    if op == "product":
        return {"op": op, "fmt": rng.randint(0, 1), "M": _odd(rng, 1, 4096), "N": 8 * _odd(rng, 1, 896), "K": _k(rng, 64, 7168),
                "f32": rng.random() < 0.3}
    if op == "experts":
        E = _odd(rng, 2, 32)
        return {"op": op, "fmt": rng.randint(0, 1), "T": _odd(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)),
                "N": 8 * _odd(rng, 16, 512), "K": _k(rng, 64, 7168)}
    E = _odd(rng, 8, 256, powers=(1, 4, 8))
    score = rng.randint(0, 1)
    case = {"op": op, "T": _odd(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E)), "score": score,
            "bias": score == 1 and rng.random() < 0.6, "dtype": rng.choice(("f32", "f32", "bf16"))}
    if op == "train":
        case["S"] = rng.choice((1, 1, 3, 17, 32))
    return case


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * sigma)


def _activation(g, shape):
    """N(0, 1) with one value in a thousand fifty times as large, as the benchmark's activations."""
    x = _normal(g, shape, 1.0)
    hit = torch.rand(shape, generator=g, device=DEV) < 1e-3
    return torch.where(hit, x * 50.0, x).to(torch.bfloat16)


def _groups(K, fmt):
    return K // (16 if fmt == 0 else 32)


def _sf_bytes(M, K, fmt):
    return (M + 127) // 128 * ((_groups(K, fmt) + 3) // 4) * 512


def _routing(g, T, E, k):
    """Distinct choices of k experts a token, expert e drawn in proportion to (e + 1)^-1.1."""
    logw = -1.1 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-30, 1 - 1e-7)
    return torch.topk(logw - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)


def _rows_cap(T, E, k):
    """Rows that the padded segments of T * k choices can take at most."""
    n = T * k + min(E, T * k) * 127
    return (n + 127) // 128 * 128


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "quantise":
        M, K, fmt, source = (case[n] for n in ("M", "K", "fmt", "source"))
        s["rows"] = None
        if source == "rows":
            s["x"] = _activation(g, (M, K))
        elif source == "gather":
            T = max(1, M // 9)
            s["x"] = _activation(g, (T, K))
            r = torch.randint(0, T, (M,), generator=g, device=DEV, dtype=torch.int32)
            pad = torch.rand((M,), generator=g, device=DEV) < 0.1
            s["rows"] = torch.where(pad, torch.full_like(r, -1), r)
        else:
            s["x"] = _normal(g, (M, 2 * K), 2.0).to(torch.bfloat16)
            pad = torch.rand((M,), generator=g, device=DEV) < 0.05
            s["rows"] = torch.where(pad, -1, 0).to(torch.int32)
        s["q"] = torch.empty((M, K // 2), dtype=torch.uint8, device=DEV)
        s["sf"] = torch.empty(_sf_bytes(M, K, fmt), dtype=torch.uint8, device=DEV)
        s["g"] = torch.empty(M, dtype=torch.float32, device=DEV) if fmt == 0 else None
        s["out"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    elif op == "product":
        M, N, K, fmt = (case[n] for n in ("M", "N", "K", "fmt"))
        s["a"] = _plain_quantise(_activation(g, (M, K)), fmt)
        s["b"] = _plain_quantise(_normal(g, (N, K), 0.02).to(torch.bfloat16), fmt)
        s["out"] = torch.empty((M, N), dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV)
    elif op == "experts":
        T, E, k, N, K, fmt = (case[n] for n in ("T", "E", "k", "N", "K", "fmt"))
        offsets, row_token, _ = _plain_layout(_routing(g, T, E, k), E)
        x = _activation(g, (T, K))
        s["a"] = _plain_quantise(x[row_token.clamp(min=0).long()], fmt, row_token)
        w = [_plain_quantise(_normal(g, (N, K), 0.02).to(torch.bfloat16), fmt) for _ in range(E)]
        s["b"] = tuple(torch.stack([t[i] for t in w]) if w[0][i] is not None else None for i in range(3))
        s["offsets"] = offsets
        s["bounds"] = offsets.tolist()
        s["out"] = torch.zeros((row_token.numel(), N), dtype=torch.bfloat16, device=DEV)
    else:
        T, E, k = case["T"], case["E"], case["k"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = (_normal(g, (T, E), 1.0) + _normal(g, (1, E), 0.5)).to(dt)
        # the selection bias moves in steps of its update rate
        s["bias"] = torch.round(_normal(g, (E,), 50.0)) * 1e-3 if case["bias"] else None
        s["idx"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        if op == "route":
            R = _rows_cap(T, E, k)
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
            s["row_token"] = torch.empty(R, dtype=torch.int32, device=DEV)
            s["row_of"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        else:
            S = case["S"]
            s["valid"] = (torch.rand(T, generator=g, device=DEV) >= 0.03).to(torch.uint8)
            cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV, dtype=torch.int32)).values
            if S > 2:
                cuts[S // 2] = cuts[S // 2 - 1]          # one empty sequence
            ends = torch.tensor([0, T], dtype=torch.int32, device=DEV)
            s["seq"] = torch.cat([ends[:1], cuts, ends[1:]])
            s["counts"] = torch.empty((S, E), dtype=torch.int32, device=DEV)
            s["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
            s["loss"] = torch.empty(1, dtype=torch.float32, device=DEV)
            s["dw"] = _normal(g, (T, k), 1.0 / T)
            s["dloss"] = torch.ones(1, dtype=torch.float32, device=DEV)
            s["dlogits"] = torch.empty((T, E), dtype=dt, device=DEV)
        # scratch memory for either call, more than it asks for
        s["ws"] = torch.empty(4 * (T * k // 256 + T // 32 + 2 * case.get("S", 1) + 64) * (E + 32), dtype=torch.uint8, device=DEV)
    return s


ALPHA, SCALE = 1e-2, 2.5     # the balance loss's factor and the factor of the gate weights


# ------------------------------------------------------------------------------------------ plain forms

def _tile_sf(sf, M, J, tail):
    """Scale bytes [M, J] in the blocked layout; unused rows and groups are `tail`."""
    mt, kg = (M + 127) // 128, (J + 3) // 4
    full = torch.full((mt * 128, kg * 4), tail, dtype=torch.uint8, device=sf.device)
    full[:M, :J] = sf
    return full.view(mt, 4, 32, kg, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile_sf(sf, M, J):
    mt, kg = (M + 127) // 128, (J + 3) // 4
    return sf.view(mt, kg, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(mt * 128, kg * 4)[:M, :J]


def _sf_values(sf, fmt):
    return sf.view(torch.float8_e4m3fn if fmt == 0 else torch.float8_e8m0fnu).to(torch.float32)


def _e2m1_code(v):
    """Nearest code of E2M1, ties to even, saturating; the sign is kept."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    for bound, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= bound) if up else (a > bound)
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _plain_quantise(x, fmt, rows=None):
    """(codes [M, K/2], blocked scale bytes, row scales or None) of x [M, K]; rows < 0 are zero rows."""
    M, K = x.shape
    v = x.to(torch.float32)
    if rows is not None:
        v = torch.where((rows >= 0)[:, None], v, torch.zeros((), device=v.device))
    J = _groups(K, fmt)
    v = v.view(M, J, -1)
    amax = v.abs().amax(dim=2)
    if fmt == 0:
        rowmax = amax.amax(dim=1)
        g = torch.clamp(rowmax / torch.full_like(rowmax, 2688.0), min=2.0 ** -100)
        s8 = (amax / (g * 6.0)[:, None]).to(torch.float8_e4m3fn)
        d = s8.to(torch.float32) * g[:, None]
        r = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
        sf = s8.view(torch.uint8)
    else:
        g = None
        m, e = torch.frexp(amax)
        k = torch.where(amax > 0, e - 3 + (m > 0.75).to(torch.int32), -127).clamp(-127, 127)
        r = ((127 - k) << 23).to(torch.int32).view(torch.float32)
        sf = (k + 127).to(torch.uint8)
    c = _e2m1_code(v * r[:, :, None]).view(M, K)
    return c[:, 0::2] | (c[:, 1::2] << 4), _tile_sf(sf, M, J, 0), g


def _plain_dequantise(q, sf, g, fmt):
    M, K = q.shape[0], q.shape[1] * 2
    J = _groups(K, fmt)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float32, device=q.device)
    c = torch.stack([q & 15, q >> 4], dim=2).view(M, J, -1)
    v = grid[c.to(torch.int32)] * _sf_values(_untile_sf(sf, M, J), fmt)[:, :, None]
    return (v if g is None else v * g[:, None, None]).view(M, K)


def _plain_swiglu(h):
    gate, up = h.to(torch.float32).chunk(2, dim=1)
    return ((gate / (1.0 + torch.exp(-gate))) * up).to(torch.bfloat16)


def _plain_scores(z, score):
    """(scores, the same divided by their sum), zero for experts with no finite logit."""
    ok = ~torch.isnan(z) & (z != -math.inf)
    if score == 0:
        top = torch.where(ok, z, torch.full_like(z, -math.inf)).amax(dim=1, keepdim=True)
        e = torch.where(ok, torch.exp(z - top), torch.zeros_like(z))
        p = e / (e.sum(dim=1, keepdim=True) + TINY)
        return ok, p, p
    s = torch.where(ok, 1.0 / (1.0 + torch.exp(-z)), torch.zeros_like(z))
    return ok, s, s / (s.sum(dim=1, keepdim=True) + TINY)


def _plain_route(z, bias, valid, score, k):
    if valid is not None:
        z = torch.where((valid != 0)[:, None], z, torch.full_like(z, -math.inf))
    ok, s, p = _plain_scores(z, score)
    # scores rise with the logits: without a bias the choice goes by the logits themselves
    key = s + bias if bias is not None else z
    key = torch.where(ok, key, torch.full_like(z, -math.inf))
    top = torch.sort(key, dim=1, descending=True, stable=True)
    idx, has = top.indices[:, :k], ok.gather(1, top.indices[:, :k])
    ws = torch.where(has, s.gather(1, idx), torch.zeros((), device=z.device))
    w = ws / (ws.sum(dim=1, keepdim=True) + TINY) * SCALE
    return ok, s, p, torch.where(has, idx, -1).to(torch.int32), w


def _plain_layout(idx, E):
    """(offsets [E + 1], row_token [cap], row_of [T, k]): the chosen pairs by expert, then by token, each
    expert's segment padded to a multiple of 128 rows."""
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, order.values, torch.ones_like(flat))
    first = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + 127) // 128 * 128
    offsets = torch.cat([padded.new_zeros(1), torch.cumsum(padded, 0)])
    here = order.values < E
    at = offsets[order.values] + torch.arange(T * k, device=idx.device) - first[order.values]
    cap = _rows_cap(T, E, k)
    row_token = torch.full((cap + 1,), -1, dtype=torch.int32, device=idx.device)
    row_token.scatter_(0, torch.where(here, at, cap), torch.where(here, order.indices // k, -1).to(torch.int32))
    row_of = torch.empty(T * k, dtype=torch.int64, device=idx.device)
    row_of.scatter_(0, order.indices, torch.where(here, at, -1))
    return offsets.to(torch.int32), row_token[:cap], row_of.view(T, k).to(torch.int32)


def _plain_train(s):
    z, seq, T, E, k, S, score = s["logits"].to(torch.float32), s["seq"], s["T"], s["E"], s["k"], s["S"], s["score"]
    ok, sc, p, idx, w = _plain_route(z, s["bias"], s["valid"], score, k)
    of = torch.bucketize(torch.arange(T, device=z.device, dtype=torch.int32), seq[1:], right=True)
    live = ok.any(dim=1)
    tokens = torch.zeros(S, dtype=torch.int32, device=z.device).scatter_add_(0, of, live.to(torch.int32))
    has = idx >= 0
    at = torch.where(has, of[:, None] * E + idx, S * E).reshape(-1)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=z.device)
    counts = counts.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:-1].view(S, E)
    n = tokens.to(torch.float32).clamp(min=1.0)[:, None]
    mean = (of[None, :] == torch.arange(S, device=z.device)[:, None]).to(torch.float32) @ p / n
    load = counts.to(torch.float32) * (E / k) / n
    loss = (load * mean).sum() * (ALPHA / S)
    # gradients: of the loss through the mean score (the load is a count), of the gate weights through theirs
    dp = (load / n * (ALPHA / S) * s["dloss"])[of]
    c = torch.where(has, idx, 0).long()
    ws = torch.where(has, sc.gather(1, c), torch.zeros((), device=z.device))
    total = ws.sum(dim=1, keepdim=True) + TINY
    dw = torch.where(has, s["dw"], torch.zeros((), device=z.device))
    dws = SCALE / total * (dw - (dw * ws).sum(dim=1, keepdim=True) / total)
    ds = torch.zeros_like(z).scatter_add_(1, c, torch.where(has, dws, torch.zeros((), device=z.device)))
    if score == 0:
        ds = ds + dp
        dz = p * (ds - (ds * p).sum(dim=1, keepdim=True))
    else:
        all_ = sc.sum(dim=1, keepdim=True) + TINY
        ds = ds + (dp - (dp * p).sum(dim=1, keepdim=True)) / all_
        dz = ds * sc * (1.0 - sc)
    dz = torch.where(ok, dz, torch.zeros_like(dz))
    return {"idx": idx, "w": w, "counts": counts, "tokens": tokens, "loss": loss.view(1), "dlogits": dz.to(s["logits"].dtype)}


def _run_plain(s):
    op = s["op"]
    if op == "quantise":
        x = s["x"]
        if s["source"] == "gather":
            x = x[s["rows"].clamp(min=0)]
        elif s["source"] == "swiglu":
            x = _plain_swiglu(x)
        q, sf, g = _plain_quantise(x, s["fmt"], s["rows"])
        out = _plain_dequantise(q, sf, g, s["fmt"]).to(torch.bfloat16)
        return {"values": out, "scales": sf.view(torch.float8_e4m3fn if s["fmt"] == 0 else torch.float8_e8m0fnu), "row": g}
    if op == "product":
        a, b = _plain_dequantise(*s["a"], s["fmt"]), _plain_dequantise(*s["b"], s["fmt"])
        return {"d": (a @ b.t()).to(s["out"].dtype)}
    if op == "experts":
        a = _plain_dequantise(*s["a"], s["fmt"])
        d = torch.zeros_like(s["out"])
        at = s["bounds"]
        for e in range(s["E"]):          # segments differ in length: one product each
            if at[e + 1] > at[e]:
                b = _plain_dequantise(*(t[e] if t is not None else None for t in s["b"]), s["fmt"])
                d[at[e]:at[e + 1]] = (a[at[e]:at[e + 1]] @ b.t()).to(d.dtype)
        return {"d": d}
    if op == "route":
        _, _, _, idx, w = _plain_route(s["logits"].to(torch.float32), s["bias"], None, s["score"], s["k"])
        offsets, row_token, row_of = _plain_layout(idx, s["E"])
        return {"idx": idx, "w": w, "offsets": offsets, "row_token": row_token, "row_of": row_of}
    return _plain_train(s)


# ------------------------------------------------------------------------------------ the package's calls

def _run_own(s):
    import fp8_fine_grained_fp8bs_gb300 as fp8bs
    op = s["op"]
    if op == "quantise":
        x, q, sf, g, fmt, M, K = s["x"], s["q"], s["sf"], s["g"], s["fmt"], s["M"], s["K"]
        if s["source"] == "swiglu":
            fp8bs.fp8bs_swiglu_quantize_fp4(x, M, K, 2 * K, s["rows"], fmt, q, sf, g)
        else:
            fp8bs.fp8bs_quantize_fp4(x, x.shape[0], K, K, s["rows"], M, fmt, q, sf, g)
        fp8bs.fp8bs_dequantize_fp4(q, sf, g, M, K, fmt, s["out"], fp8bs.OUT_BF16, K)
        return {"values": s["out"], "scales": sf.view(torch.float8_e4m3fn if fmt == 0 else torch.float8_e8m0fnu), "row": g}
    if op == "product":
        dt = fp8bs.OUT_F32 if s["f32"] else fp8bs.OUT_BF16
        fp8bs.fp8bs_gemm_fp4(*s["a"], *s["b"], s["fmt"], s["out"], dt, s["M"], s["N"], s["K"])
        return {"d": s["out"]}
    if op == "experts":
        fp8bs.fp8bs_grouped_gemm_fp4(*s["a"], s["out"].shape[0], s["offsets"], s["E"], *s["b"], s["fmt"], s["out"],
                                     fp8bs.OUT_BF16, s["N"], s["K"])
        return {"d": s["out"]}
    dt = fp8bs.IN_F32 if s["dtype"] == "f32" else fp8bs.IN_BF16
    T, E, k = s["T"], s["E"], s["k"]
    if op == "route":
        fp8bs.fp8bs_moe_route(s["logits"], dt, T, E, E, s["score"], s["bias"], None, None, 1, k, 1, SCALE, 0.0, s["idx"],
                              s["w"], None, None, None, None, 0)
        fp8bs.fp8bs_moe_layout(s["idx"], T, k, E, s["offsets"], s["row_token"], s["row_token"].numel(), s["row_of"], s["ws"],
                               s["ws"].numel())
        return {n: s[n] for n in ("idx", "w", "offsets", "row_token", "row_of")}
    fp8bs.fp8bs_moe_route(s["logits"], dt, T, E, E, s["score"], s["bias"], s["valid"], s["seq"], s["S"], k, 1, SCALE, ALPHA,
                          s["idx"], s["w"], s["counts"], s["tokens"], s["loss"], s["ws"], s["ws"].numel())
    fp8bs.fp8bs_moe_route_backward(s["logits"], dt, T, E, E, s["score"], s["valid"], s["seq"], s["S"], k, 1, SCALE, ALPHA,
                                   s["idx"], s["counts"], s["tokens"], s["dw"], s["dloss"], s["dlogits"], E)
    return {n: s[n] for n in ("idx", "w", "counts", "tokens", "loss", "dlogits")}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------- work

def _code_bytes(M, K, fmt):
    return M * (K // 2 + _groups(K, fmt) + (4 if fmt == 0 else 0))


def work(case):
    op = case["op"]
    if op == "quantise":
        M, K, fmt = case["M"], case["K"], case["fmt"]
        rows_in = max(1, M // 9) if case["source"] == "gather" else M
        read = rows_in * K * 2 * (2 if case["source"] == "swiglu" else 1) + (0 if case["source"] == "rows" else 4 * M)
        return {"bytes": read + _code_bytes(M, K, fmt) + 2 * M * K, "flops": 4 * M * K}
    if op == "product":
        M, N, K, fmt = (case[n] for n in ("M", "N", "K", "fmt"))
        return {"bytes": _code_bytes(M, K, fmt) + _code_bytes(N, K, fmt) + M * N * (4 if case["f32"] else 2),
                "flops": 2 * M * N * K}
    if op == "experts":
        T, E, k, N, K, fmt = (case[n] for n in ("T", "E", "k", "N", "K", "fmt"))
        used = min(E, T * k)
        return {"bytes": T * k * _code_bytes(1, K, fmt) + used * _code_bytes(N, K, fmt) + T * k * N * 2,
                "flops": 2 * T * k * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    z = T * E * (4 if case["dtype"] == "f32" else 2)
    if op == "route":
        return {"bytes": z + T * k * 12 + 4 * _rows_cap(T, E, k) + 4 * (E + 1), "flops": 8 * T * E}
    return {"bytes": 2 * z + T * (1 + k * 12) + case["S"] * E * 4, "flops": 24 * T * E}


# ------------------------------------------------------------------------------------------- in 64 bits

def _codes_64(q):
    """E2M1 from its bits: sign, two of exponent (bias 1), one of mantissa."""
    both = torch.cat([(q & 15).unsqueeze(-1), (q >> 4).unsqueeze(-1)], dim=-1).flatten(-2).to(torch.float64)
    sign = torch.where(both >= 8, -1.0, 1.0).to(torch.float64)
    low = both % 8
    e, m = torch.floor(low / 2), low % 2
    return sign * torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)


def _scales_64(sf, M, K, fmt):
    J = _groups(K, fmt)
    r, j = torch.arange(M, device=sf.device)[:, None], torch.arange(J, device=sf.device)[None, :]
    at = ((r // 128) * ((J + 3) // 4) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    b = sf[at].to(torch.float64)
    if fmt == 1:
        return torch.exp2(b - 127)
    e, m = torch.floor(b / 8), b % 8
    return torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m * 2.0 ** -9)


def _matrix_64(q, sf, g, fmt):
    M, K = q.shape[0], 2 * q.shape[1]
    v = _codes_64(q) * _scales_64(sf, M, K, fmt).repeat_interleave(16 if fmt == 0 else 32, dim=1)
    return v if g is None else v * g.to(torch.float64)[:, None]


def _nearest_64(v, bits, low, top):
    """|v| on the grid of `bits` mantissa bits, exponents from `low`, largest value `top`; ties to even."""
    a = v.abs()
    _, e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))
    step = torch.exp2((e.to(torch.float64) - 1).clamp(min=low) - bits)
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=top)


def _quantise_64(x, fmt, rows):
    M, K = x.shape
    if rows is not None:
        x = x * (rows >= 0).to(x.dtype)[:, None]
    x = x.view(M, _groups(K, fmt), -1)
    amax = x.abs().amax(2)
    if fmt == 0:
        g = torch.clamp(amax.amax(1) / 2688, min=2.0 ** -100)
        s = _nearest_64(amax / (6 * g[:, None]), 3, -6, 448.0)
        d = s * g[:, None]
    else:
        g = None
        s = torch.exp2(torch.ceil(torch.log2(torch.clamp(amax, min=6 * 2.0 ** -127) / 6)).clamp(-127, 127))
        d = s
    safe = torch.where(d > 0, d, torch.ones_like(d))[:, :, None]
    code = _nearest_64(torch.where((d > 0)[:, :, None], x / safe, torch.zeros_like(x)), 1, 0, 6.0)
    blocks = torch.full(((M + 127) // 128 * 128, (s.shape[1] + 3) // 4 * 4), 0.0 if fmt == 0 else 2.0 ** -127,
                        dtype=torch.float64, device=x.device)
    blocks[:M, :s.shape[1]] = s
    r = torch.arange(blocks.numel(), device=x.device)
    block, inside = r // 512, r % 512
    per = blocks.shape[1] // 4
    row = block // per * 128 + inside % 16 // 4 * 32 + inside // 16
    return {"values": (code * d[:, :, None]).view(M, K), "scales": blocks[row, block % per * 4 + inside % 4], "row": g}


def _scores_64(z, score):
    ok = torch.isfinite(z)
    if score == 0:
        p = torch.softmax(torch.where(ok, z, torch.full_like(z, -math.inf)), dim=1)
        p = torch.where(ok, p, torch.zeros_like(p))
        return ok, p, p
    s = torch.where(ok, torch.sigmoid(z), torch.zeros_like(z))
    return ok, s, s / (s.sum(1, keepdim=True) + TINY)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        x = s["x"].to(torch.float64)
        if case["source"] == "gather":
            x = x[s["rows"].clamp(min=0).long()]
        elif case["source"] == "swiglu":
            a, b = x[:, :case["K"]], x[:, case["K"]:]
            x = (a * torch.sigmoid(a) * b).to(torch.float32).to(torch.bfloat16).to(torch.float64)
        return _quantise_64(x, case["fmt"], s["rows"])
    if op == "product":
        return {"d": _matrix_64(*s["a"], case["fmt"]) @ _matrix_64(*s["b"], case["fmt"]).t()}
    if op == "experts":
        a = _matrix_64(*s["a"], case["fmt"])
        d = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                d[lo:hi] = a[lo:hi] @ _matrix_64(*(t[e] if t is not None else None for t in s["b"]), case["fmt"]).t()
        return {"d": d}
    z, k, E = s["logits"].to(torch.float64), case["k"], case["E"]
    if op == "train":
        z = z.masked_fill(s["valid"][:, None] == 0, -math.inf)
    ok, sc, p = _scores_64(z, case["score"])
    key = sc + s["bias"].to(torch.float64) if case["bias"] else z
    idx = torch.sort(key.masked_fill(~ok, -math.inf), dim=1, descending=True, stable=True).indices[:, :k]
    one = torch.zeros_like(z).scatter_(1, idx, 1.0) * ok           # the choice, as a 0/1 matrix
    total = (sc * one).sum(1, keepdim=True) + TINY
    w = (sc * one).gather(1, idx) / total * SCALE
    if op == "route":
        return {"idx": None, "w": w, "offsets": None, "row_token": None, "row_of": None}
    S, T = case["S"], case["T"]
    seq = s["seq"].to(torch.float64)
    t = torch.arange(T, device=DEV, dtype=torch.float64)[None, :]
    member = ((t >= seq[:-1, None]) & (t < seq[1:, None])).to(torch.float64)
    n = (member @ ok.any(1).to(torch.float64)).clamp(min=1)[:, None]
    load, mean = member @ one * E / (k * n), member @ p / n
    loss = ALPHA / S * (load * mean).sum()
    # d loss / d p, then through p = s / sum(s); d w / d s of the chosen ones
    dp = ALPHA / S * (member.t() @ (load / n)) * s["dloss"].to(torch.float64)
    dw = torch.zeros_like(z).scatter_(1, idx, s["dw"].to(torch.float64)) * one
    ds = one * SCALE / total * (dw - (dw * sc).sum(1, keepdim=True) / total)
    if case["score"] == 0:
        u = ds + dp
        dz = p * (u - (u * p).sum(1, keepdim=True))
    else:
        u = ds + (dp - (dp * p).sum(1, keepdim=True)) / (sc.sum(1, keepdim=True) + TINY)
        dz = u * sc * (1 - sc)
    return {"idx": None, "w": w, "counts": None, "tokens": None, "loss": loss.view(1), "dlogits": dz * ok}

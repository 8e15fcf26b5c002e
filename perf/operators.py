"""The router, expert and few-token operators as cases to time and compare.

Five operators around the dispatch and combine of this library:

  route    logits -> top-k ids and softmax weights (group-limited or not), and the gradient to the logits
  gemm     rows of each expert's segment times that expert's FP8 weights, 1 x 128 row scales and 128 x 128
           weight scales, forward or (transpose) as the gradient to the rows
  swiglu   the gate and up products of a segment's rows, SwiGLU and the E4M3 block quantisation of the result
  wgrad    the gradient of each expert's weights from bf16 rows
  layer    a whole mixture-of-experts layer for a few tokens

`run` computes them in plain torch operations in fp32, or, with `own`, through the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128
MOST_BYTES, MOST_FLOPS = 7.6e9, 3.9e12


# ---------------------------------------------------------------- cases

def listed():
    return [
        # router of a decode batch: latency alone
        dict(name="route_decode", op="route", T=1024, E=256, k=8, groups=1, keep=1, dtype="f32", masked=False, backward=False),
        # router of a training step: group-limited choice, some experts masked out, and the gradient
        dict(name="route_train", op="route", T=16384, E=128, k=8, groups=8, keep=4, dtype="bf16", masked=True, backward=True),
        # down projection of a decode step: about 32 rows an expert, bound by the weights
        dict(name="gemm_decode", op="gemm", N=2048, E=64, K=2048, M=7168, skew=0.0, transpose=False, dtype="bf16"),
        # down projection of a prefill step: uneven segments
        dict(name="gemm_prefill", op="gemm", N=65536, E=256, K=2048, M=7168, skew=0.25, transpose=False, dtype="bf16"),
        # gradient to the rows of a down projection in training: few large experts, weights read the other way, odd sizes
        dict(name="gemm_dgrad", op="gemm", N=32771, E=8, K=4096, M=2064, skew=0.5, transpose=True, dtype="bf16"),
        # gate and up products of a short batch: segments of a few rows, some of none
        dict(name="swiglu_short", op="swiglu", N=72, E=32, K=4096, M=1024, skew=0.5),
        # gate and up products of a prefill step
        dict(name="swiglu_prefill", op="swiglu", N=65536, E=128, K=7168, M=2048, skew=0.25),
        # weight gradient of a small expert: segments that end inside a tile, an expert without rows
        dict(name="wgrad_small", op="wgrad", N=1500, E=8, K=1024, M=720, skew=1.0),
        # weight gradient of a training step
        dict(name="wgrad_train", op="wgrad", N=32768, E=16, K=7168, M=4096, skew=0.25),
        # one token through a layer of 256 FP8 experts: the latency of decoding a single sequence
        dict(name="layer_one", op="layer", T=1, E=256, k=8, H=7168, I=2048, weights="fp8"),
        # a small decode batch on bf16 experts, every expert in use
        dict(name="layer_bf16", op="layer", T=16, E=8, k=2, H=4096, I=1784, weights="bf16"),
        # the largest batch of the few-token form
        dict(name="layer_batch", op="layer", T=61, E=128, k=8, H=4096, I=1408, weights="fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    while True:
        v = max(step, _log(rng, lo, hi) // step * step)
        if v not in (3072, 1536):
            return v


def draw(rng):
    op = rng.choice(["route", "gemm", "gemm", "swiglu", "wgrad", "layer", "layer"])
    while True:
        if op == "route":
            groups = rng.choice([1, 1, 4, 8])
            E = groups * rng.randint(max(1, 8 // groups), 384 // groups)
            keep = rng.randint((groups + 1) // 2, groups)
            k = rng.randint(1, min(10, E // groups * keep))
            c = dict(op=op, T=_log(rng, 1, 65536), E=E, k=k, groups=groups, keep=keep, dtype=rng.choice(["f32", "bf16"]),
                     masked=rng.random() < 0.5, backward=rng.random() < 0.5)
        elif op == "layer":
            fp8 = rng.random() < 0.6
            step = 128 if fp8 else 8
            E = _log(rng, 4, 256)
            c = dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), H=_size(rng, 512, 7168, step), I=_size(rng, 256, 4096, step),
                     weights="fp8" if fp8 else "bf16")
        else:
            E = _log(rng, 1, 128)
            M = _size(rng, 256, 4096, 128) if op == "swiglu" else _size(rng, 128, 8192, 16)
            c = dict(op=op, N=_log(rng, 1, 49152), E=E, K=_size(rng, 256, 7168, 16 if op == "wgrad" else 128), M=M, skew=rng.choice([0.0, 0.25, 0.5]))
            if op == "gemm":
                c.update(transpose=rng.random() < 0.4, dtype="bf16")
        w = work(c)
        if w["bytes"] <= MOST_BYTES / 2 and w["flops"] <= MOST_FLOPS / 4:
            return c


def _touched(E, picks, per=1):
    """Expected experts in use."""
    return E * (1 - (1 - per / E) ** picks)


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        b = c["T"] * c["E"] * size + c["T"] * c["k"] * 8
        if c["backward"]:  # ids, weights and their gradient in, the logits' gradient out
            b += c["T"] * c["k"] * 4 + c["T"] * c["E"] * size
        return {"bytes": b, "flops": 4.0 * c["T"] * c["E"]}
    if c["op"] == "layer":
        each = 3 * c["H"] * c["I"] * (1 + 4 / BLOCK ** 2 if c["weights"] == "fp8" else 2)
        return {"bytes": _touched(c["E"], c["T"], c["k"]) * each + 4 * c["T"] * c["H"] + 8 * c["T"] * c["k"], "flops": 6.0 * c["T"] * c["k"] * c["H"] * c["I"]}
    N, E, K, M = c["N"], c["E"], c["K"], c["M"]
    if c["op"] == "wgrad":
        return {"bytes": 2 * N * (K + M) + 4 * E * M * K, "flops": 2.0 * N * K * M}
    wide = 2 * M if c["op"] == "swiglu" else M
    out = N * M * (1 + 4 / BLOCK) if c["op"] == "swiglu" else N * M * 2
    return {"bytes": N * K * (1 + 4 / BLOCK) + _touched(E, N) * wide * K * (1 + 4 / BLOCK ** 2) + out, "flops": 2.0 * N * K * wide}


# ---------------------------------------------------------------- inputs

def _codes_and_scales(w):
    """E4M3 codes and fp32 scales of 128 x 128 blocks of w [e, rows, cols]."""
    e, r, c = w.shape
    rp, cp = -(-r // BLOCK) * BLOCK, -(-c // BLOCK) * BLOCK
    p = torch.nn.functional.pad(w, (0, cp - c, 0, rp - r)).view(e, rp // BLOCK, BLOCK, cp // BLOCK, BLOCK)
    s = p.abs().amax(dim=(2, 4)) / 448.0
    q = (p / s[:, :, None, :, None]).view(e, rp, cp)[:, :r, :c]
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s


def _weights(g, E, rows, cols, fan):
    """Quantised expert weights: normal values, a few experts at a time."""
    q = torch.empty((E, rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, -(-rows // BLOCK), -(-cols // BLOCK)), device="cuda")
    step = max(1, (1 << 28) // (rows * cols))
    for e in range(0, E, step):
        n = min(step, E - e)
        q[e:e + n], s[e:e + n] = _codes_and_scales(torch.randn((n, rows, cols), generator=g, device="cuda") * fan ** -0.5)
    return q, s


def _weights_bf16(g, E, rows, cols, fan):
    w = torch.empty((E, rows, cols), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = torch.randn((rows, cols), generator=g, device="cuda") * fan ** -0.5
    return w


def _rows_fp8(g, N, K):
    """Activations whose channels differ in size, as E4M3 codes and fp32 scales of 1 x 128 blocks."""
    x = torch.randn((N, K), generator=g, device="cuda") * torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5)
    b = x.view(N, K // BLOCK, BLOCK)
    s = b.abs().amax(2) / 448.0
    return (b / s[:, :, None]).view(N, K).to(torch.float8_e4m3fn).view(torch.uint8), s


def _segments(g, N, E, skew):
    """Offsets of the experts' segments of N rows, and the longest segment."""
    p = (1.0 + torch.randperm(E, generator=g, device="cuda")) ** -skew
    counts = torch.bincount(torch.multinomial(p, N, replacement=True, generator=g), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, dict(case)
    if c["op"] == "route":
        logits = torch.randn((c["T"], c["E"]), generator=g, device="cuda") * 1.5
        if c["masked"]:  # experts taken out for a token, and tokens with none left
            logits[torch.rand((c["T"], c["E"]), generator=g, device="cuda") < 0.3] = -math.inf
            logits[torch.rand(c["T"], generator=g, device="cuda") < 0.01] = -math.inf
        s["logits"] = logits.to(DTYPES[c["dtype"]])
        s["dw"] = torch.randn((c["T"], c["k"]), generator=g, device="cuda")
    elif c["op"] == "layer":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        s["x"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        top, idx = torch.randn((T, E), generator=g, device="cuda").topk(k, dim=1)
        s["idx"], s["w"] = idx.to(torch.int32), torch.softmax(top, 1)
        if c["weights"] == "fp8":
            s["w13"], s["s13"] = _weights(g, E, 2 * I, H, H)
            s["w2"], s["s2"] = _weights(g, E, H, I, I)
        else:
            s["w13"], s["s13"] = _weights_bf16(g, E, 2 * I, H, H), None
            s["w2"], s["s2"] = _weights_bf16(g, E, H, I, I), None
    else:
        N, E, K, M = c["N"], c["E"], c["K"], c["M"]
        s["offsets"], s["longest"] = _segments(g, N, E, c["skew"])
        if c["op"] == "wgrad":
            s["dy"] = torch.randn((N, M), generator=g, device="cuda").to(torch.bfloat16)
            s["x"] = torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16)
        else:
            s["a"], s["sa"] = _rows_fp8(g, N, K)
            wide = 2 * M if c["op"] == "swiglu" else M
            s["b"], s["sb"] = _weights(g, E, K, M, K) if c.get("transpose") else _weights(g, E, wide, K, K)
    return s


# ---------------------------------------------------------------- the plain forms

def _route(s):
    x = s["logits"].float()
    T, E = x.shape
    if s["groups"] > 1:
        per = x.view(T, s["groups"], -1)
        score = per.topk(min(2, per.shape[2]), dim=2).values.sum(2)
        best = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        allowed = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        x = torch.where(allowed[:, :, None], per, -math.inf).view(T, E)
    top, idx = torch.sort(x, dim=1, descending=True, stable=True)
    top, idx = top[:, :s["k"]], idx[:, :s["k"]]
    e = torch.where(top == -math.inf, 0.0, torch.exp(top - top[:, :1]))
    total = e.sum(1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0)
    if not s["backward"]:
        return idx.to(torch.int32), w
    d = w * (s["dw"] - (w * s["dw"]).sum(1, keepdim=True))
    return idx.to(torch.int32), w, torch.zeros((T, E), device=x.device).scatter_(1, idx, d).to(s["logits"].dtype)


def _values(q, s, rows, cols):
    """fp32 values of codes q [e, r, c] with a scale for each block of rows x cols."""
    f = q.view(torch.float8_e4m3fn).float()
    return f.mul_(s.repeat_interleave(rows, 1)[:, :q.shape[1]].repeat_interleave(cols, 2)[:, :, :q.shape[2]])


def _by_expert(s, *rows):
    """Rows [N, c] as [E, longest, c], zeros behind each segment's end; and where each row went."""
    at = torch.arange(s["N"], device="cuda", dtype=torch.int32)
    e = torch.searchsorted(s["offsets"], at, right=True) - 1
    p = at - s["offsets"][e]
    out = [torch.zeros((s["E"], s["longest"], r.shape[1]), device="cuda") for r in rows]
    [o.index_put_((e, p), r) for o, r in zip(out, rows)]
    return out, e, p


def _product(s):
    a = _values(s["a"][None], s["sa"][None], 1, BLOCK)[0]
    (a,), e, p = _by_expert(s, a)
    b = _values(s["b"], s["sb"], BLOCK, BLOCK)
    return torch.bmm(a, b if s.get("transpose") else b.transpose(1, 2))[e, p]


def _quantise(h):
    b = h.view(h.shape[0], -1, BLOCK)
    top = b.abs().amax(2)
    scale, inv = torch.where(top > 0, top / 448.0, 1.0), torch.where(top > 0, 448.0 / top, 0.0)
    return (b * inv[:, :, None]).view(h.shape).to(torch.float8_e4m3fn), scale


def _layer(s):
    idx, x, T = s["idx"].long(), s["x"].float(), s["T"]
    used, at = torch.unique(idx, return_inverse=True)
    share = torch.zeros((T, used.numel()), device="cuda").scatter_add_(1, at, s["w"])
    w13, w2 = s["w13"][used], s["w2"][used]
    if s["weights"] == "fp8":
        w13, w2 = _values(w13, s["s13"][used], BLOCK, BLOCK), _values(w2, s["s2"][used], BLOCK, BLOCK)
    else:
        w13, w2 = w13.float(), w2.float()
    both = torch.matmul(x, w13.transpose(1, 2))
    gate, up = both[:, :, :s["I"]], both[:, :, s["I"]:]
    h = gate / (1 + torch.exp(-gate)) * up * share.t()[:, :, None]
    return torch.bmm(h, w2.transpose(1, 2)).sum(0).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "route":
        return _route(s)
    if s["op"] == "gemm":
        return _product(s).to(DTYPES[s["dtype"]])
    if s["op"] == "swiglu":
        both = _product(s)
        gate, up = both[:, :s["M"]], both[:, s["M"]:]
        return _quantise(gate / (1 + torch.exp(-gate)) * up)
    if s["op"] == "wgrad":
        (dy, x), _, _ = _by_expert(s, s["dy"].float(), s["x"].float())
        return torch.bmm(dy.transpose(1, 2), x)
    return _layer(s)


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import combine_layout_moe_gb300 as moe

    if s["op"] == "route":
        idx, w = moe.moe_route(s["logits"], s["k"], groups=s["groups"], topk_groups=s["keep"])
        if not s["backward"]:
            return idx, w
        return idx, w, moe.moe_route_backward(idx, w, s["dw"], s["E"], out_dtype=s["logits"].dtype)
    if s["op"] == "gemm":
        return moe.moe_expert_gemm(s["a"], s["sa"], s["offsets"], s["b"], s["sb"], transpose_w=s["transpose"], out_dtype=DTYPES[s["dtype"]])
    if s["op"] == "swiglu":
        h, scale = moe.moe_expert_swiglu(s["a"], s["sa"], s["offsets"], s["b"], s["sb"])
        return h.view(torch.float8_e4m3fn), scale
    if s["op"] == "wgrad":
        return moe.moe_expert_wgrad(s["dy"], s["x"], s["offsets"])
    return moe.moe_layer_few(s["x"], s["idx"], s["w"], s["w13"], s["w2"], w13_scales=s["s13"], w2_scales=s["s2"])


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _wide(q, s, rows, cols):
    """Codes of one expert, or of rows, with their block scales, as float64."""
    v = q.view(torch.float8_e4m3fn).to(torch.float64)
    for i in range(s.shape[0] if rows > 1 else 1):
        part = v[i * rows:(i + 1) * rows] if rows > 1 else v
        factor = s[i:i + 1] if rows > 1 else s
        part *= factor.double().repeat_interleave(cols, 1)[:, :v.shape[1]]
    return v


def _silu(g):
    return g * torch.sigmoid(g)


def _exact_route(s):
    x = s["logits"].double()
    T, E = x.shape
    if s["groups"] > 1:
        size = E // s["groups"]
        score = torch.stack([x[:, i * size:(i + 1) * size].sort(1, descending=True).values[:, :2].sum(1) for i in range(s["groups"])], 1)
        order = torch.argsort(-score.float().double(), dim=1, stable=True)
        for j in range(s["keep"], s["groups"]):
            for i in range(s["groups"]):
                x[:, i * size:(i + 1) * size].masked_fill_((order[:, j] == i)[:, None], -math.inf)
    idx = torch.argsort(-x, dim=1, stable=True)[:, :s["k"]]
    w = torch.softmax(x.gather(1, idx), 1).nan_to_num(0.0)  # a row with nothing left has no weights
    if not s["backward"]:
        return None, w
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    d = (jac @ s["dw"].double()[:, :, None])[:, :, 0]
    full = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    for j in range(s["k"]):
        full[torch.arange(T, device="cuda"), idx[:, j]] = d[:, j]
    return None, w, full


def exact(case, seed):
    if work(case)["flops"] > 8e12:  # too long in 64 bits
        return None
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "layer":
        out = torch.zeros((s["T"], s["H"]), dtype=torch.float64, device="cuda")
        for e in s["idx"].unique().tolist():
            t, j = (s["idx"] == e).nonzero(as_tuple=True)
            w13 = _wide(s["w13"][e], s["s13"][e], BLOCK, BLOCK) if s["s13"] is not None else s["w13"][e].double()
            w2 = _wide(s["w2"][e], s["s2"][e], BLOCK, BLOCK) if s["s2"] is not None else s["w2"][e].double()
            both = s["x"][t].double() @ w13.t()
            y = (_silu(both[:, :s["I"]]) * both[:, s["I"]:]) @ w2.t()
            out.index_add_(0, t, y * s["w"][t, j].double()[:, None])
        return out
    ends = s["offsets"].tolist()
    if s["op"] == "wgrad":
        dw = torch.zeros((s["E"], s["M"], s["K"]), dtype=torch.float64, device="cuda")
        for e in range(s["E"]):
            dw[e] = s["dy"][ends[e]:ends[e + 1]].double().t() @ s["x"][ends[e]:ends[e + 1]].double()
        return dw
    swiglu = s["op"] == "swiglu"
    out = torch.zeros((s["N"], s["M"]), dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        a, b = _wide(s["a"][lo:hi], s["sa"][lo:hi], 1, BLOCK), _wide(s["b"][e], s["sb"][e], BLOCK, BLOCK)
        y = a @ (b if s.get("transpose") else b.t())
        out[lo:hi] = _silu(y[:, :s["M"]]) * y[:, s["M"]:] if swiglu else y
    if not swiglu:
        return out
    # the codes are numbers of 8 bits: rounded from the 64-bit values as the recipe says
    b = out.view(s["N"], -1, BLOCK)
    top = b.abs().amax(2)
    codes = (b * (448.0 / top)[:, :, None]).view(s["N"], s["M"]).float().to(torch.float8_e4m3fn).double()
    return codes, top / 448.0

"""More serving operators of a decoder block on the multi-LoRA linear, in plain form and as calls
of the library.

quant  rows in 8-bit integers with a scale per row, as they are or behind a norm:
       p = x, or p = fp32(fp32(x + residual) * weight);  top = max|p|
       y8 = rint(127 p / top) (ties to even);  s = max(top', 2^-60) / 127, top' = top, or behind the
       norm top / sqrt(mean(h^2) + eps), h = x + residual
int8   the layer on 8-bit integers, x = x_scale[m] x8[m], W = w_scale[c] W8[c]:
       y = act(x W + scale_i (x A_i) B_i + bias) * mul + residual,   i = ids[m], -1: no adapter
moe    a whole mixture-of-experts layer; e = topk_ids[m][j] (-1: none), i = ids[m], P_i[e] an
       expert's projection with its adapter, v P_i[e] = v W[e] + scale_i (v A[i][e]) B[i][e]:
       y[m] = residual[m] + sum_j topk_w[m][j] (act(x Gate_i[e]) * (x Up_i[e])) Down_i[e]
rope   rotary positions of q and k: the pair k of a head turns by the angle 2 pi pos f_k, times factor

Layouts are those of include/lora.h: W8[d_out, d_in], W[E, d_in, d_out], A[n, (E,) d_in, r_max],
B[n, (E,) r_max, d_out]; q and k [M, heads, head_dim] with a stride between rows.
"""

import math

import torch

own = False

EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------------


def listed():
    return [
        # one token in front of 8-bit projections: launch and latency only
        dict(name="quant_1_norm", op="quant", M=1, d=4096, norm=True, residual=True, weight=True, both=False),
        # a long prompt's silu(gate) * up in front of the 8-bit down projection
        dict(name="quant_4096_wide", op="quant", M=4096, d=11008, norm=False, residual=False,
             weight=False, both=False),
        # single-token decode through the down projection, residual added
        dict(name="int8_1_down", op="int8", M=1, K=11008, N=4096, n=8, r_max=16, act="none",
             bias=False, mul=False, residual=True, y="bf16"),
        # a decode batch through the gate projection: silu(gate) * up
        dict(name="int8_40_gate", op="int8", M=40, K=4096, N=11008, n=32, r_max=16, act="silu",
             bias=False, mul=True, residual=False, y="bf16"),
        # a wide decode batch, odd everywhere: rows, widths, a rank that is no power of two; fp32
        dict(name="int8_333_odd_f32", op="int8", M=333, K=4112, N=2760, n=128, r_max=24, act="none",
             bias=True, mul=False, residual=False, y="f32"),
        # a prompt through the down projection
        dict(name="int8_4096_down", op="int8", M=4096, K=11008, N=4096, n=8, r_max=16, act="none",
             bias=False, mul=False, residual=True, y="bf16"),
        # one token: four of 32 experts
        dict(name="moe_1", op="moe", M=1, top_k=4, E=32, d=2880, ff=2880, n=8, r_max=16, act="silu",
             residual=True, holes=False, y="bf16"),
        # a decode batch that meets every expert
        dict(name="moe_64", op="moe", M=64, top_k=4, E=32, d=2880, ff=2880, n=8, r_max=16, act="silu",
             residual=True, holes=False, y="bf16"),
        # odd rows and widths, many adapters, slots without an expert; fp32
        dict(name="moe_23_odd_f32", op="moe", M=23, top_k=2, E=8, d=1040, ff=2768, n=40, r_max=24,
             act="gelu", residual=False, holes=True, y="f32"),
        # one token's queries and keys
        dict(name="rope_1", op="rope", M=1, hq=32, hk=8, D=128, rot=128, layout="half", scaling="none",
             far=4096, inverse=False, y="bf16"),
        # a long prompt
        dict(name="rope_8192", op="rope", M=8192, hq=32, hk=8, D=128, rot=128, layout="half",
             scaling="yarn", far=131072, inverse=False, y="bf16"),
        # part of the head, interleaved pairs, far positions, fp32; the gradient's direction
        dict(name="rope_1021_part_f32", op="rope", M=1021, hq=12, hk=3, D=104, rot=52,
             layout="interleaved", scaling="linear", far=1000000, inverse=True, y="f32"),
    ]


def _log(rng, lo, hi):
    return min(int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))), hi)


def draw(rng):
    op = rng.choice(["quant", "int8", "moe", "rope"])
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    if op == "quant":
        d = 8 * _log(rng, 16, 1376)
        M = min(_log(rng, 1, 8192), 4096 * 11008 // (2 * d))
        norm = rng.random() < 0.6
        return dict(op=op, M=M, d=d, norm=norm, residual=norm and rng.random() < 0.7,
                    weight=norm and rng.random() < 0.9, both=norm and rng.random() < 0.3)
    y = "f32" if rng.random() < 0.25 else "bf16"
    if op == "int8":
        K, N = 16 * _log(rng, 16, 688), 8 * _log(rng, 16, 1376)
        M = max(1, min(_log(rng, 1, 4096), 4096 * 4096 * 4096 // (K * N)))
        r_max = _log(rng, 1, 64)
        return dict(op=op, M=M, K=K, N=N, n=min(_log(rng, 1, 512), 4096 // r_max), r_max=r_max,
                    act=rng.choice(acts), bias=rng.random() < 0.5, mul=rng.random() < 0.3,
                    residual=rng.random() < 0.5, y=y)
    if op == "moe":
        d, ff = 16 * _log(rng, 16, 180), 16 * _log(rng, 16, 180)
        E = min(_log(rng, 2, 64), 24 * 2880 * 2880 // (d * ff))
        top_k = rng.randint(1, min(E, 8))
        r_max = 8 * _log(rng, 1, 8)
        M = min(_log(rng, 1, 128), 512 // top_k)
        return dict(op=op, M=M, top_k=top_k, E=E, d=d, ff=ff, n=min(_log(rng, 1, 64), 512 // r_max),
                    r_max=r_max, act=rng.choice(acts), residual=rng.random() < 0.5,
                    holes=rng.random() < 0.3, y=y)
    D = 8 * rng.randint(4, 32)
    hq = _log(rng, 1, 64)
    hk = rng.choice([0, 1, max(1, hq // 4), hq])
    M = max(1, min(_log(rng, 1, 8192), 8192 * 40 * 64 // ((hq + hk) * D)))
    return dict(op=op, M=M, hq=hq, hk=hk, D=D, rot=rng.choice([D, 2 * rng.randint(1, D // 2)]),
                layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]), far=_log(rng, 64, 1000000),
                inverse=rng.random() < 0.3, y=y)


# ---- inputs ----------------------------------------------------------------------------------


def _quantised(v):
    """8-bit integers of the rows of v and the scale of each row."""
    s = v.abs().amax(1) / 127.0
    return (v / s[:, None]).round_().to(torch.int8), s


def _pool(normal, ranks, r, K, N, *expert):
    """A and B of n adapters (for each expert): rank rows past an adapter's own are zero."""
    n = len(ranks)
    kept = torch.arange(r, device="cuda") < ranks[:, None]
    if expert:
        kept = kept[:, None]
    A = (normal(n, *expert, K, r, std=K ** -0.5) * kept[..., None, :]).bfloat16()
    B = (normal(n, *expert, r, N, std=0.5 * r ** -0.5) * kept[..., None]).bfloat16()
    return A, B


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=g, dtype=torch.int32)

    out_type = torch.float32 if case.get("y") == "f32" else torch.bfloat16
    if case["op"] == "quant":
        M, d = case["M"], case["d"]
        # hidden states have a few channels far above the others
        loud = 1.0 + 15.0 * (torch.rand(d, device="cuda", generator=g) < 0.005)
        return dict(
            x=(normal(M, d, std=0.5) * loud).bfloat16(),
            residual=(normal(M, d, std=2.0) * loud).bfloat16() if case["residual"] else None,
            weight=(1.0 + normal(d, std=0.2)).bfloat16() if case["weight"] else None)

    if case["op"] == "rope":
        M, hq, hk, D = (case[k] for k in ("M", "hq", "hk", "D"))
        # q and k lie in one row of q, k and v, as one projection writes them
        qkv = normal(M, (hq + 2 * hk) * D).to(out_type)
        first = ints(0, case["far"], 1)
        return dict(qkv=qkv, positions=first + torch.arange(M, device="cuda", dtype=torch.int32))

    M, n, r = (case[k] for k in ("M", "n", "r_max"))
    ranks = ints(1, r + 1, n)
    ranks[0] = r
    s = dict(scale=16.0 / ranks.float(), ranks=ranks, ids=ints(-1, n, M))
    if case["op"] == "int8":
        K, N = case["K"], case["N"]
        s["A"], s["B"] = _pool(normal, ranks, r, K, N)
        s["x8"], s["x_scale"] = _quantised(normal(M, K))
        s["W8"], s["w_scale"] = _quantised(normal(N, K, std=K ** -0.5))
        s.update(bias=normal(N, std=0.5).bfloat16() if case["bias"] else None,
                 mul=normal(M, N).to(out_type) if case["mul"] else None,
                 residual=normal(M, N).to(out_type) if case["residual"] else None)
        return s
    E, k, d, ff = (case[k] for k in ("E", "top_k", "d", "ff"))
    # the router's choice: top_k different experts, their weights adding up to 1
    score = torch.rand(M, E, device="cuda", generator=g)
    top = score.topk(k, 1)
    s["topk_ids"] = top.indices.int()
    s["topk_w"] = torch.softmax(4.0 * top.values, 1)
    if case["holes"]:
        s["topk_ids"][torch.rand(M, k, device="cuda", generator=g) < 0.2] = -1
    s["x"] = normal(M, d).bfloat16()
    for p, (a, b) in dict(g=(d, ff), u=(d, ff), d=(ff, d)).items():
        s["W" + p] = torch.empty(E, a, b, dtype=torch.bfloat16, device="cuda").normal_(0.0, a ** -0.5, generator=g)
        s["A" + p], s["B" + p] = _pool(normal, ranks, r, a, b, E)
    s["residual"] = normal(M, d).to(out_type) if case["residual"] else None
    return s


def _freqs(case):
    """Turns per position of each pair of a head (64 bits) and the factor of the rotated values."""
    rot, base, s, length = case["rot"], 10000.0, 8.0, 4096.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    factor = 1.0
    if case["scaling"] == "ntk":
        base = base * s ** (rot / max(rot - 2, 1))
    f = base ** (-2.0 * i / rot) / (2.0 * math.pi)
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "yarn":
        kept = ((length * f - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f / s * (1.0 - kept) + f * kept
        factor = 0.1 * math.log(s) + 1.0
    return f, factor


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "rope":
        f, s["factor"] = _freqs(case)
        s["freqs"] = f.cuda()
    if own:
        s["call"] = {"quant": _own_quant, "int8": _own_int8, "moe": _own_moe, "rope": _own_rope}[case["op"]](s)
    return s


# ---- the library's calls -----------------------------------------------------------------------


def _empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _act(L, name):
    return {"none": L.LORA_ACT_NONE, "relu": L.LORA_ACT_RELU, "silu": L.LORA_ACT_SILU,
            "gelu": L.LORA_ACT_GELU, "gelu_tanh": L.LORA_ACT_GELU_TANH}[name]


def _out_type(L, s):
    f32 = s["case"]["y"] == "f32"
    return (torch.float32, L.LORA_F32) if f32 else (torch.bfloat16, L.LORA_BF16)


def _own_quant(s):
    from rank_adapter_gemm_sgmv_amd import lora as L

    c = s["case"]
    M, d = c["M"], c["d"]
    out = dict(y8=_empty(M, d, dtype=torch.int8), y_scale=_empty(M, dtype=torch.float32))
    if c["residual"]:
        out["sum"] = _empty(M, d, dtype=torch.bfloat16)
    if c["both"]:
        out["y"] = _empty(M, d, dtype=torch.bfloat16)

    def call():
        if c["norm"]:
            L.lora_rmsnorm_int8(s["x"], s["residual"], s["weight"], EPS, M, d, out.get("sum"), out.get("y"),
                                out["y8"], out["y_scale"])
        else:
            L.lora_quant_int8(s["x"], M, d, out["y8"], out["y_scale"])
        return out

    return call


def _own_int8(s):
    from rank_adapter_gemm_sgmv_amd import lora as L

    c = s["case"]
    M, K, N, n, r = (c[k] for k in ("M", "K", "N", "n", "r_max"))
    y_type, y_dtype = _out_type(L, s)
    y = _empty(M, N, dtype=y_type)
    ws, nbytes = L.int8_workspace(M, K, N, r, n)

    def call():
        epi = L.lora_epilogue(_act(L, c["act"]), s["bias"], s["mul"], s["residual"])
        L.lora_linear_int8(s["x8"], s["x_scale"], s["W8"], s["w_scale"], s["A"], s["B"], s["scale"],
                           s["ranks"], s["ids"], M, K, N, r, n, None, epi, y, y_dtype, L.LORA_MODE_AUTO,
                           ws, nbytes)
        return y

    return call


def _own_moe(s):
    from rank_adapter_gemm_sgmv_amd import lora as L

    c = s["case"]
    M, k, E, d, ff, r, n = (c[k] for k in ("M", "top_k", "E", "d", "ff", "r_max", "n"))
    y_type, y_dtype = _out_type(L, s)
    y = _empty(M, d, dtype=y_type)
    ws, nbytes = L.moe_layer_workspace(M, k, E, d, ff, r, n)
    weights = L.lora_moe_weights(*(s[m + p] for p in "gud" for m in "WAB"))

    def call():
        L.lora_moe_layer(s["x"], weights, s["scale"], s["ranks"], s["ids"], s["topk_ids"], s["topk_w"],
                         s["residual"], M, k, E, d, ff, r, n, _act(L, c["act"]), y, y_dtype,
                         L.LORA_MODE_AUTO, ws, nbytes)
        return y

    return call


def _own_rope(s):
    from rank_adapter_gemm_sgmv_amd import lora as L

    c = s["case"]
    M, hq, hk, D = (c[k] for k in ("M", "hq", "hk", "D"))
    y_type, y_dtype = _out_type(L, s)
    q, k = s["qkv"][:, :hq * D], s["qkv"][:, hq * D:(hq + hk) * D]
    row = s["qkv"].stride(0)
    out = dict(q=_empty(M, hq * D, dtype=y_type))
    if hk:
        out["k"] = _empty(M, hk * D, dtype=y_type)
    layout = L.LORA_ROPE_HALF if c["layout"] == "half" else L.LORA_ROPE_INTERLEAVED

    def call():
        L.lora_rope(q, k if hk else None, s["positions"], s["freqs"], M, hq, hk, D, c["rot"], row, row,
                    layout, s["factor"], c["inverse"], out["q"], hq * D, out.get("k"), hk * D, y_dtype)
        return out

    return call


# ---- the plain forms -----------------------------------------------------------------------------


def _plain_quant(s):
    c = s["case"]
    p = h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        p = h = h + s["residual"].float()
        out["sum"] = h.bfloat16()
    if s["weight"] is not None:
        p = p * s["weight"].float()
    top = p.abs().amax(1)
    size = top
    if c["norm"]:
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        size = top * r[:, 0]
        if c["both"]:
            out["y"] = (p * r).bfloat16()
    # (a quotient next to a border between two integers)
    out["y8"] = torch.round(p.double() * 127.0 / top.clamp_min(2.0 ** -60).double()[:, None]).to(torch.int8)
    out["y_scale"] = size.clamp_min(2.0 ** -60) / 127.0
    return out


def _plain_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _plain_int8(s):
    c = s["case"]
    M, K, N, n, r = (c[k] for k in ("M", "K", "N", "n", "r_max"))
    x = s["x8"].float()
    z = (x @ s["W8"].float().t()) * s["w_scale"]
    ids = s["ids"].long()
    if n <= 128:
        # every adapter's columns side by side, each row keeping its own adapter's
        t = (x @ s["A"].float().transpose(0, 1).reshape(K, n * r)).view(M, n, r)
        w = (ids[:, None] == torch.arange(n, device=ids.device)) * s["scale"]
        z = z + (t * w[:, :, None]).view(M, n * r) @ s["B"].float().view(n * r, N)
    else:
        # many adapters: each row's own adapter gathered
        i = ids.clamp_min(0)
        w = torch.where(ids >= 0, s["scale"][i], 0.0)
        t = torch.bmm(x[:, None, :], s["A"][i].float()) * w[:, None, None]
        z = z + torch.bmm(t, s["B"][i].float())[:, 0]
    z = z * s["x_scale"][:, None]
    if c["bias"]:
        z = z + s["bias"].float()
    z = _plain_act(z, c["act"])
    if c["mul"]:
        z = z * s["mul"].float()
    if c["residual"]:
        z = z + s["residual"].float()
    return z if c["y"] == "f32" else z.bfloat16()


def _plain_moe(s):
    c = s["case"]
    M, k, E, d, ff = (c[k] for k in ("M", "top_k", "E", "d", "ff"))
    x = s["x"].float()
    slot = s["topk_ids"].long()
    e = slot.clamp_min(0)
    m = torch.arange(M, device=e.device)[:, None].expand(M, k)
    i = s["ids"].long()
    w_ad = torch.where(i >= 0, s["scale"][i.clamp_min(0)], 0.0)[:, None, None]
    i = i.clamp_min(0)[:, None].expand(M, k)

    def delta(v, p):
        """scale (v A[i][e]) B[i][e] of every slot's row v"""
        t = torch.matmul(v[:, :, None, :], s["A" + p][i, e].float())
        return torch.matmul(t, s["B" + p][i, e].float())[:, :, 0] * w_ad

    few = M * k <= E

    def routed(p):
        # few slots: each one's expert gathered; else the rows through every expert, each slot
        # taking its own
        if few:
            z = torch.matmul(x[:, None, None, :], s["W" + p][e].float())[:, :, 0]
        else:
            z = torch.matmul(x, s["W" + p].float())[e, m]
        return z + delta(x[:, None].expand(M, k, d), p)

    h = _plain_act(routed("g"), c["act"]) * routed("u")
    w = torch.where(slot >= 0, s["topk_w"], 0.0)[:, :, None]
    if few:
        y = (torch.matmul((w * h)[:, :, None, :], s["Wd"][e].float())[:, :, 0]).sum(1)
    else:
        side = torch.zeros(M, E, ff, device=x.device).index_put((m, e), w * h, accumulate=True)
        y = side.view(M, E * ff) @ s["Wd"].float().view(E * ff, d)
    y = y + (w * delta(h, "d")).sum(1)
    if c["residual"]:
        y = y + s["residual"].float()
    return y if c["y"] == "f32" else y.bfloat16()


def _plain_rope(s):
    c = s["case"]
    M, hq, hk, D, rot = (c[k] for k in ("M", "hq", "hk", "D", "rot"))
    v = s["qkv"][:, :(hq + hk) * D].float().view(M, hq + hk, D)
    turns = s["positions"].double()[:, None] * s["freqs"]
    angle = (2.0 * math.pi) * (turns - turns.floor())
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["inverse"]:
        sin = -sin
    if c["layout"] == "half":
        a, b = v[:, :, :rot // 2], v[:, :, rot // 2:rot]
    else:
        a, b = v[:, :, 0:rot:2], v[:, :, 1:rot:2]
    turned = [(a * cos - b * sin) * s["factor"], (a * sin + b * cos) * s["factor"]]
    turned = torch.cat(turned, 2) if c["layout"] == "half" else torch.stack(turned, 3).view(M, hq + hk, rot)
    y = torch.cat([turned, v[:, :, rot:]], 2).to(s["qkv"].dtype)
    out = dict(q=y[:, :hq].reshape(M, hq * D))
    if hk:
        out["k"] = y[:, hq:].reshape(M, hk * D)
    return out


def run(s):
    if own:
        return s["call"]()
    return {"quant": _plain_quant, "int8": _plain_int8, "moe": _plain_moe, "rope": _plain_rope}[s["case"]["op"]](s)


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    y = 4 if case.get("y") == "f32" else 2
    if case["op"] == "quant":
        M, d = case["M"], case["d"]
        el = 2 + 4 * case["residual"] + 1 + 2 * case["both"]
        return dict(bytes=M * d * el + 4 * M + 2 * d * case["weight"], flops=6 * M * d)
    if case["op"] == "rope":
        el = case["M"] * (case["hq"] + case["hk"]) * case["D"]
        return dict(bytes=2 * el * y + 4 * case["M"] + 4 * case["rot"],
                    flops=3 * case["M"] * (case["hq"] + case["hk"]) * case["rot"])
    M, n, rank = case["M"], case["n"], (case["r_max"] + 1) / 2.0
    if case["op"] == "int8":
        K, N = case["K"], case["N"]
        adapters = n * (1.0 - (1.0 - 1.0 / (n + 1)) ** M)  # met by the batch, on average
        bytes_ = M * K + K * N + adapters * rank * (K + N) * 2 + M * (4 + N * y)
        bytes_ += 2 * N * case["bias"] + M * N * y * (case["mul"] + case["residual"]) + 4 * (M + N)
        return dict(bytes=bytes_, flops=2.0 * M * K * N + 2.0 * M * rank * (K + N) * n / (n + 1))
    E, k, d, ff = (case[v] for v in ("E", "top_k", "d", "ff"))
    k = k * (0.8 if case["holes"] else 1.0)
    experts = E * (1.0 - (1.0 - k / E) ** M)  # met by the batch, on average
    pools = n * E * (1.0 - (1.0 - k / (E * (n + 1.0))) ** M)
    bytes_ = 3 * experts * d * ff * 2 + 3 * pools * rank * (d + ff) * 2
    bytes_ += M * d * (2 + y + y * case["residual"]) + M * (4 + 8 * case["top_k"])
    return dict(bytes=bytes_, flops=6.0 * M * k * d * ff + 6.0 * M * k * rank * (d + ff) * n / (n + 1))


# ---- the definition in 64 bits ------------------------------------------------------------------------


def _exact_quant(case, v):
    out = {}
    h = v["x"].double()
    if case["residual"]:
        h = h + v["residual"].double()
        out["sum"] = h
    p = h.float().double()  # (p is an fp32 value by definition)
    if case["weight"]:
        p = (p * v["weight"].double()[None, :]).float().double()
    top = torch.maximum(p.max(1).values, -p.min(1).values)
    floor = torch.full_like(top, 2.0 ** -60)
    out["y8"] = torch.round(127.0 * p / torch.maximum(top, floor)[:, None]).to(torch.int8)
    if case["norm"]:
        rms = (h.square().sum(1) / case["d"] + EPS).sqrt()
        n = h / rms[:, None]
        if case["weight"]:
            n = n * v["weight"].double()[None, :]
        if case["both"]:
            out["y"] = n
        top = torch.maximum(n.max(1).values, -n.min(1).values)
    out["y_scale"] = torch.maximum(top, floor) / 127.0
    return out


def _exact_act(z, a):
    if a == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if a == "silu":
        return z * torch.sigmoid(z)
    if a == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if a == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _adapted(x, W, A, B, ids, ranks):
    """x W plus each row's own adapter, rows of one adapter at a time; A[i], B[i] by a call."""
    z = torch.mm(x, W)
    for i in sorted(set(ids.tolist()) - {-1}):
        rows = (ids == i).nonzero()[:, 0]
        r = int(ranks[i])
        low = torch.mm(x[rows], A(i)[:, :r].double())
        z[rows] += torch.mm(low, B(i)[:r].double()) * (16.0 / r)
    return z


def _exact_int8(case, v):
    x = v["x8"].double() * v["x_scale"].double()[:, None]
    W = (v["W8"].double() * v["w_scale"].double()[:, None]).t().contiguous()
    z = _adapted(x, W, lambda i: v["A"][i], lambda i: v["B"][i], v["ids"], v["ranks"])
    if case["bias"]:
        z += v["bias"].double()
    z = _exact_act(z, case["act"])
    if case["mul"]:
        z = z * v["mul"].double()
    if case["residual"]:
        z = z + v["residual"].double()
    return z


def _exact_moe(case, v):
    x = v["x"].double()
    y = v["residual"].double().clone() if case["residual"] else torch.zeros_like(x)
    for e in sorted(set(v["topk_ids"].flatten().tolist()) - {-1}):
        m, j = (v["topk_ids"] == e).nonzero(as_tuple=True)
        ids = v["ids"][m]

        def through(rows, p):
            return _adapted(rows, v["W" + p][e].double(), lambda i: v["A" + p][i, e],
                            lambda i: v["B" + p][i, e], ids, v["ranks"])

        h = _exact_act(through(x[m], "g"), case["act"]) * through(x[m], "u")
        y.index_add_(0, m, through(h, "d") * v["topk_w"][m, j].double()[:, None])
    return y


def _exact_rope(case, v):
    M, hq, hk, D, rot = (case[k] for k in ("M", "hq", "hk", "D", "rot"))
    f, factor = _freqs(case)
    # the remainder of the turns first, then the complex number that it stands for
    turns = torch.fmod(v["positions"].double()[:, None] * f.cuda()[None, :], 1.0)
    way = -1.0 if case["inverse"] else 1.0
    turn = torch.polar(torch.full_like(turns, factor), way * 2.0 * math.pi * turns)[:, None, :]
    x = v["qkv"].double().view(M, hq + 2 * hk, D)[:, :hq + hk].clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :rot].reshape(M, hq + hk, rot // 2, 2)) * turn
        x[..., :rot] = torch.view_as_real(z).reshape(M, hq + hk, rot)
    out = dict(q=x[:, :hq].reshape(M, -1))
    if hk:
        out["k"] = x[:, hq:].reshape(M, -1)
    return out


def exact(case, seed):
    v = _inputs(case, seed)
    return {"quant": _exact_quant, "int8": _exact_int8, "moe": _exact_moe, "rope": _exact_rope}[case["op"]](case, v)

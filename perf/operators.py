"""The serving operators around the multi-LoRA linear, in plain form and as calls of the library.

norm  residual addition, root-mean-square norm, output in bf16 or in 8 bits with a scale per row:
      h = x + residual;  n = h / sqrt(mean(h^2) + eps) * weight;  sum = bf16(h);  y = bf16(n);
      s = max(max|n|, 2^-60) / 448;  y8 = E4M3(n / s)
act   the layer with its epilogue:
      y = act(x W + scale_i (x A_i) B_i + bias) * mul + residual,   i = ids[m], -1: no adapter
fp8   the same on 8-bit operands, x = x_scale[m] dec(x8[m]), W = w_scale[c] dec(W8[c])

Layouts are those of include/lora.h: x[M, d_in], W[d_in, d_out], W8[d_out, d_in],
A[n, d_in, r_max], B[n, r_max, d_out], y[M, d_out].
"""

import math

import torch

own = False

EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------------


def listed():
    return [
        # one token of one request: launch and latency only
        dict(name="norm_1_bf16", op="norm", M=1, d=4096, out="bf16", residual=True, weight=True),
        # a decode batch in front of an 8-bit projection
        dict(name="norm_64_e4m3", op="norm", M=64, d=4096, out="e4m3", residual=True, weight=True),
        # an odd number of rows at the MLP's inner width, a norm without residual
        dict(name="norm_1023_wide_bf16", op="norm", M=1023, d=11008, out="bf16", residual=False, weight=True),
        # a long prompt in front of 8-bit projections; both outputs (the bf16 one feeds others)
        dict(name="norm_8192_both", op="norm", M=8192, d=4096, out="both", residual=True, weight=True),
        # single-token decode through an output projection, residual added
        dict(name="act_1_residual", op="act", M=1, K=4096, N=4096, n=8, r_max=16, act="none",
             bias=False, mul=False, residual=True, y="bf16"),
        # the gate projection of a decode batch: silu(gate) * up; every row its own adapter
        dict(name="act_64_gate", op="act", M=64, K=4096, N=11008, n=32, r_max=16, act="silu",
             bias=False, mul=True, residual=False, y="bf16"),
        # the down projection of a wide decode batch over a large pool; odd rows, a rank that is
        # no power of two, fp32 output
        dict(name="act_509_down_f32", op="act", M=509, K=11008, N=4096, n=256, r_max=24, act="none",
             bias=True, mul=False, residual=True, y="f32"),
        # a prompt through a biased GELU projection
        dict(name="act_4096_gelu", op="act", M=4096, K=4096, N=4096, n=4, r_max=16, act="gelu",
             bias=True, mul=False, residual=True, y="bf16"),
        # single-token decode on the 8-bit base
        dict(name="fp8_1_gate", op="fp8", M=1, K=4096, N=11008, n=8, r_max=16, act="silu",
             bias=False, mul=True, residual=False, y="bf16"),
        # a decode batch, odd rows, ragged width
        dict(name="fp8_117_residual", op="fp8", M=117, K=4096, N=4104, n=64, r_max=16, act="none",
             bias=True, mul=False, residual=True, y="bf16"),
        # a wide decode batch over many adapters
        dict(name="fp8_512_down", op="fp8", M=512, K=11008, N=4096, n=256, r_max=16, act="none",
             bias=False, mul=False, residual=True, y="bf16"),
        # a prompt through the gate projection
        dict(name="fp8_4096_gate", op="fp8", M=4096, K=4096, N=11008, n=8, r_max=16, act="silu",
             bias=False, mul=True, residual=False, y="bf16"),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["norm", "act", "fp8"])
    M = min(_log(rng, 1, 8192), 8192)
    if op == "norm":
        d = 8 * min(_log(rng, 16, 1376), 1376)
        M = min(M, 8192 * 4096 // d)
        return dict(op=op, M=M, d=d, out=rng.choice(["bf16", "e4m3", "both"]),
                    residual=rng.random() < 0.7, weight=rng.random() < 0.9)
    q = 8 if op == "act" else 16
    K = q * min(_log(rng, 256 // q, 11008 // q), 11008 // q)
    N = 8 * min(_log(rng, 16, 1376), 1376)
    M = max(1, min(M, 4096 * 4096 * 4096 // (K * N), 4096))
    r_max = min(_log(rng, 1, 64), 64)
    n = min(_log(rng, 1, 512), max(1, 4096 // r_max))
    return dict(op=op, M=M, K=K, N=N, n=n, r_max=r_max,
                act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                bias=rng.random() < 0.5, mul=rng.random() < 0.3, residual=rng.random() < 0.5,
                y="f32" if rng.random() < 0.2 else "bf16")


# ---- inputs ----------------------------------------------------------------------------------


def _quantised(v):
    """E4M3 codes of the rows of v and the scale of each row."""
    s = v.abs().amax(1).clamp_min(2.0 ** -60) / 448.0
    return (v / s[:, None]).to(torch.float8_e4m3fn), s


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g)

    if case["op"] == "norm":
        M, d = case["M"], case["d"]
        # hidden states have a few channels far above the others
        loud = 1.0 + 15.0 * (torch.rand(d, device="cuda", generator=g) < 0.005)
        return dict(
            x=(normal(M, d, std=0.5) * loud).bfloat16(),
            residual=(normal(M, d, std=2.0) * loud).bfloat16() if case["residual"] else None,
            weight=(1.0 + normal(d, std=0.2)).bfloat16() if case["weight"] else None)

    M, K, N, n, r = (case[k] for k in ("M", "K", "N", "n", "r_max"))
    ranks = torch.randint(1, r + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    ranks[0] = r
    kept = torch.arange(r, device="cuda") < ranks[:, None]  # rank rows past an adapter's own are zero
    out_type = torch.float32 if case["y"] == "f32" else torch.bfloat16
    s = dict(
        A=(normal(n, K, r, std=K ** -0.5) * kept[:, None, :]).bfloat16(),
        B=(normal(n, r, N, std=0.5 * r ** -0.5) * kept[:, :, None]).bfloat16(),
        scale=16.0 / ranks.float(), ranks=ranks,
        ids=torch.randint(-1, n, (M,), device="cuda", generator=g, dtype=torch.int32),
        bias=normal(N, std=0.5).bfloat16() if case["bias"] else None,
        mul=normal(M, N).to(out_type) if case["mul"] else None,
        residual=normal(M, N).to(out_type) if case["residual"] else None)
    if case["op"] == "act":
        s.update(x=normal(M, K).bfloat16(), W=normal(K, N, std=K ** -0.5).bfloat16())
    else:
        s["x8"], s["x_scale"] = _quantised(normal(M, K))
        s["W8"], s["w_scale"] = _quantised(normal(N, K, std=K ** -0.5))
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if own:
        s["call"] = _own_norm(s) if case["op"] == "norm" else _own_linear(s)
    return s


# ---- the library's calls -----------------------------------------------------------------------


def _own_norm(s):
    from rank_adapter_gemm_sgmv_amd import lora as L

    c = s["case"]
    M, d = c["M"], c["d"]
    out = {}
    if c["residual"]:
        out["sum"] = torch.empty(M, d, dtype=torch.bfloat16, device="cuda")
    if c["out"] != "e4m3":
        out["y"] = torch.empty(M, d, dtype=torch.bfloat16, device="cuda")
    if c["out"] != "bf16":
        out["y8"] = torch.empty(M, d, dtype=torch.float8_e4m3fn, device="cuda")
        out["y_scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
    to = [out.get(k) for k in ("sum", "y", "y8", "y_scale")]

    def call():
        L.lora_rmsnorm(s["x"], s["residual"], s["weight"], EPS, M, d, *to)
        return out

    return call


def _own_linear(s):
    from rank_adapter_gemm_sgmv_amd import lora as L

    c = s["case"]
    M, K, N, n, r = (c[k] for k in ("M", "K", "N", "n", "r_max"))
    f32 = c["y"] == "f32"
    y = torch.empty(M, N, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    y_dtype = L.LORA_F32 if f32 else L.LORA_BF16
    act = {"none": L.LORA_ACT_NONE, "relu": L.LORA_ACT_RELU, "silu": L.LORA_ACT_SILU,
           "gelu": L.LORA_ACT_GELU, "gelu_tanh": L.LORA_ACT_GELU_TANH}[c["act"]]
    lora = (s["A"], s["B"], s["scale"], s["ranks"], s["ids"], M, K, N, r, n, None)
    if c["op"] == "act":
        ws, nbytes = L.workspace(M, K, N, r, n)

        def call():
            epi = L.lora_epilogue(act, s["bias"], s["mul"], s["residual"])
            L.lora_linear_act(s["x"], s["W"], *lora, epi, y, y_dtype, L.LORA_MODE_AUTO, ws, nbytes)
            return y
    else:
        ws, nbytes = L.fp8_workspace(M, K, N, r, n)

        def call():
            epi = L.lora_epilogue(act, s["bias"], s["mul"], s["residual"])
            L.lora_linear_fp8(s["x8"], s["x_scale"], s["W8"], s["w_scale"], *lora, epi, y, y_dtype,
                              L.LORA_MODE_AUTO, ws, nbytes)
            return y
    return call


# ---- the plain forms -----------------------------------------------------------------------------


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["sum"] = h.bfloat16()
    n = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    if s["weight"] is not None:
        n = n * s["weight"].float()
    if s["case"]["out"] != "e4m3":
        out["y"] = n.bfloat16()
    if s["case"]["out"] != "bf16":
        scale = n.abs().amax(1).clamp_min(2.0 ** -60) / 448.0
        out["y8"] = (n / scale[:, None]).to(torch.float8_e4m3fn)
        out["y_scale"] = scale
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


def _plain_linear(s):
    c = s["case"]
    M, K, N, n, r = (c[k] for k in ("M", "K", "N", "n", "r_max"))
    if c["op"] == "act":
        x = s["x"].float()
        z = x @ s["W"].float()
    else:
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
    if c["op"] == "fp8":
        z = z * s["x_scale"][:, None]
    if c["bias"]:
        z = z + s["bias"].float()
    z = _plain_act(z, c["act"])
    if c["mul"]:
        z = z * s["mul"].float()
    if c["residual"]:
        z = z + s["residual"].float()
    return z if c["y"] == "f32" else z.bfloat16()


def run(s):
    if own:
        return s["call"]()
    return _plain_norm(s) if s["case"]["op"] == "norm" else _plain_linear(s)


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    if case["op"] == "norm":
        el = case["M"] * case["d"]
        out = {"bf16": 2, "e4m3": 1, "both": 3}[case["out"]]
        rows = 0 if case["out"] == "bf16" else 4 * case["M"]
        return dict(bytes=el * (2 + 4 * case["residual"] + out) + rows + 2 * case["d"] * case["weight"],
                    flops=6 * el)
    M, K, N, n, r = (case[k] for k in ("M", "K", "N", "n", "r_max"))
    w = 2 if case["op"] == "act" else 1
    y = 4 if case["y"] == "f32" else 2
    adapters = n * (1.0 - (1.0 - 1.0 / (n + 1)) ** M)  # met by the batch, on average
    rank = (r + 1) / 2.0
    bytes_ = w * (M * K + K * N) + adapters * rank * (K + N) * 2 + M * (4 + N * y)
    bytes_ += 2 * N * case["bias"] + M * N * y * (case["mul"] + case["residual"])
    if case["op"] == "fp8":
        bytes_ += 4 * (M + N)
    return dict(bytes=bytes_, flops=2.0 * M * K * N + 2.0 * M * rank * (K + N) * n / (n + 1))


# ---- the definition in 64 bits ------------------------------------------------------------------------


def _exact_norm(case, v):
    out = {}
    h = v["x"].double()
    if case["residual"]:
        h.add_(v["residual"].double())
        out["sum"] = h.clone()
    rms = (h.square().sum(1) / case["d"] + EPS).sqrt()
    n = h / rms[:, None]
    if case["weight"]:
        n *= v["weight"].double()[None, :]
    if case["out"] in ("bf16", "both"):
        out["y"] = n
    if case["out"] in ("e4m3", "both"):
        top = torch.maximum(n.max(1).values, -n.min(1).values)
        top = torch.clamp(top, min=2.0 ** -60)
        out["y8"] = (n * (448.0 / top)[:, None]).to(torch.float8_e4m3fn)
        out["y_scale"] = top / 448.0
    return out


def _exact_linear(case, v):
    if case["op"] == "act":
        x, W = v["x"].double(), v["W"].double()
    else:
        x = v["x8"].double() * v["x_scale"].double()[:, None]
        W = (v["W8"].double() * v["w_scale"].double()[:, None]).t().contiguous()
    z = torch.mm(x, W)
    del W
    for i in sorted(set(v["ids"].tolist()) - {-1}):
        rows = (v["ids"] == i).nonzero()[:, 0]
        r = int(v["ranks"][i])
        low = torch.mm(x[rows], v["A"][i, :, :r].double())
        z[rows] += torch.mm(low, v["B"][i, :r].double()) * (16.0 / r)
    if case["bias"]:
        z += v["bias"].double()
    a = case["act"]
    if a == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif a == "silu":
        z = z * torch.sigmoid(z)
    elif a == "gelu":
        z = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    elif a == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if case["mul"]:
        z = z * v["mul"].double()
    if case["residual"]:
        z = z + v["residual"].double()
    return z


def exact(case, seed):
    v = _inputs(case, seed)
    return _exact_norm(case, v) if case["op"] == "norm" else _exact_linear(case, v)

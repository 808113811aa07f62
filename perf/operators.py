"""Measured cases of the 16-bit operators that stand around the W4A4 layer: the
matrix product with bias, activation and residual in its epilogue, layer
normalisation, and the backward passes of both.

  linear                Z = X W + b;  Y = act(Z) + R
  linear_backward       dZ = dY * act'(Z);  dX = dZ W^T, dW = X^T dZ, db = sum_m dZ
  layer_norm            Y = (X - mean) * rstd * w + b, per row; w and b per group of rows
  layer_norm_backward   dX, and dw, db summed over the rows of a group

Shapes are those of the layers this repository is benchmarked on (PixArt-Sigma,
SANA-1.6B, Qwen3-8B) and generic odd ones.  ``own`` selects the library's
entry points; otherwise ``run`` computes the plain form in 32 bits.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# Largest products of the cases: 2048 tokens of Qwen3-8B's up or down projection.
_MAX_MKN = 2048 * 4096 * 12288


def listed():
    return [
        # one token through an up projection of Qwen3-8B: the weights are read once, latency counts
        dict(name="linear_1tok_up_silu", op="linear", M=1, K=4096, N=12288, act="silu", bias=False,
             residual=False, preact=False, dtype="bf16", y_dtype="bf16"),
        # sixteen tokens in flight, down projection added onto the residual stream
        dict(name="linear_16tok_down_residual", op="linear", M=16, K=12288, N=4096, act="identity",
             bias=False, residual=True, preact=False, dtype="bf16", y_dtype="bf16"),
        # PixArt-Sigma's MLP up projection at 4096 image tokens, keeping Z for a backward pass
        dict(name="linear_pixart_up_gelu", op="linear", M=4096, K=1152, N=4608, act="gelu_tanh", bias=True,
             residual=False, preact=True, dtype="bf16", y_dtype="bf16"),
        # ragged in every size: a short prompt batch through a layer of unusual widths, fp32 residual stream
        dict(name="linear_odd_gelu_f16", op="linear", M=333, K=1001, N=777, act="gelu", bias=True,
             residual=True, preact=False, dtype="f16", y_dtype="f32"),
        # Qwen3-8B's up projection over a 2048-token prompt: the largest forward product
        dict(name="linear_qwen3_up_silu", op="linear", M=2048, K=4096, N=12288, act="silu", bias=False,
             residual=False, preact=False, dtype="bf16", y_dtype="bf16"),
        # training or calibration step through PixArt-Sigma's up projection
        dict(name="linear_bwd_pixart_up_gelu", op="linear_backward", M=4096, K=1152, N=4608, act="gelu_tanh",
             bias=True, dtype="bf16"),
        # Qwen3-8B's down projection, 2048 tokens: the largest backward products
        dict(name="linear_bwd_qwen3_down", op="linear_backward", M=2048, K=12288, N=4096, act="identity",
             bias=False, dtype="bf16"),
        # ragged backward pass in fp16
        dict(name="linear_bwd_odd_silu_f16", op="linear_backward", M=257, K=515, N=1023, act="silu",
             bias=True, dtype="f16"),
        # one token's normalisation before a Qwen3-width projection: pure latency
        dict(name="ln_1tok", op="layer_norm", M=1, C=4096, groups=1, affine=True, stats=False, dtype="bf16",
             y_dtype="bf16", p_dtype="bf16"),
        # two images of 4096 tokens, scale and shift per image (PixArt-Sigma's modulated norm), training forward
        dict(name="ln_pixart_modulated", op="layer_norm", M=8192, C=1152, groups=2, affine=True, stats=True,
             dtype="bf16", y_dtype="bf16", p_dtype="f32"),
        # its backward pass: dX and the gradients of the per-image scale and shift
        dict(name="ln_bwd_pixart_modulated", op="layer_norm_backward", M=8192, C=1152, groups=2, affine=True,
             dtype="bf16", y_dtype="bf16", p_dtype="f32"),
        # fp32 residual stream of an odd width into a 16-bit layer input, one weight for every row
        dict(name="ln_bwd_odd_f32", op="layer_norm_backward", M=1537, C=2241, groups=1, affine=True,
             dtype="f32", y_dtype="bf16", p_dtype="f32"),
    ]


def _log_size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    # half of the sizes as they fall (mostly odd), half on the multiples that models use
    step = 64 if n >= 512 else 8
    if rng.random() < 0.5 and n >= step:
        n = n // step * step
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "layer_norm", "layer_norm_backward"])
    if op in ("linear", "linear_backward"):
        half = rng.choice(["bf16", "bf16", "f16"])
        limit = _MAX_MKN if op == "linear_backward" else 2 * _MAX_MKN
        while True:
            M, K, N = _log_size(rng, 1, 8192), _log_size(rng, 48, 12288), _log_size(rng, 48, 12288)
            if M * K * N <= limit:
                break
        c = dict(op=op, M=M, K=K, N=N, act=rng.choice(["identity", "gelu_tanh", "gelu", "silu"]),
                 bias=rng.random() < 0.6, dtype=half)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, preact=rng.random() < 0.3,
                     y_dtype=rng.choice([half, half, "f32"]))
        return c
    dtype = rng.choice(["bf16", "f16", "f32"])
    y = dtype if dtype != "f32" else rng.choice(["f32", "bf16", "f16"])
    C = _log_size(rng, 48, 12288)
    groups = rng.choice([1, 1, 2, 5])
    M = groups * _log_size(rng, 1, max(1, min(16384, (1 << 26) // C) // groups))
    c = dict(op=op, M=M, C=C, groups=groups, affine=rng.random() < 0.8, dtype=dtype, y_dtype=y,
             p_dtype=rng.choice([y, "f32"]))
    if op == "layer_norm":
        c["stats"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, C):
    """Rows as they reach a linear layer: channel-varying spread, a few wide channels."""
    spread = 0.5 + _rand(g, C)
    wide = _rand(g, C) < 0.004
    return _randn(g, M, C) * torch.where(wide, spread * 8.0, spread)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("linear", "linear_backward"):
        M, K, N, dt = case["M"], case["K"], case["N"], _DT[case["dtype"]]
        s["X"] = _activations(g, M, K).to(dt)
        s["W"] = (_randn(g, K, N) / math.sqrt(K)).to(dt)
        s["bias"] = (0.2 * _randn(g, N)).to(dt) if case["bias"] else None
        if case["op"] == "linear":
            s["residual"] = _randn(g, M, N).to(_DT[case["y_dtype"]]) if case["residual"] else None
        else:
            s["dY"] = (0.1 * _randn(g, M, N)).to(dt)
            s["Z"] = None
            if case["act"] != "identity":   # what the forward pass kept
                z = s["X"].float() @ s["W"].float()
                s["Z"] = (z if s["bias"] is None else z + s["bias"].float()).to(dt)
        if own:
            import w4a4_rank_assisted_amd as hsq

            need = (hsq.linear_workspace_bytes(M, K, N) if case["op"] == "linear"
                    else hsq.linear_backward_workspace_bytes(M, K, N))
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        return s
    M, C, G = case["M"], case["C"], case["groups"]
    s["X"] = (_activations(g, M, C) + 0.5 * _randn(g, M, 1)).to(_DT[case["dtype"]])
    s["w"] = s["b"] = None
    if case["affine"]:
        s["w"] = (1.0 + 0.2 * _randn(g, G, C)).to(_DT[case["p_dtype"]])
        s["b"] = (0.2 * _randn(g, G, C)).to(_DT[case["p_dtype"]])
    if case["op"] == "layer_norm_backward":
        s["dY"] = (0.1 * _randn(g, M, C)).to(_DT[case["y_dtype"]])
        x = s["X"].double()
        mean = x.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = ((x - mean[:, None]).square().mean(1) + 1e-6).rsqrt().float()
        if own:
            import w4a4_rank_assisted_amd as hsq

            s["workspace"] = torch.empty(max(hsq.layer_norm_backward_workspace_bytes(M, C, G), 16),
                                         dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def _act(z, kind):
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, kind):
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    sg = 1.0 / (1.0 + torch.exp(-z))    # silu
    return sg * (1.0 + z * (1.0 - sg))


def _own(s):
    import w4a4_rank_assisted_amd as hsq

    c = s["case"]
    if c["op"] == "linear":
        return hsq.linear(s["X"], s["W"], s["bias"], s["residual"], act=c["act"], y_dtype=c["y_dtype"],
                          return_preact=c["preact"], workspace=s["workspace"])
    if c["op"] == "linear_backward":
        dX, dW, db = hsq.linear_backward(s["dY"], s["X"], s["W"], s["Z"], act=c["act"], need_bias=c["bias"],
                                         workspace=s["workspace"])
        return (dX, dW, db) if c["bias"] else (dX, dW)
    if c["op"] == "layer_norm":
        return hsq.layer_norm(s["X"], s["w"], s["b"], eps=1e-6, y_dtype=c["y_dtype"], return_stats=c["stats"])
    dX, dw, db = hsq.layer_norm_backward(s["dY"], s["X"], s["mean"], s["rstd"], s["w"], need_params=c["affine"],
                                         workspace=s["workspace"])
    return (dX, dw, db) if c["affine"] else dX


def run(state):
    if own:
        return _own(state)
    s, c = state, state["case"]
    if c["op"] == "linear":
        z = s["X"].float() @ s["W"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = y.to(_DT[c["y_dtype"]])
        return (y, z.to(s["X"].dtype)) if c["preact"] else y
    if c["op"] == "linear_backward":
        dt = s["X"].dtype
        dz = s["dY"].float()
        if c["act"] != "identity":
            dz = dz * _act_grad(s["Z"].float(), c["act"])
        dX = (dz @ s["W"].float().t()).to(dt)
        dW = (s["X"].float().t() @ dz).to(dt)
        return (dX, dW, dz.sum(0).to(dt)) if c["bias"] else (dX, dW)
    M, C, G = c["M"], c["C"], c["groups"]
    x = s["X"].float().view(G, M // G, C)
    if c["op"] == "layer_norm":
        mean = x.mean(2, keepdim=True)
        d = x - mean
        rstd = torch.rsqrt((d * d).mean(2, keepdim=True) + 1e-6)
        y = d * rstd
        if c["affine"]:
            y = y * s["w"].float()[:, None] + s["b"].float()[:, None]
        y = y.view(M, C).to(_DT[c["y_dtype"]])
        return (y, mean.view(M), rstd.view(M)) if c["stats"] else y
    dy = s["dY"].float().view(G, M // G, C)
    rstd = s["rstd"].view(G, -1, 1)
    xh = (x - s["mean"].view(G, -1, 1)) * rstd
    gr = dy * s["w"].float()[:, None] if c["affine"] else dy
    dX = (gr - gr.mean(2, keepdim=True) - xh * (gr * xh).mean(2, keepdim=True)) * rstd
    dX = dX.view(M, C).to(s["X"].dtype)
    if not c["affine"]:
        return dX
    return dX, (dy * xh).sum(1).to(s["w"].dtype), dy.sum(1).to(s["w"].dtype)


# ------------------------------------------------------------------ 64 bits
def _silu64(z):
    return z * torch.sigmoid(z)


def _normal_cdf(z):
    return torch.special.ndtr(z)


def exact(case, seed):
    """The definition in 64 bits, on the inputs of ``prepare``."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.mm(s["X"].double(), s["W"].double())
        if case["bias"]:
            z += s["bias"].double()
        kind = case["act"]
        if kind == "identity":
            y = z.clone()
        elif kind == "silu":
            y = _silu64(z)
        elif kind == "gelu":
            y = z * _normal_cdf(z)
        else:   # 0.5 (1 + tanh u) = sigmoid(2 u)
            y = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        if case["residual"]:
            y += s["residual"].double()
        return (y, z) if case["preact"] else y
    if case["op"] == "linear_backward":
        dz = s["dY"].double()
        kind = case["act"]
        if kind != "identity":
            z = s["Z"].double()
            if kind == "silu":
                p = torch.sigmoid(z)
                dz *= p + z * p * torch.sigmoid(-z)
            elif kind == "gelu":
                dz *= _normal_cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
            else:   # y = z sigmoid(2u): y' = sigmoid(2u) + 2 z u' sigmoid(2u) sigmoid(-2u)
                k = math.sqrt(2.0 / math.pi)
                u = k * (z + 0.044715 * z ** 3)
                p, q = torch.sigmoid(2 * u), torch.sigmoid(-2 * u)
                dz *= p + 2 * z * (k + 3 * k * 0.044715 * z ** 2) * p * q
        dX = torch.mm(dz, s["W"].double().t().contiguous())
        dW = torch.mm(s["X"].double().t().contiguous(), dz)
        if case["bias"]:
            return dX, dW, torch.mv(dz.t().contiguous(), torch.ones(case["M"], dtype=torch.float64, device="cuda"))
        return dX, dW
    M, C, G = case["M"], case["C"], case["groups"]
    x = s["X"].double()
    rows = M // G
    if case["op"] == "layer_norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + 1e-6)
        y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
        if case["affine"]:
            w = s["w"].double().repeat_interleave(rows, 0)
            y = y * w + s["b"].double().repeat_interleave(rows, 0)
        return (y, mean, rstd) if case["stats"] else y
    rstd = s["rstd"].double().unsqueeze(1)
    xh = (x - s["mean"].double().unsqueeze(1)) * rstd
    dy = s["dY"].double()
    gr = dy * s["w"].double().repeat_interleave(rows, 0) if case["affine"] else dy
    dX = rstd / C * (C * gr - gr.sum(1, keepdim=True) - xh * (gr * xh).sum(1, keepdim=True))
    if not case["affine"]:
        return dX
    dw = torch.stack([(dy[i * rows:(i + 1) * rows] * xh[i * rows:(i + 1) * rows]).sum(0) for i in range(G)])
    db = torch.stack([dy[i * rows:(i + 1) * rows].sum(0) for i in range(G)])
    return dX, dw, db


def work(case):
    """Bytes of the inputs and outputs, each once, and the operations of one pass."""
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] in ("linear", "linear_backward"):
        M, K, N, h = case["M"], case["K"], case["N"], size[case["dtype"]]
        if case["op"] == "linear":
            ysz = size[case["y_dtype"]]
            b = h * (M * K + K * N + (N if case["bias"] else 0) + (M * N if case["preact"] else 0))
            b += ysz * M * N * (2 if case["residual"] else 1)
            return {"bytes": b, "flops": 2 * M * K * N}
        b = h * (M * N * (1 if case["act"] == "identity" else 2) + 2 * M * K + 2 * K * N + (N if case["bias"] else 0))
        return {"bytes": b, "flops": 4 * M * K * N}
    M, C, G = case["M"], case["C"], case["groups"]
    x, y, p = size[case["dtype"]], size[case["y_dtype"]], size[case["p_dtype"]]
    if case["op"] == "layer_norm":
        b = M * C * (x + y) + (2 * G * C * p if case["affine"] else 0) + (8 * M if case["stats"] else 0)
        return {"bytes": b, "flops": 8 * M * C}
    b = M * C * (2 * x + y) + 8 * M + (3 * G * C * p if case["affine"] else 0)
    return {"bytes": b, "flops": 14 * M * C}

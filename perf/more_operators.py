"""Measured cases of the operators of a 4-bit decoding step: the W4A4 layer's
weights under activations that stay in 16 bits, a key / value cache that is
quantised to 4 bits as it is written and read back, and attention over it.

  linear      xh = X / lambda
              Y  = sum_g sw[g] sum_{k in g} xh[k] qw[k] + (xh L1) L2 + bias + residual
  kv_cache    per token, head and 64 channels x:
                asym  lo = min(0, min x), hi = max(0, max x), s = fp16((hi - lo) / 15),
                      z = clamp(rint(-lo / s), 0, 15), n = clamp(rint(x / s) + z, 0, 15)
                sym   s = fp16(max |x| / 7), z = 8, n = clamp(rint(x / s), -8, 7) + 8
              the value held is s (n - z); a pass writes new tokens and reads them
              back, or reads back what is held
  attention   Y[i] = sum_t p[i,t] v[t], p = softmax over the visible t of scale q[i] k[t];
              query i of n sits at position len - n + i and sees what is not after it
              (causal) and less than `window` before it

Sizes are those of the Qwen3-8B projections this repository is benchmarked on
and generic ones, odd and ragged among them.  ``own`` selects the library's
entry points; otherwise ``run`` computes the plain form in 32 bits.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}

# Limits of drawn cases, those of the largest listed ones: weights of a linear,
# channels held per side of a cache and written or read in a pass, operations of
# an attention.
_MAX_KN = 4096 * 12288
_MAX_HELD = 64 * 4000 * 8 * 128
_MAX_MOVED = 16384 * 8 * 128
_MAX_FLOPS = 2e11


def listed():
    return [
        # one token through Qwen3-8B's up projection, weights only: the read of 25 MB
        dict(name="linear_1tok_up", op="linear", M=1, K=4096, N=12288, batch=1, group=64, r=0, smooth=False,
             bias=False, residual=False, dtype="bf16", y_dtype="bf16"),
        # one token through a whole rank-16 layer, Q, K and V at once: smoothing, three rank branches
        dict(name="linear_1tok_qkv_rank16", op="linear", M=1, K=4096, N=4096, batch=3, group=128, r=16, smooth=True,
             bias=True, residual=False, dtype="bf16", y_dtype="bf16"),
        # sixteen tokens in flight, down projection added onto an fp32 residual stream
        dict(name="linear_16tok_down_residual", op="linear", M=16, K=12288, N=4096, batch=1, group=64, r=4,
             smooth=True, bias=False, residual=True, dtype="bf16", y_dtype="f32"),
        # speculative tokens of several sequences through a layer of unusual widths, fp16
        dict(name="linear_odd_f16", op="linear", M=37, K=1088, N=1003, batch=1, group=64, r=5, smooth=False,
             bias=True, residual=True, dtype="f16", y_dtype="f16"),
        # a prompt of 8192 tokens enters the cache, all heads of a layer
        dict(name="cache_prompt", op="kv_cache", write=True, B=1, q=8192, ragged=False, lo=8192, hi=8192, Hkv=8,
             D=128, page=64, quant="asym", dtype="bf16"),
        # one new token of each of 64 sequences: latency
        dict(name="cache_append_64", op="kv_cache", write=True, B=64, q=1, ragged=False, lo=100, hi=4000, Hkv=8,
             D=128, page=64, quant="asym", dtype="bf16"),
        # ragged prompts behind what is held already, narrow heads of an odd number, symmetric, fp16
        dict(name="cache_odd_f16", op="kv_cache", write=True, B=5, q=333, ragged=True, lo=400, hi=1777, Hkv=5, D=64,
             page=32, quant="sym", dtype="f16"),
        # a shared prefix of 16384 tokens is read back for a path that wants 16 bits
        dict(name="cache_read_prefix", op="kv_cache", write=False, B=1, q=16384, ragged=False, lo=16384, hi=16384,
             Hkv=8, D=128, page=256, quant="asym", dtype="bf16"),
        # one sequence, one token, a short history: pure latency
        dict(name="attention_1seq_short", op="attention", B=1, q=1, ragged=False, lo=777, hi=777, Hq=32, Hkv=8,
             D=128, page=64, quant="asym", causal=True, window=0, lse=False, dtype="bf16", y_dtype="bf16"),
        # a full decoding batch: 64 sequences of 100 to 8000 tokens
        dict(name="attention_batch_64", op="attention", B=64, q=1, ragged=False, lo=100, hi=8000, Hq=32, Hkv=8,
             D=128, page=64, quant="asym", causal=True, window=0, lse=False, dtype="bf16", y_dtype="bf16"),
        # four drafted tokens a sequence, a head of its own for each query, sliding window, narrow heads, fp16
        dict(name="attention_draft_window_f16", op="attention", B=24, q=4, ragged=True, lo=5, hi=5001, Hq=7, Hkv=7,
             D=64, page=32, quant="sym", causal=True, window=1000, lse=True, dtype="f16", y_dtype="f32"),
        # the last 2048 tokens of a prompt attend to all of it: the most operations
        dict(name="attention_prompt_chunk", op="attention", B=2, q=2048, ragged=True, lo=6001, hi=8192, Hq=32, Hkv=8,
             D=128, page=64, quant="asym", causal=True, window=0, lse=False, dtype="bf16", y_dtype="bf16"),
    ]


def _log_size(rng, lo, hi, step=8):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    # half of the sizes as they fall (mostly odd), half on the multiples that models use
    if rng.random() < 0.5 and n >= step:
        n = n // step * step
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["linear", "linear", "kv_cache", "attention", "attention"])
    half = rng.choice(["bf16", "bf16", "f16"])
    if op == "linear":
        group = rng.choice([64, 64, 128])
        while True:
            batch = rng.choice([1, 1, 1, 2, 3])
            K, N = group * _log_size(rng, 1, 12288 // group), _log_size(rng, 16, 12288, 64)
            if batch * K * N <= _MAX_KN:
                break
        return dict(op=op, M=_log_size(rng, 1, 64), K=K, N=N, batch=batch, group=group,
                    r=rng.choice([0, 0, 4, 16, 32, rng.randint(1, 32)]), smooth=rng.random() < 0.5,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.4, dtype=half,
                    y_dtype=rng.choice([half, half, "f32"]))
    while True:
        c = dict(op=op, B=_log_size(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 5, 8, 8, 16]), D=rng.choice([64, 128, 128, 256]),
                 page=rng.choice([32, 64, 64, 128, 256]), quant=rng.choice(["asym", "asym", "sym"]), dtype=half)
        c["q"] = rng.choice([1, 1, rng.randint(2, 8), _log_size(rng, 9, 4096)])
        c["ragged"] = c["q"] > 1 and rng.random() < 0.6
        c["lo"] = c["q"] + _log_size(rng, 1, 8192) - 1
        c["hi"] = min(c["lo"] * _log_size(rng, 1, 16), 131072)
        if op == "kv_cache":
            c["write"] = rng.random() < 0.7
            if not c["write"] and rng.random() < 0.5:
                c["q"] = c["lo"]
            if sum(_queries(c)) * c["Hkv"] * c["D"] > _MAX_MOVED:
                continue
        else:
            c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 4, 8])
            c["causal"] = rng.random() < 0.8
            c["window"] = _log_size(rng, 1, 4096) if c["causal"] and rng.random() < 0.3 else 0
            c["lse"] = rng.random() < 0.4
            c["y_dtype"] = rng.choice([half, half, "f32"])
            if max(_queries(c)) * max(_lens(c)) * c["Hq"] > 1 << 29 or work(c)["flops"] > _MAX_FLOPS:
                continue
        if sum(_lens(c)) * c["Hkv"] * c["D"] <= _MAX_HELD:
            return c


# ------------------------------------------------------------------ lengths
def _spread(lo, hi, n):
    """n lengths from lo to hi in no order."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.5) % 1.0)) for i in range(n)]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["B"])


def _queries(c):
    return _spread(max(1, c["q"] // 3), c["q"], c["B"])[::-1] if c["ragged"] else [c["q"]] * c["B"]


def _seen(c):
    """Sum over the queries of the tokens each sees, and tokens that any sees."""
    pairs = held = 0
    for n, q in zip(_lens(c), _queries(c)):
        w = c["window"]
        if not c["causal"]:
            pairs, held = pairs + n * q, held + n
            continue
        for i in (range(q) if w else ()):
            pairs += min(n - q + i + 1, w)
        pairs += 0 if w else q * (n - q) + q * (q + 1) // 2
        held += min(n, w + q - 1) if w else n
    return pairs, held


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
    """Rows as they reach a layer: channel-varying spread, a few wide channels."""
    spread = 0.5 + _rand(g, C)
    wide = _rand(g, C) < 0.004
    return _randn(g, M, C) * torch.where(wide, spread * 8.0, spread)


def _linear_inputs(c, seed):
    g = _gen(seed)
    M, K, N, b, r, dt = c["M"], c["K"], c["N"], c["batch"], c["r"], _DT[c["dtype"]]
    s = dict(case=c)
    s["X"] = _activations(g, M, K).to(dt)
    s["lam"] = (0.5 + 2.0 * _rand(g, K)).half() if c["smooth"] else None
    s["codes"] = torch.randint(-8, 8, (b, K, N), generator=g, device="cuda", dtype=torch.int8)
    s["sw"] = ((0.5 + _rand(g, b, K // c["group"], N)) * (0.25 / math.sqrt(K))).half()
    s["L1"] = (_randn(g, b, K, r) / math.sqrt(K)).to(dt) if r else None
    s["L2"] = (_randn(g, b, r, N) / math.sqrt(r)).to(dt) if r else None
    s["bias"] = (0.2 * _randn(g, b, N)).to(dt) if c["bias"] else None
    s["residual"] = _randn(g, b, M, N).to(_DT[c["y_dtype"]]) if c["residual"] else None
    return s


def _kv(c, seed):
    """Keys and values of every token held, in the order of the sequences:
    keys with a few wide channels off centre, as projections give them."""
    g = _gen(seed)
    T, H, D = sum(_lens(c)), c["Hkv"], c["D"]
    k = _randn(g, T, H, D)
    wide = _rand(g, H, D) < 0.03
    k *= torch.where(wide, 3.0, 0.7 + 0.6 * _rand(g, H, D))
    k += torch.where(wide, 6.0 * _randn(g, H, D), 0.0 * _rand(g, H, D))
    k = k.to(_DT[c["dtype"]])
    v = _randn(g, T, H, D)
    v *= 0.5 + _rand(g, H, D)
    return g, k, v.to(_DT[c["dtype"]])


def _query(c, g):
    return _randn(g, sum(_queries(c)), c["Hq"], c["D"]).to(_DT[c["dtype"]])


def _last(c):
    """Rows of the new tokens among all held ones."""
    rows, off = [], 0
    for n, q in zip(_lens(c), _queries(c)):
        rows.append(torch.arange(off + n - q, off + n, device="cuda"))
        off += n
    return torch.cat(rows)


def _quantise(x, quant):
    """(..., D) -> n (..., D) uint8, s (..., D / 64) fp16, z (..., D / 64) uint8.
    In 64 bits: values next to the border of two codes."""
    shape = x.shape
    x = x.double().view(*shape[:-1], shape[-1] // 64, 64)
    if quant == "asym":
        lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / 15.0).clamp(max=65504.0).half()
    else:
        s = (x.abs().amax(-1) / 7.0).clamp(max=65504.0).half()
    d = torch.where(s > 0, s.double(), math.inf)
    if quant == "asym":
        z = (-lo / d).round().clamp(0, 15)
        n = ((x / d[..., None]).round() + z[..., None]).clamp(0, 15)
    else:
        z = torch.full_like(d, 8.0)
        n = (x / d[..., None]).round().clamp(-8, 7) + 8.0
    return n.view(shape).to(torch.uint8), s, z.to(torch.uint8)


def _values(n, s, z):
    shape = n.shape
    v = n.float().view(*shape[:-1], shape[-1] // 64, 64) - z.float()[..., None]
    return (v * s.float()[..., None]).view(shape)


def _pieces(t):
    """Runs of rows that keep 64-bit temporaries small."""
    step = max(1, (1 << 25) // max(1, t[0].numel()))
    return [slice(i, min(i + step, t.shape[0])) for i in range(0, t.shape[0], step)]


def prepare(case, seed):
    c = case
    if c["op"] == "linear":
        s = _linear_inputs(c, seed)
        if own:
            import w4a4_rank_assisted_amd as hsq

            s["packed"] = torch.cat([hsq.pack_weights(w)[0] for w in s.pop("codes")])
            need = hsq.w4a16_workspace_bytes(c["M"], c["K"], c["N"], c["r"], c["batch"], c["group"],
                                             smooth=c["smooth"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        return s
    g, k, v = _kv(c, seed)
    B, H, D, page, lens, queries = c["B"], c["Hkv"], c["D"], c["page"], _lens(c), _queries(c)
    s = dict(case=c, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    s["cu"] = None
    if c["ragged"]:
        s["cu"] = torch.tensor([0] + queries, device="cuda").cumsum(0).to(torch.int32)
    # pages in no order, with room to grow by a few that have no number yet
    need = [-(-n // page) for n in lens]
    pages = sum(need)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(need) + 3), -1, dtype=torch.int32, device="cuda")
    off = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[off:off + m]
        off += m
    s["table"] = table
    held = None      # slots of all held tokens, in the order of the sequences
    if not own or c["op"] != "kv_cache" or not c["write"]:
        held = torch.cat([table[b, :need[b]].long().repeat_interleave(page)[:n] * page
                          + torch.arange(n, device="cuda") % page for b, n in enumerate(lens)])
    if c["op"] == "attention":
        s["Q"] = _query(c, g)
        s["scale"] = 1.0 / math.sqrt(D)
    elif c["write"]:
        new = _last(c)
        s["K"], s["V"] = k[new], v[new]
    if own:
        import w4a4_rank_assisted_amd as hsq

        s["cache"] = hsq.kv_cache(pages, H, D, page)
        if c["op"] == "attention" or not c["write"]:
            cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
            hsq.kv_cache_write(k, v, s["cache"], table, s["lens"], cu, quant=c["quant"], max_tokens=max(lens))
        if c["op"] == "attention":
            need = hsq.kv_attention_workspace_bytes(s["Q"].shape[0], c["Hq"], H, D, B, c["q"],
                                                    table.shape[1] * page)
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        return s
    for name, x in (("k", k), ("v", v)):
        s[name + "n"] = torch.zeros(pages * page, H, D, dtype=torch.uint8, device="cuda")
        s[name + "s"] = torch.zeros(pages * page, H, D // 64, dtype=torch.float16, device="cuda")
        s[name + "z"] = torch.zeros(pages * page, H, D // 64, dtype=torch.uint8, device="cuda")
        if c["op"] == "attention" or not c["write"]:
            for p in _pieces(x):
                for part, t in zip("nsz", _quantise(x[p], c["quant"])):
                    s[name + part][held[p]] = t
    if c["op"] == "kv_cache":
        s["slots"] = held[_last(c)]
    return s


# ------------------------------------------------------------------ one pass
def _own(s):
    import w4a4_rank_assisted_amd as hsq

    c = s["case"]
    if c["op"] == "linear":
        return hsq.w4a16_lowrank_linear(s["X"], s["packed"], s["sw"], s["lam"], s["L1"], s["L2"], s["bias"],
                                        s["residual"], N=c["N"], batch=c["batch"], group=c["group"],
                                        y_dtype=c["y_dtype"], workspace=s["workspace"])
    if c["op"] == "kv_cache":
        if c["write"]:
            hsq.kv_cache_write(s["K"], s["V"], s["cache"], s["table"], s["lens"], s["cu"], quant=c["quant"],
                               max_tokens=c["q"])
        tokens = sum(_queries(c)) if c["ragged"] else c["B"] * c["q"]
        return hsq.kv_cache_read(s["cache"], s["table"], s["lens"], s["cu"], tokens=tokens, head_dim=c["D"],
                                 dtype=c["dtype"], max_tokens=c["q"])
    return hsq.kv_attention(s["Q"], s["cache"], s["table"], s["lens"], s["cu"], scale=s["scale"], causal=c["causal"],
                            window=c["window"], y_dtype=c["y_dtype"], return_lse=c["lse"], max_tokens=c["q"],
                            workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    s, c = state, state["case"]
    if c["op"] == "linear":
        xh = s["X"].float()
        if c["smooth"]:
            xh = xh * (1.0 / s["lam"].float())
        ys = []
        for b in range(c["batch"]):
            w = s["codes"][b].float().view(-1, c["group"], c["N"]) * s["sw"][b].float()[:, None]
            y = xh @ w.view(c["K"], c["N"])
            if c["r"]:
                y = y + (xh @ s["L1"][b].float()) @ s["L2"][b].float()
            if c["bias"]:
                y = y + s["bias"][b].float()
            if c["residual"]:
                y = y + s["residual"][b].float()
            ys.append(y.to(_DT[c["y_dtype"]]))
        return torch.stack(ys)
    if c["op"] == "kv_cache":
        if c["write"]:
            for name, x in (("k", s["K"]), ("v", s["V"])):
                for part, t in zip("nsz", _quantise(x, c["quant"])):
                    s[name + part][s["slots"]] = t
        return tuple(_values(s[a + "n"][s["slots"]], s[a + "s"][s["slots"]], s[a + "z"][s["slots"]]).to(_DT[c["dtype"]])
                     for a in "kv")
    H, D, G, page = c["Hkv"], c["D"], c["Hq"] // c["Hkv"], c["page"]
    ys, lses, off = [], [], 0
    for b, (n, q) in enumerate(zip(_lens(c), _queries(c))):
        at = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[at // page] * page + at % page
        k = _values(s["kn"][slots], s["ks"][slots], s["kz"][slots]).transpose(0, 1).contiguous()      # H, n, D
        v = _values(s["vn"][slots], s["vs"][slots], s["vz"][slots]).transpose(0, 1).contiguous()
        Q = s["Q"][off:off + q].float().view(q, H, G, D).permute(1, 2, 0, 3).reshape(H, G * q, D)
        logits = torch.bmm(Q, k.transpose(1, 2).contiguous()).view(H, G, q, n) * s["scale"]
        if c["causal"]:
            pos = torch.arange(n - q, n, device="cuda")[:, None]
            hide = at[None] > pos
            if c["window"]:
                hide = hide | (at[None] <= pos - c["window"])
            logits = logits.masked_fill_(hide, -math.inf)
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - top)
        total = p.sum(-1, keepdim=True)
        y = torch.bmm(p.view(H, G * q, n), v).view(H, G, q, D) / total
        ys.append(y.permute(2, 0, 1, 3).reshape(q, H * G, D).to(_DT[c["y_dtype"]]))
        lses.append((top + torch.log(total)).squeeze(-1).permute(2, 0, 1).reshape(q, H * G))
        off += q
    y = torch.cat(ys)
    return (y, torch.cat(lses)) if c["lse"] else y


# ------------------------------------------------------------------ 64 bits
def _held64(x, quant):
    """What the cache holds of x (T, H, D): the definition, group by group."""
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for g in range(x.shape[2] // 64):
        part = slice(64 * g, 64 * g + 64)
        v = x[:, :, part].double()
        if quant == "sym":
            s = torch.maximum(v.amax(2), -v.amin(2)) / 7
            low, high, zero = -8.0, 7.0, torch.zeros_like(s)
        else:
            s = (torch.relu(v.amax(2)) + torch.relu(-v.amin(2))) / 15
            low, high = 0.0, 15.0
        s = torch.clamp(s, max=65504.0).to(torch.float16).double()
        inv = torch.where(s == 0, torch.ones_like(s), s)
        if quant != "sym":
            zero = torch.clamp(torch.round(torch.relu(-v.amin(2)) / inv), low, high)
        q = torch.clamp(torch.round(v / inv.unsqueeze(2)) + zero.unsqueeze(2), low, high)
        out[:, :, part] = s.unsqueeze(2) * (q - zero.unsqueeze(2))
    return out


def exact(case, seed):
    """The definition in 64 bits, on the inputs of ``prepare``."""
    c = case
    if c["op"] == "linear":
        s = _linear_inputs(c, seed)
        x = s["X"].double()
        if c["smooth"]:
            x = x / s["lam"].double()
        out = torch.zeros(c["batch"], c["M"], c["N"], dtype=torch.float64, device="cuda")
        for b in range(c["batch"]):
            scale = s["sw"][b].double().repeat_interleave(c["group"], 0)
            out[b] = torch.mm(x, s["codes"][b].double() * scale)
            if c["r"]:
                out[b] += torch.mm(torch.mm(x, s["L1"][b].double()), s["L2"][b].double())
            if c["bias"]:
                out[b] += s["bias"][b].double()
            if c["residual"]:
                out[b] += s["residual"][b].double()
        return out
    g, k, v = _kv(c, seed)
    if c["op"] == "kv_cache":
        new = _last(c)
        return _held64(k[new], c["quant"]), _held64(v[new], c["quant"])
    # the permutation of the pages is drawn before the queries
    torch.randperm(sum(-(-n // c["page"]) for n in _lens(c)), generator=g, device="cuda")
    Q = _query(c, g)
    G, w = c["Hq"] // c["Hkv"], c["window"]
    y = torch.empty(Q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(Q.shape[:2], dtype=torch.float64, device="cuda")
    row = tok = 0
    for n, q in zip(_lens(c), _queries(c)):
        ks, vs = _held64(k[tok:tok + n], c["quant"]), _held64(v[tok:tok + n], c["quant"])
        t = torch.arange(n, device="cuda").view(1, n)
        i = torch.arange(q, device="cuda").view(q, 1) + (n - q)
        seen = t <= i if c["causal"] else torch.ones(q, n, dtype=torch.bool, device="cuda")
        if w:
            seen &= i - t < w
        for h in range(c["Hq"]):
            kh, vh = ks[:, h // G].contiguous(), vs[:, h // G].contiguous()
            e = torch.mm(Q[row:row + q, h].double(), kh.t().contiguous()) / math.sqrt(c["D"])
            e = torch.where(seen, e, torch.full_like(e, -math.inf))
            l = torch.logsumexp(e, 1)
            y[row:row + q, h] = torch.mm(torch.exp(e - l.unsqueeze(1)), vh)
            lse[row:row + q, h] = l
        row, tok = row + q, tok + n
    return (y, lse) if c["lse"] else y


def work(case):
    """Bytes of the inputs and outputs, each once, and the operations of one pass."""
    c = case
    if c["op"] == "linear":
        M, K, N, b, r, h, y = c["M"], c["K"], c["N"], c["batch"], c["r"], _SIZE[c["dtype"]], _SIZE[c["y_dtype"]]
        n = M * K * h + b * (K * N // 2 + K // c["group"] * N * 2 + (K + N) * r * h)
        n += (2 * K if c["smooth"] else 0) + (b * N * h if c["bias"] else 0)
        n += b * M * N * y * (2 if c["residual"] else 1)
        return {"bytes": n, "flops": 2 * b * M * (K * N + r * (K + N))}
    per = c["Hkv"] * 2 * (c["D"] // 2 + c["D"] // 64 * 3)      # codes, scale and zero of one token
    if c["op"] == "kv_cache":
        T = sum(_queries(c))
        raw = T * c["Hkv"] * c["D"] * 2 * _SIZE[c["dtype"]]
        # a pass that writes reads the tokens, writes the cache, reads it and writes the values
        return {"bytes": 2 * (raw + T * per) if c["write"] else raw + T * per,
                "flops": T * c["Hkv"] * c["D"] * 2 * (6 if c["write"] else 2)}
    pairs, held = _seen(c)
    T = sum(_queries(c))
    n = held * per + T * c["Hq"] * (c["D"] * (_SIZE[c["dtype"]] + _SIZE[c["y_dtype"]]) + (4 if c["lse"] else 0))
    return {"bytes": n, "flops": 4 * c["D"] * c["Hq"] * pairs}

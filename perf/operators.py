"""Cases of the operators that stand around the routed experts of a decoder block, each in two forms.

    norm     a norm behind a block and the norm before the next one, with the block's gate and the residual scale
    int8     products in 8-bit integers with a scale for each token and each output channel
    grouped  products grouped by expert with ragged sizes (bf16 experts), plain or with clamp-SwiGLU behind
    combine  the weighted sum of a token's k expert rows, taken from the expert-grouped order

`run` is one pass: in elementary torch operations where `own` is false, through the package's entry points where it
is true.  `exact` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one token between two blocks: a channel gate, both norms; latency is all that counts
        {"name": "norm_token", "op": "norm", "M": 1, "H": 7168, "gate": "channel", "post": True, "pre": True},
        # an odd batch of tokens, gated per element (a gate computed from a condition), wide-decode hidden size
        {"name": "norm_batch_333", "op": "norm", "M": 333, "H": 2048, "gate": "full", "post": True, "pre": True},
        # a long prompt: nothing but memory traffic
        {"name": "norm_prompt", "op": "norm", "M": 16384, "H": 7168, "gate": "token", "post": True, "pre": True},
        # a linear layer for one token: quantise the row, stream the int8 weights once
        {"name": "int8_token", "op": "int8_linear", "M": 1, "K": 7168, "N": 4096},
        # a shared expert for an odd decode batch: quantise, gate_up, SwiGLU and quantise, down, plus the routed output
        {"name": "int8_mlp_33", "op": "int8_mlp", "M": 33, "H": 2048, "I": 768},
        # a prompt's product from rows that are quantised already
        {"name": "int8_prompt", "op": "int8_gemm", "M": 4096, "K": 7168, "N": 4096},
        # decode of one token: 8 experts of 128 with a row each, x gathered by the routing, SwiGLU behind
        {"name": "grouped_token", "op": "grouped", "M": 1, "k": 8, "E": 128, "K": 2048, "N": 768, "swiglu": True,
         "gather": True, "skew": 0.0},
        # decode of 32 tokens: most of 256 experts touched with one or two rows, down projection
        {"name": "grouped_decode_32", "op": "grouped", "M": 32, "k": 8, "E": 256, "K": 2048, "N": 7168,
         "swiglu": False, "gather": False, "skew": 0.0},
        # skewed routing: some experts with hundreds of rows, many with none to a few
        {"name": "grouped_skew_1024", "op": "grouped", "M": 1024, "k": 8, "E": 128, "K": 1536, "N": 4096,
         "swiglu": False, "gather": False, "skew": 1.5},
        # a prompt of 2048 tokens over 16 experts: a dense contraction with ragged groups
        {"name": "grouped_prompt", "op": "grouped", "M": 2048, "k": 8, "E": 16, "K": 7168, "N": 2048, "swiglu": True,
         "gather": True, "skew": 0.3},
        # the end of a decode step's layer
        {"name": "combine_8", "op": "combine", "M": 8, "k": 8, "H": 2048, "add": False},
        # the end of a prompt's layer, with the shared expert's output added
        {"name": "combine_2048", "op": "combine", "M": 2048, "k": 8, "H": 7168, "add": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "int8_linear", "int8_mlp", "int8_gemm", "grouped", "grouped", "grouped",
                     "combine"])
    if op == "norm":
        H = _log(rng, 512, 8192, 32)
        return {"op": op, "M": _log(rng, 1, min(16384, 16384 * 7168 // H)), "H": H,
                "gate": rng.choice(["none", "channel", "token", "full"]), "post": rng.random() < 0.7,
                "pre": rng.random() < 0.8}
    if op == "int8_linear":
        return {"op": op, "M": _log(rng, 1, 512), "K": _log(rng, 256, 7168, 32), "N": _log(rng, 512, 4096, 8)}
    if op == "int8_mlp":
        return {"op": op, "M": _log(rng, 1, 1024), "H": _log(rng, 512, 4096, 32), "I": _log(rng, 256, 1536, 32)}
    if op == "int8_gemm":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 256, 7168, 32), "N": _log(rng, 512, 4096, 8)}
    if op == "combine":
        return {"op": op, "M": _log(rng, 1, 2048), "k": rng.choice([1, 2, 4, 6, 8]), "H": _log(rng, 512, 7168, 32),
                "add": rng.random() < 0.5}
    k = rng.choice([1, 2, 4, 6, 8])
    E = rng.choice([8, 16, 32, 60, 64, 128])
    return {"op": op, "M": _log(rng, 1, 1024), "k": k, "E": E, "K": _log(rng, 256, 4096, 32),
            "N": _log(rng, 256, 2048, 32), "swiglu": rng.random() < 0.5, "gather": rng.random() < 0.5,
            "skew": rng.choice([0.0, 0.5, 1.5])}


def _randn(g, shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _int8_weights(g, N, K):
    """Per-channel int8 weights as a checkpoint holds them: near-normal codes and one scale for each output row."""
    q = torch.randn((N, K), generator=g, device="cuda").mul_(30.0).round_().clamp_(-127, 127).to(torch.int8)
    s = torch.rand(N, generator=g, device="cuda").add_(0.5).mul_(1.0 / (30.0 * math.sqrt(K)))
    return q, s


def _routing(g, c):
    """Expert-grouped order of M*k assignments, and the group sizes that the plain form pads to."""
    M, k, E = c["M"], c["k"], c["E"]
    u = torch.rand((M, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    bias = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    ids = (bias - torch.log(-torch.log(u))).topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    active = counts.nonzero().flatten()
    slot_of = torch.zeros(E, dtype=torch.int64, device="cuda")
    slot_of[active] = torch.arange(active.numel(), device="cuda")
    expert = ids[order]
    return {"offsets": offsets.to(torch.int32), "sorted_ids": order.to(torch.int32), "active": active,
            "slot": slot_of[expert], "row": torch.arange(M * k, device="cuda") - offsets[expert],
            "cap": int(counts.max())}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op == "norm":
        M, H = c["M"], c["H"]
        s["x"] = _randn(g, (M, H), 0.7)
        s["residual"] = _randn(g, (M, H), 2.0)
        s["w_post"] = _randn(g, (H,), 0.2).add_(1.0) if c["post"] else None
        s["w_pre"] = _randn(g, (H,), 0.2).add_(1.0) if c["pre"] else None
        if c["gate"] == "channel":
            s["gate"] = _randn(g, (H,), 0.5)
        elif c["gate"] == "token":
            s["gate"] = torch.rand(M, generator=g, device="cuda")
        elif c["gate"] == "full":
            s["gate"] = _randn(g, (M, H), 0.5)
        else:
            s["gate"] = None
        s["residual_scale"], s["block_scale"] = 0.875, 1.25
    elif op in ("int8_linear", "int8_gemm"):
        x = _randn(g, (c["M"], c["K"]))
        if op == "int8_linear":
            s["x"] = x
        else:
            s["q"] = torch.randn((c["M"], c["K"]), generator=g, device="cuda").mul_(35.0).round_().clamp_(-127, 127) \
                .to(torch.int8)
            s["qs"] = torch.rand(c["M"], generator=g, device="cuda").add_(0.5).mul_(1.0 / 35.0)
        s["w"], s["ws"] = _int8_weights(g, c["N"], c["K"])
    elif op == "int8_mlp":
        s["x"] = _randn(g, (c["M"], c["H"]))
        s["routed"] = _randn(g, (c["M"], c["H"]))
        s["w13"], s["ws13"] = _int8_weights(g, 2 * c["I"], c["H"])
        s["w2"], s["ws2"] = _int8_weights(g, c["H"], c["I"])
    elif op == "grouped":
        s.update(_routing(g, c))
        s["x"] = _randn(g, (c["M"] if c["gather"] else c["M"] * c["k"], c["K"]))
        s["w"] = _randn(g, (c["E"], (2 if c["swiglu"] else 1) * c["N"], c["K"]), 1.0 / math.sqrt(c["K"]))
    else:
        R = c["M"] * c["k"]
        s["y"] = _randn(g, (R, c["H"]))
        s["topk_w"] = torch.softmax(torch.randn((c["M"], c["k"]), generator=g, device="cuda"), 1)
        s["inv_pos"] = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
        s["add"] = _randn(g, (c["M"], c["H"])) if c["add"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _rms(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    z = s["x"].float()
    if s["w_post"] is not None:
        z = z * _rms(z) * s["w_post"].float()
    if s["gate"] is not None:
        z = z * (s["gate"][:, None] if s["case"]["gate"] == "token" else s["gate"].float())
    r = s["residual_scale"] * s["residual"].float() + s["block_scale"] * z
    if s["w_pre"] is None:
        return [r.bfloat16()]
    return [r.bfloat16(), (r * _rms(r) * s["w_pre"].float()).bfloat16()]


def _plain_quantize(v):
    scale = v.abs().amax(-1) / 127.0
    q = torch.where(scale[:, None] > 0, v / scale[:, None], torch.zeros_like(v)).round().clamp(-127, 127)
    return q, scale


def _plain_int8(q, qs, w, ws):
    # sums of up to K * 127^2 pass 24 bits: the products are summed in 64
    return (q.double() @ w.double().t()).float() * qs[:, None] * ws[None, :]


def _swiglu(gu):
    g, u = gu.chunk(2, -1)
    g, u = g.clamp(max=7.0), u.clamp(-7.0, 7.0)
    return g / (1 + torch.exp(-g)) * u


def _plain_grouped(s):
    c = s["case"]
    x = s["x"].float()
    if c["gather"]:
        x = x[torch.div(s["sorted_ids"].long(), c["k"], rounding_mode="floor")]
    padded = x.new_zeros((s["active"].numel(), s["cap"], c["K"]))
    padded[s["slot"], s["row"]] = x
    y = torch.bmm(padded, s["w"][s["active"]].float().transpose(1, 2))[s["slot"], s["row"]]
    return (_swiglu(y) if c["swiglu"] else y).bfloat16()


def _plain_combine(s):
    c = s["case"]
    rows = s["y"].float()[s["inv_pos"].long()].view(c["M"], c["k"], c["H"])
    out = (rows * s["topk_w"][:, :, None]).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.bfloat16()


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "int8_gemm":
        return _plain_int8(s["q"], s["qs"], s["w"], s["ws"]).bfloat16()
    if op == "int8_linear":
        return _plain_int8(*_plain_quantize(s["x"].float()), s["w"], s["ws"]).bfloat16()
    if op == "int8_mlp":
        gu = _plain_int8(*_plain_quantize(s["x"].float()), s["w13"], s["ws13"]).bfloat16()
        y = _plain_int8(*_plain_quantize(_swiglu(gu.float())), s["w2"], s["ws2"])
        return (y + s["routed"].float()).bfloat16()
    if op == "grouped":
        return _plain_grouped(s)
    return _plain_combine(s)


# ------------------------------------------------------------------ the package's calls

def _run_own(s):
    import decode_moe_layer_b200 as moe

    c = s["case"]
    op = c["op"]
    if op == "norm":
        r, h = moe.moe_block_norm(s["x"], residual=s["residual"], w_post=s["w_post"], gate=s["gate"],
                                  w_pre=s["w_pre"], residual_scale=s["residual_scale"],
                                  block_scale=s["block_scale"], eps=EPS)
        return [r] if h is None else [r, h]
    if op == "int8_gemm":
        return moe.moe_int8_gemm(s["q"], s["qs"], s["w"], s["ws"])
    if op == "int8_linear":
        q, qs = moe.moe_int8_quantize(s["x"])
        return moe.moe_int8_gemm(q, qs, s["w"], s["ws"])
    if op == "int8_mlp":
        q, qs = moe.moe_int8_quantize(s["x"])
        gu = moe.moe_int8_gemm(q, qs, s["w13"], s["ws13"])
        q, qs = moe.moe_int8_quantize(gu, swiglu=True)
        return moe.moe_int8_gemm(q, qs, s["w2"], s["ws2"], add=s["routed"])
    if op == "grouped":
        return moe.moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["sorted_ids"] if c["gather"] else None, k=c["k"],
                                    swiglu=c["swiglu"])
    return moe.moe_combine(s["y"], s["topk_w"], s["inv_pos"], add=s["add"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    if op == "norm":
        M, H = c["M"], c["H"]
        rows = 3 + int(c["pre"]) + int(c["gate"] == "full")           # x, residual, residual out, next input, gate
        vecs = int(c["post"]) + int(c["pre"]) + int(c["gate"] == "channel")
        return {"bytes": 2 * rows * M * H + 2 * vecs * H + (4 * M if c["gate"] == "token" else 0), "flops": 10 * M * H}
    if op in ("int8_linear", "int8_gemm"):
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": N * K + 4 * N + M * K * (2 if op == "int8_linear" else 1) + 4 * M + 2 * M * N,
                "flops": 2 * M * N * K}
    if op == "int8_mlp":
        M, H, I = c["M"], c["H"], c["I"]
        return {"bytes": 3 * H * I + 4 * (2 * I + H) + 2 * M * H * 3, "flops": 6 * M * H * I}
    if op == "grouped":
        M, k, E, K, N = c["M"], c["k"], c["E"], c["K"], c["N"]
        rows = (2 if c["swiglu"] else 1) * N
        # expected number of experts that a draw of M*k assignments touches (uniform routing)
        touched = E * (1 - (1 - k / E) ** M) if c["skew"] == 0 else min(E, M * k)
        return {"bytes": int(touched * rows * K * 2 + (M if c["gather"] else M * k) * K * 2 + M * k * N * 2),
                "flops": 2 * M * k * rows * K}
    M, k, H = c["M"], c["k"], c["H"]
    return {"bytes": 2 * M * k * H + 8 * M * k + 2 * M * H * (2 if c["add"] else 1), "flops": 2 * M * k * H}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_int8(q, qs, w, ws):
    acc = torch.matmul(q.to(torch.float64), w.to(torch.float64).T)
    return acc * qs.to(torch.float64).reshape(-1, 1) * ws.to(torch.float64).reshape(1, -1)


def _exact_codes(v):
    """Row-wise symmetric codes of v (float64): (codes, scale), the scale being the row's largest magnitude / 127."""
    top = v.abs().max(dim=1).values
    scale = top / 127
    safe = torch.where(top == 0, torch.ones_like(top), scale)
    return torch.round(v / safe.reshape(-1, 1)), scale


def exact(case, seed):
    c, d = case, torch.float64
    s = prepare(case, seed)
    op = c["op"]
    if op == "norm":
        x, res = s["x"].to(d), s["residual"].to(d)
        if c["post"]:
            x = x / torch.sqrt((x * x).sum(1, keepdim=True) / c["H"] + EPS) * s["w_post"].to(d)
        if c["gate"] == "token":
            x = x * s["gate"].to(d).reshape(-1, 1)
        elif c["gate"] != "none":
            x = x * s["gate"].to(d)
        out = res * s["residual_scale"] + x * s["block_scale"]
        if not c["pre"]:
            return [out]
        return [out, out / torch.sqrt((out * out).sum(1, keepdim=True) / c["H"] + EPS) * s["w_pre"].to(d)]
    if op == "int8_gemm":
        return _exact_int8(s["q"], s["qs"], s["w"], s["ws"])
    if op == "int8_linear":
        q, qs = _exact_codes(s["x"].to(d))
        return _exact_int8(q, qs, s["w"], s["ws"])
    if op == "int8_mlp":
        q, qs = _exact_codes(s["x"].to(d))
        # the exchange between the two products is bf16 by definition
        gu = _exact_int8(q, qs, s["w13"], s["ws13"]).to(torch.bfloat16).to(d)
        a, b = gu[:, :c["I"]].clamp(max=7), gu[:, c["I"]:].clamp(min=-7, max=7)
        q, qs = _exact_codes(a * torch.sigmoid(a) * b)
        return _exact_int8(q, qs, s["w2"], s["ws2"]) + s["routed"].to(d)
    if op == "grouped":
        bounds = s["offsets"].tolist()
        ids = s["sorted_ids"].tolist()
        out = torch.empty((c["M"] * c["k"], c["N"]), dtype=d, device="cuda")
        for e in range(c["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            if lo == hi:
                continue
            rows = s["x"][[f // c["k"] for f in ids[lo:hi]]] if c["gather"] else s["x"][lo:hi]
            y = rows.to(d) @ s["w"][e].to(d).T
            if c["swiglu"]:
                a, b = y[:, :c["N"]].clamp(max=7), y[:, c["N"]:].clamp(min=-7, max=7)
                y = a * torch.sigmoid(a) * b
            out[lo:hi] = y
        return out
    out = torch.zeros((c["M"], c["H"]), dtype=d, device="cuda")
    pos = s["inv_pos"].reshape(c["M"], c["k"]).long()
    for j in range(c["k"]):
        out += s["y"][pos[:, j]].to(d) * s["topk_w"][:, j].to(d).reshape(-1, 1)
    return out + s["add"].to(d) if c["add"] else out

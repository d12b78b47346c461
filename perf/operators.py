"""Measured cases of the 8-bit integer projections and of the 8-bit mixture-of-experts layer.

Weights are whole numbers in [-127, 127] with one f32 scale per output channel, activations are
quantized per token inside the pass: s = max|x| / 127, q = round-half-even(127 x / max|x|).

  linear   y = (q . Wq^T) * s_token * s_channel + bias, from bf16 / f16 / f32 rows
  experts  one projection of the routed experts over a CSR of routed rows: gate_up with the
           clamped SwiGLU (bf16 rows out) or down (f32 rows out)
  decode   the whole layer of a few tokens: top-k routing, gate_up, SwiGLU, down, weighted sum
"""
import math

import torch

own = False

ALPHA, LIMIT = 1.702, 7.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LARGEST = 2.0 * 4096 * 8192 * 8192        # multiply-adds x 2 of the largest listed case


def listed():
    return [
        # one token through a small odd projection: nothing but latency
        {"name": "linear_1x1003_517", "kind": "linear", "rows": 1, "k": 1003, "n": 517,
         "x": "bf16", "out": "bf16", "bias": True},
        # one decoded token through a projection of the layer's own width: a stream of weights
        {"name": "linear_1x2880_5760", "kind": "linear", "rows": 1, "k": 2880, "n": 5760,
         "x": "bf16", "out": "bf16", "bias": True},
        # a batch of 64 decoding sequences
        {"name": "linear_64x2880_5760", "kind": "linear", "rows": 64, "k": 2880, "n": 5760,
         "x": "f16", "out": "f16", "bias": False},
        # a short prompt, f32 in and out
        {"name": "linear_509x2880_2880", "kind": "linear", "rows": 509, "k": 2880, "n": 2880,
         "x": "f32", "out": "f32", "bias": True},
        # a long prompt through a wide model's square projection: the matrix cores
        {"name": "linear_4096x8192_8192", "kind": "linear", "rows": 4096, "k": 8192, "n": 8192,
         "x": "bf16", "out": "bf16", "bias": False},
        # batched decoding: every expert has a handful of rows
        {"name": "gate_up_t64", "kind": "experts", "act": "swiglu", "tokens": 64, "experts": 32,
         "top": 4, "d": 2880, "f": 2880, "tile": 16},
        # a 512-token prompt, both projections of the layer
        {"name": "gate_up_t512", "kind": "experts", "act": "swiglu", "tokens": 512, "experts": 32,
         "top": 4, "d": 2880, "f": 2880, "tile": 16},
        {"name": "down_t512", "kind": "experts", "act": "none", "tokens": 512, "experts": 32,
         "top": 4, "d": 2880, "f": 2880, "tile": 16},
        # a 2048-token prompt over many experts
        {"name": "gate_up_t2048_e128", "kind": "experts", "act": "swiglu", "tokens": 2048,
         "experts": 128, "top": 4, "d": 2880, "f": 2880, "tile": 16},
        # one token through the whole layer: four experts are read
        {"name": "decode_t1", "kind": "decode", "tokens": 1, "experts": 32, "top": 4, "d": 2880,
         "f": 2880, "y": "bf16"},
        # five drafted tokens over many experts: nearly every pick is another expert
        {"name": "decode_t5_e128", "kind": "decode", "tokens": 5, "experts": 128, "top": 4,
         "d": 2880, "f": 2880, "y": "bf16"},
        # sixteen sequences: most experts are picked by more than one of them
        {"name": "decode_t16", "kind": "decode", "tokens": 16, "experts": 32, "top": 4, "d": 2880,
         "f": 2880, "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "experts", "experts", "decode"])
    if kind == "linear":
        while True:
            c = {"kind": kind, "rows": _log(rng, 1, 8192), "k": _log(rng, 33, 8192),
                 "n": _log(rng, 17, 8192), "x": rng.choice(["bf16", "f16", "f32"]),
                 "out": rng.choice(["bf16", "f16", "f32"]), "bias": rng.random() < 0.5}
            if 2.0 * c["rows"] * c["k"] * c["n"] <= LARGEST:
                return c
    experts = _log(rng, 4, 128)
    c = {"kind": kind, "experts": experts, "d": _log(rng, 64, 2880), "f": _log(rng, 64, 2880)}
    if kind == "experts":
        c["act"] = rng.choice(["swiglu", "none"])
        c["tokens"] = _log(rng, 16, 2048)
        c["top"] = rng.randint(1, min(8, experts))
        c["tile"] = rng.choice([1, 4, 16, 32])
    else:
        c["tokens"] = rng.randint(1, 16)
        c["top"] = rng.randint(1, min(8, experts))
        c["y"] = "bf16"
    return c


def _distinct(c):
    """Experts that are expected to be picked by at least one of the tokens."""
    return c["experts"] * (1.0 - (1.0 - c["top"] / c["experts"]) ** c["tokens"])


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["kind"] == "linear":
        m, k, n = c["rows"], c["k"], c["n"]
        return {"bytes": m * k * size[c["x"]] + n * k + n * 4 * (2 if c["bias"] else 1) +
                m * n * size[c["out"]], "flops": 2.0 * m * k * n}
    d, f, r = c["d"], c["f"], c["tokens"] * c["top"]
    live = _distinct(c)
    if c["kind"] == "experts":
        if c["act"] == "swiglu":
            return {"bytes": c["tokens"] * d * 2 + live * 2 * f * (d + 8) + r * f * 2 + r * 4,
                    "flops": 2.0 * r * d * 2 * f}
        return {"bytes": r * f * 2 + live * d * (f + 8) + r * d * 4, "flops": 2.0 * r * d * f}
    return {"bytes": c["tokens"] * (4 * c["experts"] + 2 * d + 2 * d + 8 * c["top"]) +
            r * f * 2 + live * (2 * f * (d + 8) + d * (f + 8)), "flops": 2.0 * r * d * 3 * f}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + stream)
    return g


def _rows(seed, stream, rows, k, dtype):
    """Rows as a layer sees them: normal values, and a few channels that are much larger."""
    g = _gen(seed, stream)
    x = torch.randn(rows, k, generator=g, device="cuda")
    x *= 1.0 + 12.0 * (torch.rand(k, generator=g, device="cuda") < 0.004)
    return x.to(dtype)


def _weights(seed, stream, e, n, k, bias):
    """Whole-number weights [e][n][k], channel scales and biases [e][n] of a quantized stack."""
    g = _gen(seed, stream)
    q = torch.empty(e, n, k, dtype=torch.int8, device="cuda")
    for i in range(0, e, 8):            # a few experts at a time: the normals take four bytes
        w = torch.randn(min(8, e - i), n, k, generator=g, device="cuda")
        q[i:i + 8] = w.mul_(127.0 / 4.0).round_().clamp_(-127, 127)
    s = torch.exp(0.2 * torch.randn(e, n, generator=g, device="cuda")) * (4.0 / 127.0 / k ** 0.5)
    b = 0.02 * torch.randn(e, n, generator=g, device="cuda")
    return q, s, (b if bias else None)


def _logits(seed, tokens, experts):
    """Router logits: some experts are more popular than others."""
    g = _gen(seed, 3)
    z = torch.randn(tokens, experts, generator=g, device="cuda")
    return z + 0.4 * torch.randn(experts, generator=g, device="cuda")


def _csr(c, seed):
    """The CSR of routed rows (rows of an expert together, in token order, each run padded to a
    multiple of the tile) and, for the plain forms, where each live row stands."""
    tokens, experts, top, tile = c["tokens"], c["experts"], c["top"], c["tile"]
    ids = torch.topk(_logits(seed, tokens, experts), top, dim=1).indices
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=experts)
    padded = (counts + tile - 1) // tile * tile
    basep = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    basep[1:] = torch.cumsum(padded, 0)
    routed = tokens * top
    mpad = -(-(routed + min(experts, routed) * (tile - 1)) // tile) * tile
    order = torch.argsort(flat, stable=True)          # expert by expert, tokens ascending
    expert = flat[order]
    first = torch.cumsum(counts, 0) - counts
    nth = torch.arange(routed, device="cuda") - first[expert]
    row = basep[expert] + nth
    row_tok = torch.full((mpad,), -1, dtype=torch.int32, device="cuda")
    row_tok[row] = (order // top).to(torch.int32)
    return {"counts": counts.to(torch.int32), "basep": basep.to(torch.int32), "row_tok": row_tok,
            "mpad": mpad, "tile": tile, "row": row, "expert": expert, "nth": nth,
            "token": order // top, "most": int(counts.max())}


def _inputs(case, seed):
    c = case
    if c["kind"] == "linear":
        q, s, b = _weights(seed, 1, 1, c["n"], c["k"], c["bias"])
        return {"x": _rows(seed, 0, c["rows"], c["k"], DTYPES[c["x"]]), "q": q, "s": s, "b": b}
    d, f = c["d"], c["f"]
    if c["kind"] == "decode":
        gq, gs, gb = _weights(seed, 1, c["experts"], 2 * f, d, True)
        dq, ds, db = _weights(seed, 2, c["experts"], d, f, True)
        return {"x": _rows(seed, 0, c["tokens"], d, torch.bfloat16),
                "logits": _logits(seed, c["tokens"], c["experts"]),
                "gq": gq, "gs": gs, "gb": gb, "dq": dq, "ds": ds, "db": db}
    state = _csr(c, seed)
    if c["act"] == "swiglu":
        q, s, b = _weights(seed, 1, c["experts"], 2 * f, d, True)
        x = _rows(seed, 0, c["tokens"], d, torch.bfloat16)
    else:
        # the rows that a SwiGLU leaves: products of two normal values
        q, s, b = _weights(seed, 1, c["experts"], d, f, True)
        g = _gen(seed, 0)
        x = (torch.randn(state["mpad"], f, generator=g, device="cuda") *
             torch.randn(state["mpad"], f, generator=g, device="cuda")).to(torch.bfloat16)
    return {**state, "x": x, "q": q, "s": s, "b": b}


def prepare(case, seed):
    state = {**_inputs(case, seed), "case": case}
    c = case
    if c["kind"] == "linear":
        state["out"] = torch.zeros(c["rows"], c["n"], dtype=DTYPES[c["out"]], device="cuda")
    elif c["kind"] == "experts":
        width, dtype = (c["f"], torch.bfloat16) if c["act"] == "swiglu" else (c["d"], torch.float32)
        state["out"] = torch.zeros(state["mpad"], width, dtype=dtype, device="cuda")
    if own:
        import mxfp4_mixture_experts_route_amd as moe

        state["moe"] = moe
        if c["kind"] == "decode":
            state["gate_up"] = moe.I8Experts(state["gq"], state["gs"], state["gb"], glu=True)
            state["down"] = moe.I8Experts(state["dq"], state["ds"], state["db"])
        else:
            glu = c["kind"] == "experts" and c["act"] == "swiglu"
            state["w"] = moe.I8Experts(state["q"], state["s"], state["b"], glu=glu)
            state["ws"] = moe.i8_row_buffers(state["x"].shape[0], state["x"].shape[1], "cuda")
    return state


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _quantize(x):
    """Per-row whole numbers and scales. In 64 bits: 127 x / max may lie on a rounding border."""
    x = x.double()
    top = x.abs().amax(dim=-1, keepdim=True)
    q = torch.where(top > 0, torch.round(127.0 * x / top), torch.zeros_like(x))
    return q.float(), (top / 127.0).float()


def _swiglu(g, f):
    gate = torch.clamp(g[..., :f], max=LIMIT)
    up = torch.clamp(g[..., f:], -LIMIT, LIMIT)
    return gate / (1.0 + torch.exp(-ALPHA * gate)) * (up + 1.0)


def _plain_linear(state):
    q, s = _quantize(state["x"])
    y = torch.matmul(q, state["q"][0].float().t()) * (s * state["s"][0])
    if state["b"] is not None:
        y = y + state["b"][0]
    state["out"].copy_(y)
    return state["out"]


def _plain_experts(state):
    c = state["case"]
    q, s = _quantize(state["x"])
    source = state["token"] if c["act"] == "swiglu" else state["row"]
    e, nth = state["expert"], state["nth"]
    a = torch.zeros(c["experts"], state["most"], q.shape[1], device="cuda")
    a[e, nth] = q[source]
    g = torch.bmm(state["q"].float(), a.transpose(1, 2).contiguous())      # [E][N][rows]
    g = g.transpose(1, 2)[e, nth] * (s[source] * state["s"][e]) + state["b"][e]
    state["out"][state["row"]] = (_swiglu(g, c["f"]) if c["act"] == "swiglu" else g).to(
        state["out"].dtype)
    return state["out"]


def _plain_decode(state):
    c = state["case"]
    t, k, d, f = c["tokens"], c["top"], c["d"], c["f"]
    logits, ids = torch.sort(state["logits"], dim=1, descending=True, stable=True)
    ids, top = ids[:, :k], logits[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(dim=1, keepdim=True)
    pick = ids.reshape(-1)
    q, s = _quantize(state["x"])
    q, s = q.repeat_interleave(k, dim=0), s.repeat_interleave(k, dim=0)
    g = torch.bmm(state["gq"][pick].float(), q.unsqueeze(2)).squeeze(2)
    h = _swiglu(g * (s * state["gs"][pick]) + state["gb"][pick], f).to(torch.bfloat16)
    q, s = _quantize(h)
    y = torch.bmm(state["dq"][pick].float(), q.unsqueeze(2)).squeeze(2)
    y = (y * (s * state["ds"][pick]) + state["db"][pick]).reshape(t, k, d)
    y = (w.unsqueeze(2) * y).sum(dim=1).to(DTYPES[c["y"]])
    return {"ids": ids.to(torch.int32), "w": w, "h": h, "y": y}


def run(state):
    c = state["case"]
    if not own:
        if c["kind"] == "linear":
            return _plain_linear(state)
        return _plain_experts(state) if c["kind"] == "experts" else _plain_decode(state)
    moe = state["moe"]
    if c["kind"] == "linear":
        return moe.i8_linear(state["x"], state["w"], out=state["out"], ws=state["ws"])
    if c["kind"] == "experts":
        swiglu = c["act"] == "swiglu"
        live = None if swiglu else state["row_tok"]
        q, s = moe.i8_quantize(state["x"], live=live, out=state["ws"])
        return moe.i8_moe_gemm(q, s, state["row_tok"] if swiglu else None, state["w"],
                               state["counts"], state["basep"], state["tile"], state["mpad"],
                               moe.MOE_ACT_SWIGLU_OAI if swiglu else moe.MOE_ACT_NONE, ALPHA,
                               LIMIT, out=state["out"])
    o = moe.i8_moe_decode(state["logits"], state["x"], state["gate_up"], state["down"], c["top"],
                          ALPHA, LIMIT, y_dtype=DTYPES[c["y"]])
    return {"ids": o["ids"], "w": o["w"], "h": o["h"], "y": o["y"]}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, expert by expert
# ---------------------------------------------------------------------------------------------

def _exact_rows(x):
    """The values that quantized rows stand for: s q, with the scale as it is stored."""
    x = x.to(torch.float64)
    most = x.abs().max(dim=1).values
    scale = (most / 127.0).to(torch.float32).to(torch.float64)
    steps = torch.round(x * 127.0 / torch.where(most > 0, most, torch.ones_like(most))[:, None])
    return steps * scale[:, None]


def _exact_project(x, q, s, b):
    y = x @ (q.to(torch.float64) * s.to(torch.float64)[:, None]).T.contiguous()
    return y if b is None else y + b.to(torch.float64)


def _exact_act(g, f):
    gate = torch.minimum(g[:, :f], torch.tensor(LIMIT, dtype=torch.float64, device=g.device))
    up = g[:, f:].clamp(-LIMIT, LIMIT)
    return gate * torch.sigmoid(ALPHA * gate) * (up + 1.0)


def exact(case, seed):
    c = case
    state = _inputs(case, seed)
    if c["kind"] == "linear":
        bias = None if state["b"] is None else state["b"][0]
        return _exact_project(_exact_rows(state["x"]), state["q"][0], state["s"][0], bias)
    if c["kind"] == "experts":
        swiglu = c["act"] == "swiglu"
        rows = _exact_rows(state["x"])
        out = torch.zeros(state["mpad"], c["f"] if swiglu else c["d"], dtype=torch.float64,
                          device="cuda")
        counts, base = state["counts"].tolist(), state["basep"].tolist()
        for e in range(c["experts"]):
            if counts[e] == 0:
                continue
            span = slice(base[e], base[e] + counts[e])
            x = rows[state["row_tok"][span].long()] if swiglu else rows[span]
            g = _exact_project(x, state["q"][e], state["s"][e], state["b"][e])
            out[span] = _exact_act(g, c["f"]) if swiglu else g
        return out
    logits = state["logits"].to(torch.float64)
    order = torch.argsort(-logits, dim=1, stable=True)[:, :c["top"]]
    w = torch.softmax(torch.gather(logits, 1, order), dim=1)
    rows = _exact_rows(state["x"])
    y = torch.zeros(c["tokens"], c["d"], dtype=torch.float64, device="cuda")
    hidden = torch.zeros(c["tokens"] * c["top"], c["f"], dtype=torch.float64, device="cuda")
    for t, picks in enumerate(order.tolist()):
        for slot, e in enumerate(picks):
            g = _exact_project(rows[t:t + 1], state["gq"][e], state["gs"][e], state["gb"][e])
            h = _exact_act(g, c["f"])
            hidden[t * c["top"] + slot] = h[0]
            # the layer quantizes the rows as they are stored, in bf16
            h = _exact_rows(h.to(torch.bfloat16))
            y[t:t + 1] += w[t, slot] * _exact_project(h, state["dq"][e], state["ds"][e],
                                                      state["db"][e])
    return {"ids": order.to(torch.int32), "w": w, "h": hidden, "y": y}

"""Cases of the 8-bit floating point and grouped matrix products, with their plain forms.

Three operators of a served model:

dense    y = X W^T for e4m3 X and W with one fp32 scale per 128 values of a row of X and per
         128 x 128 block of W (a dense layer's projections, from one decoded token to a long prompt)
grouped  the same product with one matrix per expert over ragged runs of rows, rows optionally
         gathered through an index; in e4m3 and in bf16 (the experts' products of a routed layer)
quant    rows of activations to e4m3 with a scale per 128 values, plain or as silu(gate) * up
         (what feeds the two products)
"""

import math

import torch

own = False

FP8 = torch.float8_e4m3fn
MAX8 = 448.0
TINY = 2.0 ** -126
BLOCK = 128


def blocks(k):
    return -(-k // BLOCK)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token through a dense FFN's up projection: the weights are streamed once
        {"name": "dense decode", "op": "dense", "m": 1, "n": 17408, "k": 5120, "out": "f32"},
        # a short ragged prompt through an odd projection: rows, columns and the last K block are partial
        {"name": "dense ragged", "op": "dense", "m": 77, "n": 1000, "k": 2064, "out": "f32"},
        # a prompt of 512 tokens through the down projection
        {"name": "dense prompt", "op": "dense", "m": 512, "n": 5120, "k": 17408, "out": "bf16"},
        # a long prompt through the up projection: bound by the matrix cores
        {"name": "dense long prompt", "op": "dense", "m": 4096, "n": 17408, "k": 5120, "out": "bf16"},
        # one decoded token, top 8 of 128 experts, gate and up in one matrix
        {"name": "grouped fp8 decode", "op": "grouped", "type": "fp8", "tokens": 1, "experts": 128, "top": 8,
         "n": 1536, "k": 2048, "gather": True, "spare": 0, "out": "f32"},
        # a prompt of 512 tokens through the same layer, rows gathered by token, some rows spare
        {"name": "grouped fp8 prompt", "op": "grouped", "type": "fp8", "tokens": 512, "experts": 128, "top": 8,
         "n": 1536, "k": 2048, "gather": True, "spare": 40, "out": "bf16"},
        # the down product of 8192 tokens, rows already in expert order
        {"name": "grouped fp8 long", "op": "grouped", "type": "fp8", "tokens": 8192, "experts": 128, "top": 8,
         "n": 2048, "k": 768, "gather": False, "spare": 0, "out": "bf16"},
        # a few tokens through bf16 experts: a speculative verify step
        {"name": "grouped bf16 verify", "op": "grouped", "type": "bf16", "tokens": 4, "experts": 128, "top": 8,
         "n": 2048, "k": 768, "gather": False, "spare": 0, "out": "f32"},
        # few large experts over a long prompt
        {"name": "grouped bf16 long", "op": "grouped", "type": "bf16", "tokens": 8191, "experts": 8, "top": 2,
         "n": 2816, "k": 2048, "gather": True, "spare": 0, "out": "bf16"},
        # one token's activations: latency
        {"name": "quant token", "op": "quant", "m": 1, "k": 5120, "gated": False, "x": "bf16"},
        # a long prompt's activations: bandwidth
        {"name": "quant long", "op": "quant", "m": 4096, "k": 5120, "gated": False, "x": "bf16"},
        # the hidden rows of a prompt of 512 tokens x 8 experts from the gate/up product's fp32 output, ragged
        {"name": "quant gated", "op": "quant", "m": 4099, "k": 776, "gated": True, "x": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: a multiple of 16, of 128 two times in three."""
    step = rng.choice((16, 128, 128))
    return max(step, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(("dense", "dense", "dense", "grouped", "grouped", "grouped", "quant", "quant"))
    out = rng.choice(("f32", "bf16"))
    if op == "dense":
        n, k = _log(rng, 64, 17408), _width(rng, 256, 17408)
        most = min(4096, max(1, 4096 * 17408 * 5120 // (2 * n * k)))
        return {"op": op, "m": _log(rng, 1, most), "n": n, "k": k, "out": out}
    if op == "grouped":
        kind = rng.choice(("fp8", "fp8", "bf16"))
        experts = rng.choice((2, 5, 8, 16, 32, 60, 64, 100, 128))
        top = rng.choice([t for t in (1, 2, 4, 6, 8) if t <= experts])
        n = _log(rng, 128, 4096)
        k = _width(rng, 256, 4096 if kind == "fp8" else 2048)
        while experts * n * k > 128 * 1536 * 2048:
            n = max(64, n // 2)
        most = min(8192, max(1, 8192 * 8 * 2048 * 768 // (2 * top * n * k)))
        return {"op": op, "type": kind, "tokens": _log(rng, 1, most), "experts": experts, "top": top, "n": n, "k": k,
                "gather": rng.random() < 0.6, "spare": rng.choice((0, 0, 1, 17)), "out": out}
    k = _width(rng, 128, 17408)
    return {"op": op, "m": _log(rng, 1, max(1, min(8192, 4096 * 5120 // k))), "k": k, "gated": rng.random() < 0.5,
            "x": rng.choice(("bf16", "f32"))}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, m, k):
    """Normal rows of differing size with a few strong channels."""
    x = _normal(g, m, k) * torch.exp(0.5 * _normal(g, m, 1))
    strong = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x * strong


def _rows8(x):
    """Rows to e4m3 with one scale per 128 values: what the program's earlier step left."""
    m, k = x.shape
    pad = torch.nn.functional.pad(x, (0, blocks(k) * BLOCK - k)).view(m, blocks(k), BLOCK)
    scale = (pad.abs().amax(2).double() / MAX8).clamp_min(TINY).float()   # 64 bits: a scale one step off moves borders
    q = (pad / scale[:, :, None]).clamp(-MAX8, MAX8).view(m, -1)[:, :k].to(FP8).contiguous()
    return q, scale.t().contiguous()


def _weights8(g, *shape):
    """e4m3 weights that fill the type's range, and scales as a checkpoint's blocks of 128 x 128 have them."""
    w = (_normal(g, *shape) * 110.0).clamp_(-MAX8, MAX8).to(FP8)
    lead, n, k = shape[:-2], shape[-2], shape[-1]
    return w, 2e-4 * torch.exp(0.3 * _normal(g, *lead, blocks(n), blocks(k)))


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "dense":
        m, n, k = case["m"], case["n"], case["k"]
        s["w"], s["ws"] = _weights8(g, n, k)
        s["x"], s["xs"] = _rows8(_activations(g, m, k))
        s["y"] = torch.zeros(m, n, device="cuda", dtype=_out(case))
    elif case["op"] == "grouped":
        t, e, top, n, k = case["tokens"], case["experts"], case["top"], case["n"], case["k"]
        scores = _normal(g, t, e) + 0.5 * _normal(g, 1, e)         # some experts are more popular than others
        ids = scores.topk(top, dim=1).indices.flatten()
        order = torch.argsort(ids, stable=True)
        counts = torch.bincount(ids, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
        rows = t * top + case["spare"]
        s["index"] = None
        if case["gather"]:
            s["index"] = torch.cat([order // top, order.new_zeros(case["spare"])]).to(torch.int32)
        x = _activations(g, t if case["gather"] else rows, k)
        if case["type"] == "fp8":
            s["w"], s["ws"] = _weights8(g, e, n, k)
            s["x"], s["xs"] = _rows8(x)
        else:
            s["w"] = (_normal(g, e, n, k) * 0.02).to(torch.bfloat16)
            s["x"] = x.to(torch.bfloat16)
        s["y"] = torch.full((rows, n), -1.0, device="cuda", dtype=_out(case))
    else:
        m, k = case["m"], case["k"]
        x = _activations(g, m, 2 * k if case["gated"] else k)
        s["x"] = x if case["x"] == "f32" else x.to(torch.bfloat16)
        s["q"] = torch.zeros(m, k, device="cuda", dtype=FP8)
        s["qs"] = torch.zeros(blocks(k), m, device="cuda")
    return s


def _out(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


# ------------------------------------------------------------------ one pass

def _spread_rows(x, xs, k):
    """fp32 values of e4m3 rows: xs[b][r] times the code."""
    return x.float() * xs.t().repeat_interleave(BLOCK, 1)[:, :k]


def _spread_weights(w, ws, n, k):
    return w.float() * ws.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _dense(s):
    x = _spread_rows(s["x"], s["xs"], s["k"])
    w = _spread_weights(s["w"], s["ws"], s["n"], s["k"])
    return (x @ w.t()).to(s["y"].dtype)


def _grouped(s):
    """Each expert's rows side by side in one batch, as long as the longest expert's run."""
    e, n, k, y, off = s["experts"], s["n"], s["k"], s["y"], s["offsets"].long()
    row = torch.arange(y.shape[0], device="cuda")
    used = row < off[-1]
    expert = (torch.searchsorted(off, row, right=True) - 1).clamp(max=e - 1)
    place = torch.where(used, row - off[expert], s["most"])       # rows behind the last expert go to a spare place
    x = _spread_rows(s["x"], s["xs"], k) if s["type"] == "fp8" else s["x"].float()
    w = _spread_weights(s["w"], s["ws"], n, k) if s["type"] == "fp8" else s["w"].float()
    if s["index"] is not None:
        x = x[s["index"].long()]
    batch = torch.zeros(e, s["most"] + 1, k, device="cuda")
    batch[expert, place] = x
    product = torch.bmm(w, batch.transpose(1, 2).contiguous()).transpose(1, 2)
    return torch.where(used[:, None], product[expert, place].to(y.dtype), y)


def _quant(s):
    x, k = s["x"].float(), s["k"]
    if s["gated"]:
        gate, up = x[:, :k], x[:, k:]
        x = gate / (1 + torch.exp(-gate)) * up
    return _rows8(x)


def run(s):
    if own:
        import gguf_block_quantized_qmv_amd as q
        if s["op"] == "dense":
            return q.qmm_fp8(s["w"], s["ws"], s["x"], s["xs"], s["n"], s["k"], y=s["y"])
        if s["op"] == "grouped" and s["type"] == "fp8":
            return q.qmm_fp8_grouped(s["w"], s["ws"], s["x"], s["xs"], s["offsets"], s["n"], s["k"],
                                     row_index=s["index"], y=s["y"])
        if s["op"] == "grouped":
            return q.qmm_bf16_grouped(s["w"], s["x"], s["offsets"], s["n"], s["k"], row_index=s["index"], y=s["y"])
        if s["gated"]:
            return q.qmm_fp8_quant_silu_mul(s["x"], xq=s["q"], xs=s["qs"])
        return q.qmm_fp8_quant(s["x"], xq=s["q"], xs=s["qs"])
    if s["op"] == "dense":
        return _dense(s)
    if s["op"] == "grouped":
        return _grouped(s)
    return _quant(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 4 if case.get("out") == "f32" else 2
    if case["op"] == "dense":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * (blocks(n) * blocks(k) + m * blocks(k))
        return {"bytes": n * k + m * k + scales + size * m * n, "flops": 2 * m * n * k}
    if case["op"] == "grouped":
        t, e, n, k, rows = case["tokens"], case["experts"], case["n"], case["k"], case["tokens"] * case["top"]
        active = e * (1 - (1 - case["top"] / e) ** t)              # experts with a row, were all equally likely
        wide = 1 if case["type"] == "fp8" else 2
        inputs = (t if case["gather"] else rows) * k * wide + 4 * (e + 1 + (rows if case["gather"] else 0))
        if case["type"] == "fp8":
            inputs += 4 * blocks(k) * (active * blocks(n) + (t if case["gather"] else rows))
        return {"bytes": active * n * k * wide + inputs + size * rows * n, "flops": 2 * rows * n * k}
    m, k = case["m"], case["k"]
    wide = 4 if case["x"] == "f32" else 2
    return {"bytes": m * k * (wide * (2 if case["gated"] else 1) + 1) + 4 * m * blocks(k),
            "flops": (12 if case["gated"] else 4) * m * k}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _e4m3_table():
    """The 256 values of e4m3: sign, four exponent bits with bias 7, three mantissa bits; 0x7F and 0xFF are NaN."""
    code = torch.arange(256, device="cuda")
    exponent, mantissa = (code >> 3) & 15, (code & 7).double()
    size = torch.where(exponent == 0, mantissa / 8 * 2.0 ** -6, (1 + mantissa / 8) * torch.exp2(exponent.double() - 7))
    size = torch.where((code & 127) == 127, torch.full_like(size, math.nan), size)
    return torch.where(code >= 128, -size, size)


def _codes(t):
    return _e4m3_table()[t.view(torch.uint8).int()]


def _to_e4m3(v):
    """Nearest e4m3 value, ties to even, of finite 64-bit values up to 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (v / step).round() * step


def exact(case, seed):
    s = prepare(case, seed)
    k = case["k"]
    at = torch.arange(k, device="cuda") // BLOCK
    if case["op"] == "quant":
        x = s["x"].double()
        if case["gated"]:
            x = x[:, :k] * torch.sigmoid(x[:, :k]) * x[:, k:]
        scale = torch.zeros(x.shape[0], blocks(k), device="cuda", dtype=torch.float64)
        scale = scale.index_reduce(1, at, x.abs(), "amax") / MAX8
        scale = scale.clamp_min(TINY)
        # a code is that of the fp32 quotient by the scale as it is stored: bf16 values often lie on the borders
        quotient = (x / scale.float().double()[:, at]).float().double()
        return _to_e4m3(quotient), scale.t()
    n = case["n"]
    if case["op"] == "dense":
        of = torch.arange(n, device="cuda") // BLOCK
        w = _codes(s["w"]) * s["ws"].double()[of][:, at]
        return (_codes(s["x"]) * s["xs"].double()[at].t()) @ w.t()
    y = s["y"].double()
    bounds = s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        rows = torch.arange(lo, hi, device="cuda") if s["index"] is None else s["index"][lo:hi].long()
        if case["type"] == "fp8":
            of = torch.arange(n, device="cuda") // BLOCK
            w = _codes(s["w"][e]) * s["ws"][e].double()[of][:, at]
            x = _codes(s["x"][rows]) * s["xs"].double()[at][:, rows].t()
        else:
            w, x = s["w"][e].double(), s["x"][rows].double()
        y[lo:hi] = x @ w.t()
    return y

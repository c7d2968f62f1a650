"""Cases of the operators around a served layer's products, with their plain forms.

sort      tokens sorted by expert: row ranges per expert, the token of each row, the row of each choice, and
          the tokens' values spread over those rows (what the grouped products read)
combine   back again: each token's rows summed, with the router's weights or without (the latter is the
          gradient of the spread)
grad      the gradient of the weighted sum: by row and by weight
adapters  low-rank adapters of many requests added to a shared projection's result
verify    drafted tokens held against the target's probabilities, and the token that follows them
"""

import math

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four rows of a verify step, top 8 of 128 experts: a launch's own time counts
        {"name": "sort verify", "op": "sort", "tokens": 4, "top": 8, "experts": 128, "h": 0, "type": "bf16", "drop": 0.0},
        # a long prompt's tokens, spread for the experts' products
        {"name": "sort long prompt", "op": "sort", "tokens": 8192, "top": 8, "experts": 128, "h": 2048, "type": "bf16",
         "drop": 0.0},
        # odd counts, and a third of the choices on experts that another process holds
        {"name": "sort ragged", "op": "sort", "tokens": 1021, "top": 3, "experts": 60, "h": 1003, "type": "f32",
         "drop": 0.35},
        # four rows of a verify step back from the down product
        {"name": "combine verify", "op": "combine", "tokens": 4, "top": 8, "experts": 128, "h": 2048, "type": "f32",
         "out": "bf16", "weights": True, "drop": 0.0},
        # a long prompt back from the experts
        {"name": "combine long prompt", "op": "combine", "tokens": 8192, "top": 8, "experts": 128, "h": 2048,
         "type": "bf16", "out": "bf16", "weights": True, "drop": 0.0},
        # the gradient of a training batch's weighted sum
        {"name": "grad batch", "op": "grad", "tokens": 4096, "top": 8, "experts": 128, "h": 2048, "type": "bf16",
         "drop": 0.0},
        # the same in fp32 with odd rows and experts held elsewhere
        {"name": "grad ragged", "op": "grad", "tokens": 777, "top": 2, "experts": 8, "h": 1003, "type": "f32", "drop": 0.3},
        # one decoded token with its request's adapter
        {"name": "adapter token", "op": "adapters", "rows": 1, "adapters": 8, "rank": 16, "mixed": False, "n": 5120,
         "k": 5120, "out": "f32", "none": 0.0},
        # 64 requests decode at once, adapters of several ranks, some requests without one
        {"name": "adapters decode", "op": "adapters", "rows": 64, "adapters": 24, "rank": 32, "mixed": True, "n": 17408,
         "k": 5120, "out": "f32", "none": 0.2},
        # prompts of a few requests, long runs of one adapter each
        {"name": "adapters prompt", "op": "adapters", "rows": 4096, "adapters": 5, "rank": 64, "mixed": False, "n": 5120,
         "k": 5120, "out": "bf16", "none": 0.0},
        # one request, three drafts
        {"name": "verify one", "op": "verify", "requests": 1, "drafts": 3, "vocab": 131072, "type": "f32",
         "sampled": True, "cut": False, "ragged": False},
        # a large batch of requests with fewer or more drafts each, an odd vocabulary, rare tokens cut off
        {"name": "verify batch", "op": "verify", "requests": 128, "drafts": 3, "vocab": 100003, "type": "f32",
         "sampled": True, "cut": True, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sort", "combine", "grad", "adapters", "adapters", "verify", "verify"))
    if op in ("sort", "combine", "grad"):
        experts = rng.choice((2, 7, 8, 16, 60, 64, 128, 256, 1000))
        top = rng.choice([t for t in (1, 2, 3, 4, 6, 8) if t <= experts])
        h = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            h = max(64, h // 64 * 64)
        kind = rng.choice(("f32", "bf16"))
        most = 8192 * 8 * 2048 // (top * h * (2 if op == "grad" else 1) * (2 if kind == "f32" else 1))
        case = {"op": op, "tokens": _log(rng, 1, max(1, min(16384, most))), "top": top, "experts": experts, "h": h,
                "type": kind, "drop": rng.choice((0.0, 0.0, 0.3, 0.9))}
        if op == "sort":
            case["h"] = rng.choice((0, h))
        if op == "combine":
            case["out"], case["weights"] = rng.choice(("f32", "bf16")), rng.random() < 0.7
        return case
    if op == "adapters":
        n, k = _log(rng, 64, 17408), max(64, _log(rng, 64, 17408) // 8 * 8)
        if rng.random() < 0.7:
            n = max(64, n // 64 * 64)
        rank = rng.choice((8, 16, 16, 24, 32, 64, 128))
        out = rng.choice(("f32", "bf16"))
        most = min(4096 * 3 * 5120 * 2 // (2 * k + (8 if out == "f32" else 4) * n), 4096 * 64 * 2 // rank)
        return {"op": op, "rows": _log(rng, 1, max(1, min(8192, most))), "adapters": rng.choice((1, 3, 8, 24, 64)),
                "rank": rank, "mixed": rng.random() < 0.5, "n": n, "k": k, "out": out,
                "none": rng.choice((0.0, 0.0, 0.2))}
    vocab, drafts = _log(rng, 1000, 262144), rng.choice((1, 2, 3, 3, 5, 8))
    most = 128 * 4 * 100003 // (vocab * (drafts + 1))
    return {"op": op, "requests": _log(rng, 1, max(1, min(256, most))), "drafts": drafts, "vocab": vocab,
            "type": rng.choice(("f32", "bf16")), "sampled": rng.random() < 0.7, "cut": rng.random() < 0.5,
            "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _rows(g, m, k, kind):
    """Normal rows of differing size with a few strong channels."""
    x = _normal(g, m, k) * torch.exp(0.5 * _normal(g, m, 1))
    return (x * torch.where(_uniform(g, k) < 0.01, 20.0, 1.0)).to(kind)


def _choices(g, case):
    """The router's choices, some experts more popular than others, and their weights."""
    t, e, top = case["tokens"], case["experts"], case["top"]
    scores = _normal(g, t, e) + 0.5 * _normal(g, 1, e)
    best, ids = scores.topk(top, dim=1)
    ids = torch.where(_uniform(g, t, top) < case["drop"], -1, ids).to(torch.int32)
    return ids, torch.softmax(best, 1).contiguous()


def _adapter_plan(ids, adapters):
    """Runs of rows by adapter: what a step's program sorts once for all of its layers."""
    key = torch.where(ids < 0, adapters, ids.long())
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=adapters + 1)[:adapters]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    row = torch.arange(len(ids), device="cuda")
    index = torch.where(row < offsets[-1], order, -1)
    return offsets.to(torch.int32), index.to(torch.int32), int(counts.max())


def _probabilities(logits, cut):
    """Their softmax; cut: without the tokens of less than a twentieth of the likeliest one's probability."""
    p = torch.softmax(logits, -1)
    if cut:
        p = torch.where(p < 0.05 * p.amax(-1, keepdim=True), 0.0, p)
        p = p / p.sum(-1, keepdim=True)
    return p


def _workspace(sizes, *shape):
    """Device memory that the framework's call needs, where it does: a program keeps it from step to step."""
    if not own:
        return None
    import gguf_block_quantized_qmv_amd as q
    size = getattr(q, sizes)(*shape)
    return torch.empty(size, device="cuda", dtype=torch.uint8) if size else None


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] in ("sort", "combine", "grad"):
        t, top, h, kind = case["tokens"], case["top"], case["h"], _type(case["type"])
        s["ids"], s["w"] = _choices(g, case)
        if case["op"] == "sort":
            s["offsets"] = torch.zeros(case["experts"] + 1, device="cuda", dtype=torch.int32)
            s["index"] = torch.zeros(t * top, device="cuda", dtype=torch.int32)
            s["places"] = torch.zeros(t, top, device="cuda", dtype=torch.int32)
            s["ws"] = _workspace("qmm_rows_sort_workspace", t, top, case["experts"])
            if h:
                s["x"] = _rows(g, t, h, kind)
                s["rows"] = torch.full((t * top, h), -1.0, device="cuda", dtype=kind)
            return s
        s["places"] = _sorted(s["ids"], case["experts"])[2].contiguous()
        s["z"] = _rows(g, t * top, h, kind)
        if case["op"] == "combine":
            s["y"] = torch.zeros(t, h, device="cuda", dtype=_type(case["out"]))
            if not case["weights"]:
                s["w"] = None
        else:
            s["dy"] = (_normal(g, t, h) * 0.1).to(kind)
            s["dz"] = torch.full((t * top, h), -1.0, device="cuda", dtype=kind)
            s["dw"] = torch.zeros(t, top, device="cuda")
        return s
    if case["op"] == "adapters":
        m, na, rank, n, k = case["rows"], case["adapters"], case["rank"], case["n"], case["k"]
        run = max(1, m // 16) if m > 256 else 1                      # a prompt's rows stand side by side
        owner = torch.randint(0, na, (-(-m // run),), generator=g, device="cuda").repeat_interleave(run)[:m]
        owner = torch.where(_uniform(g, m) < case["none"], -1, owner)
        s["offsets"], s["index"], s["most"] = _adapter_plan(owner, na)
        s["x"] = _rows(g, m, k, torch.bfloat16)
        s["a"] = (_normal(g, na, rank, k) / math.sqrt(k)).to(torch.bfloat16)
        s["b"] = (_normal(g, na, n, rank) / math.sqrt(rank)).to(torch.bfloat16)
        s["scale"] = 0.25 + _uniform(g, na)
        s["ranks"] = None
        if case["mixed"]:                                            # adapters of fewer dimensions, filled up
            s["ranks"] = torch.randint(1, rank + 1, (na,), generator=g, device="cuda", dtype=torch.int32)
        s["base"] = _normal(g, m, n).to(_type(case["out"]))
        s["y"] = s["base"].clone()
        s["ws"] = _workspace("qmm_lora_workspace", m, n, k, rank, na)
        return s
    r, d, v = case["requests"], case["drafts"], case["vocab"]
    logits = 3.0 * _normal(g, r, d + 1, v)
    s["p"] = _probabilities(logits, case["cut"]).to(_type(case["type"]))
    drafter = logits[:, :d] + 0.7 * _normal(g, r, d, v)
    if case["sampled"]:
        s["q"] = _probabilities(drafter, case["cut"]).to(_type(case["type"]))
        drafter = s["q"].float().log() - torch.log(-torch.log(_uniform(g, r, d, v).clamp(1e-30, 1 - 2.0 ** -24)))
    else:
        s["q"] = None
    s["tokens"] = drafter.argmax(-1).to(torch.int32)
    s["u"] = _uniform(g, r, d + 1)
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(0, d + 1, (r,), generator=g, device="cuda", dtype=torch.int32)
    s["accepted"] = torch.zeros(r, device="cuda", dtype=torch.int32)
    s["out"] = torch.zeros(r, d + 1, device="cuda", dtype=torch.int32)
    s["ws"] = _workspace("qmv_verify_drafts_workspace", r, v)
    return s


# ------------------------------------------------------------------ one pass

def _sorted(ids, experts):
    t, top = ids.shape
    flat = ids.flatten().long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, device="cuda", dtype=torch.int64).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:experts].cumsum(0)])
    row = torch.arange(t * top, device="cuda")
    index = torch.where(row < offsets[-1], order // top, -1)
    place = torch.empty_like(order)
    place[order] = row
    place = torch.where(key < experts, place, -1).view(t, top)
    return offsets.to(torch.int32), index.to(torch.int32), place.to(torch.int32)


def _put(rows, places, values):
    """rows with values [tokens, top, h] at their places; choices without a place go to a row that is dropped."""
    n = rows.shape[0]
    at = torch.where(places < 0, n, places.long()).flatten()
    wide = torch.cat([rows, rows[:1]])
    wide[at] = values.reshape(at.numel(), -1).to(rows.dtype)
    return wide[:n]


def _take(z, places):
    """fp32 rows [tokens, top, h] of z at their places, zeros without one."""
    return torch.where(places[:, :, None] < 0, 0.0, z[places.clamp(min=0).long()].float())


def _lora(s):
    """Each adapter's rows side by side in one batch, as long as the longest run."""
    na, rank, index, off, base = s["adapters"], s["rank"], s["index"], s["offsets"].long(), s["base"]
    m = s["rows"]
    row = torch.arange(m, device="cuda")
    used = row < off[-1]
    adapter = (torch.searchsorted(off, row, right=True) - 1).clamp(max=na - 1)
    place = torch.where(used, row - off[adapter], s["most"])
    at = torch.where(used, index.long(), m)                          # rows without an adapter: one that is dropped
    batch = torch.zeros(na, s["most"] + 1, s["k"], device="cuda")
    batch[adapter, place] = s["x"][at.clamp(max=m - 1)].float()
    h = torch.bmm(batch, s["a"].float().transpose(1, 2).contiguous())
    if s["ranks"] is not None:
        h = torch.where(torch.arange(rank, device="cuda") < s["ranks"].long()[:, None, None], h, 0.0)
    delta = torch.bmm(h, s["b"].float().transpose(1, 2).contiguous()) * s["scale"][:, None, None]
    sums = torch.cat([base.float(), torch.zeros(1, s["n"], device="cuda")])
    sums[at] = sums[at] + delta[adapter, place]
    return sums[:m].to(base.dtype)


def _verify(s):
    """In 64 bits: a product of two inputs is exact there, and a token is found in a long running sum."""
    r, d, v = s["requests"], s["drafts"], s["vocab"]
    p, u, tokens = s["p"], s["u"].double(), s["tokens"].long()
    length = torch.full((r,), d, device="cuda") if s["lengths"] is None else s["lengths"].long()
    there = p[:, :d].gather(2, tokens[:, :, None])[:, :, 0].double()
    drafted = torch.ones_like(there) if s["q"] is None else s["q"].gather(2, tokens[:, :, None])[:, :, 0].double()
    good = (u[:, :d] * drafted < there) & (torch.arange(d, device="cuda") < length[:, None])
    accepted = good.long().cumprod(1).sum(1)
    each = torch.arange(r, device="cuda")
    left = p[each, accepted].double()
    refused = (accepted < length)[:, None]
    last = accepted.clamp(max=d - 1)
    if s["q"] is None:
        taken = (torch.arange(v, device="cuda") == tokens[each, last][:, None]).double() * left
    else:
        taken = s["q"][each, last].double()
    rest = torch.where(refused, (left - taken).clamp_min(0.0), left)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, left)
    run = rest.cumsum(1)
    total = run[:, -1:]
    below = (run <= u[:, d:] * total) | (run <= 0)
    pick = below.long().sum(1).clamp(max=v - 1)
    at = torch.arange(d + 1, device="cuda")
    padded = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(at < accepted[:, None], padded, torch.where(at == accepted[:, None], pick[:, None], -1))
    return accepted.to(torch.int32), out.to(torch.int32)


def _run_own(s):
    import gguf_block_quantized_qmv_amd as q
    if s["op"] == "sort":
        plan = q.qmm_rows_sort(s["ids"], s["experts"], offsets=s["offsets"], row_index=s["index"], places=s["places"],
                               ws=s["ws"])
        return plan if not s["h"] else (*plan, q.qmm_rows_spread(s["x"], s["places"], out=s["rows"]))
    if s["op"] == "combine":
        return q.qmm_rows_combine(s["z"], s["places"], s["w"], y=s["y"])
    if s["op"] == "grad":
        return q.qmm_rows_combine_grad(s["dy"], s["z"], s["places"], s["w"], dz=s["dz"], dw=s["dw"])
    if s["op"] == "adapters":
        return q.qmm_lora(s["x"], s["a"], s["b"], s["offsets"], s["y"], row_index=s["index"], scale=s["scale"],
                          ranks=s["ranks"], base=s["base"], ws=s["ws"])
    return q.qmv_verify_drafts(s["p"], s["tokens"], s["u"], q=s["q"], lengths=s["lengths"], accepted=s["accepted"],
                               tokens=s["out"], ws=s["ws"])


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "sort":
        plan = _sorted(s["ids"], s["experts"])
        if not s["h"]:
            return plan
        return (*plan, _put(s["rows"], plan[2], s["x"][:, None].expand(-1, s["top"], -1)))
    if s["op"] == "combine":
        rows = _take(s["z"], s["places"])
        if s["w"] is not None:
            rows = rows * s["w"][:, :, None]
        return rows.sum(1).to(s["y"].dtype)
    if s["op"] == "grad":
        dy = s["dy"].float()[:, None]
        return _put(s["dz"], s["places"], dy * s["w"][:, :, None]), (dy * _take(s["z"], s["places"])).sum(2)
    if s["op"] == "adapters":
        return _lora(s)
    return _verify(s)


# ------------------------------------------------------------------ what a pass cannot do without

ACCEPT = 0.75   # of the drafts that _probabilities' pairs give


def work(case):
    wide = 4 if case.get("type", case.get("out")) == "f32" else 2
    if case["op"] in ("sort", "combine", "grad"):
        t, choices, h = case["tokens"], case["tokens"] * case["top"], case["h"]
        held = choices * (1 - case["drop"])
        if case["op"] == "sort":
            return {"bytes": 12 * choices + 4 * (case["experts"] + 1) + wide * h * (t + held), "flops": choices}
        if case["op"] == "combine":
            out = 4 if case["out"] == "f32" else 2
            return {"bytes": (8 if case["weights"] else 4) * choices + wide * h * held + out * h * t,
                    "flops": 2 * h * held}
        return {"bytes": 12 * choices + wide * h * (t + 2 * held), "flops": 3 * h * held}
    if case["op"] == "adapters":
        m, na, n, k = case["rows"] * (1 - case["none"]), case["adapters"], case["n"], case["k"]
        rank = case["rank"] / 2 if case["mixed"] else case["rank"]
        groups = case["rows"] if case["rows"] <= 256 else 16
        busy = na * (1 - (1 - 1 / na) ** groups)                     # adapters with a row
        return {"bytes": 2 * m * k + 2 * busy * rank * (n + k) + 2 * wide * m * n, "flops": 2 * m * rank * (n + k)}
    r, d, v = case["requests"], case["drafts"], case["vocab"]
    lengths = range(d + 1) if case["ragged"] else [d]
    refused = sum(1 - ACCEPT ** n for n in lengths) / len(lengths) if case["sampled"] else 0
    return {"bytes": r * v * wide * (1 + refused), "flops": 2 * r * v}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify" or case["op"] == "sort" and not case["h"]:
        return None                                                  # whole numbers
    if case["op"] == "sort":
        ids = s["ids"].flatten().tolist()
        held = sorted((e, i) for i, e in enumerate(ids) if 0 <= e < case["experts"])
        rows = s["rows"].double()
        if held:
            rows[:len(held)] = s["x"].double()[torch.tensor([i // case["top"] for _, i in held], device="cuda")]
        return None, None, None, rows
    if case["op"] == "combine":
        y = torch.zeros(case["tokens"], case["h"], device="cuda", dtype=torch.float64)
        for j in range(case["top"]):
            here = (s["places"][:, j] >= 0).nonzero()[:, 0]
            rows = s["z"][s["places"][here, j].long()].double()
            y[here] += rows if s["w"] is None else rows * s["w"][here, j, None].double()
        return y
    if case["op"] == "grad":
        dz, dw = s["dz"].double(), s["dw"].double()
        for j in range(case["top"]):
            here = (s["places"][:, j] >= 0).nonzero()[:, 0]
            at = s["places"][here, j].long()
            dy = s["dy"][here].double()
            dz[at] = dy * s["w"][here, j, None].double()
            dw[here, j] = (dy * s["z"][at].double()).sum(1)
        return dz, dw
    y, bounds = s["base"].double(), s["offsets"].tolist()
    for e in range(case["adapters"]):
        rows = s["index"][bounds[e]:bounds[e + 1]].long()
        rank = case["rank"] if s["ranks"] is None else int(s["ranks"][e])
        h = s["x"][rows].double() @ s["a"][e, :rank].double().t()
        y[rows] += float(s["scale"][e]) * (h @ s["b"][e, :, :rank].double().t())
    return y

"""One verify step of several requests, as a program makes it: drafted rows through a shared e4m3 projection with each
request's adapter, through a routed layer of e4m3 experts, through a head, and to the decision on the drafts. Every new
step is held to the fp64 oracle on its own inputs (tolerances of test_gpu_rows.py and test_gpu_lora.py); then the whole
step is replayed from a graph under other routings, adapters and drafts."""

import numpy as np
import pytest

from gpu_util import device, host
from oracle import rows_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q():
    import gguf_block_quantized_qmv_amd as mod
    return mod


@pytest.fixture(scope="module")
def dev():
    return device()


def codes(g, *shape):
    c = g.integers(0, 256, shape, dtype=np.uint8)
    return np.where((c & 127) > 0x70, c ^ 0x40, c)              # no NaN, moderate sizes


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def blocks(k):
    return -(-k // 128)


class Model:
    def __init__(self, g, dev, h, ffn, experts, vocab, adapters, rank):
        def weights(*shape):
            n, k = shape[-2:]
            s = 2e-4 * np.exp(0.2 * g.standard_normal((*shape[:-2], blocks(n), blocks(k)))).astype(np.float32)
            return up(codes(g, *shape), dev), up(s.astype(np.float32), dev)

        self.h, self.ffn, self.experts, self.vocab, self.adapters, self.rank = h, ffn, experts, vocab, adapters, rank
        self.proj, self.gate_up, self.down = weights(h, h), weights(experts, 2 * ffn, h), weights(experts, h, ffn)
        self.head = weights(vocab, h)
        small = lambda *s: up((g.standard_normal(s) / np.sqrt(s[-1])).astype(np.float32), dev).to(torch.bfloat16)
        self.a, self.b = small(adapters, rank, h), small(adapters, h, rank)
        self.scale = up(g.uniform(0.5, 2, adapters).astype(np.float32), dev)
        self.ranks = up(g.integers(1, rank + 1, adapters).astype(np.int32), dev)


class Batch:
    """What changes from step to step."""

    def __init__(self, g, dev, m, requests, drafts, top):
        rows = requests * (drafts + 1)
        self.x = up(g.standard_normal((rows, m.h)).astype(np.float32), dev).to(torch.bfloat16)
        owner = g.integers(-1, m.adapters, requests)
        self.adapter = up(np.repeat(owner, drafts + 1)[:, None].astype(np.int32), dev)
        self.ids = up(np.argsort(g.random((rows, m.experts)), 1)[:, :top].astype(np.int32), dev)
        self.weights = up(g.dirichlet(np.ones(top), rows).astype(np.float32), dev)
        self.drafts = up(g.integers(0, m.vocab, (requests, drafts)).astype(np.int32), dev)
        self.u = up((g.random((requests, drafts + 1)) ** 8).astype(np.float32), dev)   # small ones, so that some drafts stand
        self.lengths = up(g.integers(0, drafts + 1, requests).astype(np.int32), dev)

    def copy_(self, other):
        for k, v in vars(self).items():
            v.copy_(getattr(other, k))


def step(q, m, b):
    s = {}
    s["runs"], s["rows"], _ = q.qmm_rows_sort(b.adapter, m.adapters)
    xq, xs = q.qmm_fp8_quant(b.x)
    s["shared"] = q.qmm_fp8(*m.proj, xq, xs, m.h, m.h)
    s["y"] = q.qmm_lora(b.x, m.a, m.b, s["runs"], s["shared"].clone(), row_index=s["rows"], scale=m.scale, ranks=m.ranks)
    hidden = torch.tanh(s["y"] * 0.01).to(torch.bfloat16)
    s["plan"] = q.qmm_rows_sort(b.ids, m.experts)
    hq, hs = q.qmm_fp8_quant(hidden)
    gu = q.qmm_fp8_grouped(*m.gate_up, hq, hs, s["plan"][0], 2 * m.ffn, m.h, row_index=s["plan"][1])
    fq, fs = q.qmm_fp8_quant_silu_mul(gu)
    s["z"] = q.qmm_fp8_grouped(*m.down, fq, fs, s["plan"][0], m.h, m.ffn, out_dtype=torch.bfloat16)
    s["out"] = q.qmm_rows_combine(s["z"], s["plan"][2], b.weights, out_dtype=torch.bfloat16)
    oq, os_ = q.qmm_fp8_quant(s["out"])
    logits = q.qmm_fp8(*m.head, oq, os_, m.vocab, m.h)
    scaled = 8 * logits / logits.abs().amax(1, keepdim=True)
    requests, drafts = b.drafts.shape
    s["p"] = torch.softmax(scaled, 1).view(requests, drafts + 1, m.vocab)
    s["accepted"], s["tokens"] = q.qmv_verify_drafts(s["p"], b.drafts, b.u, lengths=b.lengths)
    return s


def f64(t):
    return t.double().cpu().numpy()


SHAPES = [(1, 3, 256, 128, 8, 2, 1000, 2, 8), (5, 3, 512, 256, 16, 4, 20011, 3, 16), (40, 2, 384, 128, 6, 3, 5003, 5, 40)]


@pytest.mark.parametrize("requests,drafts,h,ffn,experts,top,vocab,adapters,rank", SHAPES)
def test_every_step_against_the_oracle(q, dev, requests, drafts, h, ffn, experts, top, vocab, adapters, rank):
    g = np.random.default_rng(requests)
    m = Model(g, dev, h, ffn, experts, vocab, adapters, rank)
    b = Batch(g, dev, m, requests, drafts, top)
    s = step(q, m, b)
    torch.cuda.synchronize()
    for got, want in zip((s["runs"], s["rows"]), o.sort(host(b.adapter), adapters)):
        assert np.array_equal(host(got), want)
    for got, want in zip(s["plan"], o.sort(host(b.ids), experts)):
        assert np.array_equal(host(got), want)
    exact, mag = o.lora(f64(b.x), f64(m.a), f64(m.b), host(s["runs"]), host(s["rows"]), host(m.scale), host(m.ranks),
                        f64(s["shared"]))
    tol = (2 * h + 48 + 6 * 128 + 8) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(exact)
    assert (np.abs(f64(s["y"]) - exact) <= tol).all()
    assert not np.array_equal(f64(s["y"]), f64(s["shared"])) or (host(b.adapter) < 0).all()
    exact, mag = o.combine(f64(s["z"]), host(s["plan"][2]), host(b.weights))
    tol = top * 2.0 ** -24 * mag
    assert (np.abs(f64(s["out"]) - exact) <= tol + 2.0 ** -8 * (np.abs(exact) + tol)).all() and np.isfinite(exact).all()
    accepted, tokens = o.verify(f64(s["p"]), None, host(b.drafts), host(b.lengths), host(b.u))
    assert np.array_equal(host(s["accepted"]), accepted) and np.array_equal(host(s["tokens"]), tokens)


def test_the_step_replayed_from_a_graph(q, dev):
    g = np.random.default_rng(9)
    m = Model(g, dev, 512, 256, 16, 20011, 3, 16)
    b = Batch(g, dev, m, 6, 3, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(q, m, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kept = step(q, m, b)
    for _ in range(4):
        b.copy_(Batch(g, dev, m, 6, 3, 4))
        eager = step(q, m, b)                                  # the same inputs, eagerly, between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("runs", "rows", "y", "out", "p", "accepted", "tokens"):
            assert torch.equal(kept[k], eager[k]), k


def test_a_gradient_through_the_experts(q, dev):
    # a routed layer of bf16 experts between spread and weighted sum, and its gradient by the way back: the products with the
    # transposed weights are the library's own grouped products. Against the formula in fp64 on the steps' inputs.
    g = np.random.default_rng(10)
    tokens, h, n, experts, top = 50, 64, 48, 5, 3
    x = up(g.standard_normal((tokens, h)).astype(np.float32), dev).to(torch.bfloat16)
    ids = np.argsort(g.random((tokens, experts)), 1)[:, :top].astype(np.int32)
    ids[g.random(ids.shape) < 0.2] = -1
    w = up((g.standard_normal((experts, n, h)) / 8).astype(np.float32), dev).to(torch.bfloat16)
    weights = up(g.dirichlet(np.ones(top), tokens).astype(np.float32), dev)
    dy = up(g.standard_normal((tokens, n)).astype(np.float32), dev).to(torch.bfloat16)
    offsets, index, places = q.qmm_rows_sort(up(ids, dev), experts)
    rows = q.qmm_rows_spread(x, places)
    z = q.qmm_bf16_grouped(w, rows, offsets, n, h, out_dtype=torch.bfloat16)
    assert torch.equal(z, q.qmm_bf16_grouped(w, x, offsets, n, h, row_index=index, out_dtype=torch.bfloat16))
    y = q.qmm_rows_combine(z, places, weights)
    dz, dweights = q.qmm_rows_combine_grad(dy, z, places, weights)
    drows = q.qmm_bf16_grouped(w.transpose(1, 2).contiguous(), dz, offsets, h, n, out_dtype=torch.bfloat16)
    dx = q.qmm_rows_combine(drows, places)
    # fp64, with the roundings to bf16 between the steps: half a step each, and the products' fp32 sums
    x64, w64, dy64, p = f64(x), f64(w), f64(dy), f64(weights)
    ref_y, ref_dx, ref_dp = np.zeros((tokens, n)), np.zeros((tokens, h)), np.zeros((tokens, top))
    mag_y, mag_dx, mag_dp = np.zeros_like(ref_y), np.zeros_like(ref_dx), np.zeros_like(ref_dp)
    for t, j in np.ndindex(*ids.shape):
        if ids[t, j] < 0:
            continue
        e = w64[ids[t, j]]
        zz, back = e @ x64[t], p[t, j] * (dy64[t] @ e)
        ref_y[t] += p[t, j] * zz
        ref_dp[t, j] = dy64[t] @ zz
        ref_dx[t] += back
        mag_y[t] += p[t, j] * (np.abs(e) @ np.abs(x64[t]))
        mag_dp[t, j] = np.abs(dy64[t]) @ (np.abs(e) @ np.abs(x64[t]))
        mag_dx[t] += p[t, j] * (np.abs(dy64[t]) @ np.abs(e))
    one = 2.0 ** -8 + (2 * 64 + 40 + 16) * 2.0 ** -24          # a rounding to bf16 and a product's fp32 sums
    assert (np.abs(f64(y) - ref_y) <= (one + 4 * 2.0 ** -24) * mag_y).all()
    assert (np.abs(f64(dweights) - ref_dp) <= (one + 40 * 2.0 ** -24) * mag_dp).all()
    assert (f64(dweights)[ids < 0] == 0).all()
    assert (np.abs(f64(dx) - ref_dx) <= (2 * one + 2.0 ** -15) * mag_dx).all()   # dz's rounding, and the rows'

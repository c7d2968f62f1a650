"""The e4m3 and grouped products give the same bits from call to call, whatever the workspace held, and an expert's
rows the same bits wherever its matrix and rows lie. Sizes with the plan each takes: tests/fp8_plans.py (whole tiles,
tiles cut along k, both in one call, every grouped tile)."""

import numpy as np
import pytest

from fp8_plans import DENSE, GROUPED, LEAD, RUNS, rows_of
from gpu_util import device
from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
KINDS = [("fp8", False, F32), ("fp8", False, BF16), ("fp8", True, BF16), ("bf16", False, F32), ("bf16", False, BF16)]


@pytest.fixture(scope="module")
def q():
    import gguf_block_quantized_qmv_amd as mod
    return mod


@pytest.fixture(scope="module")
def dev():
    return device()


def codes(g, dev, *shape):
    c = torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8)
    return torch.where((c & 127) == 127, c ^ 1, c)


def scales(g, dev, *shape):
    return torch.rand(*shape, generator=g, device=dev) + 0.5


def same_bits(a, b):
    return bool((a.view(torch.uint8) == b.view(torch.uint8)).all())


@pytest.mark.parametrize("m,n,k,fast,out", [
    pytest.param(m, n, k, fast, out, id=f"{m}x{n}x{k}-{'fast' if fast else str(out)[6:]}")
    for m, n, k, fast, _ in DENSE for out in ((BF16,) if fast else (F32, BF16))])
def test_dense_repeats(q, dev, m, n, k, fast, out):
    g = torch.Generator(device=dev).manual_seed(m + n + k)
    w, x = codes(g, dev, n, k), codes(g, dev, m, k)
    ws, xs = scales(g, dev, o.blocks(n), o.blocks(k)), scales(g, dev, o.blocks(k), m)
    plan = next(p for *shape, p in DENSE if shape == [m, n, k, fast])
    need = q.qmm_fp8_workspace(m, n, k, out, fast)
    assert (need > 0) == (plan[3] > 0)
    first = q.qmm_fp8(w, ws, x, xs, n, k, out_dtype=out, fast_sums=fast)
    space = torch.empty(need + 256, dtype=torch.uint8, device=dev)
    for fill in (0xFF, 0x00, 0x3C):
        space.fill_(fill)
        y = torch.empty_like(first)
        q.qmm_fp8(w, ws, x, xs, n, k, y=y, ws=space[:need] if need else None, fast_sums=fast)
        assert same_bits(y, first) and bool((space[need:] == fill).all())


def grouped(q, kind, fast, w, ws, x, xs, off, n, k, y, index=None):
    if kind == "fp8":
        return q.qmm_fp8_grouped(w, ws, x, xs, off, n, k, row_index=index, y=y, fast_sums=fast)
    return q.qmm_bf16_grouped(w, x, off, n, k, row_index=index, y=y)


def operands(g, dev, kind, e, n, k, x_rows):
    if kind == "bf16":
        return (torch.randn(e, n, k, generator=g, device=dev).to(BF16), None,
                torch.randn(x_rows, k, generator=g, device=dev).to(BF16), None)
    return (codes(g, dev, e, n, k), scales(g, dev, e, o.blocks(n), o.blocks(k)), codes(g, dev, x_rows, k),
            scales(g, dev, o.blocks(k), x_rows))


@pytest.mark.parametrize("kind,fast,out", KINDS)
@pytest.mark.parametrize("runs,n,k", [c[:3] for c in GROUPED])
def test_grouped_repeats_and_does_not_see_the_other_experts(q, dev, runs, n, k, kind, fast, out):
    # a row's sums go block after block of k in every tile, so its expert's matrix alone gives the same bits
    g = torch.Generator(device=dev).manual_seed(n + k)
    counts, rows = RUNS[runs], rows_of(runs)
    w, ws, x, xs = operands(g, dev, kind, len(counts), n, k, 70)
    index = torch.randint(-3, 75, (rows,), generator=g, device=dev, dtype=torch.int32)
    bounds = (np.concatenate([[0], np.cumsum(counts)]) + LEAD).tolist()
    off = torch.tensor(bounds, dtype=torch.int32, device=dev)
    first = grouped(q, kind, fast, w, ws, x, xs, off, n, k, torch.full((rows, n), -7.0, dtype=out, device=dev), index)
    again = grouped(q, kind, fast, w, ws, x, xs, off, n, k, torch.full((rows, n), -7.0, dtype=out, device=dev), index)
    assert same_bits(first, again)
    for e in np.argsort(counts)[-4:]:
        lo, hi = bounds[e], bounds[e + 1]
        alone = torch.empty(hi - lo, n, dtype=out, device=dev)
        grouped(q, kind, fast, w[e:e + 1], None if ws is None else ws[e:e + 1], x, xs,
                torch.tensor([0, hi - lo], dtype=torch.int32, device=dev), n, k, alone, index[lo:hi].contiguous())
        assert same_bits(alone, first[lo:hi]), int(e)


@pytest.mark.parametrize("kind,fast,out", KINDS)
def test_a_bank_beyond_4_gib(q, dev, kind, fast, out):
    e, n, k, rows = (66 if kind == "fp8" else 34), 8192, 8192, 40
    g = torch.Generator(device=dev).manual_seed(3)
    if kind == "fp8":
        w = torch.randint(0, 120, (e, n, k), dtype=torch.uint8, device=dev, generator=g)
        ws, xs = scales(g, dev, e, 64, 64), scales(g, dev, 64, rows)
        x = codes(g, dev, rows, k)
    else:
        w, ws, xs = torch.randn(e, n, k, dtype=BF16, device=dev, generator=g), None, None
        x = torch.randn(rows, k, dtype=BF16, device=dev, generator=g)
    off = torch.zeros(e + 1, dtype=torch.int32, device=dev)
    off[-1] = rows
    y = grouped(q, kind, fast, w, ws, x, xs, off, n, k, torch.zeros(rows, n, dtype=out, device=dev))
    alone = torch.zeros(rows, n, dtype=out, device=dev)
    grouped(q, kind, fast, w[-1:].clone(), None if ws is None else ws[-1:].clone(), x, xs,
            torch.tensor([0, rows], dtype=torch.int32, device=dev), n, k, alone)
    assert same_bits(y, alone) and bool(torch.isfinite(alone).all()) and bool((alone != 0).any())


@pytest.mark.parametrize("out", [F32, BF16])
def test_an_empty_batch_runs_through_a_layer(q, dev, out):
    w, ws = torch.zeros(256, 128, dtype=E4M3, device=dev), torch.ones(2, 1, device=dev)
    down, ds = torch.zeros(64, 128, dtype=E4M3, device=dev), torch.ones(1, 1, device=dev)
    y = q.qmm_fp8(w, ws, *q.qmm_fp8_quant(torch.empty(0, 128, dtype=out, device=dev)), 256, 128, out_dtype=out)
    z = q.qmm_fp8(down, ds, *q.qmm_fp8_quant_silu_mul(y), 64, 128, out_dtype=out)
    assert y.shape == (0, 256) and z.shape == (0, 64) and z.dtype == out


@pytest.mark.parametrize("kind,fast,out", KINDS)
def test_a_captured_call_follows_the_routing_that_it_finds(q, dev, kind, fast, out):
    # offsets and row indexes are read on the device: a replay takes those that are there by then
    n, k, rows, e = 520, 400, 700, 9
    g = torch.Generator(device=dev).manual_seed(5)
    w, ws, x, xs = operands(g, dev, kind, e, n, k, 200)
    index, off = torch.zeros(rows, dtype=torch.int32, device=dev), torch.zeros(e + 1, dtype=torch.int32, device=dev)
    y = torch.empty(rows, n, dtype=out, device=dev)
    off[1:] = rows
    grouped(q, kind, fast, w, ws, x, xs, off, n, k, y, index)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        grouped(q, kind, fast, w, ws, x, xs, off, n, k, y, index)
    routings = ([0] * 10, [0, 700] + [700] * 8, [3, 3, 4, 260, 260, 517, 580, 581, 690, 695], list(range(0, 700, 70)),
                [0] * 9 + [700])
    for bounds in routings:
        off.copy_(torch.tensor(bounds, dtype=torch.int32))
        index.copy_(torch.randint(-3, 205, (rows,), generator=g, device=dev, dtype=torch.int32))
        want = torch.full_like(y, -7.0)
        grouped(q, kind, fast, w, ws, x, xs, off, n, k, want, index)
        y.fill_(-7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(y, want), bounds
        assert bool((want[:bounds[0]] == -7.0).all() and (want[bounds[-1]:] == -7.0).all())

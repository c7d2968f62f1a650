"""GPU parity of the low-rank adapters with the fp64 oracle.

Tolerance, from the arithmetic. A product of two bf16 values is exact in fp32. A x[r] adds k of them, and fewer than 24
parts' sums, each add off by at most one fp32 step (2^-23 of the running magnitude, which covers truncation); the scale
rounds once. The result goes through the matrix cores in three bf16 parts that add up to it exactly, three products for
each of `rank` dimensions; each add is off by at most a step. All of that acts on sums no larger than
M = |scale| sum |b| sum |a x|, so the delta is within (2 k + 48 + 6 * 128 + 8) * 2^-24 * M for ranks up to 128 (padded by
zeros, which add nothing). The sum with base rounds once: 2^-24 of the value. A bf16 result adds half a step, 2^-8.
"""

import numpy as np
import pytest

import lora_cases as cases
from gpu_util import device, guarded, guards_intact, host
from oracle import rows_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    import gguf_block_quantized_qmv_amd as mod
    return mod


@pytest.fixture(scope="module")
def dev():
    return device()


def rng(*seed):
    return np.random.default_rng(seed)


def bf16(g, *shape):
    v = (g.standard_normal(shape) * 10.0 ** g.uniform(-1, 1, (*shape[:-1], 1))).astype(np.float32)
    return torch.from_numpy(v).to(torch.bfloat16)


def up(a, dev):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def tolerance(exact, mag, k, out):
    t = (2 * k + 48 + 6 * 128 + 8) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(exact)
    return t + (2.0 ** -8 * (np.abs(exact) + t) if out == "bf16" else 0)


def check(got, exact, tol):
    bad = ~(np.abs(got - exact) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4].tolist(), exact[bad][:4].tolist(),
                           tol[bad][:4].tolist())


class Case:
    """Rows by adapter (-1: none), sorted; weights, and what the call needs."""

    def __init__(self, g, rows, n, k, rank, adapters, out, mixed=True, scaled=True, owner=None):
        if owner is None:
            owner = g.integers(-1, adapters, rows)
        self.owner = np.asarray(owner)
        self.offsets, self.index, _ = o.sort(self.owner[:, None].astype(np.int32), adapters)
        self.x, self.a, self.b = bf16(g, rows, k), bf16(g, adapters, rank, k), bf16(g, adapters, n, rank)
        self.scale = g.uniform(-2, 2, adapters).astype(np.float32) if scaled else None
        self.ranks = g.integers(0, rank + 2, adapters).astype(np.int32) if mixed else None
        self.base = torch.from_numpy(g.standard_normal((rows, n)).astype(np.float32) * 30).to(TYPES[out])
        self.n, self.k, self.rank, self.adapters, self.rows, self.out = n, k, rank, adapters, rows, out

    def exact(self):
        return o.lora(f64(self.x), f64(self.a), f64(self.b), self.offsets, self.index, self.scale, self.ranks, f64(self.base))

    def args(self, dev):
        return dict(x=self.x.to(dev), a=self.a.to(dev), b=self.b.to(dev), offsets=up(self.offsets, dev),
                    row_index=up(self.index, dev), scale=up(self.scale, dev), ranks=up(self.ranks, dev))

    def run(self, q, dev):
        y, buf = guarded((self.rows, self.n), TYPES[self.out], dev)
        y.copy_(self.base)
        q.qmm_lora(y=y, **self.args(dev))
        torch.cuda.synchronize()
        assert guards_intact(buf)
        return f64(y)

    def holds(self, got):
        exact, mag = self.exact()
        check(got, exact, tolerance(exact, mag, self.k, self.out))
        assert np.array_equal(got[self.owner < 0], f64(self.base)[self.owner < 0])


@pytest.mark.parametrize("rows,n,k,rank,adapters", [
    (1, 1, 8, 8, 1), (1, 5120, 512, 16, 8), (2, 64, 64, 16, 2), (5, 65, 72, 8, 3), (16, 257, 200, 24, 5), (17, 300, 136, 32, 4),
    (40, 129, 1000, 40, 40), (64, 1000, 512, 64, 24), (63, 260, 264, 128, 3), (130, 190, 520, 72, 2), (300, 333, 200, 16, 3),
    (700, 259, 136, 64, 2), (400, 1100, 72, 104, 1), (100, 70, 64, 8, 1024), (530, 130, 72, 128, 1), (1100, 75, 64, 8, 2),
    (1030, 66, 80, 24, 5), (1500, 40, 64, 8, 700)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_against_the_oracle(q, dev, rows, n, k, rank, adapters, out):
    for mixed in (True, False):
        c = Case(rng(rows, n, k, rank), rows, n, k, rank, adapters, out, mixed=mixed, scaled=mixed)
        c.holds(c.run(q, dev))


@pytest.mark.parametrize("k", [8, 56, 64, 248, 256, 264, 4096, 17408])
def test_lengths_of_k(q, dev, k):
    for rows, rank in ((3, 16), (40, 16), (5, 40), (40, 40), (5, 24)):   # one launch up to some k, or two
        c = Case(rng(k, rows), rows, 96, k, rank, 3, "f32")
        c.holds(c.run(q, dev))


@pytest.mark.parametrize("rank", [16, 40, 96])
@pytest.mark.parametrize("rows,parts", [(1000, 4), (2049, 4), (3000, 4), (4200, 3)])
def test_long_runs_in_several_parts_of_k(q, dev, rows, rank, parts):
    assert rank != 40 or q.qmm_lora_workspace(rows, 70, 2600, rank, 5) == parts * rows * rank * 4
    c = Case(rng(rows, rank), rows, 70, 2600, rank, 5, "bf16")
    c.holds(c.run(q, dev))


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("rank", [16, 40, 128])
def test_one_adapter_for_all(q, dev, rows, rank):   # tiles of 16 rows, and of 32 from 128 (512) rows on
    c = Case(rng(rows, rank), rows, 100, 96, rank, 1, "f32", owner=np.zeros(rows), mixed=False)
    c.holds(c.run(q, dev))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("adapters", [3, 40])
@pytest.mark.parametrize("rank,n", [(16, 18901), (40, 18896), (72, 18904)])
def test_results_larger_than_the_caches(q, dev, out, adapters, rank, n):
    c = Case(rng(n, adapters), 1800 if rank > 64 else 900, n, 64, rank, adapters, out)
    c.holds(c.run(q, dev))


def test_uneven_runs(q, dev):
    g = rng(3)
    owner = np.concatenate([np.full(150, 4), np.full(1, 0), np.full(64, 6), np.full(30, -1), np.full(33, 2)])
    for adapters in (7, 300):                                  # tiles of many rows, and of few
        c = Case(g, len(owner), 200, 128, 32, adapters, "bf16", owner=g.permutation(owner))
        c.holds(c.run(q, dev))


def test_rows_in_order_without_an_index(q, dev):
    g = rng(4)
    c = Case(g, 50, 90, 80, 16, 3, "f32", owner=np.sort(g.integers(0, 3, 50)))
    y = c.base.to(dev)
    a = c.args(dev)
    a["row_index"] = None
    q.qmm_lora(y=y, **a)
    c.holds(f64(y))
    a["offsets"] = torch.tensor([2, 10, 10, 41], dtype=torch.int32, device=dev)   # rows before the first and behind the last
    y2 = c.base.to(dev)
    q.qmm_lora(y=y2, **a)
    exact, mag = o.lora(f64(c.x), f64(c.a), f64(c.b), [2, 10, 10, 41], None, c.scale, c.ranks, f64(c.base))
    check(f64(y2), exact, tolerance(exact, mag, c.k, "f32"))
    assert torch.equal(y2[:2].cpu(), c.base[:2]) and torch.equal(y2[41:].cpu(), c.base[41:])


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_base_apart_from_y(q, dev, out):
    for rank in (24, 40):
        apart(q, dev, out, Case(rng(5), 45, 131, 64, rank, 4, out))


def apart(q, dev, out, c):
    c.ranks[0] = 0                                             # no dimension at all: base as it is
    y, buf = guarded((45, 131), TYPES[out], dev)
    y.fill_(7.0)
    q.qmm_lora(y=y, base=c.base.to(dev), **c.args(dev))
    torch.cuda.synchronize()
    assert guards_intact(buf)
    assert (f64(y)[c.owner < 0] == 7).all()
    there = c.run(q, dev)
    assert np.array_equal(f64(y)[c.owner >= 0], there[c.owner >= 0])


def test_what_lies_behind_a_rank_does_not_matter(q, dev):
    for rank in (8, 24, 40, 64, 128):
        c = Case(rng(6, rank), 30, 140, 200, rank, 5, "f32")
        c.ranks[:5] = [0, 1, rank // 2 + 1, rank - 1, rank + 9]
        clean = c.run(q, dev)
        c.holds(clean)
        a, b = c.a.clone(), c.b.clone()
        for e in range(5):
            used = min(int(c.ranks[e]), rank)
            a[e, used:], b[e, :, used:] = float("nan"), float("inf")
        c.a, c.b = a, b
        assert np.array_equal(c.run(q, dev), clean)
        c.ranks[:] = -3                                        # below zero: none
        assert np.array_equal(c.run(q, dev), f64(c.base))


def test_rows_that_are_not_finite_touch_no_other(q, dev):
    for rows, rank in ((20, 16), (20, 40), (300, 16), (500, 40)):
        c = Case(rng(7, rows), rows, 150, 136, rank, 3, "f32", mixed=False)
        clean = c.run(q, dev)
        owned = np.flatnonzero(c.owner >= 0)
        bad = owned[[0, 7, -1]]
        c.x[bad[0], 3], c.x[bad[1], 135], c.x[bad[2], 0] = float("nan"), float("inf"), -float("inf")
        got = c.run(q, dev)
        keep = np.setdiff1d(np.arange(rows), bad)
        assert np.array_equal(got[keep], clean[keep]) and not np.isfinite(got[bad]).any()
        c.x[bad] = 0
        clean = c.run(q, dev)
        c.b[1, 40, 2] = float("nan")
        got, hit = c.run(q, dev), c.owner == 1
        hit[bad] &= True
        cols = np.arange(150) != 40
        assert np.array_equal(got[:, cols], clean[:, cols]) and np.isnan(got[hit, 40]).all()
        assert np.array_equal(got[~hit], clean[~hit])


def test_large_and_small_values_keep_their_bits(q, dev):
    # sums whose upper and lower bits both count: 2^20 + 1 through one dimension, against whole numbers
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 2.0 ** 20, 1.0
    x[1, 5], x[1, 9] = -(2.0 ** 23), 1.0
    x[2, 0], x[2, 63] = 3.0e38, 1.0
    a = torch.ones((1, 8, 64), dtype=torch.bfloat16)
    b = torch.zeros((1, 40, 8), dtype=torch.bfloat16)
    b[0, :, 0], b[0, 1, 0] = 1.0, 3.0
    y = torch.zeros((3, 40), device=dev)
    q.qmm_lora(x.to(dev), a.to(dev), b.to(dev), torch.tensor([0, 3], dtype=torch.int32, device=dev), y,
               ranks=torch.ones(1, dtype=torch.int32, device=dev))
    big = float(torch.tensor(3.0e38).to(torch.bfloat16))
    assert host(y)[0, :2].tolist() == [2.0 ** 20 + 1, 3 * (2.0 ** 20 + 1)] and host(y)[1, 0] == 1 - 2.0 ** 23
    assert host(y)[2, 0] == np.float32(big) and host(y)[2, 1] == np.inf


def test_a_rows_bits_whatever_stands_beside_it(q, dev):
    # up to 16 rows: the same bits alone, in company and under other adapters beside it
    for rank in (32, 40):                                      # one launch, and two
        same_bits(q, dev, Case(rng(8), 16, 300, 1000, rank, 4, "f32", owner=np.arange(16) % 4, mixed=False))
    big = Case(rng(9), 900, 300, 520, 64, 5, "f32")            # and from call to call
    assert np.array_equal(big.run(q, dev), big.run(q, dev))


def same_bits(q, dev, c):
    full = c.run(q, dev)
    a = c.args(dev)
    for r in (0, 5, 15):
        off = np.zeros(5, np.int32)
        off[c.owner[r] + 1:] = 1
        y = c.base[r:r + 1].to(dev)
        q.qmm_lora(a["x"][r:r + 1].contiguous(), a["a"], a["b"], up(off, dev), y, scale=a["scale"])
        assert np.array_equal(f64(y)[0], full[r])
        alone = c.owner[r]
        y = c.base[r:r + 1].to(dev)
        q.qmm_lora(a["x"][r:r + 1].contiguous(), a["a"][alone:alone + 1], a["b"][alone:alone + 1],
                   torch.tensor([0, 1], dtype=torch.int32, device=dev), y, scale=a["scale"][alone:alone + 1])
        assert np.array_equal(f64(y)[0], full[r])


def test_indexes_and_offsets_outside(q, dev):
    c = Case(rng(10), 30, 70, 64, 8, 2, "f32", owner=np.repeat([0, 1], 15), mixed=False)
    a = c.args(dev)
    a["row_index"] = torch.tensor([0, -1, 30, 5, 1 << 30, -(1 << 31), 7], dtype=torch.int32, device=dev)
    a["offsets"] = torch.tensor([-4, 4, 99], dtype=torch.int32, device=dev)        # clamped to 0 and 7
    y, buf = guarded((30, 70), torch.float32, dev)
    y.copy_(c.base)
    q.qmm_lora(y=y, **a)
    torch.cuda.synchronize()
    assert guards_intact(buf)
    exact, mag = o.lora(f64(c.x), f64(c.a), f64(c.b), [0, 4, 7], host(a["row_index"]), c.scale, None, f64(c.base))
    check(f64(y), exact, tolerance(exact, mag, c.k, "f32"))
    a["offsets"] = torch.tensor([5, 2, 0], dtype=torch.int32, device=dev)          # decreasing: nothing outside is touched
    q.qmm_lora(y=y, **a)
    torch.cuda.synchronize()
    assert guards_intact(buf)


def test_nothing_to_do(q, dev):
    a = torch.zeros((2, 8, 16), dtype=torch.bfloat16, device=dev)
    b = torch.zeros((2, 10, 8), dtype=torch.bfloat16, device=dev)
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    y = torch.empty((0, 10), device=dev)
    assert q.qmm_lora(torch.empty((0, 16), dtype=torch.bfloat16, device=dev), a, b, off, y) is y
    y = torch.full((4, 10), float("nan"), device=dev)          # rows, and all without an adapter
    q.qmm_lora(torch.zeros((4, 16), dtype=torch.bfloat16, device=dev), a, b, off, y)
    assert bool(torch.isnan(y).all())


def test_past_4_gib(q, dev):
    # x, and a bank whose last adapter lies behind 4 GiB
    k, adapters, rows = 16384, 1024, 5
    a = torch.zeros((adapters, 128, k), dtype=torch.bfloat16, device=dev)
    a[-1, 3, -8:] = 1.0
    b = torch.zeros((adapters, 24, 128), dtype=torch.bfloat16, device=dev)
    b[-1, 7, 3] = 2.0
    x_rows = (1 << 17) + 3
    x = torch.zeros((x_rows, k), dtype=torch.bfloat16, device=dev)
    x[-1, -8:] = 3.0
    y = torch.zeros((x_rows, 24), device=dev)
    off = torch.zeros(adapters + 1, dtype=torch.int32, device=dev)
    off[-1] = rows
    q.qmm_lora(x, a, b, off, y, row_index=torch.tensor([0, x_rows - 1, 7, 1, 2], dtype=torch.int32, device=dev))
    want = torch.zeros((x_rows, 24))
    want[-1, 7] = 48.0
    assert torch.equal(y.cpu(), want)


def test_graph_and_streams(q, dev):
    c = Case(rng(11), 64, 500, 640, 40, 6, "bf16")            # a rank that needs the workspace
    a = c.args(dev)
    base = c.base.to(dev)
    ws = torch.empty(q.qmm_lora_workspace(64, 500, 640, 40, 6), dtype=torch.uint8, device=dev)
    y = base.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q.qmm_lora(y=y, base=base, ws=ws, **a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q.qmm_lora(y=y, base=base, ws=ws, **a)
    g = rng(12)
    for turn in range(4):
        owner = g.integers(-1, 6, 64)
        off, idx, _ = o.sort(owner[:, None].astype(np.int32), 6)
        a["offsets"].copy_(up(off, dev))
        a["row_index"].copy_(up(idx, dev))
        a["x"].copy_(bf16(g, 64, 640))
        y.copy_(base)
        torch.cuda.synchronize()
        eager = q.qmm_lora(y=base.clone(), base=base, **a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
    other = torch.cuda.Stream()                                # a stream by name
    late = base.clone()
    other.wait_stream(torch.cuda.current_stream())             # after the copy that the call writes over
    q.qmm_lora(y=late, base=base, stream=other, **a)
    other.synchronize()
    assert torch.equal(late, eager)


def test_refusals_of_the_binding(q, dev):
    c = Case(rng(13), 6, 40, 64, 40, 2, "f32")
    a = c.args(dev)
    y = c.base.to(dev)

    def call(**kw):
        return q.qmm_lora(**{**a, "y": y, **kw})

    for bad in ({"x": a["x"].float()}, {"a": a["a"].half()}, {"scale": a["scale"].double()}, {"ranks": a["ranks"].long()},
                {"base": y.to(torch.bfloat16)}, {"y": y.half()}, {"offsets": a["offsets"].long()}):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in ({"a": a["a"][:, :, :32]}, {"a": a["a"][:1]}, {"b": a["b"][..., :4].contiguous()}, {"y": y[:5]},
                {"offsets": a["offsets"][:2]}, {"scale": a["scale"][:1]}, {"y": y[0]}):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in ({"ws": torch.empty(16, dtype=torch.uint8, device=dev)}, {"row_index": a["row_index"][:0], "ws": None, "y": y}):
        if "row_index" in bad:
            assert call(**bad) is y                            # no rows: nothing to do
            continue
        with pytest.raises(q.QmvError):
            call(**bad)
    with pytest.raises(q.QmvError):                            # y in part over its own base
        both = torch.zeros((8, 40), device=dev)
        call(y=both[:6], base=both[2:])


@pytest.mark.parametrize("rank", [16, 40])                     # one launch, and two
def test_small_values_keep_their_bits_down_to_the_smallest_bf16_value(q, dev, rank):
    # scale times A x of 24 bits down to below bf16's smallest value: every bit from 2^-133 on comes out, none below
    g = rng(14)
    n = 64
    scale = (g.integers(1 << 23, 1 << 24, n) * 2.0 ** g.integers(-70, -20, n)).astype(np.float32)
    x = torch.full((n, 8), 2.0 ** -40, dtype=torch.bfloat16)
    a, b = torch.zeros((n, rank, 8), dtype=torch.bfloat16), torch.zeros((n, 9, rank), dtype=torch.bfloat16)
    a[:, 3, 5], b[:, :, 3] = 2.0 ** -50, 2.0 ** 110
    y = torch.zeros((n, 9), device=dev)
    q.qmm_lora(x.to(dev), a.to(dev), b.to(dev), torch.arange(n + 1, dtype=torch.int32, device=dev), y, scale=up(scale, dev))
    h = scale.astype(np.float64) * 2.0 ** -90
    h = np.where(h < 2.0 ** -126, h.astype(np.float32).astype(np.float64), h)   # fp32's own smallest values
    cut = np.floor(h * 2.0 ** 133) * 2.0 ** -133
    assert 5 < (cut != h).sum() < 40 and (cut == 0).any() and (cut > 2.0 ** -105).any()
    assert np.array_equal(f64(y), np.tile(cut[:, None] * 2.0 ** 110, (1, 9)))


@pytest.mark.parametrize("k", cases.KS)
@pytest.mark.parametrize("rows,rank", cases.ROWS_RANKS)
def test_whole_numbers(q, dev, rows, rank, k):
    # no tolerance: a block of k that is lost, taken twice or from elsewhere changes some result
    for n, out in ((67, "f32"), (1, "f32"), (130, "bf16")):
        c = cases.whole_numbers(rows, n, k, rank)
        want = torch.from_numpy(cases.result(c)).float().to(TYPES[out])
        assert n == 1 or bool((want != torch.from_numpy(c["base"])).any())
        y, buf = guarded((rows, n), TYPES[out], dev)
        y.copy_(torch.from_numpy(c["base"]))
        x, a, b = (torch.from_numpy(c[v]).to(dev).bfloat16() for v in "xab")
        q.qmm_lora(x, a, b, up(c["offsets"], dev), y, row_index=up(c["index"], dev), scale=up(c["scale"], dev),
                   ranks=up(c["ranks"], dev))
        torch.cuda.synchronize()
        assert guards_intact(buf)
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("k", [8, 64, 2600])
@pytest.mark.parametrize("rank", [8, 16, 40, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_one_row_and_one_column(q, dev, k, rank, out):
    for rows, n in ((1, 1), (1, 64), (3, 1), (3, 2)):
        c = Case(rng(k, rank, rows), rows, n, k, rank, 2, out, owner=np.zeros(rows), mixed=False)
        c.base.mul_(2.0 ** -20)                                # the adapter's part is what counts
        assert c.exact()[1].min() > 0
        c.holds(c.run(q, dev))

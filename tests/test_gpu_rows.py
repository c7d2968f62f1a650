"""GPU parity of the rows' operators with the fp64 oracle.

Sorting and spreading move whole numbers and bytes: equal. Sums, from the arithmetic: a token's top_k terms enter an fp32
sum by one fma each, so |y - exact| <= top_k * 2^-24 * sum |w z|. A gradient's row is one product: 2^-24 of its value. A
weight's gradient is a chain of fma in a lane, at most 8 * ceil(h / 256) of them, and fewer than 16 additions over the lanes:
(8 * ceil(h / 256) + 16) * 2^-24 * sum |dy z|. A bf16 result adds half a step, 2^-8 of its value, to the fp32 one.
"""

import numpy as np
import pytest

from gpu_util import device, guarded, guards_intact, host
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


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def rng(*seed):
    return np.random.default_rng(seed)


def values(g, kind, *shape):
    """Rows of differing size, as a tensor of the type and as fp64."""
    v = g.standard_normal(shape) * 10.0 ** g.uniform(-2, 2, (*shape[:-1], 1))
    t = torch.from_numpy(v.astype(np.float32)).to(TYPES[kind])
    return t, t.double().numpy()


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def rounded(exact, tol, kind):
    return tol + (2.0 ** -8 * (np.abs(exact) + tol) if kind == "bf16" else 0)


def check(got, exact, tol):
    bad = ~(np.abs(got - exact) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4].tolist(), exact[bad][:4].tolist())


def f64(t):
    return t.double().cpu().numpy()


def choices(g, tokens, top_k, experts, dropped=0.2):
    ids = g.integers(0, experts, (tokens, top_k))
    ids[g.random((tokens, top_k)) < dropped] = -1
    ids[g.random((tokens, top_k)) < dropped / 4] = experts + int(g.integers(0, 1 << 30))
    return ids.astype(np.int32)


def np_sort(ids, experts):
    """As the oracle, by numpy's own stable sort, for long lists."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])])
    row_index = np.full(len(flat), -1)
    row_index[:offsets[-1]] = order[:offsets[-1]] // ids.shape[1]
    places = np.empty(len(flat), np.int64)
    places[order] = np.arange(len(flat))
    places[key == experts] = -1
    return offsets, row_index, places.reshape(ids.shape)


# ------------------------------------------------------------------ sort

def sort_into_guards(q, dev, ids, experts, ws=None):
    tokens, top_k = ids.shape
    bufs = [guarded(s, torch.int32, dev, fill=77) for s in ((experts + 1,), (tokens * top_k,), (tokens, top_k))]
    q.qmm_rows_sort(up(ids, dev), experts, *(v for v, _ in bufs), ws=ws)
    torch.cuda.synchronize()
    for _, b in bufs:
        assert guards_intact(b) and int(b[0]) == 77
    return [host(v) for v, _ in bufs]


@pytest.mark.parametrize("tokens,top_k,experts", [
    (1, 1, 1), (1, 8, 128), (4, 8, 128), (3, 2, 3), (64, 1, 5), (65, 1, 64), (21, 3, 65), (128, 32, 1024), (512, 8, 128),
    (4096, 1, 1), (1365, 3, 60), (513, 8, 128), (4097, 1, 2), (1025, 4, 1), (1024, 5, 1024), (2500, 2, 255), (2100, 2, 256),
    (2100, 2, 257), (6000, 8, 17), (16384, 1, 7), (16385, 1, 2), (3300, 5, 1024), (17000, 1, 1),
    (9000, 2, 257), (20, 32, 1024), (640, 1, 1024)])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_sort(q, dev, tokens, top_k, experts, dropped):
    g = rng(tokens, top_k, experts, int(dropped * 10))
    ids = choices(g, tokens, top_k, experts, dropped)
    want = o.sort(ids, experts) if tokens * top_k < 5000 else np_sort(ids, experts)
    for got, exact in zip(sort_into_guards(q, dev, ids, experts), want):
        assert np.array_equal(got, exact)


@pytest.mark.parametrize("tokens", [7, 700, 70000])
@pytest.mark.parametrize("which", ["none", "one", "first", "last", "alternating", "descending"])
def test_sort_of_uneven_choices(q, dev, tokens, which):
    e = 100
    ids = {"none": np.full((tokens, 2), -5), "one": np.full((tokens, 2), 41), "first": np.zeros((tokens, 2)),
           "last": np.full((tokens, 2), e - 1), "alternating": np.tile([3, 97], (tokens, 1)),
           "descending": (e - 1 - np.arange(2 * tokens) * e // (2 * tokens)).reshape(tokens, 2)}[which].astype(np.int32)
    for got, exact in zip(sort_into_guards(q, dev, ids, e), np_sort(ids, e)):
        assert np.array_equal(got, exact)


def test_sort_of_many_choices_and_extreme_ids(q, dev):
    # more than a tile for each of the most parts, and every id that a sign or a bit could spoil
    g = rng(8)
    ids = choices(g, 300001, 1, 1000)
    ids[::7, 0] = g.choice([-1, -(1 << 31), (1 << 31) - 1, 1000, 1023, 1024, 1 << 10, 999, 0], len(ids[::7]))
    for got, exact in zip(sort_into_guards(q, dev, ids, 1000), np_sort(ids, 1000)):
        assert np.array_equal(got, exact)


def test_sort_of_more_than_a_tile_a_part(q, dev):
    ids = choices(rng(11), 1500001, 1, 77)
    for got, exact in zip(sort_into_guards(q, dev, ids, 77), np_sort(ids, 77)):
        assert np.array_equal(got, exact)


def test_sort_without_tokens_or_some_outputs(q, dev):
    off, idx, pl = q.qmm_rows_sort(torch.empty((0, 4), dtype=torch.int32, device=dev), 3)
    assert host(off).tolist() == [0, 0, 0, 0] and idx.shape == (0,) and pl.shape == (0, 4)
    for tokens in (50, 5000, 10000):                           # the C entry takes null for either
        ids = choices(rng(tokens), tokens, 2, 9)
        want = np_sort(ids, 9)
        d, ws = up(ids, dev), torch.empty(max(1, q.qmm_rows_sort_workspace(tokens, 2, 9)), dtype=torch.uint8, device=dev)
        for keep in (0, 1, 2):
            out = [torch.full((n,), 55, dtype=torch.int32, device=dev) for n in (10, 2 * tokens, 2 * tokens)]
            rc = q.lib.qmm_rows_sort(d.data_ptr(), out[0].data_ptr(), out[1].data_ptr() if keep == 1 else None,
                                     out[2].data_ptr() if keep == 2 else None, tokens, 2, 9, ws.data_ptr(), ws.numel(),
                                     torch.cuda.current_stream().cuda_stream)
            assert rc == 0
            assert np.array_equal(host(out[0]), want[0])
            for k in (1, 2):
                assert np.array_equal(host(out[k]), want[k].reshape(-1)) if k == keep else bool((out[k] == 55).all())


# ------------------------------------------------------------------ spread, combine, gradient

SHAPES = [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (4, 8, 16), (5, 3, 1003), (17, 9, 64), (2, 32, 33), (130, 2, 260), (7, 4, 5000),
          (33, 8, 513), (64, 1, 2047), (9, 17, 24)]


def layout(g, tokens, top_k, spare, dropped=0.2):
    """Places of a sorted routing, and one row more than it needs, its rows in no place."""
    places = o.sort(choices(g, tokens, top_k, 6, dropped), 6)[2]
    return places, tokens * top_k + spare


@pytest.mark.parametrize("tokens,top_k,h", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_spread(q, dev, tokens, top_k, h, kind):
    g = rng(1, tokens, top_k, h)
    places, rows = layout(g, tokens, top_k, 3)
    x, x64 = values(g, kind, tokens, h)
    out, buf = guarded((rows, h), TYPES[kind], dev)
    out.fill_(5.0)
    q.qmm_rows_spread(x.to(dev), up(places, dev), out=out)
    torch.cuda.synchronize()
    assert guards_intact(buf)
    assert np.array_equal(f64(out), o.spread(x64, places, np.full((rows, h), 5.0)))


@pytest.mark.parametrize("tokens,top_k,h", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(q, dev, tokens, top_k, h, kind, out, weighted):
    g = rng(2, tokens, top_k, h)
    places, rows = layout(g, tokens, top_k, 2)
    z, z64 = values(g, kind, rows, h)
    w = (g.standard_normal((tokens, top_k)) * 3).astype(np.float32) if weighted else None
    y, buf = guarded((tokens, h), TYPES[out], dev)
    q.qmm_rows_combine(z.to(dev), up(places, dev), None if w is None else up(w, dev), y=y)
    torch.cuda.synchronize()
    assert guards_intact(buf)
    exact, mag = o.combine(z64, places, w)
    check(f64(y), exact, rounded(exact, top_k * 2.0 ** -24 * mag, out))


@pytest.mark.parametrize("tokens,top_k,h", SHAPES + [(4097, 2, 96), (4100, 1, 515)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(q, dev, tokens, top_k, h, kind, weighted):
    g = rng(3, tokens, top_k, h)
    places, rows = layout(g, tokens, top_k, 2)
    z, z64 = values(g, kind, rows, h)
    dy, dy64 = values(g, kind, tokens, h)
    w = (g.standard_normal((tokens, top_k)) * 3).astype(np.float32) if weighted else None
    dz, zbuf = guarded((rows, h), TYPES[kind], dev)
    dz.fill_(5.0)
    dw, wbuf = guarded((tokens, top_k), torch.float32, dev)
    q.qmm_rows_combine_grad(dy.to(dev), z.to(dev), up(places, dev), None if w is None else up(w, dev), dz=dz, dw=dw)
    torch.cuda.synchronize()
    assert guards_intact(zbuf) and guards_intact(wbuf)
    edz, edw, mag = o.combine_grad(dy64, z64, places, w, np.full((rows, h), 5.0))
    check(f64(dz), edz, rounded(edz, 2.0 ** -24 * np.abs(edz), kind))
    check(f64(dw), edw, (8 * -(-h // 256) + 16) * 2.0 ** -24 * mag)
    only, none = q.qmm_rows_combine_grad(dy.to(dev), None, up(places, dev), None if w is None else up(w, dev), rows=rows)
    assert none is None
    named = np.zeros(rows, bool)
    named[places[places >= 0]] = True
    assert np.array_equal(f64(only)[named], f64(dz)[named]) and (f64(only)[~named] == 0).all()


def test_gradient_is_that_of_differences(q, dev):
    # y is linear in each of z and w: steps of 2^-2 on values with few bits are exact in fp32
    g = rng(4)
    places = o.sort(choices(g, 9, 3, 4), 4)[2]
    z, w, dy = (g.integers(-8, 9, s).astype(np.float32) / 4 for s in ((27, 40), (9, 3), (9, 40)))
    d = lambda a: up(a, dev)
    dz, dw = (f64(t) for t in q.qmm_rows_combine_grad(d(dy), d(z), d(places), d(w)))
    y = lambda z, w: float((q.qmm_rows_combine(d(z), d(places), d(w)).double() * d(dy).double()).sum())
    base = y(z, w)
    for at in ((0, 0), (13, 39), (26, 5), (8, 17)):
        step = z.copy()
        step[at] += 0.25
        assert (y(step, w) - base) / 0.25 == dz[at]
    for at in ((0, 0), (4, 1), (8, 2)):
        step = w.copy()
        step[at] += 0.25
        assert (y(z, step) - base) / 0.25 == dw[at]


def test_rows_that_are_not_finite_touch_no_other(q, dev):
    g = rng(5)
    for kind in ("f32", "bf16"):
        places = o.sort(choices(g, 20, 4, 6, 0.3), 6)[2]
        z, z64 = values(g, kind, 80, 72)
        w = g.random((20, 4)).astype(np.float32)
        dead = set(range(80)) - set(places[places >= 0].tolist())
        z64 = z64.copy()
        for r in dead | {0}:                                   # row 0 stands in for choices without a place
            z64[r] = np.nan
        z64[int(places[places >= 0].max()), 5] = np.inf
        w[places < 0] = np.nan                                 # a weight without a row
        zt = torch.from_numpy(z64).to(TYPES[kind])
        y = f64(q.qmm_rows_combine(zt.to(dev), up(places, dev), up(w, dev), out_dtype=torch.float32))
        with np.errstate(invalid="ignore"):
            exact, mag = o.combine(zt.double().numpy(), places, w)
        ok = np.isfinite(exact)
        assert np.array_equal(np.isnan(y), np.isnan(exact)) and np.array_equal(y[~ok], exact[~ok], equal_nan=True)
        check(y[ok], exact[ok], 4 * 2.0 ** -24 * mag[ok])
        dy, dy64 = values(g, kind, 20, 72)
        dz, dw = q.qmm_rows_combine_grad(dy.to(dev), zt.to(dev), up(places, dev), up(w, dev))
        with np.errstate(invalid="ignore"):
            edz, edw, _ = o.combine_grad(dy64, zt.double().numpy(), places, w, np.zeros((80, 72)))
        assert np.array_equal(np.isnan(f64(dw)), np.isnan(edw)) and (f64(dw)[places < 0] == 0).all()
        assert np.isfinite(f64(dz)).all() and (f64(dz)[sorted(dead)] == 0).all()


def test_nothing_to_sum(q, dev):
    none = torch.full((3, 4), -1, dtype=torch.int32, device=dev)
    z = torch.full((5, 10), float("nan"), device=dev)
    assert bool((q.qmm_rows_combine(z, none) == 0).all())
    empty = torch.empty((0, 10), device=dev)
    zeros = torch.zeros((3, 4), dtype=torch.int32, device=dev)
    assert bool((q.qmm_rows_combine(empty, zeros, out_dtype=torch.bfloat16) == 0).all())   # no row: every place lies outside
    dz, dw = q.qmm_rows_combine_grad(torch.ones((3, 10), device=dev), empty, zeros)
    assert dz.shape == (0, 10) and bool((dw == 0).all())
    assert q.qmm_rows_spread(torch.ones((3, 10), device=dev), zeros, rows=0).shape == (0, 10)
    no = torch.empty((0, 4), dtype=torch.int32, device=dev)
    assert q.qmm_rows_combine(z, no).shape == (0, 10)
    out = torch.ones((2, 10), device=dev)
    assert bool((q.qmm_rows_spread(empty, no, out=out) == 1).all())


def test_places_outside_are_passed_over(q, dev):
    places = torch.tensor([[0, 5], [-(1 << 31), (1 << 31) - 1], [4, 6]], dtype=torch.int32, device=dev)
    x = torch.arange(1, 31, device=dev, dtype=torch.float32).view(3, 10)
    out, buf = guarded((5, 10), torch.float32, dev)
    out.fill_(0.0)
    q.qmm_rows_spread(x, places, out=out)
    torch.cuda.synchronize()
    assert guards_intact(buf)
    assert torch.equal(out[0], x[0]) and torch.equal(out[4], x[2]) and bool((out[1:4] == 0).all())
    y = q.qmm_rows_combine(out, places)
    assert torch.equal(y[0], x[0]) and torch.equal(y[2], x[2]) and bool((y[1] == 0).all())


@pytest.mark.parametrize("top_k,h", [(2, 16384), (4, 8192), (9, 4096)])
def test_rows_larger_than_the_caches(q, dev, top_k, h):
    # from 64 MiB of rows on they go past the caches: bf16, and the same in fp32, against sums of whole numbers
    g = rng(9, top_k)
    tokens = -(-(64 << 20) // (top_k * h * 2)) + 1
    places = np_sort(choices(g, tokens, top_k, 50, 0.1), 50)[2].astype(np.int32)
    x = torch.from_numpy(g.integers(-8, 9, (tokens, h)).astype(np.float32)).to(dev)
    w = torch.from_numpy(g.integers(-4, 5, (tokens, top_k)).astype(np.float32)).to(dev)
    at = up(places, dev)
    held = (at >= 0).float()
    for kind in (torch.bfloat16, torch.float32):
        z = q.qmm_rows_spread(x.to(kind), at)
        ids = torch.where(at < 0, 0, at).long()
        assert torch.equal(z[ids] * held[:, :, None].to(kind), x.to(kind)[:, None] * held[:, :, None].to(kind))
        y = q.qmm_rows_combine(z, at, w)
        assert torch.equal(y, x * (w * held).sum(1, keepdim=True))         # below 2^24: exact
        dz, dw = q.qmm_rows_combine_grad(x.to(kind), z, at, w)
        assert torch.equal(dz[ids] * held[:, :, None].to(kind), (x[:, None] * (w * held)[:, :, None]).to(kind))
        assert torch.equal(dw, (x * x).sum(1, keepdim=True) * held)        # at most 64 * 2^14


def test_rows_past_4_gib(q, dev):
    # 2^21 + 5 rows of 1024 fp32 values: the last rows' addresses pass 2^32 bytes, and 2^31 values
    rows, h = (1 << 21) + 5, 1024
    z = torch.zeros((rows, h), device=dev)
    z[-1], z[-2], z[3] = 2.0, 3.0, 5.0
    places = torch.tensor([[rows - 1, 3], [rows - 2, rows - 1]], dtype=torch.int32, device=dev)
    y = q.qmm_rows_combine(z, places)
    assert bool((y[0] == 7).all()) and bool((y[1] == 5).all())
    q.qmm_rows_spread(torch.full((2, h), 9.0, device=dev), places[:, :1].contiguous(), out=z)
    assert bool((z[-1] == 9).all()) and bool((z[-2] == 9).all()) and bool((z[4:-2] == 0).all())
    dz, dw = q.qmm_rows_combine_grad(torch.ones((2, h), device=dev), z, places[:, :1].contiguous(), dz=z.clone())
    assert host(dw).tolist() == [[9 * h], [9 * h]] and bool((dz[-1] == 1).all()) and bool((dz[4:-2] == 0).all())


def test_more_tokens_than_workgroups(q, dev):
    # 2^20 + 3 tokens of 256 pieces each: the kernels take several tokens a workgroup
    tokens, h = (1 << 20) + 3, 1024
    z = torch.arange(tokens, device=dev, dtype=torch.float32)[:, None] + torch.arange(h, device=dev) / 2048
    places = torch.arange(tokens - 1, -1, -1, device=dev, dtype=torch.int32)[:, None]
    y = q.qmm_rows_combine(z, places)
    assert torch.equal(y, z.flip(0))
    assert torch.equal(q.qmm_rows_spread(y, places), z)
    weights = torch.full((tokens, 1), 0.5, device=dev)
    dz, dw = q.qmm_rows_combine_grad(torch.ones_like(z), z.flip(0).contiguous().sign_(), places, weights)
    assert bool((dz == 0.5).all())
    assert int((dw != h).sum()) == 1 and float(dw.min()) == h - 1            # ones, but for the first value of all


# ------------------------------------------------------------------ calls as a program makes them

def test_another_stream_and_a_graph(q, dev):
    g = rng(6)
    tokens = 2100                                              # enough for the sort to need its workspace
    ids = [choices(g, tokens, 8, 128, 0.1) for _ in range(4)]
    x, x64 = values(g, "bf16", tokens, 256)
    w = g.random((tokens, 8)).astype(np.float32)
    xd, wd, idsd = x.to(dev), up(w, dev), up(ids[0], dev)
    ws = torch.empty(q.qmm_rows_sort_workspace(tokens, 8, 128), dtype=torch.uint8, device=dev)
    state = {}

    def layer():
        state["plan"] = q.qmm_rows_sort(idsd, 128, ws=ws)
        state["z"] = q.qmm_rows_spread(xd, state["plan"][2])
        state["y"] = q.qmm_rows_combine(state["z"], state["plan"][2], wd)
        state["grad"] = q.qmm_rows_combine_grad(xd, state["z"], state["plan"][2], wd)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer()
    captured = {k: v for k, v in state.items()}
    for new in ids:
        idsd.copy_(up(new, dev))
        layer()                                                # eager, between the replays
        eager = {k: v for k, v in state.items()}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        used = int(eager["plan"][0][-1])
        for a, b in zip((*captured["plan"], captured["z"][:used], captured["y"], captured["grad"][0][:used], captured["grad"][1]),
                        (*eager["plan"], eager["z"][:used], eager["y"], eager["grad"][0][:used], eager["grad"][1])):
            assert torch.equal(a, b)
        for a, b in zip(eager["plan"], np_sort(new, 128)):
            assert np.array_equal(host(a), b)


def test_refusals_of_the_binding(q, dev):
    f, i = torch.zeros((4, 8), device=dev), torch.zeros((4, 2), dtype=torch.int32, device=dev)
    with pytest.raises(TypeError):
        q.qmm_rows_sort(i.long(), 4)
    with pytest.raises(ValueError, match="contiguous"):
        q.qmm_rows_sort(torch.zeros((2, 8), dtype=torch.int32, device=dev).t(), 4)
    with pytest.raises(ValueError, match="offsets has shape"):
        q.qmm_rows_sort(i, 4, offsets=torch.zeros(4, dtype=torch.int32, device=dev))
    with pytest.raises(q.QmvError):
        q.qmm_rows_sort(i, 0)
    with pytest.raises(q.QmvError):
        q.qmm_rows_sort(i, 1025)
    with pytest.raises(TypeError):
        q.qmm_rows_spread(f.half(), i)
    with pytest.raises(TypeError):
        q.qmm_rows_spread(f, i, out=torch.zeros((8, 8), dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError, match="places has shape"):
        q.qmm_rows_spread(f, i[:3])
    with pytest.raises(ValueError, match="expected 9"):
        q.qmm_rows_spread(f, i, rows=9, out=f)
    with pytest.raises(q.QmvError):
        q.qmm_rows_spread(f, i, out=f)                         # the rows read are the rows written
    with pytest.raises(ValueError, match="weights has shape"):
        q.qmm_rows_combine(f, i, torch.ones((4, 3), device=dev))
    with pytest.raises(TypeError):
        q.qmm_rows_combine(f, i, torch.ones((4, 2), device=dev, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="needs z"):
        q.qmm_rows_combine_grad(f, None, i, dw=torch.zeros((4, 2), device=dev))
    with pytest.raises(q.QmvError):
        q.qmm_rows_combine_grad(f, f.clone(), i, dz=f)


def test_the_most_choices_and_the_widest_rows(q, dev):
    n = 1 << 24
    ids = choices(rng(12), n // 32, 32, 1024, 0.1)
    for got, exact in zip(sort_into_guards(q, dev, ids, 1024), np_sort(ids, 1024)):
        assert np.array_equal(got, exact)
    h, top_k = 1 << 20, 3
    places = torch.tensor([[5, 0, -1], [2, 6, 3]], dtype=torch.int32, device=dev)
    at, held = places.clamp(min=0).long(), (places >= 0).float()
    w = torch.tensor([[2.0, -1.0, 9.0], [3.0, 0.5, 4.0]], device=dev)
    for width in (h, h - 3):                                   # whole pieces, and rows that start anywhere
        x = ((torch.arange(2 * width, device=dev) * 7 % 17).float() - 8).view(2, width)
        for kind in (torch.float32, torch.bfloat16):
            z = q.qmm_rows_spread(x.to(kind), places, rows=7)
            assert torch.equal(z[at] * held[:, :, None].to(kind), x.to(kind)[:, None] * held[:, :, None].to(kind))
            assert bool((z[[1, 4]] == 0).all())
            assert torch.equal(q.qmm_rows_combine(z, places, w), x * (w * held).sum(1, keepdim=True))
            dz, dw = q.qmm_rows_combine_grad(x.to(kind), z, places, w)
            want = (x[:, None] * (w * held)[:, :, None]).to(kind)
            assert torch.equal(dz[at] * held[:, :, None].to(kind), want)
            got = (x.double() ** 2).sum(1, keepdim=True) * held   # whole numbers up to 2^25: the last additions round
            assert bool(((dw - got).abs() <= 16 * 2.0 ** -24 * got).all())

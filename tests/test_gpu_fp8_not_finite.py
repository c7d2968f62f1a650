"""A NaN or an infinity among the operands or scales of the e4m3 and grouped products reaches the results it enters
and no other, on every kernel and tile, whole and cut along k (tests/fp8_plans.py).

The same call without them gives the bits that all other results must keep.
"""

import numpy as np
import pytest

from fp8_plans import DENSE, GROUPED, LEAD, RUNS, rows_of
from gpu_util import device
from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q():
    import gguf_block_quantized_qmv_amd as mod
    return mod


@pytest.fixture(scope="module")
def dev():
    return device()


def values(g, dev, *shape):
    """No value is 0, so that no product with an infinity is accidentally one with 0."""
    return (torch.rand(*shape, generator=g, device=dev) + 0.5) * torch.where(
        torch.rand(*shape, generator=g, device=dev) < 0.5, -16.0, 16.0)


def scales(g, dev, *shape):
    return torch.rand(*shape, generator=g, device=dev) + 0.5


def same_bits(a, b):
    return bool((a.view(torch.uint8) == b.view(torch.uint8)).all())


@pytest.mark.parametrize("m,n,k,fast,out", [
    pytest.param(m, n, k, fast, out, id=f"{m}x{n}x{k}-{'fast' if fast else str(out)[6:]}")
    for m, n, k, fast, _ in DENSE for out in ((BF16,) if fast else (F32, BF16))])
def test_dense(q, dev, m, n, k, fast, out):
    g = torch.Generator(device=dev).manual_seed(m * 7 + n + k)
    w, x = values(g, dev, n, k).to(E4M3), values(g, dev, m, k).to(E4M3)
    ws, xs = scales(g, dev, o.blocks(n), o.blocks(k)), scales(g, dev, o.blocks(k), m)
    ws[-1] = 1.0
    clean = q.qmm_fp8(w, ws, x, xs, n, k, out_dtype=out, fast_sums=fast)
    assert bool(torch.isfinite(clean).all())
    hit = torch.zeros(m, n, dtype=torch.bool, device=dev)
    x.view(torch.uint8)[m - 1, k - 1] = 0x7F                 # the last row, in the partial block
    hit[m - 1] = True
    xs[0, 1] = np.inf                                        # a row inside the first tile
    hit[1] = True
    w.view(torch.uint8)[n - 1, 3] = 0xFF
    hit[:, n - 1] = True
    w.view(torch.uint8)[n // 2, k // 2] = 0x7F
    hit[:, n // 2] = True
    if n > 256:                                              # 128 columns under one scale
        ws[1, -1] = np.nan
        hit[:, 128:256] = True
    y = q.qmm_fp8(w, ws, x, xs, n, k, out_dtype=out, fast_sums=fast)
    assert not bool(torch.isfinite(y[hit]).any())
    assert same_bits(y[~hit], clean[~hit])


@pytest.mark.parametrize("gather", [True, False], ids=["gathered", "in order"])
@pytest.mark.parametrize("kind,fast,out", [("fp8", False, F32), ("fp8", False, BF16), ("fp8", True, BF16),
                                           ("bf16", False, F32), ("bf16", False, BF16)])
@pytest.mark.parametrize("runs,n,k", [c[:3] for c in GROUPED])
def test_grouped(q, dev, runs, n, k, kind, fast, out, gather):
    g = torch.Generator(device=dev).manual_seed(n + k + len(RUNS[runs]))
    counts, rows = RUNS[runs], rows_of(runs)
    e, x_rows = len(counts), 90 if gather else rows
    bounds = (np.concatenate([[0], np.cumsum(counts)]) + LEAD).tolist()
    off = torch.tensor(bounds, dtype=torch.int32, device=dev)
    index = torch.randint(0, x_rows, (rows,), generator=g, device=dev, dtype=torch.int32) if gather else None
    src = index.long() if gather else torch.arange(rows, device=dev)
    w, x = values(g, dev, e, n, k), values(g, dev, x_rows, k)
    w, x = (w.to(E4M3), x.to(E4M3)) if kind == "fp8" else (w.to(BF16), x.to(BF16))
    ws, xs = scales(g, dev, e, o.blocks(n), o.blocks(k)), scales(g, dev, o.blocks(k), x_rows)

    def call():
        y = torch.full((rows, n), -7.0, dtype=out, device=dev)
        if kind == "fp8":
            return q.qmm_fp8_grouped(w, ws, x, xs, off, n, k, row_index=index, y=y, fast_sums=fast)
        return q.qmm_bf16_grouped(w, x, off, n, k, row_index=index, y=y)

    clean = call()
    assert bool(torch.isfinite(clean).all())
    hit = torch.zeros(rows, n, dtype=torch.bool, device=dev)
    full = [i for i, c in enumerate(counts) if c > 1]
    first, last = full[len(full) // 2], full[-1]
    # the first row of a run (behind another run's last tile), the last of another, and a row of no run
    for r in (bounds[first], bounds[last + 1] - 1, rows - 1):
        if kind == "fp8":
            x.view(torch.uint8)[int(src[r]), k - 1] = 0x7F
        else:
            x[int(src[r]), k - 1] = np.nan
        hit |= (src == src[r])[:, None]
    if kind == "fp8":                                        # a row's scale
        r = bounds[full[0]]
        xs[-1, int(src[r])] = np.inf
        hit |= (src == src[r])[:, None]
    # one weight of one expert, in its last column; a scale of another's first columns
    if kind == "fp8":
        w.view(torch.uint8)[first, n - 1, k // 2] = 0xFF
        ws[last, 0, 0] = np.inf
        hit[bounds[last]:bounds[last + 1], :128] = True
    else:
        w[first, n - 1, k // 2] = np.inf
        w[last, 0, 0] = np.nan
        hit[bounds[last]:bounds[last + 1], 0] = True
    hit[bounds[first]:bounds[first + 1], n - 1] = True
    hit[:bounds[0]] = False
    hit[bounds[-1]:] = False
    y = call()
    assert not bool(torch.isfinite(y[hit]).any())
    assert same_bits(y[~hit], clean[~hit])

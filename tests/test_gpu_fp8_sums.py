"""The sums of the e4m3 and grouped products, on every kernel and tile (tests/fp8_plans.py).

Whole numbers. Operands are whole numbers; scales are 1 and 2 for x, 1/2 and 1 for w.
Every partial sum, in any order, is then a whole number of halves, at most 2 * sum |w x|;
while that is under 2^24 halves (checked in `whole`) fp32 holds each of them, so fp32
sums give the result itself: y in fp32 equals it and y in bf16 is it rounded once, with
no tolerance. Pairs of +-240 * 240 that cancel stand in one group of eight
neighbours with small products, which a sum cut 13 bits below 240 * 240 loses.

Fast sums: of each eight neighbouring products the seven others lose less than 2^-13
of the largest each, so a result is off by less than 7 * 2^-13 * sum of the groups'
largest products, and fp32's (2 * 128 + blocks + 40) * 2^-24 * sum |w x|, before its
rounding to bf16 (2^-8 of its value).

Norms. With errors e before the rounding, the part of the bf16 results that are not the
nearest to the exact value is the mean of min(1, e / step), step >= 2^-8 |y|: for
normal y of size s and e = c s / 2^8 that is below 0.8 c (log(1 / c) + 0.6). Fast sums
with 1.5e-5 s on normal data: c = 0.0038, below 2 %, with 4e-5 s where a few channels
are strong: c = 0.01, below 5 %; fp32 sums with 2e-7 s or less: c = 5e-5, below 0.05 %
(and four deviations of a count with that mean, and 4 for the smallest). An fp32 result
adds one rounding, 2^-24 of the running sum, a block, and inside a block eight of them at
most of its size: (blocks + 8) * 2^-24 of the norm.
"""

import numpy as np
import pytest

from fp8_plans import DENSE, GROUPED, LEAD, RUNS, SPARE, rows_of
from gpu_util import device, guards_intact, guarded
from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def q():
    import gguf_block_quantized_qmv_amd as mod
    return mod


@pytest.fixture(scope="module")
def dev():
    return device()


def pick(g, dev, values, *shape):
    v = torch.tensor(values, device=dev)
    return v[torch.randint(0, len(values), shape, generator=g, device=dev)]


def whole(g, dev, lead, rows, k, second):
    """Whole numbers -15..15 with a pair of 240 every 256 values; the second operand's pair cancels the first's."""
    v = torch.randint(-15, 16, (*lead, rows, k), generator=g, device=dev).float()
    sign = pick(g, dev, [-240.0, 240.0], *lead, rows, 1)
    at = torch.arange(0, k, 256, device=dev)
    v[..., at], v[..., at + 1] = sign, -sign if second else sign
    assert 2 * (2 * (len(at) * 2 * 240 * 240 + 225 * k)) < 1 << 24   # under scales of 2, in halves
    return v


def scales_of(g, dev, second, *shape):
    return pick(g, dev, [0.5, 1.0] if second else [1.0, 2.0], *shape)


def spread(v, s, k):
    """Values times their scales, fp64: s [..., blocks] for each row."""
    return v.double() * s.double().repeat_interleave(128, -1)[..., :k]


def spread_rows(v, s, k):
    return spread(v, s.t(), k)


def spread_weights(v, s, n, k):
    return spread(v, s.repeat_interleave(128, -2)[..., :n, :], k)


def generator(dev, *seed):
    return torch.Generator(device=dev).manual_seed(int(np.random.SeedSequence(seed).generate_state(1)[0]))


E4M3 = torch.float8_e4m3fn


def dense_cases():
    for m, n, k, fast, plan in DENSE:
        for out in ((BF16,) if fast else (F32, BF16)):
            name = f"{m}x{n}x{k}-{'fast' if fast else 'f32' if out is F32 else 'bf16'}"
            yield pytest.param(m, n, k, fast, out, id=name)


def within_groups(x, w, k, got, exact):
    """Holds rows of fast results to the bound above; x, w fp64 with their scales in."""
    pad = -k % 8
    xg = torch.nn.functional.pad(x, (0, pad)).abs().view(len(x), -1, 8)
    wg = torch.nn.functional.pad(w, (0, pad)).abs().view(len(w), -1, 8)
    top, mag = torch.zeros_like(exact), torch.zeros_like(exact)
    for i in range(len(x)):
        for c in range(0, len(w), 4096):
            p = xg[i] * wg[c:c + 4096]
            top[i, c:c + 4096], mag[i, c:c + 4096] = p.amax(2).sum(1), p.sum((1, 2))
    tol = 7 * 2.0 ** -13 * top + (2 * 128 + k // 128 + 41) * 2.0 ** -24 * mag
    tol = tol + 2.0 ** -8 * (exact.abs() + tol)
    bad = ~((got.double() - exact).abs() <= tol)
    assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("m,n,k,fast,out", dense_cases())
def test_dense_sums_of_whole_numbers(q, dev, m, n, k, fast, out):
    g = generator(dev, 1, m, n, k)
    x, w = whole(g, dev, (), m, k, False), whole(g, dev, (), n, k, True)
    xs, ws = scales_of(g, dev, False, o.blocks(k), m), scales_of(g, dev, True, o.blocks(n), o.blocks(k))
    y, buf = guarded((m, n), out, dev)
    q.qmm_fp8(w.to(E4M3), ws, x.to(E4M3), xs, n, k, y=y, fast_sums=fast)
    torch.cuda.synchronize()
    assert guards_intact(buf)
    x, w = spread_rows(x, xs, k), spread_weights(w, ws, n, k)
    exact = x @ w.t()
    if fast:
        rows = sorted({0, m // 2, m - 1})
        within_groups(x[rows], w, k, y[rows], exact[rows])
    else:
        assert torch.equal(y, exact.to(out))


def grouped_data(dev, kind, runs, n, k, seed):
    g = generator(dev, seed, n, k, len(RUNS[runs]))
    rows, e, x_rows = rows_of(runs), len(RUNS[runs]), 300
    off = torch.tensor(np.concatenate([[0], np.cumsum(RUNS[runs])]) + LEAD, dtype=torch.int32, device=dev)
    index = torch.randint(0, x_rows, (rows,), generator=g, device=dev, dtype=torch.int32)
    index[::97], index[50::97] = -1, x_rows                  # rows of zeros
    x, w = whole(g, dev, (), x_rows, k, False), whole(g, dev, (e,), n, k, True)
    if kind == "bf16":
        return off, index, x, w, None, None
    return (off, index, x, w, scales_of(g, dev, False, o.blocks(k), x_rows),
            scales_of(g, dev, True, e, o.blocks(n), o.blocks(k)))


def call_grouped(q, kind, off, index, x, w, xs, ws, n, k, y, fast):
    if kind == "bf16":
        return q.qmm_bf16_grouped(w.to(BF16), x.to(BF16), off, n, k, row_index=index, y=y)
    return q.qmm_fp8_grouped(w.to(E4M3), ws, x.to(E4M3), xs, off, n, k, row_index=index, y=y, fast_sums=fast)


@pytest.mark.parametrize("gather", [True, False], ids=["gathered", "in order"])
@pytest.mark.parametrize("kind,fast,out", [("fp8", False, F32), ("fp8", False, BF16), ("fp8", True, BF16),
                                           ("bf16", False, F32), ("bf16", False, BF16)])
@pytest.mark.parametrize("runs,n,k", [c[:3] for c in GROUPED])
def test_grouped_sums_of_whole_numbers(q, dev, runs, n, k, kind, fast, out, gather):
    off, index, x, w, xs, ws = grouped_data(dev, kind, runs, n, k, 2)
    inside = (index >= 0) & (index < len(x))
    at = index.clamp(0, len(x) - 1).long()
    rows = x[at] * inside[:, None]                           # what each row of y multiplies
    row_scales = None if xs is None else xs[:, at] * inside
    y, buf = guarded((len(index), n), out, dev)
    y.fill_(-7.0)
    if gather:
        call_grouped(q, kind, off, index, x, w, xs, ws, n, k, y, fast)
    else:
        call_grouped(q, kind, off, None, rows, w, None if xs is None else row_scales.contiguous(), ws, n, k, y, fast)
    torch.cuda.synchronize()
    assert guards_intact(buf)
    a = rows.double() if xs is None else spread_rows(rows, row_scales, k)
    b = w.double() if xs is None else spread_weights(w, ws, n, k)
    exact = torch.full(y.shape, -7.0, dtype=torch.float64, device=dev)
    bounds = off.tolist()
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        exact[lo:hi] = a[lo:hi] @ b[e].t()
        if fast and hi > lo:
            r = sorted({lo, hi - 1})
            within_groups(a[r], b[e], k, y[r], exact[r])
    if fast:
        assert bool((y[:LEAD] == -7).all() and (y[-SPARE:] == -7).all())
    else:
        assert torch.equal(y, exact.to(out))


@pytest.mark.parametrize("fast", [False, True], ids=["fp32 sums", "fast"])
def test_a_group_that_cancels(q, dev, fast):
    # 448 * 448 - 448 * 448 + 6 * (2 * 2) a group of eight: 24 a group of exact sums; fast ones may lose the 4s
    m, n, k = 130, 5391, 2048
    x, w = torch.full((m, k), 2.0, device=dev), torch.full((n, k), 2.0, device=dev)
    x[:, ::8], x[:, 1::8] = 448.0, 448.0
    w[:, ::8], w[:, 1::8] = 448.0, -448.0
    one = torch.ones
    y = q.qmm_fp8(w.to(E4M3), one(o.blocks(n), 16, device=dev), x.to(E4M3), one(16, m, device=dev), n, k, out_dtype=BF16,
                  fast_sums=fast)
    if fast:
        assert bool(((y >= 0) & (y <= 3 * k)).all())
    else:
        assert bool((y == 3 * k).all())


def normal_case(dev, m, n, k, strong):
    g = generator(dev, 3, m, n, k)
    x = torch.randn(m, k, generator=g, device=dev)
    if strong:
        x = x * torch.where(torch.rand(k, generator=g, device=dev) < 0.01, 20.0, 1.0)
    w = (torch.randn(n, k, generator=g, device=dev) * 110).clamp(-448, 448).to(E4M3)
    return x, w, 2e-4 * torch.exp(0.3 * torch.randn(o.blocks(n), o.blocks(k), generator=g, device=dev))


@pytest.mark.parametrize("strong", [False, True], ids=["normal", "strong channels"])
@pytest.mark.parametrize("m,n,k,fast,out", dense_cases())
def test_norms(q, dev, m, n, k, fast, out, strong):
    x, w, ws = normal_case(dev, m, n, k, strong)
    xq, xs = q.qmm_fp8_quant(x)
    y = q.qmm_fp8(w, ws, xq, xs, n, k, out_dtype=out, fast_sums=fast)
    exact = spread_rows(xq, xs, k) @ spread_weights(w, ws, n, k).t()
    if out == F32:
        assert float((y - exact).norm() / exact.norm()) <= (o.blocks(k) + 8) * 2.0 ** -24
        return
    other, most = int((y != exact.to(BF16)).sum()), y.numel() * ((0.05 if strong else 0.02) if fast else 5e-4)
    assert other <= most + 4 * most ** 0.5 + 4, (other, y.numel())


def test_fast_sums_go_with_bf16_results_alone(q, dev):
    w, x = torch.zeros(64, 128, dtype=E4M3, device=dev), torch.zeros(20, 128, dtype=E4M3, device=dev)
    ws, xs = torch.ones(1, 1, device=dev), torch.ones(1, 20, device=dev)
    with pytest.raises(ValueError, match="bfloat16"):
        q.qmm_fp8(w, ws, x, xs, 64, 128, fast_sums=True)
    with pytest.raises(ValueError, match="bfloat16"):
        q.qmm_fp8_grouped(w[None], ws[None], x, xs, torch.tensor([0, 20], dtype=torch.int32, device=dev), 64, 128,
                          out_dtype=F32, fast_sums=True)
    y = torch.ones(20, 64, dtype=BF16, device=dev)
    q.qmm_fp8(w, ws, x, xs, 64, 128, y=y, fast_sums=True)
    assert bool((y == 0).all())

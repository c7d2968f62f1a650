"""The verification of drafted tokens against the fp64 oracle: whole numbers, so equal.

The oracle's running sums and the kernel's add in another order, in 64 bits: borders move by less than 2^-53 * vocab of the
whole, and no random number below lies that near to one (but for sums of few bits, which both hold exactly)."""

import numpy as np
import pytest

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


def up(a, dev):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def softmax(v):
    e = np.exp(v - v.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def case(g, requests, drafts, vocab, kind, sampled=True, cut=False, ragged=True):
    logits = 2.5 * g.standard_normal((requests, drafts + 1, vocab))
    p = softmax(logits)
    if cut:
        p[p < 0.1 * p.max(-1, keepdims=True)] = 0
        p /= p.sum(-1, keepdims=True)
    p = torch.from_numpy(p).to(TYPES[kind])
    qq, lengths = None, None
    near = logits[:, :drafts] + 0.6 * g.standard_normal((requests, drafts, vocab))
    if sampled:
        qq = torch.from_numpy(softmax(near)).to(TYPES[kind])
        near = near + g.gumbel(size=near.shape)
    tokens = near.argmax(-1).astype(np.int32) if drafts else np.zeros((requests, 0), np.int32)
    u = g.random((requests, drafts + 1)).astype(np.float32)
    if ragged:
        lengths = g.integers(-1, drafts + 2, requests).astype(np.int32)
    return p, qq, tokens, lengths, u


def call(q, dev, p, qq, tokens, lengths, u, **kw):
    acc, abuf = guarded((len(p),), torch.int32, dev, fill=-7)
    out, obuf = guarded(u.shape, torch.int32, dev, fill=-7)
    q.qmv_verify_drafts(p.to(dev), up(tokens, dev), up(u, dev), q=None if qq is None else qq.to(dev), lengths=up(lengths, dev),
                        accepted=acc, tokens=out, **kw)
    torch.cuda.synchronize()
    for b in (abuf, obuf):
        assert guards_intact(b) and int(b[0]) == -7
    return host(acc), host(out)


def wanted(p, qq, tokens, lengths, u):
    return o.verify(p.double().numpy(), None if qq is None else qq.double().numpy(), tokens, lengths, u)


@pytest.mark.parametrize("requests,drafts,vocab", [(1, 3, 32768), (1, 1, 1), (7, 3, 2), (5, 4, 1000), (3, 2, 4095), (3, 2, 4096),
                                                   (3, 2, 4097), (40, 3, 5003), (2, 32, 777), (6, 0, 9001), (2, 8, 50001),
                                                   (3, 3, 16384), (3, 3, 16385), (9, 2, 17403), (1, 2, 131075)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sampled", [True, False])
def test_against_the_oracle(q, dev, requests, drafts, vocab, kind, sampled):
    for cut in (False, True):
        c = case(rng(requests, drafts, vocab, cut), requests, drafts, vocab, kind, sampled, cut, ragged=cut)
        got, want = call(q, dev, *c), wanted(*c)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("stride", [1, 97])
def test_every_border_of_small_sums(q, dev, stride):
    # weights of few bits: every sum is exact, and u stands on, just below and just above each border
    g = rng(1)
    w = g.integers(0, 4, 300) / 1024
    w[[0, 5, 299]] = 0
    total, run = w.sum(), np.cumsum(w)
    scale = 2.0 ** np.ceil(np.log2(total)) / total             # whole sum a power of two: u * sum is exact
    w[7] += total * scale - total
    total, run = w.sum(), np.cumsum(w)
    assert np.log2(total) == np.round(np.log2(total)) and np.array_equal(w, w.astype(np.float32))
    us = np.unique(np.concatenate([run / total, np.nextafter((run / total).astype(np.float32), np.float32(0)),
                                   np.nextafter((run / total).astype(np.float32), np.float32(2))]).astype(np.float32))
    us = us[us < 1]
    p = torch.zeros((len(us), 1, 300 * stride))
    p[:, :, ::stride] = torch.from_numpy(w).float()            # side by side, and spread over chunks
    c = (p, None, np.zeros((len(us), 0), np.int32), None, us[:, None])
    got, want = call(q, dev, *c), wanted(*c)
    assert np.array_equal(got[1], want[1]) and len(np.unique(got[1])) > 150


@pytest.mark.parametrize("v", [9000, 70000])
def test_random_numbers_at_and_outside_their_ends(q, dev, v):
    p = np.zeros((6, 1, v), np.float32)
    p[:, 0, [17, 4096, 4500, 8191, 8192, v - 10]] = 0.125
    u = np.array([0.0, 1.0, 1.5, -1.0, np.nan, 1 - 2.0 ** -24], np.float32)[:, None]
    acc, out = call(q, dev, torch.from_numpy(p), None, np.zeros((6, 0), np.int32), None, u)
    assert out[:, 0].tolist() == [17, v - 10, v - 10, 17, v - 10, v - 10]
    one = torch.zeros((3, 1, v))
    one[0, 0, 0], one[1, 0, v - 1], one[2, 0, 4095] = 1.0, 1e-38, 3e38
    for x in (0.0, 0.5, 0.99999994):
        _, out = call(q, dev, one, None, np.zeros((3, 0), np.int32), None, np.full((3, 1), x, np.float32))
        assert out[:, 0].tolist() == [0, v - 1, 4095]


def test_tests_of_drafts_are_exact(q, dev):
    # u q against p where fp32 would round the product onto the border
    g = rng(2)
    n = 4000
    u, b = g.random(n).astype(np.float32), g.random(n).astype(np.float32)
    at = (u * b).astype(np.float32)                            # within half a step of u q, on either side or on it
    p = np.zeros((n, 2, 3), np.float32)
    qq = np.zeros((n, 1, 3), np.float32)
    p[:, 0, 1], p[:, 1, 2], qq[:, 0, 1] = at, 1.0, b
    stands = u.astype(np.float64) * b.astype(np.float64) < at.astype(np.float64)
    assert 1000 < stands.sum() < 3000
    acc, out = call(q, dev, torch.from_numpy(p), torch.from_numpy(qq), np.ones((n, 1), np.int32), None,
                    np.stack([u, np.full(n, 0.5, np.float32)], 1))
    assert np.array_equal(acc, stands.astype(np.int32))
    assert np.array_equal(out[stands], np.tile([1, 2], (stands.sum(), 1)))


@pytest.mark.parametrize("more", [0, 40000])
def test_nothing_left_and_values_that_are_not_finite(q, dev, more):
    v = 5000 + more                                            # zeros behind the 5000
    nan, inf = float("nan"), float("inf")
    p = torch.full((7, 2, v), 1.0 / 8192)
    p[:, :, 5000:] = 0
    qq = p[:, :1].clone()
    tokens = np.full((7, 1), 3, np.int32)
    u = np.tile(np.float32([1.0, 0.5]), (7, 1))                # 1 * q < p fails where they are equal
    p[1, 0] = 0                                                # nothing left at all
    p[2, 0, :] = nan
    p[3, 0, 100], p[3, 0, 200] = inf, nan                      # left out, the rest as it was
    qq[4, 0, 4000] = nan                                       # of this draft's weights none is positive, so p picks
    qq[5, 0, 4097] = 0                                         # one weight
    qq[6, 0, 10], p[6, 0, 20] = -inf, 1.0                      # inf does not count, 1 - 1/8192 does
    acc, out = call(q, dev, p, qq, tokens, None, u)
    want = wanted(p, qq, tokens, None, u)
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])
    assert acc.tolist() == [0] * 7 and out[:, 0].tolist() == [2500, -1, -1, 2501, 2500, 4097, 20]
    assert (out[:, 1] == -1).all()


def test_drafts_outside_the_vocabulary(q, dev):
    g = rng(3)
    for sampled in (True, False):
        p, qq, tokens, _, u = case(g, 5, 3, 100, "f32", sampled, ragged=False)
        tokens[0, 0], tokens[1, 1], tokens[2, 2], tokens[3, 0] = -1, 100, 1 << 30, -(1 << 31)
        u[:, :3] = 0                                           # any other draft with a probability stands
        got, want = call(q, dev, p, qq, tokens, None, u), wanted(p, qq, tokens, None, u)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert got[0].tolist() == [0, 1, 2, 0, 3]


@pytest.mark.parametrize("v", [8200, 30000])
def test_a_likeliest_draft_is_zeroed_wherever_it_stands(q, dev, v):
    for d in (0, 1, 1023, 1024, 4095, 4096, 8191, v - 1):
        p = torch.zeros((1, 2, v))
        p[0, 0, d], p[0, 0, (d + 5) % v] = 0.5, 0.5
        got = call(q, dev, p, None, np.array([[d]], np.int32), None, np.float32([[0.9, 0.1]]))
        assert got[0].tolist() == [0] and got[1][0].tolist() == [(d + 5) % v, -1]


def test_distribution_is_the_targets(q, dev):
    # over many random numbers the token that follows one draft from q has p's distribution
    g = rng(4)
    n, v = 60000, 5
    p, qq = np.float32([0.5, 0.2, 0.15, 0.1, 0.05]), np.float32([0.1, 0.4, 0.3, 0.05, 0.15])
    drafts = g.choice(v, (n, 1), p=qq / qq.sum()).astype(np.int32)
    pt = torch.from_numpy(np.tile(p, (n, 2, 1)))
    qt = torch.from_numpy(np.tile(qq, (n, 1, 1)))
    _, out = call(q, dev, pt, qt, drafts, None, g.random((n, 2)).astype(np.float32))
    seen = np.bincount(out[:, 0], minlength=v) / n
    assert np.abs(seen - p).max() < 5 * np.sqrt(0.25 / n)      # five standard deviations


def test_nothing_to_do_and_more_requests(q, dev):
    e = torch.empty
    acc, out = q.qmv_verify_drafts(e((0, 3, 10), device=dev), e((0, 2), dtype=torch.int32, device=dev), e((0, 3), device=dev))
    assert acc.shape == (0,) and out.shape == (0, 3)
    c = case(rng(5), 3000, 1, 33, "bf16")
    got, want = call(q, dev, *c), wanted(*c)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_the_most_requests(q, dev):
    c = case(rng(8), 65535, 1, 3, "f32")
    got, want = call(q, dev, *c), wanted(*c)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    p = torch.zeros((65535, 1, 16385))
    p[:, 0, 16384] = 1
    _, out = call(q, dev, p, None, np.zeros((65535, 0), np.int32), None, np.full((65535, 1), 0.3, np.float32))
    assert (out == 16384).all()


def test_rows_past_4_gib(q, dev):
    # p of 2^32 + values: the last request's rows lie behind 16 GiB
    r, v = 1030, 1 << 22
    p = torch.zeros((r, 1, v), dtype=torch.bfloat16, device=dev)
    p[r - 1, 0, v - 3], p[r - 1, 0, 5], p[0, 0, 9] = 0.5, 0.25, 1.0
    acc, out = q.qmv_verify_drafts(p, torch.empty((r, 0), dtype=torch.int32, device=dev),
                                   torch.full((r, 1), 0.4, device=dev))
    o_ = host(out)[:, 0]
    assert o_[0] == 9 and o_[r - 1] == v - 3 and (o_[1:r - 1] == -1).all()


def test_graph_and_streams(q, dev):
    cs = [case(rng(6, i), 4, 3, 20011, "f32", ragged=True) for i in range(4)]
    bufs = [cs[0][0].to(dev), cs[0][1].to(dev), *(up(a, dev) for a in cs[0][2:])]
    ws = torch.empty(q.qmv_verify_drafts_workspace(4, 20011), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()

    def step(**kw):
        return q.qmv_verify_drafts(bufs[0], bufs[2], bufs[4], q=bufs[1], lengths=bufs[3], **kw)

    with torch.cuda.stream(s):
        step(ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        acc, out = step(ws=ws)
    for c in cs:
        for b, v in zip(bufs, (c[0], c[1], *(torch.from_numpy(a) for a in c[2:]))):
            b.copy_(v)
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = wanted(*c)
        assert torch.equal(acc, eager[0]) and torch.equal(out, eager[1])
        assert np.array_equal(host(acc), want[0]) and np.array_equal(host(out), want[1])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    late = step(stream=other)
    other.synchronize()
    assert torch.equal(late[1], eager[1])


def test_refusals_of_the_binding(q, dev):
    p, qq, tokens, lengths, u = case(rng(7), 2, 2, 50, "f32")
    a = dict(p=p.to(dev), q=qq.to(dev), drafts=up(tokens, dev), lengths=up(lengths, dev), u=up(u, dev))
    for bad in ({"p": a["p"].half()}, {"q": a["q"].to(torch.bfloat16)}, {"drafts": a["drafts"].long()}, {"u": a["u"].double()},
                {"lengths": a["lengths"].long()}):
        with pytest.raises(TypeError):
            q.qmv_verify_drafts(**{**a, **bad})
    for bad in ({"p": a["p"][:, :2]}, {"q": a["q"][:1]}, {"u": a["u"][:, :2].contiguous()}, {"lengths": a["lengths"][:1]},
                {"p": a["p"][0]}, {"p": a["p"][:, :0]}):
        with pytest.raises(ValueError):
            q.qmv_verify_drafts(**{**a, **bad})
    wide = torch.zeros((2, 1, 20000), device=dev)
    with pytest.raises(q.QmvError):
        q.qmv_verify_drafts(wide, torch.empty((2, 0), dtype=torch.int32, device=dev), a["u"][:, :1].contiguous(),
                            ws=torch.empty(8, dtype=torch.uint8, device=dev))
    with pytest.raises(q.QmvError):
        q.qmv_verify_drafts(**a, accepted=a["lengths"])


@pytest.mark.parametrize("v", [8000, 32768])
@pytest.mark.parametrize("left", ["all", "rest"])
def test_a_random_number_of_one_picks_the_last_weight_of_any(q, dev, v, left):
    # sums that round: the whole may lie below a running sum of another order, and weights at the end below half its last bit
    g = rng(9, v)
    n = 64
    p = softmax(4 * g.standard_normal((n, 2, v)))
    p[:, :, v - 9:] = 0
    last = g.integers(v - 9, v, n)
    p[np.arange(n), 0, last] = 1e-30
    p = torch.from_numpy(p.astype(np.float32))
    tokens, u = np.zeros((n, 1), np.int32), np.ones((n, 2), np.float32)
    u[::3, 1] = np.float32([1 + 2.0 ** -23, np.inf, np.nan])[np.arange(len(u[::3])) % 3]
    qq = None
    if left == "rest":                                         # 1 * q < p does not hold, and half of p is left of every token
        p[:, 0, 0] = 0
        qq = p[:, :1] / 2
    lengths = np.full(n, 0 if left == "all" else 1, np.int32)
    c = (p, qq, tokens, lengths, u)
    got, want = call(q, dev, *c), wanted(*c)
    assert want[0].tolist() == got[0].tolist() == [0] * n
    assert want[1][:, 0].tolist() == last.tolist()
    assert got[1][:, 0].tolist() == last.tolist()

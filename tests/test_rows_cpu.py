"""The rows' operators and the verification of drafts without a GPU: the library exports what include/qmm_rows.h and
include/qmv_verify.h declare, refuses every malformed call before any HIP call, and the fp64 oracle that the GPU tests
use is pinned by values worked out by hand."""

import ctypes
import math
import os
import re
import weakref

import numpy as np
import pytest
import torch

import gguf_block_quantized_qmv_amd as q
import lora_cases as cases
from oracle import rows_oracle as o

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = q.lib

OK, NULL, SHAPE, SIZE, ALIGN, RANGE, WORKSPACE, ALIAS = 0, -1, -2, -3, -4, -5, -6, -7
F32, BF16 = 0, 1

# Fake, never dereferenced device addresses, 4 GiB apart: every call below is refused first.
A0 = 0x7F0000000000
X, Z, Y, TMP, IDS, OFF, IDX, PL, W, DW, SC, RK, A, B, U, LEN = (A0 + (i << 32) for i in range(16))
V = ctypes.c_void_p


@pytest.mark.parametrize("header,table,count", [("qmm_rows.h", "ROWS_EXPORTS", 7), ("qmv_verify.h", "VERIFY_EXPORTS", 2)])
def test_library_exports_what_the_headers_declare(header, table, count):
    with open(os.path.join(ROOT, "include", header)) as f:
        names = set(re.findall(r"^(?:int|size_t)\s+(qm[mv]_[a-z_0-9]+)\s*\(", f.read(), re.M))
    assert names == set(getattr(q, table)) and len(names) == count
    for name in names:
        assert hasattr(L, name) and callable(getattr(q, name)) and name in q.__all__


# ------------------------------------------------------------------ refusals

def sort(ids=IDS, off=OFF, idx=IDX, pl=PL, t=5000, k=8, e=128, ws=TMP, wn=1 << 30):
    return L.qmm_rows_sort(V(ids), V(off), V(idx), V(pl), t, k, e, V(ws), wn, None)


def test_sort_refusals():
    assert sort(ids=0) == NULL and sort(off=0) == NULL
    for bad in ({"t": -1}, {"k": 0}, {"k": 33}, {"e": 0}, {"e": 1025}, {"t": (1 << 24) // 8 + 1}, {"t": (1 << 31) - 1}):
        assert sort(**bad) == RANGE, bad
    assert sort(ids=IDS + 2) == ALIGN and sort(off=OFF + 1) == ALIGN and sort(idx=IDX + 2) == ALIGN
    assert sort(pl=PL + 2) == ALIGN and sort(ws=TMP + 128) == ALIGN
    need = L.qmm_rows_sort_workspace(5000, 8, 128)
    assert need > 0 and sort(ws=0) == WORKSPACE and sort(wn=need - 1) == WORKSPACE
    for pair in ({"off": IDS}, {"idx": IDS + 4}, {"pl": IDS}, {"pl": IDX}, {"off": IDX}, {"off": PL + 512}, {"ws": IDS},
                 {"ws": IDX}, {"ws": OFF - 256}):
        assert sort(**pair) == ALIAS, pair
    assert sort(off=IDS - 4 * 129) != ALIAS or need == 0       # side by side, no byte shared


def test_sort_workspaces():
    assert L.qmm_rows_sort_workspace(4, 8, 128) == 0 and L.qmm_rows_sort_workspace(2048, 8, 1024) == 0
    for bad in ((-1, 8, 128), (4, 0, 128), (4, 33, 128), (4, 8, 0), (4, 8, 1025), (1 << 22, 8, 128)):
        assert L.qmm_rows_sort_workspace(*bad) == 0, bad
    for t in (2049, 2500, 8192, 1 << 20, 1 << 21):
        b = L.qmm_rows_sort_workspace(t, 8, 128)
        assert 0 < b <= 256 * 128 * 4 and b % 512 == 0, t
    assert q.qmm_rows_sort_workspace((1 << 32) + 4, 8, 128) == 0


def spread(x=X, ty=F32, pl=PL, out=Y, t=10, k=4, h=100, rows=40):
    return L.qmm_rows_spread(V(x), ty, V(pl), V(out), t, k, h, rows, None)


def combine(z=Z, zt=F32, pl=PL, w=W, y=Y, yt=F32, t=10, k=4, h=100, rows=40):
    return L.qmm_rows_combine(V(z), zt, V(pl), V(w), V(y), yt, t, k, h, rows, None)


def grad(dy=X, z=Z, ty=F32, pl=PL, w=W, dz=Y, dw=DW, t=10, k=4, h=100, rows=40):
    return L.qmm_rows_combine_grad(V(dy), V(z), ty, V(pl), V(w), V(dz), V(dw), t, k, h, rows, None)


@pytest.mark.parametrize("call", [spread, combine, grad])
def test_move_refusals(call):
    for bad in ({"t": -1}, {"k": 0}, {"k": 33}, {"rows": -1}, {"rows": (1 << 24) + 1}, {"t": 1 << 23}, {"h": (1 << 20) + 1}):
        assert call(**bad) == RANGE, bad
    assert call(h=0) == SHAPE and call(h=-5) == SHAPE
    assert call(pl=0) == NULL and call(pl=PL + 2) == ALIGN
    assert call(t=0) == OK


def test_spread_refusals():
    assert spread(ty=2) == RANGE and spread(x=0) == NULL and spread(out=0) == NULL
    assert spread(x=X + 8) == ALIGN and spread(out=Y + 4) == ALIGN
    assert spread(out=X) == ALIAS and spread(out=PL) == ALIAS and spread(out=X + 10 * 400 - 16) == ALIAS
    assert spread(rows=0) == OK


def test_combine_refusals():
    assert combine(zt=2) == RANGE and combine(yt=-1) == RANGE and combine(z=0) == NULL and combine(y=0) == NULL
    assert combine(z=Z + 8) == ALIGN and combine(y=Y + 8) == ALIGN and combine(w=W + 1) == ALIGN
    for base in (Z, PL, W):
        assert combine(y=base) == ALIAS


def test_combine_grad_refusals():
    assert grad(ty=3) == RANGE
    for name in ("dy", "z", "dw", "dz"):                       # z and dw go together
        assert grad(**{name: 0}) == NULL, name
    for name, base in (("dy", X), ("z", Z), ("dz", Y)):
        assert grad(**{name: base + 8}) == ALIGN, name
    assert grad(w=W + 2) == ALIGN and grad(dw=DW + 2) == ALIGN
    for base in (X, Z, PL, W, DW):
        assert grad(dz=base & ~15) == ALIAS, base
    for base in (X, Z, PL, W):
        assert grad(dw=base) == ALIAS, base
    assert grad(rows=0, z=0, dw=0, dz=0) == OK                 # nothing to do


def lora(a=A, an=None, b=B, bn=None, sc=SC, rk=RK, x=X, off=OFF, idx=IDX, base=Z, y=Y, ty=F32, rows=40, x_rows=50, n=200,
         k=256, rank=40, e=4, ws=TMP, wn=1 << 30):
    an = 2 * e * rank * k if an is None else an
    bn = 2 * e * rank * n if bn is None else bn
    return L.qmm_lora(V(a), an, V(b), bn, V(sc), V(rk), V(x), V(off), V(idx), V(base), V(y), ty, rows, x_rows, n, k, rank, e,
                      V(ws), wn, None)


def test_lora_refusals():
    for name in ("a", "b", "x", "off", "base", "y"):
        assert lora(**{name: 0}) == NULL, name
    for bad in ({"ty": 2}, {"rows": -1}, {"rows": (1 << 24) + 1}, {"x_rows": -1}, {"x_rows": (1 << 24) + 1}, {"e": 0},
                {"e": 1025}, {"n": (1 << 20) + 1}, {"k": (1 << 20) + 8}, {"rank": 136}):
        assert lora(**bad) == RANGE, bad
    for bad in ({"n": 0}, {"k": 0}, {"k": 12}, {"rank": 0}, {"rank": 12}, {"rank": -8}, {"idx": 0}):
        assert lora(**bad) == SHAPE, bad
    assert lora(an=0) == SIZE and lora(bn=2 * 4 * 40 * 200 - 1) == SIZE and lora(an=2 * 4 * 40 * 256 + 2) == SIZE
    for name, base in (("a", A), ("b", B), ("x", X), ("base", Z), ("y", Y)):
        assert lora(**{name: base + 8}) == ALIGN, name
    assert lora(sc=SC + 2) == ALIGN and lora(rk=RK + 1) == ALIGN and lora(off=OFF + 2) == ALIGN
    assert lora(idx=IDX + 2) == ALIGN and lora(ws=TMP + 64) == ALIGN
    need = L.qmm_lora_workspace(40, 200, 256, 40, 4)
    assert need > 0 and lora(ws=0) == WORKSPACE and lora(wn=need - 1) == WORKSPACE
    for at in (A, B, SC, RK, X, OFF, IDX, Z + 16, TMP):
        assert lora(y=at) == ALIAS, hex(at)
    for at in (A, B, SC, RK, X, OFF, IDX, Z, Y):
        assert lora(ws=at) == ALIAS, hex(at)
    assert lora(rows=0) == OK and lora(x_rows=0) == OK         # nothing to do
    assert lora(rows=0, an=1) == SIZE


def test_lora_workspaces():
    for bad in ((-1, 64, 64, 16, 1), (4, 0, 64, 16, 1), (4, 64, 60, 16, 1), (4, 64, 64, 12, 1), (4, 64, 64, 16, 0), (0, 64, 64, 16, 1)):
        assert L.qmm_lora_workspace(*bad) == 0, bad
    for rows in (1, 16, 17, 64, 300, 4096, 1 << 20):
        for k in (8, 64, 1000, 5120, 17408):
            for e in (1, 24, 1024):
                b = L.qmm_lora_workspace(rows, 5120, k, 64, e)
                # at most 16 parts of k, none without a block of 64
                assert b % (rows * 64 * 4) == 0 and 1 <= b // (rows * 64 * 4) <= max(1, min(16, -(-k // 64))), (rows, k, e)
    assert L.qmm_lora_workspace(1, 5120, 2048, 16, 8) == 0     # a small A: one launch
    # many: parts of k that fill the CUs evenly, 130 tiles by 3
    assert L.qmm_lora_workspace(4096, 5120, 5120, 64, 5) == 3 * 4096 * 64 * 4
    # few rows: the parts of k, and so a row's bits, go by k alone
    assert {L.qmm_lora_workspace(r, 5120, 5120, 64, e) // r for r in (1, 2, 7, 16) for e in (1, 3, 1024)} == {8 * 256}


def test_lora_with_more_workgroups_than_a_grid_takes():
    # (rows / 16 + min(rows, adapters)) * ceil(n / 256) up to 2^28: 65536 tiles by 4096
    n, rows = 1 << 20, (65536 - 4) * 16
    assert lora(n=n, rows=rows, ws=0) == WORKSPACE             # in range: the next check speaks
    assert lora(n=n, rows=rows + 16, ws=0) == RANGE and L.qmm_lora_workspace(rows + 16, n, 256, 40, 4) == 0


def test_lora_in_one_launch():
    def one(rows, n, k, rank, e):
        return L.qmm_lora_workspace(rows, n, k, rank, e) == 0

    ks, ns = range(8, 9000, 56), (1, 1024, 1025, 5120, 16384, 17408, 18432, 18433, 20480, 1 << 20)
    # a rank of 8 takes a rank of 16's time, 24 that of 32: as many lines of A are loaded
    for rows, e in ((1, 8), (16, 16), (64, 5), (64, 64), (1000, 5)):
        for lower, upper in ((8, 16), (24, 32)):
            assert [one(rows, 2048, k, lower, e) for k in ks] == [one(rows, 2048, k, upper, e) for k in ks], (rows, lower)
    # few rows: the choice, and so a row's bits, goes by n, k and rank alone
    for n in ns:
        for k in (64, 2048, 3624, 3632, 5120, 5440, 5448, 8192):
            for rank in (8, 16, 24, 32, 40):
                assert len({one(rows, n, k, rank, e) for rows in (1, 2, 9, 16) for e in (1, 8, 16, 1024)}) == 1, (n, k, rank)
    # one launch up to some length, then two; and none above rank 32
    for rows, e in ((1, 8), (16, 1024), (17, 3), (64, 5), (1000, 5)):
        for rank in (8, 16, 24, 32):
            took = [one(rows, 1024, k, rank, e) for k in ks]
            assert took[0] and not took[-1] and took == sorted(took, reverse=True), (rows, rank)
        assert not one(rows, 64, 64, 40, e)
    # more workgroups than CUs would wait for each other
    assert one(300, 5120, 1024, 16, 5) and not one(2000, 5120, 1024, 16, 5) and not one(100, 5120, 1024, 16, 100)


def verify(p=X, qq=Z, ty=F32, tok=IDS, ln=LEN, u=U, acc=DW, out=Y, r=3, d=4, v=20000, ws=TMP, wn=1 << 30):
    return L.qmv_verify_drafts(V(p), V(qq), ty, V(tok), V(ln), V(u), V(acc), V(out), r, d, v, V(ws), wn, None)


def test_verify_refusals():
    for name in ("p", "tok", "u", "acc", "out"):
        assert verify(**{name: 0}) == NULL, name
    for bad in ({"ty": 2}, {"d": -1}, {"d": 33}, {"r": -1}, {"r": 65536}, {"v": (1 << 22) + 1}):
        assert verify(**bad) == RANGE, bad
    assert verify(v=0) == SHAPE and verify(v=-3) == SHAPE
    for name, base, by in (("p", X, 8), ("qq", Z, 4), ("tok", IDS, 2), ("ln", LEN, 1), ("u", U, 2), ("acc", DW, 2), ("out", Y, 2),
                           ("ws", TMP, 128)):
        assert verify(**{name: base + by}) == ALIGN, name
    need = L.qmv_verify_drafts_workspace(3, 20000)
    assert need > 0 and verify(ws=0) == WORKSPACE and verify(wn=need - 1) == WORKSPACE
    for at in (X, Z, IDS, LEN, U):
        assert verify(acc=at) == ALIAS and verify(out=at) == ALIAS and verify(ws=at) == ALIAS
    assert verify(acc=Y) == ALIAS
    assert verify(r=0, p=0, u=0, acc=0, out=0) == OK
    assert L.qmv_verify_drafts_workspace(3, 16384) == 0 and L.qmv_verify_drafts_workspace(3, 16385) == 3 * 17 * 16
    assert L.qmv_verify_drafts_workspace(3, 0) == 0 and L.qmv_verify_drafts_workspace(-1, 10) == 0
    assert q.qmv_verify_drafts_workspace(3, (1 << 32) + 10) == 0


def test_binding_refuses_what_is_not_on_a_gpu():
    i, f = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 8)
    bank = torch.zeros(1, 8, 8, dtype=torch.bfloat16)
    for call in (lambda: q.qmm_rows_sort(i, 4), lambda: q.qmm_rows_spread(f, i), lambda: q.qmm_rows_combine(f, i),
                 lambda: q.qmm_rows_combine_grad(f, f, i), lambda: q.qmm_lora(bank[0], bank, bank, i[0], f),
                 lambda: q.qmv_verify_drafts(bank, i, f)):
        with pytest.raises(ValueError, match="device memory"):
            call()
    with pytest.raises(TypeError, match="torch tensor"):
        q.qmm_rows_sort([[1]], 4)


class Fake:
    """A contiguous device tensor by its attributes alone."""

    def __init__(self, shape, dtype=torch.int32, address=1 << 20):
        self.shape, self.dtype, self.device, self.address = torch.Size(shape), dtype, 0, address

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()


HUGE = (1 << 32) + 5   # a C int of this value is 5


def test_sizes_that_a_c_int_does_not_hold_are_refused(monkeypatch):
    calls = []
    monkeypatch.setattr(q, "_run", lambda *a: calls.append(a))
    f, bf = torch.float32, torch.bfloat16
    plan = (Fake((5,)), Fake((12,)), Fake((4, 3)))

    def refused(call):
        with pytest.raises(q.QmvError) as e:
            call()
        assert e.value.code == RANGE and calls == []

    for t, k, e in ((HUGE, 3, 4), (4, HUGE, 4), (4, 3, HUGE)):
        refused(lambda: q.qmm_rows_sort(Fake((t, k)), e, *plan))
    for t, k, h, r in ((HUGE, 3, 8, 9), (4, HUGE, 8, 9), (4, 3, HUGE, 9), (4, 3, 8, HUGE)):
        x, z, pl, w = Fake((t, h), f), Fake((r, h), f), Fake((t, k)), Fake((t, k), f)
        refused(lambda: q.qmm_rows_spread(x, pl, out=z))
        refused(lambda: q.qmm_rows_combine(z, pl, w, y=x))
        refused(lambda: q.qmm_rows_combine_grad(x, z, pl, w, dz=z, dw=w))
    for x_rows, rows, n, k, rank, e in ((HUGE, 7, 8, 8, 8, 1), (9, HUGE, 8, 8, 8, 1), (9, 7, HUGE, 8, 8, 1), (9, 7, 8, HUGE, 8, 1),
                                        (9, 7, 8, 8, HUGE, 1), (9, 7, 8, 8, 8, HUGE)):
        refused(lambda: q.qmm_lora(Fake((x_rows, k), bf), Fake((e, rank, k), bf), Fake((e, n, rank), bf), Fake((e + 1,)),
                                   Fake((x_rows, n), f), row_index=Fake((rows,)), ws=Fake((1 << 20,), torch.uint8)))
    for r, d, v in ((HUGE, 3, 100), (2, HUGE, 100), (2, 3, HUGE)):
        refused(lambda: q.qmv_verify_drafts(Fake((r, d + 1, v), f), Fake((r, d)), Fake((r, d + 1), f), accepted=Fake((r,)),
                                            tokens=Fake((r, d + 1))))
    assert q.qmm_lora_workspace(HUGE, 64, 64, 16, 1) == 0 and q.qmm_lora_workspace(4, 64, HUGE + 3, 16, 1) == 0


def test_what_may_be_left_out(monkeypatch):
    calls = []
    monkeypatch.setattr(q, "_run", lambda fn, name, index, stream, *a: calls.append(a))
    f, bf = torch.float32, torch.bfloat16
    x, z, pl = Fake((4, 8), f, 16), Fake((9, 8), f, 32), Fake((4, 3), address=48)
    q.qmm_rows_combine(z, pl, y=x)
    assert calls.pop()[3] is None
    q.qmm_rows_combine_grad(x, None, pl, dz=z)
    assert calls[-1][1] is None and calls[-1][4] is None and calls.pop()[6] is None
    ws = Fake((1 << 20,), torch.uint8, 64)
    a, b, off, y = Fake((2, 8, 16), bf), Fake((2, 10, 8), bf), Fake((3,)), Fake((4, 10), f, 80)
    q.qmm_lora(Fake((4, 16), bf), a, b, off, y, ws=ws)
    got = calls.pop()
    assert got[4] is None and got[5] is None and got[8] is None and got[9] == got[10] == 80 and got[-2:] == (64, 1 << 20)
    q.qmm_lora(Fake((4, 16), bf), a, b, off, y, row_index=Fake((0,), address=0), ws=ws)   # no rows: nothing is launched
    assert calls == []
    q.qmv_verify_drafts(Fake((2, 4, 100), f), Fake((2, 3)), Fake((2, 4), f), accepted=Fake((2,)), tokens=Fake((2, 4)))
    got = calls.pop()
    assert got[1] is None and got[4] is None and got[8:] == (2, 3, 100, None, 0)
    for missing in ("z", "places"):
        with pytest.raises(TypeError):
            q.qmm_rows_combine(**{**dict(z=z, places=pl, y=x), missing: None})


def test_a_workspace_that_the_binding_makes_lives_until_the_call_has_been_made(monkeypatch):
    # let go of before, another thread's call on the same stream could be given its memory in between
    made, calls = [], []

    def new(shape, dtype, *a, **kw):
        t = Fake(shape, dtype)
        if dtype == torch.uint8:
            made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(q, "_new", new)
    monkeypatch.setattr(q, "_run", lambda fn, name, *a: calls.append((name, [m() is not None for m in made])))
    f, bf = torch.float32, torch.bfloat16
    q.qmm_rows_sort(Fake((5000, 8)), 128)
    q.qmm_lora(Fake((40, 256), bf), Fake((4, 40, 256), bf), Fake((4, 200, 40), bf), Fake((5,)), Fake((40, 200), f))
    q.qmv_verify_drafts(Fake((3, 5, 20000), f), Fake((3, 4)), Fake((3, 5), f))
    assert [c[0] for c in calls] == ["qmm_rows_sort", "qmm_lora", "qmv_verify_drafts"]
    assert [c[1][-1] for c in calls] == [True] * 3 and len(made) == 3
    assert [m() for m in made] == [None] * 3                   # and no longer


def test_what_is_no_tensor_is_refused_by_name(monkeypatch):
    calls = []
    monkeypatch.setattr(q, "_run", lambda *a: calls.append(a))
    f, bf = torch.float32, torch.bfloat16
    lora_args = dict(x=Fake((40, 256), bf), a=Fake((4, 40, 256), bf), b=Fake((4, 200, 40), bf), offsets=Fake((5,)),
                     y=Fake((40, 200), f), ws=Fake((1 << 20,), torch.uint8))
    z, places, y = Fake((9, 8), f), Fake((4, 3)), Fake((4, 8), f)
    for name, call in (("row_index", lambda v: q.qmm_lora(**{**lora_args, "row_index": v})),
                       ("ws", lambda v: q.qmm_lora(**{**lora_args, "ws": v})),
                       ("scale", lambda v: q.qmm_lora(**{**lora_args, "scale": v})),
                       ("base", lambda v: q.qmm_lora(**{**lora_args, "base": v})),
                       ("y", lambda v: q.qmm_lora(**{**lora_args, "y": v})),
                       ("y", lambda v: q.qmm_rows_combine(z, places, y=v)),
                       ("weights", lambda v: q.qmm_rows_combine(z, places, v, y=y)),
                       ("out", lambda v: q.qmm_rows_spread(y, places, out=v)),
                       ("dz", lambda v: q.qmm_rows_combine_grad(y, z, places, dz=v, dw=Fake((4, 3), f))),
                       ("ws", lambda v: q.qmm_rows_sort(Fake((4, 8)), 9, Fake((10,)), Fake((32,)), Fake((4, 8)), ws=v)),
                       ("ws", lambda v: q.qmv_verify_drafts(Fake((2, 4, 100), f), Fake((2, 3)), Fake((2, 4), f),
                                                            accepted=Fake((2,)), tokens=Fake((2, 4)), ws=v))):
        for bad in ([0] * 4, 7):
            with pytest.raises(TypeError, match=f"{name} must be a torch tensor"):
                call(bad)
    assert calls == []


# ------------------------------------------------------------------ the oracle

def test_sort_by_hand():
    off, idx, pl = o.sort([[2, 0], [7, 2], [0, 0], [-1, 1]], 3)
    assert off.tolist() == [0, 3, 4, 6]
    assert idx.tolist() == [0, 2, 2, 3, 0, 1, -1, -1]
    assert pl.tolist() == [[4, 0], [-1, 5], [1, 2], [-1, 3]]


def test_there_and_back_by_hand():
    x, pl = np.array([[1.0, 2.0], [3.0, 4.0]]), np.array([[2, 0], [-1, 3]])
    out = o.spread(x, pl, np.full((5, 2), 9.0))
    assert out.tolist() == [[1, 2], [9, 9], [1, 2], [3, 4], [9, 9]]
    w = np.array([[0.5, 2.0], [7.0, -1.0]])
    y, mag = o.combine(out, pl, w)
    assert y.tolist() == [[2.5, 5], [-3, -4]] and mag.tolist() == [[2.5, 5], [3, 4]]
    dz, dw, _ = o.combine_grad([[1.0, 0.0], [0.0, 2.0]], out, pl, w, np.full((5, 2), 9.0))
    assert dz.tolist() == [[2, 0], [9, 9], [0.5, 0], [0, -2], [9, 9]] and dw.tolist() == [[1, 1], [0, 8]]


def test_gradient_against_differences():
    g = np.random.default_rng(1)
    off, idx, pl = o.sort(g.integers(-1, 4, (6, 3)), 4)
    z, w, dy = g.standard_normal((18, 5)), g.standard_normal((6, 3)), g.standard_normal((6, 5))
    dz, dw, _ = o.combine_grad(dy, z, pl, w, np.zeros((18, 5)))
    # y is linear in z and in w: a difference of one step is the gradient
    for at in ((0, 0), (3, 4), (17, 2), (8, 1)):
        step = np.zeros_like(z)
        step[at] = 1
        assert abs(((o.combine(z + step, pl, w)[0] - o.combine(z, pl, w)[0]) * dy).sum() - dz[at]) < 1e-12
    for at in ((0, 0), (5, 2), (2, 1)):
        step = np.zeros_like(w)
        step[at] = 1
        assert abs(((o.combine(z, pl, w + step)[0] - o.combine(z, pl, w)[0]) * dy).sum() - dw[at]) < 1e-12
    # the spread's gradient: rows summed back without weights
    x, dout = g.standard_normal((6, 5)), g.standard_normal((18, 5))
    assert abs((o.spread(x, pl, np.zeros((18, 5))) * dout).sum() - (x * o.combine(dout, pl, None)[0]).sum()) < 1e-12


def test_lora_by_hand():
    a = np.array([[[1.0, 0], [0, 1]], [[2.0, 0], [0, 0]]])
    b = np.array([[[1.0, 1], [0, 1]], [[1.0, 9], [3, 9]]])
    x = np.array([[1.0, 2], [3, 4], [5, 6]])
    y, mag = o.lora(x, a, b, [0, 1, 2], [2, 0], [1.0, 10.0], [2, 1], np.ones((3, 2)))
    assert y.tolist() == [[21, 61], [1, 1], [12, 7]] and mag[0].tolist() == [20, 60]


def test_verify_by_hand():
    p = [[0.5, 0.5, 0.0], [0.1, 0.2, 0.7], [0.25, 0.25, 0.5]]
    qq = [[1.0, 0.0, 0.0], [0.6, 0.0, 0.4]]
    # 0.4 * 1 < 0.5 stands, 0.2 * 0.6 >= 0.1 does not: max(p - q, 0) = (0, 0.2, 0.3), 0.3 * 0.5 falls on token 1
    assert o.verify_one(p, qq, [0, 0], [0.4, 0.2, 0.3]) == (1, 1)
    assert o.verify_one(p, qq, [0, 0], [0.4, 0.1, 0.25]) == (2, 1)         # all stand: a sum of 0.25 is not above it
    assert o.verify_one(p, qq, [1, 0], [0.0, 0, 0]) == (2, 0)              # 0 < 0.5 and 0 < 0.1 stand; p[2] from 0
    assert o.verify_one(p, qq, [2, 0], [0.0, 0, 0.9]) == (0, 1)            # 0 < 0 does not; (0, 0.5, 0)
    assert o.verify_one(p, None, [0, 2], [0.4, 0.75, 0.4]) == (1, 1)       # without q: (0.1, 0.2, 0)
    assert o.verify_one(p, qq, [], [0.99]) == (0, 1)
    assert o.verify_one([[0.5, 0.5]] * 2, [[0.5, 0.5]], [1], [1.0, 0.6]) == (0, 1)   # nothing left: p itself
    assert o.verify_one([[0.0, np.nan]], None, [], [0.5]) == (0, -1)
    acc, out = o.verify([p], [qq], [[0, 0]], [1], [[0.4, 0.9, 0.3]])       # 0.1 + 0.2 lies above 0.3 in 64 bits
    assert acc.tolist() == [1] and out.tolist() == [[0, 1, -1]]


def test_verify_picks_the_last_weight_from_one_on():
    # 0.8 + 0.9 + 0.7 added one by one lies above their sum rounded once
    w = [0.8, 0.9, 0.7, 1e-30, 0.0]
    assert w[0] + w[1] + w[2] > math.fsum(w)
    for u in (1.0, 1 + 2.0 ** -23, 7.0, math.inf, math.nan):
        assert o.verify_one([w], None, [], [u]) == (0, 3), u
    assert o.verify_one([w], None, [], [1 - 2.0 ** -24]) == (0, 2)


@pytest.mark.parametrize("rows,rank", cases.ROWS_RANKS)
def test_every_block_of_k_counts_in_the_whole_numbers(rows, rank):
    # a block of 64 lost, taken twice, or a row's blocks taken from their neighbour's places: some result differs
    for k in cases.KS:
        c = cases.whole_numbers(rows, 67, k, rank)
        y, adds = cases.result(c), cases.by_block(c, 0)
        assert np.array_equal(adds.sum(0) + c["base"][0], y[0]) and len(adds) == -(-k // 64)
        assert adds.any(axis=1).all(), k
        assert np.abs(y).max() < 1 << 24
        if k > 64:
            assert (cases.result(c, np.roll(c["a"], 64, axis=2))[0] != y[0]).any()
        e, rows_of = c["owner"], np.abs(c["x"]).sum(1).max()
        assert 2 * rows_of * rank + 8 < 1 << 24 and (e == 0).any()


def test_whole_numbers_take_both_plans():
    one = {(rows, k, rank): q.qmm_lora_workspace(rows, 67, k, rank, cases.ADAPTERS) == 0 for rows, rank in cases.ROWS_RANKS
           for k in cases.KS}
    assert set(one.values()) == {True, False}
    for rows in (1, 16, 40, 300):                              # the change from one to two launches lies within
        assert {v for (r, _, rank), v in one.items() if r == rows and rank <= 32} == {True, False}, rows

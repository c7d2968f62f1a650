"""The e4m3 binding without a GPU, on stand-in tensors and a stand-in library: what reaches the C entry points."""

import os
import subprocess
import sys

import pytest
import torch

import gguf_block_quantized_qmv_amd as q


class Fake:
    """A contiguous device tensor by its attributes alone."""

    def __init__(self, shape, dtype=torch.uint8, device=0, address=1 << 20):
        self.shape, self.dtype, self.device, self.address = torch.Size(shape), dtype, device, address

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()


@pytest.fixture
def calls(monkeypatch):
    """Records what _run is given."""
    seen = []
    monkeypatch.setattr(q, "_run", lambda fn, name, index, stream, *args: seen.append((name, args)))
    return seen


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HUGE = (1 << 32) + 5   # a C int of this value is 5


@pytest.fixture
def refused():
    """A context in which one call has to be refused as out of range."""
    def check(call):
        with pytest.raises(q.QmvError) as e:
            call()
        assert e.value.code == -5
    return check


def test_more_rows_than_a_c_int_are_refused(calls, refused):
    ws, off = Fake((1, 1), torch.float32), Fake((2,), torch.int32)
    refused(lambda: q.qmm_fp8(Fake((64, 128)), ws, Fake((HUGE, 128)), Fake((1, HUGE), torch.float32), 64, 128,
                              y=Fake((HUGE, 64), torch.float32)))
    refused(lambda: q.qmm_fp8_quant(Fake((HUGE, 128), torch.float32), xq=Fake((HUGE, 128)),
                                    xs=Fake((1, HUGE), torch.float32)))
    refused(lambda: q.qmm_fp8_quant_silu_mul(Fake((HUGE, 256), torch.float32), xq=Fake((HUGE, 128)),
                                             xs=Fake((1, HUGE), torch.float32)))
    bank = Fake((1, 64, 128), torch.bfloat16)
    for x_rows, index in ((HUGE, None), (HUGE, Fake((7,), torch.int32)), (4, Fake((HUGE,), torch.int32))):
        rows = HUGE if index is None else index.numel()
        refused(lambda: q.qmm_bf16_grouped(bank, Fake((x_rows, 128), torch.bfloat16), off, 64, 128, row_index=index,
                                           y=Fake((rows, 64), torch.float32)))
    assert calls == []
    for shape in ((HUGE + 300, 5120, 17408), (300, HUGE + 5120, 17408), (300, 5120, HUGE + 17403)):
        assert q.qmm_fp8_workspace(*shape) == 0
    assert q.qmm_fp8_workspace(300, 5120, 17408) > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_empty_batch_gives_an_empty_result(calls, dtype):
    # as the grouped products and the quantisers: the C entry is for m >= 1
    y = Fake((0, 64), dtype, address=0)
    assert q.qmm_fp8(Fake((64, 128)), Fake((1, 1), torch.float32), Fake((0, 128), address=0),
                     Fake((1, 0), torch.float32, address=0), 64, 128, y=y) is y
    assert calls == []
    with pytest.raises(ValueError, match="w has shape"), pytest.MonkeyPatch.context() as p:
        p.setattr(q, "_dev", lambda *a: None)
        q.qmm_fp8(Fake((65, 128)), Fake((1, 1), torch.float32), Fake((0, 128)), Fake((1, 0), torch.float32), 64, 128, y=y)


def test_workspace_of_a_type_that_is_no_result(calls):
    for dtype in (torch.float16, torch.uint8, "bf16"):
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            q.qmm_fp8_workspace(300, 5120, 17408, dtype)
    assert q.qmm_fp8_workspace(300, 5120, 17408, torch.bfloat16) == q.qmm_fp8_workspace(300, 5120, 17408)


def test_the_binding_needs_no_private_name_of_torch():
    # the current stream's handle by torch's public call when its short one is gone
    code = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import gguf_block_quantized_qmv_amd as q
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda index: Stream() if index == 3 else None
torch.cuda.current_device = lambda: 3
seen = []
q._run(lambda *a: seen.append(a) or 0, "call", 3, None, 1, 2)
assert seen == [(1, 2, 77)], seen
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr

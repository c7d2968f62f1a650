"""Python binding of the gfx950 block-quantized matrix-vector library (libqmv.so).

Argument marshalling only: every function below checks tensor dtypes/devices,
takes device pointers and torch's current stream, and calls the C entry point of
the same name declared in include/qmv.h or include/qmm_fp8.h. All computation happens in the HIP
kernels of the library; there is no fallback path. Importing this package
without a built library raises ImportError.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "QmvError", "lib", "LIB_PATH", "version",
    "qmv_q8_0", "qmv_q4_k", "qmv_q4_k_pair", "qmv_iq4_xs", "qmv_q4_k_moe", "qmv_q4_k_moe_workspace", "qmv_q4_k_moe_prefill",
    "qmv_q4_k_moe_noalloc",
    "qmv_q4_k_moe_prefill_workspace", "qmv_iq4_xs_moe",
    "qmv_iq4_xs_moe_workspace", "qmm_q4_k_prefill_workspace",
    "qmm_q4_k_prefill", "qmv_dequant_q4_k_f32", "qmv_dequant_q4_k_bf16", "qmv_dequant_q8_0_f32",
    "qmv_dequant_iq4_xs_f32", "qmv_q5_k", "qmv_dequant_q5_k_f32", "qmv_q6_k", "qmv_dequant_q6_k_f32", "qmv_q4_0",
    "qmv_dequant_q4_0_f32", "qmv_stream_read", "q4_0_bytes",
    "q4_k_bytes", "q5_k_bytes", "q6_k_bytes", "q8_0_bytes",
    "iq4_xs_bytes", "EXPORTS",
    "qmm_fp8_quant", "qmm_fp8_quant_silu_mul", "qmm_fp8", "qmm_fp8_workspace", "qmm_fp8_grouped", "qmm_bf16_grouped",
    "FP8_EXPORTS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmv.so")

_c_int, _c_size, _vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p

# name -> (restype, argtypes); mirrors include/qmv.h
EXPORTS = {
    "qmv_version": (_c_int, []),
    "qmv_strerror": (ctypes.c_char_p, [_c_int]),
    "qmv_last_error": (ctypes.c_char_p, []),
    "qmv_q8_0": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_q4_k": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_q4_k_pair": (_c_int, [_vp, _vp, _c_size, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_iq4_xs": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_q5_k": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_q6_k": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_q4_0": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "qmv_q4_k_moe_workspace": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "qmv_q4_k_moe": (_c_int, [_vp, _vp, _vp, _c_size, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_size,
                              _c_int, _c_int, _c_int, _c_int, _c_int, _vp]),
    "qmv_q4_k_moe_noalloc": (_c_int, [_vp, _vp, _vp, _c_size, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _c_int, _c_int, _c_int, _c_int, _c_int, _vp]),
    "qmv_q4_k_moe_prefill_workspace": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "qmv_q4_k_moe_prefill": (_c_int, [_vp, _vp, _vp, _c_size, _vp, _vp, _vp, _vp, _vp, _vp, _c_size,
                                      _c_int, _c_int, _c_int, _c_int, _c_int, _vp]),
    "qmv_iq4_xs_moe_workspace": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "qmv_iq4_xs_moe": (_c_int, [_vp, _vp, _vp, _c_size, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_size,
                                _c_int, _c_int, _c_int, _c_int, _c_int, _vp]),
    "qmm_q4_k_prefill_workspace": (_c_size, [_c_int, _c_int, _c_int]),
    "qmm_q4_k_prefill": (_c_int, [_vp, _c_size, _vp, _vp, _c_int, _c_int, _c_int, _vp, _c_size, _vp]),
    "qmv_dequant_q4_k_f32": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_dequant_q4_k_bf16": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_dequant_q8_0_f32": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_dequant_iq4_xs_f32": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_dequant_q5_k_f32": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_dequant_q6_k_f32": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_dequant_q4_0_f32": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _vp]),
    "qmv_stream_read": (_c_int, [_vp, _c_size, _vp, _c_int, _c_int, _c_int, _vp]),
}

# name -> (restype, argtypes); mirrors include/qmm_fp8.h
FP8_EXPORTS = {
    "qmm_fp8_quant": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _c_int, _vp]),
    "qmm_fp8_quant_silu_mul": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _c_int, _vp]),
    "qmm_fp8_workspace": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "qmm_fp8": (_c_int, [_vp, _c_size, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _c_size, _vp]),
    "qmm_fp8_grouped": (_c_int, [_vp, _c_size, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                 _c_int, _vp]),
    "qmm_bf16_grouped": (_c_int, [_vp, _c_size, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _vp]),
}


def _load():
    # torch's HIP build ships its own libamdhip64 (same soname as the system one).
    # Loading torch first makes libqmv.so bind to that already-loaded runtime, so
    # the process holds exactly one HIP runtime; two runtimes in one process do
    # not share a device (the second reports that no device is present).
    import torch  # noqa: F401

    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python gguf_block_quantized_qmv_amd/build.py` "
            "(or __graft_entry__.build()) first")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in (*EXPORTS.items(), *FP8_EXPORTS.items()):
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


lib = _load()


class QmvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = lib.qmv_last_error().decode() if code == -8 else ""
        super().__init__(f"{where}: {lib.qmv_strerror(code).decode()} (code {code})" + (f" [{detail}]" if detail else ""))


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise QmvError(rc, where)


def version() -> int:
    return lib.qmv_version()


def q4_k_bytes(n: int, k: int) -> int:
    return n * (k // 256) * 144


def q5_k_bytes(n: int, k: int) -> int:
    return n * (k // 256) * 176


def q6_k_bytes(n: int, k: int) -> int:
    return n * (k // 256) * 210


def q4_0_bytes(n: int, k: int) -> int:
    return n * (k // 32) * 18


def q8_0_bytes(n: int, k: int) -> int:
    return n * (k // 32) * 34


# ---------------------------------------------------------------- marshalling helpers

def _torch():
    import torch
    return torch


def _dev(t, name, dtypes):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be in device memory (got {t.device})")
    if dtypes and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _nbytes(t):
    return t.numel() * t.element_size() if t is not None else 0


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _bf16_types():
    torch = _torch()
    return (torch.bfloat16, torch.int16, torch.uint16)


# ---------------------------------------------------------------- entry points

def qmv_q8_0(w, x, n: int, k: int, y=None, stream=None):
    """y[m, n] = x[m, k] @ dequant(w)^T for a Q8_0 matrix w (uint8 bytes) and fp32 x."""
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", (torch.float32,))
    m = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    _check(lib.qmv_q8_0(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)), "qmv_q8_0")
    return y


def qmv_q4_k(w, x, n: int, k: int, y=None, stream=None):
    """y[m, n] = x[m, k] @ dequant(w)^T for a Q4_K matrix w (uint8 bytes) and bf16 x (1 <= m <= 4)."""
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    m = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    _check(lib.qmv_q4_k(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)), "qmv_q4_k")
    return y


def qmv_q4_k_pair(w0, w1, x, n: int, k: int, y0=None, y1=None, stream=None):
    """(x @ dequant(w0)^T, x @ dequant(w1)^T) for two Q4_K matrices of one shape, in one launch."""
    torch = _torch()
    _dev(w0, "w0", (torch.uint8,))
    _dev(w1, "w1", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    if _nbytes(w0) != _nbytes(w1):
        raise ValueError("qmv_q4_k_pair: w0 and w1 must have the same size")
    m = x.shape[0] if x.dim() == 2 else 1
    if y0 is None:
        y0 = torch.empty((m, n), dtype=torch.float32, device=x.device)
    if y1 is None:
        y1 = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y0, "y0", (torch.float32,))
    _dev(y1, "y1", (torch.float32,))
    _check(lib.qmv_q4_k_pair(_ptr(w0), _ptr(w1), _nbytes(w0), _ptr(x), _ptr(y0), _ptr(y1), m, n, k, _stream(stream)),
           "qmv_q4_k_pair")
    return y0, y1


def qmv_q4_k_moe_workspace(t: int, hidden: int, ffn: int, n_experts: int, top_k: int) -> int:
    return lib.qmv_q4_k_moe_workspace(t, hidden, ffn, n_experts, top_k)


def _moe(fn, ws_fn, name, w_gate, w_up, w_down, logits, x, hidden, ffn, n_experts, top_k, y, ws, routing, stream):
    torch = _torch()
    for wname, t in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _dev(t, wname, (torch.uint8,))
    _dev(logits, "logits", (torch.float32,))
    _dev(x, "x", _bf16_types())
    tc = x.shape[0] if x.dim() == 2 else 1
    dev = x.device
    if y is None:
        y = torch.empty((tc, hidden), dtype=torch.float32, device=dev)
    _dev(y, "y", (torch.float32,))
    need = ws_fn(tc, hidden, ffn, n_experts, top_k)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(ws, "ws", (torch.uint8,))
    ids = wts = pairs = None
    if routing:
        ids = torch.empty((tc, top_k), dtype=torch.int32, device=dev)
        wts = torch.empty((tc, top_k), dtype=torch.float32, device=dev)
        pairs = torch.empty((tc * top_k, 2), dtype=torch.int32, device=dev)
    rc = fn(_ptr(w_gate), _ptr(w_up), _ptr(w_down), _nbytes(w_gate), _ptr(logits), _ptr(x),
            _ptr(y), _ptr(ids), _ptr(wts), _ptr(pairs), _ptr(ws), _nbytes(ws),
            tc, hidden, ffn, n_experts, top_k, _stream(stream))
    _check(rc, name)
    return y, ids, wts, pairs


def qmv_q4_k_moe(w_gate, w_up, w_down, logits, x, hidden: int, ffn: int, n_experts: int, top_k: int,
                 y=None, ws=None, routing: bool = True, stream=None):
    """Routed-expert MoE FFN; returns (y, topk_ids, topk_w, pairs) (the last three None if not routing)."""
    return _moe(lib.qmv_q4_k_moe, qmv_q4_k_moe_workspace, "qmv_q4_k_moe", w_gate, w_up, w_down, logits, x,
                hidden, ffn, n_experts, top_k, y, ws, routing, stream)


def qmv_q4_k_moe_prefill_workspace(t: int, hidden: int, ffn: int, n_experts: int, top_k: int) -> int:
    return lib.qmv_q4_k_moe_prefill_workspace(t, hidden, ffn, n_experts, top_k)


def qmv_q4_k_moe_prefill(w_gate, w_up, w_down, logits, x, hidden: int, ffn: int, n_experts: int, top_k: int,
                         y=None, ws=None, routing: bool = True, stream=None):
    """Routed-expert MoE FFN over a prompt's tokens; returns (y, topk_ids, topk_w) (the last two None if not routing)."""
    torch = _torch()
    for wname, t in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _dev(t, wname, (torch.uint8,))
    _dev(logits, "logits", (torch.float32,))
    _dev(x, "x", _bf16_types())
    tc = x.shape[0] if x.dim() == 2 else 1
    dev = x.device
    if y is None:
        y = torch.empty((tc, hidden), dtype=torch.float32, device=dev)
    _dev(y, "y", (torch.float32,))
    need = qmv_q4_k_moe_prefill_workspace(tc, hidden, ffn, n_experts, top_k)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(ws, "ws", (torch.uint8,))
    ids = wts = None
    if routing:
        ids = torch.empty((tc, top_k), dtype=torch.int32, device=dev)
        wts = torch.empty((tc, top_k), dtype=torch.float32, device=dev)
    _check(lib.qmv_q4_k_moe_prefill(_ptr(w_gate), _ptr(w_up), _ptr(w_down), _nbytes(w_gate), _ptr(logits), _ptr(x),
                                    _ptr(y), _ptr(ids), _ptr(wts), _ptr(ws), _nbytes(ws), tc, hidden, ffn, n_experts,
                                    top_k, _stream(stream)), "qmv_q4_k_moe_prefill")
    return y, ids, wts


def qmv_iq4_xs_moe_workspace(t: int, hidden: int, ffn: int, n_experts: int, top_k: int) -> int:
    return lib.qmv_iq4_xs_moe_workspace(t, hidden, ffn, n_experts, top_k)


def qmv_iq4_xs_moe(w_gate, w_up, w_down, logits, x, hidden: int, ffn: int, n_experts: int, top_k: int,
                   y=None, ws=None, routing: bool = True, stream=None):
    """Routed-expert MoE FFN on IQ4_XS expert banks; returns (y, topk_ids, topk_w, pairs)."""
    return _moe(lib.qmv_iq4_xs_moe, qmv_iq4_xs_moe_workspace, "qmv_iq4_xs_moe", w_gate, w_up, w_down, logits, x,
                hidden, ffn, n_experts, top_k, y, ws, routing, stream)


def qmm_q4_k_prefill_workspace(m: int, n: int, k: int) -> int:
    return lib.qmm_q4_k_prefill_workspace(m, n, k)


def qmm_q4_k_prefill(w, x, n: int, k: int, y=None, ws=None, stream=None):
    """Y[m, n] = X[m, k] @ bf16(dequant(w))^T on bf16 matrix cores, fp32 accumulation.

    ws: None allocates the workspace the shape's K split needs (if any), or a
    uint8 device tensor of at least qmm_q4_k_prefill_workspace(m, n, k) bytes to reuse.
    """
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    if ws is None:
        need = qmm_q4_k_prefill_workspace(m, n, k)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    if ws is not None:
        _dev(ws, "ws", (torch.uint8,))
    _check(lib.qmm_q4_k_prefill(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _ptr(ws), _nbytes(ws),
                                _stream(stream)), "qmm_q4_k_prefill")
    return y


def qmv_q5_k(w, x, n: int, k: int, y=None, stream=None):
    """y[m, n] = x[m, k] @ dequant(w)^T for a Q5_K matrix w (uint8 bytes) and bf16 x (1 <= m <= 4)."""
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    m = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    _check(lib.qmv_q5_k(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)), "qmv_q5_k")
    return y


def qmv_dequant_q5_k_f32(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _dev(out, "out", (torch.float32,))
    _check(lib.qmv_dequant_q5_k_f32(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)), "qmv_dequant_q5_k_f32")
    return out


def qmv_dequant_q4_k_f32(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _dev(out, "out", (torch.float32,))
    _check(lib.qmv_dequant_q4_k_f32(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)), "qmv_dequant_q4_k_f32")
    return out


def qmv_dequant_q4_k_bf16(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.int16, device=w.device)
    _dev(out, "out", _bf16_types())
    _check(lib.qmv_dequant_q4_k_bf16(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)),
           "qmv_dequant_q4_k_bf16")
    return out


def qmv_dequant_q8_0_f32(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _dev(out, "out", (torch.float32,))
    _check(lib.qmv_dequant_q8_0_f32(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)), "qmv_dequant_q8_0_f32")
    return out


def qmv_iq4_xs(w, x, n: int, k: int, y=None, stream=None):
    """y[m, n] = x[m, k] @ dequant_iq4_xs(w)^T for m = 1..4 bf16 rows (fp32 out)."""
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    m = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    _check(lib.qmv_iq4_xs(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)), "qmv_iq4_xs")
    return y


def qmv_dequant_iq4_xs_f32(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _dev(out, "out", (torch.float32,))
    _check(lib.qmv_dequant_iq4_xs_f32(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)),
           "qmv_dequant_iq4_xs_f32")
    return out


def iq4_xs_bytes(n: int, k: int) -> int:
    """Byte size of an n x k IQ4_XS matrix (136-byte blocks of 256 weights along k)."""
    return n * (k // 256) * 136


def qmv_q6_k(w, x, n: int, k: int, y=None, stream=None):
    """y[m, n] = x[m, k] @ dequant(w)^T for a Q6_K matrix w (uint8 bytes) and bf16 x (1 <= m <= 4)."""
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    m = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    _check(lib.qmv_q6_k(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)), "qmv_q6_k")
    return y


def qmv_dequant_q6_k_f32(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _dev(out, "out", (torch.float32,))
    _check(lib.qmv_dequant_q6_k_f32(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)), "qmv_dequant_q6_k_f32")
    return out


def qmv_q4_0(w, x, n: int, k: int, y=None, stream=None):
    """y[m, n] = x[m, k] @ dequant(w)^T for a Q4_0 matrix w (uint8 bytes) and bf16 x (1 <= m <= 4)."""
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    _dev(x, "x", _bf16_types())
    m = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(y, "y", (torch.float32,))
    _check(lib.qmv_q4_0(_ptr(w), _nbytes(w), _ptr(x), _ptr(y), m, n, k, _stream(stream)), "qmv_q4_0")
    return y


def qmv_dequant_q4_0_f32(w, n: int, k: int, out=None, stream=None):
    torch = _torch()
    _dev(w, "w", (torch.uint8,))
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _dev(out, "out", (torch.float32,))
    _check(lib.qmv_dequant_q4_0_f32(_ptr(w), _nbytes(w), _ptr(out), n, k, _stream(stream)), "qmv_dequant_q4_0_f32")
    return out


def qmv_stream_read(buf, grid: int = 1024, depth: int = 4, nontemporal: bool = False, sink=None, stream=None):
    """Plain streaming read of a device buffer (a measurement aid); returns the
    per-workgroup XOR words (uint32 as int32, [grid])."""
    torch = _torch()
    if sink is None:
        sink = torch.empty(grid, dtype=torch.int32, device=buf.device)
    _check(lib.qmv_stream_read(_ptr(buf), _nbytes(buf), _ptr(sink), grid, depth, int(nontemporal), _stream(stream)),
           "qmv_stream_read")
    return sink


# ---------------------------------------------------------------- e4m3 and grouped products
#
# A decode step calls these between kernels of a few microseconds, so the checks
# of a correct call are a handful of attribute reads; a refused one is explained
# afterwards.

def _blocks(k: int) -> int:
    return -(-k // 128)


_F32 = (_torch().float32,)
_I32 = (_torch().int32,)
_U8 = (_torch().uint8,)
_E4M3 = (_torch().float8_e4m3fn, _torch().uint8)
_BF16 = _bf16_types()
_FLOATS = {_torch().float32: 0, _torch().bfloat16: 1}   # QMM_F32, QMM_BF16
_FAST_SUMS = 16                                         # QMM_FAST_SUMS
_MAX_ROWS = 1 << 24                                     # QMM_MAX_ROWS


def _explain(t, name, types, shape, index):
    _dev(t, name, tuple(types))
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{index}")


def _take(t, name, types, shape, index):
    """Device address of a contiguous tensor of one of `types` and of `shape` on device `index`."""
    try:
        if t.dtype in types and t.shape == shape and t.is_contiguous() and t.get_device() == index:   # host: -1
            return t.data_ptr()
    except AttributeError:
        pass
    _explain(t, name, types, shape, index)


def _rows_in_range(rows, where):
    # refused here as the C entry does: a C int would take rows modulo 2^32
    if rows > _MAX_ROWS:
        raise QmvError(-5, where)


def _first(x, name, types, dims, where):
    """Device index and shape of the tensor that the others go by (its address is taken, and checked, later)."""
    try:
        index, shape = x.get_device(), x.shape
    except AttributeError:
        index = -1
    if index < 0 or len(shape) != dims:
        _dev(x, name, tuple(types))
        raise ValueError(f"{name} has {x.dim()} dimensions, expected {dims}")
    _rows_in_range(shape[0], where)
    return index, shape


def _current_stream(index):
    return _torch().cuda.current_stream(index).cuda_stream


# the same without the stream's object, where torch has it: a decode step makes many calls
_current_stream = getattr(_torch()._C, "_cuda_getCurrentRawStream", _current_stream)


def _run(fn, name, index, stream, *args):
    """Calls the C entry point on the tensors' own device, on its current stream unless one is given."""
    torch = _torch()
    if stream is None:
        raw = _current_stream(index)
    elif stream.device_index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc:
        raise QmvError(rc, name)


def _quant(fn, name, x, gated, xq, xs, stream):
    torch = _torch()
    index, (m, k) = _first(x, "x", _FLOATS, 2, name)
    if gated:
        if k % 2:
            raise ValueError(f"{name}: x must be [m, 2 k], got {(m, k)}")
        k //= 2
    if xq is None or xs is None:
        with torch.cuda.stream(stream):   # memory of the stream that writes it
            if xq is None:
                xq = torch.empty((m, k), dtype=torch.float8_e4m3fn, device=x.device)
            if xs is None:
                xs = torch.empty((_blocks(k), m), dtype=torch.float32, device=x.device)
    xp = _take(x, "x", _FLOATS, x.shape, index)
    _run(fn, name, index, stream, xp, _FLOATS[x.dtype], _take(xq, "xq", _E4M3, (m, k), index),
         _take(xs, "xs", _F32, (_blocks(k), m), index), m, k)
    return xq, xs


def qmm_fp8_quant(x, xq=None, xs=None, stream=None):
    """Rows x [m, k] (fp32 or bf16) as e4m3 codes xq [m, k] with fp32 scales xs [ceil(k/128), m]; returns (xq, xs)."""
    return _quant(lib.qmm_fp8_quant, "qmm_fp8_quant", x, False, xq, xs, stream)


def qmm_fp8_quant_silu_mul(x, xq=None, xs=None, stream=None):
    """As qmm_fp8_quant on silu(gate) * up [m, k], where x [m, 2 k] holds a row's gate values and then its up values."""
    return _quant(lib.qmm_fp8_quant_silu_mul, "qmm_fp8_quant_silu_mul", x, True, xq, xs, stream)


def _type_code(dtype, fast_sums):
    code = _FLOATS[dtype]
    if not fast_sums:
        return code
    if code != 1:
        raise ValueError("fast_sums goes with a bfloat16 result")
    return code | _FAST_SUMS


def qmm_fp8_workspace(m: int, n: int, k: int, out_dtype=None, fast_sums: bool = False) -> int:
    """Bytes of ws a qmm_fp8 call of this shape needs (y fp32 unless out_dtype says bf16)."""
    if out_dtype is not None and out_dtype not in _FLOATS:
        raise TypeError(f"out_dtype is {out_dtype}, expected float32 or bfloat16")
    code = _type_code(out_dtype or _F32[0], fast_sums)
    return 0 if max(m, n, k) > _MAX_ROWS else lib.qmm_fp8_workspace(m, n, k, code)   # out of range: 0, as in C


def _y_type(y, out_dtype, fast_sums=False):
    if y.dtype not in _FLOATS:
        raise TypeError(f"y has dtype {y.dtype}, expected float32 or bfloat16")
    if out_dtype is not None and y.dtype != out_dtype:
        raise TypeError(f"y has dtype {y.dtype}, out_dtype is {out_dtype}")
    return _type_code(y.dtype, fast_sums)


def qmm_fp8(w, w_scale, x, x_scale, n: int, k: int, y=None, out_dtype=None, ws=None, stream=None,
            fast_sums: bool = False):
    """y[m, n] = x @ w^T for e4m3 w [n, k] and x [m, k] with scales w_scale [ceil(n/128), ceil(k/128)] and
    x_scale [ceil(k/128), m] (as qmm_fp8_quant gives them); y is fp32 unless y or out_dtype says bf16. Without rows
    (m = 0) nothing is launched.

    ws: None allocates the workspace the shape needs (if any), or a uint8 device
    tensor of at least qmm_fp8_workspace(m, n, k, y.dtype, fast_sums) bytes to reuse.
    fast_sums (bf16 y): the e4m3 matrix instruction, twice the rate for many rows,
    which cuts partial sums (QMM_FAST_SUMS in qmm_fp8.h).
    """
    torch = _torch()
    index, (m, _) = _first(x, "x", _E4M3, 2, "qmm_fp8")
    if y is None:
        with torch.cuda.stream(stream):   # memory of the stream that writes it
            y = torch.empty((m, n), dtype=out_dtype or torch.float32, device=x.device)
    y_type = _y_type(y, out_dtype, fast_sums)
    if ws is None:
        need = lib.qmm_fp8_workspace(m, n, k, y_type)
        if need:
            with torch.cuda.stream(stream):
                ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    args = (_take(w, "w", _E4M3, (n, k), index), n * k, _take(w_scale, "w_scale", _F32, (_blocks(n), _blocks(k)), index),
            _take(x, "x", _E4M3, (m, k), index), _take(x_scale, "x_scale", _F32, (_blocks(k), m), index),
            _take(y, "y", _FLOATS, (m, n), index), y_type, m, n, k,
            None if ws is None else _take(ws, "ws", _U8, ws.shape, index), 0 if ws is None else ws.numel())
    if m:   # no rows: y is empty, as from the grouped products
        _run(lib.qmm_fp8, "qmm_fp8", index, stream, *args)
    return y


def _grouped(fn, name, types, w, w_scale, x, x_scale, offsets, n, k, row_index, y, out_dtype, stream, fast_sums=False):
    torch = _torch()
    index, (x_rows, _) = _first(x, "x", types, 2, name)
    _, (e, _, _) = _first(w, "w", types, 3, name)
    rows = x_rows
    found = None
    if row_index is not None:
        rows = row_index.numel()
        _rows_in_range(rows, name)
        found = _take(row_index, "row_index", _I32, (rows,), index)
    if y is None:
        # rows that belong to no expert are not written: zeros there rather than what the memory held
        with torch.cuda.stream(stream):
            y = torch.zeros((rows, n), dtype=out_dtype or torch.float32, device=x.device)
    y_type = _y_type(y, out_dtype, fast_sums)
    wp, xp = _take(w, "w", types, (e, n, k), index), _take(x, "x", types, (x_rows, k), index)
    op, yp = _take(offsets, "offsets", _I32, (e + 1,), index), _take(y, "y", _FLOATS, (rows, n), index)
    if types is _E4M3:
        wsp = _take(w_scale, "w_scale", _F32, (e, _blocks(n), _blocks(k)), index)
        xsp = _take(x_scale, "x_scale", _F32, (_blocks(k), x_rows), index)
        if rows:
            _run(fn, name, index, stream, wp, e * n * k, wsp, xp, xsp, op, found, yp, y_type, rows, x_rows, n, k, e)
    elif rows:
        _run(fn, name, index, stream, wp, 2 * e * n * k, xp, op, found, yp, y_type, rows, x_rows, n, k, e)
    return y


def qmm_fp8_grouped(w, w_scale, x, x_scale, offsets, n: int, k: int, row_index=None, y=None, out_dtype=None,
                    stream=None, fast_sums: bool = False):
    """Rows offsets[e] .. offsets[e+1] - 1 of y [rows, n] = x rows @ w[e]^T for e4m3 w [experts, n, k] and x, scales as
    in qmm_fp8 with one more leading dimension for w_scale; offsets int32 [experts + 1] on the device.

    row_index (int32, one per row of y): the row of x to take, outside x for a row of zeros; None: the same row.
    Rows of y that belong to no expert are left as they were (zeros when y is None). fast_sums as in qmm_fp8.
    """
    return _grouped(lib.qmm_fp8_grouped, "qmm_fp8_grouped", _E4M3, w, w_scale, x, x_scale, offsets, n, k, row_index, y,
                    out_dtype, stream, fast_sums)


def qmm_bf16_grouped(w, x, offsets, n: int, k: int, row_index=None, y=None, out_dtype=None, stream=None):
    """As qmm_fp8_grouped on bf16 w [experts, n, k] and x [x_rows, k]."""
    return _grouped(lib.qmm_bf16_grouped, "qmm_bf16_grouped", _BF16, w, None, x, None, offsets, n, k, row_index, y,
                    out_dtype, stream)

"""ctypes binding of libqmoe.so: the C ABI of include/qmoe.h under the same names.

Argument marshalling only. Tensor arguments are torch CUDA tensors (their data
pointers are passed); ``stream`` defaults to torch's current stream. A call
that returns a non-OK status raises :class:`QmoeError`. There is no fallback:
if the library is missing, importing this module's functions raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmoe.so")

OK = 0
Q2, Q4 = 2, 4
F32, BF16, I8 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
GATE_UP, DOWN = 0, 1
STACK_TIMING = 1
STACK_LAYERWISE = 2
PATH_LAYERWISE, PATH_FUSED = 0, 1

STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "GEOMETRY", 3: "UNSUPPORTED", 4: "WORKSPACE",
                5: "CUDA", 6: "TIMEOUT", 7: "DEVICE_STATUS", 8: "RANGE"}


class QmoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}")


class qmoe_experts(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int), ("fmt", ctypes.c_int),
                ("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("gate_up_bytes", ctypes.c_size_t), ("down_bytes", ctypes.c_size_t)]


class qmoe_stack_desc(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("T", ctypes.c_int), ("k", ctypes.c_int), ("eps", ctypes.c_float),
                ("Wr", ctypes.POINTER(ctypes.c_void_p)), ("bias", ctypes.POINTER(ctypes.c_void_p)),
                ("layers", ctypes.POINTER(qmoe_experts)), ("flags", ctypes.c_int)]


_VP, _I, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "qmoe_packed_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "qmoe_pack": (_I, [_I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "qmoe_route_workspace_bytes": (_SZ, [_I, _I]),
    "qmoe_route": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "qmoe_route_fixed": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP, _VP]),
    "qmoe_residual_route": (_I, [_VP, _VP, _F, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "qmoe_rmsnorm_residual": (_I, [_VP, _VP, _F, _VP, _I, _I, _VP]),
    "qmoe_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "qmoe_ffn_decode": (_I, [ctypes.POINTER(qmoe_experts), _VP, _I, _VP, _VP, _I, _VP, _VP, _SZ, _VP, _VP]),
    "qmoe_bucket_workspace_bytes": (_SZ, [_I, _I, _I]),
    "qmoe_bucket": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "qmoe_prefill_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "qmoe_ffn_prefill": (_I, [ctypes.POINTER(qmoe_experts), _VP, _I, _VP, _VP, _I, _VP, _VP, _SZ, _VP, _VP]),
    "qmoe_ffn_prefill_timed": (_I, [ctypes.POINTER(qmoe_experts), _VP, _I, _VP, _VP, _I, _VP, _VP, _SZ, _VP, _VP,
                                    ctypes.POINTER(_VP), _I]),
    "qmoe_stack_workspace_bytes": (_SZ, [ctypes.POINTER(qmoe_stack_desc)]),
    "qmoe_stack_create": (_I, [ctypes.POINTER(qmoe_stack_desc), _VP, _SZ, _VP, ctypes.POINTER(_VP)]),
    "qmoe_stack_destroy": (_I, [_VP]),
    "qmoe_stack_buffers": (_I, [_VP, ctypes.POINTER(_VP), ctypes.POINTER(_VP), ctypes.POINTER(_VP),
                                ctypes.POINTER(_VP), ctypes.POINTER(_VP)]),
    "qmoe_stack_barrier_word": (_VP, [_VP]),
    "qmoe_stack_trace": (_I, [_VP, _VP, _SZ, _VP, _VP]),
    "qmoe_stack_kernels_per_replay": (_I, [_VP]),
    "qmoe_stack_path": (_I, [_VP]),
    "qmoe_stack_decode": (_I, [_VP, _VP]),
    "qmoe_stack_layer_times": (_I, [_VP, _VP, _VP]),
    "qmoe_stack_decode_host": (_I, [_VP, _VP, _VP, _VP]),
    "qmoe_ngram_gather": (_I, [_VP, _I, ctypes.c_uint64, _VP, _VP, ctypes.c_int64, _I, _VP, _VP, _VP]),
    "qmoe_rmsnorm_residual_q8": (_I, [_VP, _VP, _I, _VP, _F, _I, _I, _I, _VP, _VP, _VP, _VP, _VP]),
    "qmoe_quantise_rows": (_I, [_VP, _I, _I, _I, _I, _VP, _VP, _VP]),
    "qmoe_linear": (_I, [_VP, _I, _VP, _I, _I, _I, _VP, _VP, _VP, _I, _VP, _VP, _I, ctypes.c_int64, ctypes.c_int64,
                         ctypes.c_int64, ctypes.c_int64, _VP, _VP]),
    "qmoe_sample": (_I, [_VP, _I, _I, _I, ctypes.c_int64, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "qmoe_read_status": (_I, [_VP]),
    "qmoe_status_string": (ctypes.c_char_p, [_I]),
    "qmoe_launch_count": (ctypes.c_uint64, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libqmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python quantised_expert_decode_b200/build.py` (there is no CPU fallback)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


# ------------------------------------------------------------------ helpers --
def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _s(stream) -> int | None:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # (a Stream object takes 3 us to make)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name: str, code: int) -> None:
    if code != OK:
        raise QmoeError(name, code)


# ---------------------------------------------------------------- the ABI --
def qmoe_packed_bytes(fmt: int, kind: int, E: int, H: int, I: int) -> int:
    return lib().qmoe_packed_bytes(fmt, kind, E, H, I)


def qmoe_pack(fmt, kind, E, H, I, codes_a, scales_a, codes_up, scales_up, dst, stream=None) -> None:
    _check("qmoe_pack", lib().qmoe_pack(fmt, kind, E, H, I, _p(codes_a), _p(scales_a), _p(codes_up),
                                        _p(scales_up), _p(dst), dst.numel() * dst.element_size(), _s(stream)))


def qmoe_route_workspace_bytes(T: int, E: int) -> int:
    return lib().qmoe_route_workspace_bytes(T, E)


def qmoe_route(Wr, bias, x, x_dtype, T, H, E, k, idx, gate, workspace, dev_status, stream=None) -> None:
    _check("qmoe_route", lib().qmoe_route(_p(Wr), _p(bias), _p(x), x_dtype, T, H, E, k, _p(idx), _p(gate),
                                          _p(workspace), workspace.numel() * workspace.element_size(),
                                          _p(dev_status), _s(stream)))


def qmoe_route_fixed(Wr, bias, x, T, H, E, k, idx, gate, dev_status, stream=None) -> None:
    """The decode router with its scratch in a fixed device array (no workspace)."""
    _check("qmoe_route_fixed", lib().qmoe_route_fixed(_p(Wr), _p(bias), _p(x), T, H, E, k, _p(idx), _p(gate),
                                                      _p(dev_status), _s(stream)))


def qmoe_residual_route(x_in, y, eps, x_out, Wr, bias, T, H, E, k, idx, gate, workspace, dev_status,
                        stream=None) -> None:
    _check("qmoe_residual_route", lib().qmoe_residual_route(
        _p(x_in), _p(y), float(eps), _p(x_out), _p(Wr), _p(bias), T, H, E, k, _p(idx), _p(gate),
        _p(workspace), workspace.numel() * workspace.element_size(), _p(dev_status), _s(stream)))


def qmoe_rmsnorm_residual(x_in, y, eps, x_out, T, H, stream=None) -> None:
    _check("qmoe_rmsnorm_residual",
           lib().qmoe_rmsnorm_residual(_p(x_in), _p(y), float(eps), _p(x_out), T, H, _s(stream)))


def qmoe_decode_workspace_bytes(T: int, k: int, H: int, I: int) -> int:
    return lib().qmoe_decode_workspace_bytes(T, k, H, I)


def qmoe_ffn_decode(experts: qmoe_experts, x, T, idx, gate, k, y, workspace, dev_status, stream=None) -> None:
    _check("qmoe_ffn_decode", lib().qmoe_ffn_decode(
        ctypes.byref(experts), _p(x), T, _p(idx), _p(gate), k, _p(y), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(dev_status), _s(stream)))


def qmoe_bucket_workspace_bytes(T: int, k: int, E: int) -> int:
    return lib().qmoe_bucket_workspace_bytes(T, k, E)


def qmoe_bucket(idx, T, k, E, offsets, perm, active, nactive, workspace, dev_status, stream=None) -> None:
    _check("qmoe_bucket", lib().qmoe_bucket(_p(idx), T, k, E, _p(offsets), _p(perm), _p(active), _p(nactive),
                                            _p(workspace), workspace.numel() * workspace.element_size(),
                                            _p(dev_status), _s(stream)))


def qmoe_prefill_workspace_bytes(T: int, k: int, E: int, H: int, I: int) -> int:
    return lib().qmoe_prefill_workspace_bytes(T, k, E, H, I)


def qmoe_ffn_prefill(experts: qmoe_experts, x, T, idx, gate, k, y, workspace, dev_status, stream=None) -> None:
    _check("qmoe_ffn_prefill", lib().qmoe_ffn_prefill(
        ctypes.byref(experts), _p(x), T, _p(idx), _p(gate), k, _p(y), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(dev_status), _s(stream)))


def qmoe_ngram_gather(ngrams, T, seed, codes, scales, R, D, out, rows=None, stream=None) -> None:
    """``ngrams`` int32 [T, 3]; ``codes`` uint8 [R, D/2]; ``scales`` int16/uint16 [R, D/32, 2];
    ``out`` fp32 [T, 16, D]; ``rows`` int32 [T, 16] or None."""
    _check("qmoe_ngram_gather", lib().qmoe_ngram_gather(_p(ngrams), T, seed & ((1 << 64) - 1), _p(codes), _p(scales),
                                                        R, D, _p(out), _p(rows), _s(stream)))


_TORCH_TYPES: dict = {}
_DTYPES = {F32: "float32", BF16: "bfloat16", I8: "int8"}


def _misfit(t, rows, cols, ld) -> str | None:
    """Why a tensor's own shape and strides are not ``rows`` rows of ``cols`` dense elements, ``ld`` elements from
    one to the next (0: a vector of ``cols``). What lies in its storage beside it does not count."""
    def run(dims):   # (size, stride) of dimensions that are one run, outermost first; sizes of 1 have no stride
        dims = [d for d in dims if d[0] > 1]
        if any(a[1] != b[0] * b[1] for a, b in zip(dims, dims[1:])):
            return None
        size = 1
        for d in dims:
            size *= d[0]
        return size, dims[-1][1] if dims else None
    shape, strides = t.shape, t.stride()
    if ld and len(shape) == 2 and strides == (ld, 1) and shape[0] >= rows and shape[1] >= cols:   # (most that get here)
        return None
    dims = list(zip(shape, strides))
    lead, width = dims[:-1], dims[-1] if dims else (1, 1)
    if ld and any(n > 1 for n, _ in lead):
        at = run(lead)
        if width[1] != 1 and width[0] > 1:
            return "whose rows are not contiguous"
        if at is None or at[1] != ld:
            return "whose row stride is not the one given"
        return None if at[0] >= rows and width[0] >= cols else "smaller than the call's sizes"
    # one run: a vector, a single row, or a flat buffer of rows
    at = run(dims)
    if at is None or at[1] not in (None, 1):
        return "whose rows are not contiguous"
    return None if t.numel() >= (rows - 1) * (ld or cols) + cols else "smaller than the call's sizes"


def _fits(fn: str, *wants) -> list:
    """(tensor or None, type, rows, columns, row stride) each: on the current device, of the type, rows dense and
    at one stride, and large enough by its own shape for what the call reads or writes. A plain address (int) is
    the caller's word. Returns their addresses (one pass over the tensors: a short kernel takes less time than
    asking them twice)."""
    import torch
    if not _TORCH_TYPES:
        _TORCH_TYPES.update((name, getattr(torch, name)) for name in ("float32", "bfloat16", "int8", "int32"))
    dev, tensor, types, out = torch.cuda.current_device(), torch.Tensor, _TORCH_TYPES, []
    for t, dtype, rows, cols, ld in wants:
        if t is None:
            out.append(None)
            continue
        # a packed tensor of its own rows, as most are, with few questions to it; the others one by one
        if (type(t) is tensor and t.dtype is types[dtype] and t.get_device() == dev and t.is_contiguous()
                and t.numel() >= rows * cols and (not ld or (ld == cols and (t.dim() < 2 or t.size(-1) == ld)))):
            out.append(t.data_ptr())
            continue
        if isinstance(t, int):
            out.append(t)
            continue
        if t.dtype != types[dtype]:
            raise QmoeError(fn + f" (a {t.dtype} tensor in the place of a {dtype} one)", 1)
        if t.get_device() != dev:
            raise QmoeError(fn + " (a tensor on another device than the current one)", 1)
        wrong = _misfit(t, rows, cols, ld)
        if wrong:
            raise QmoeError(f"{fn} (a tensor {wrong})", 1)
        out.append(t.data_ptr())
    return out


def qmoe_rmsnorm_residual_q8(x_in, y, dtype, gain, eps, T, H, group, z_out, norm_out, codes, scales, stream=None) -> None:
    """``x_in``, ``y``, ``z_out`` fp32 or bf16 [T, H] (``dtype``); ``gain`` fp32 [H]; ``norm_out`` bf16 [T, H];
    ``codes`` int8 [T, H]; ``scales`` fp32 [T] (``group`` 0) or [T, H / group]. Any of y, gain, z_out, norm_out
    and (codes, scales) may be None."""
    dt = _DTYPES.get(dtype, "float32")
    x, y, g, z, n, c, s = _fits(
        "qmoe_rmsnorm_residual_q8", (x_in, dt, T, H, H), (y, dt, T, H, H), (gain, "float32", 1, H, 0),
        (z_out, dt, T, H, H), (norm_out, "bfloat16", T, H, H), (codes, "int8", T, H, H),
        (scales, "float32", 1, T * (H // group if group > 0 else 1), 0))
    _check("qmoe_rmsnorm_residual_q8", lib().qmoe_rmsnorm_residual_q8(x, y, dtype, g, eps, T, H, group, z, n, c, s,
                                                                      _s(stream)))


def qmoe_quantise_rows(x, dtype, T, H, group, codes, scales, stream=None) -> None:
    """``x`` fp32 or bf16 [T, H] -> ``codes`` int8 [T, H] and ``scales`` fp32 [T] or [T, H / group]."""
    x, c, s = _fits("qmoe_quantise_rows", (x, _DTYPES.get(dtype, "float32"), T, H, H), (codes, "int8", T, H, H),
                    (scales, "float32", 1, T * (H // group if group > 0 else 1), 0))
    _check("qmoe_quantise_rows", lib().qmoe_quantise_rows(x, dtype, T, H, group, c, s, _s(stream)))


def qmoe_linear(a, in_dtype, w, M, N, K, a_scale, w_scale, bias, act, residual, out, out_dtype, dev_status, lda=0,
                ldw=0, ldr=0, ldo=0, stream=None) -> None:
    """out = act(a w^T scaled + bias) + residual. ``a`` [M, K] and ``w`` [N, K] bf16 (``in_dtype`` BF16) or int8
    with ``a_scale`` fp32 [M] and ``w_scale`` fp32 [N] (I8); ``bias`` fp32 [N] or None; ``residual`` and ``out``
    [M, N] of ``out_dtype``; strides in elements, 0 = packed."""
    dt, odt = _DTYPES.get(in_dtype, "bfloat16"), _DTYPES.get(out_dtype, "float32")
    a, w, sa, sw, b, r, o, st = _fits(
        "qmoe_linear", (a, dt, M, K, lda or K), (w, dt, N, K, ldw or K), (a_scale, "float32", 1, M, 0),
        (w_scale, "float32", 1, N, 0), (bias, "float32", 1, N, 0), (residual, odt, M, N, ldr or N),
        (out, odt, M, N, ldo or N), (dev_status, "int32", 1, 1, 0))
    _check("qmoe_linear", lib().qmoe_linear(a, in_dtype, w, M, N, K, sa, sw, b, act, r, o, out_dtype, lda, ldw, ldr, ldo,
                                            st, _s(stream)))


def qmoe_sample(logits, dtype, T, V, temperature, top_k, top_p, min_p, u, token, prob, dev_status, ld=0,
                stream=None) -> None:
    """``logits`` fp32 or bf16 [T, V] (row stride ``ld`` elements, 0 = V); ``temperature``, ``top_p``, ``min_p``
    fp32 [T] or None, ``top_k`` int32 [T] or None, ``u`` fp32 [T]; ``token`` int32 [T], ``prob`` fp32 [T] or None."""
    x, t, k, p, m, u, tok, pr, st = _fits(
        "qmoe_sample", (logits, _DTYPES.get(dtype, "float32"), T, V, ld or V), (temperature, "float32", 1, T, 0),
        (top_k, "int32", 1, T, 0), (top_p, "float32", 1, T, 0), (min_p, "float32", 1, T, 0), (u, "float32", 1, T, 0),
        (token, "int32", 1, T, 0), (prob, "float32", 1, T, 0), (dev_status, "int32", 1, 1, 0))
    _check("qmoe_sample", lib().qmoe_sample(x, dtype, T, V, ld, t, k, p, m, u, tok, pr, st, _s(stream)))


PREFILL_ATOMIC_COMBINE = 1


def qmoe_ffn_prefill_timed(experts: qmoe_experts, x, T, idx, gate, k, y, workspace, dev_status, events,
                           stream=None, flags=0) -> None:
    """``events``: three torch.cuda.Event(enable_timing=True) objects."""
    for e in events:
        if not e.cuda_event:   # torch creates the CUDA event at its first record
            e.record()
    arr = (_VP * 3)(*[e.cuda_event for e in events])
    _check("qmoe_ffn_prefill_timed", lib().qmoe_ffn_prefill_timed(
        ctypes.byref(experts), _p(x), T, _p(idx), _p(gate), k, _p(y), _p(workspace),
        workspace.numel() * workspace.element_size(), _p(dev_status), _s(stream), arr, flags))


def qmoe_stack_workspace_bytes(desc: qmoe_stack_desc) -> int:
    return lib().qmoe_stack_workspace_bytes(ctypes.byref(desc))


def qmoe_stack_create(desc: qmoe_stack_desc, workspace, stream=None) -> int:
    out = ctypes.c_void_p()
    _check("qmoe_stack_create", lib().qmoe_stack_create(
        ctypes.byref(desc), _p(workspace), workspace.numel() * workspace.element_size(), _s(stream),
        ctypes.byref(out)))
    return out.value


def qmoe_stack_destroy(stack: int) -> None:
    _check("qmoe_stack_destroy", lib().qmoe_stack_destroy(stack))


def qmoe_stack_buffers(stack: int) -> dict:
    ptrs = [ctypes.c_void_p() for _ in range(5)]
    _check("qmoe_stack_buffers", lib().qmoe_stack_buffers(stack, *[ctypes.byref(p) for p in ptrs]))
    return dict(zip(("x_in", "x_out", "idx", "gate", "dev_status"), (p.value for p in ptrs)))


def qmoe_stack_kernels_per_replay(stack: int) -> int:
    return lib().qmoe_stack_kernels_per_replay(stack)


def qmoe_stack_trace(stack: int, L: int, max_ctas: int = 1024, points: int = 16):
    """Phase stamps (SM cycles) of the last replay: numpy int64 [L, ctas, points]."""
    import numpy as np
    buf = np.zeros(L * max_ctas * points, dtype=np.int64)
    g, p = ctypes.c_int(0), ctypes.c_int(0)
    _check("qmoe_stack_trace", lib().qmoe_stack_trace(stack, buf.ctypes.data, buf.size, ctypes.byref(g),
                                                      ctypes.byref(p)))
    return buf[:L * g.value * p.value].reshape(L, g.value, p.value)


def qmoe_stack_barrier_word(stack: int) -> int | None:
    return lib().qmoe_stack_barrier_word(stack)


def qmoe_stack_path(stack: int) -> int:
    return lib().qmoe_stack_path(stack)


def qmoe_stack_layer_times(stack: int, L: int):
    """(route_ms, ffn_ms) lists of the last completed replay of a timing stack."""
    r = (ctypes.c_float * L)()
    f = (ctypes.c_float * L)()
    _check("qmoe_stack_layer_times", lib().qmoe_stack_layer_times(stack, r, f))
    return list(r), list(f)


def qmoe_stack_decode(stack: int, stream=None) -> None:
    _check("qmoe_stack_decode", lib().qmoe_stack_decode(stack, _s(stream)))


def qmoe_stack_decode_host(stack: int, x_host, x_out_host, stream=None) -> None:
    _check("qmoe_stack_decode_host", lib().qmoe_stack_decode_host(stack, _p(x_host), _p(x_out_host), _s(stream)))


def qmoe_read_status(dev_status) -> int:
    return lib().qmoe_read_status(_p(dev_status))


def qmoe_status_string(code: int) -> str:
    return lib().qmoe_status_string(code).decode()


def qmoe_launch_count() -> int:
    return lib().qmoe_launch_count()

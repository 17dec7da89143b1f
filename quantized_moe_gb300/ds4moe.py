"""ctypes binding of libds4moe.so (argument marshalling only; every step runs in the library).

The names mirror the C ABI in include/ds4moe.h. Pointers are plain integers (for example
``tensor.data_ptr()``) or numpy arrays, which are passed by address and must stay alive for
the duration of the call. Streams are raw cudaStream_t values (``torch.cuda.current_stream()
.cuda_stream``); 0 is the legacy default stream.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libds4moe.so")

DS4MOE_OK = 0
DS4MOE_ERR_INVALID_ARG = -1
DS4MOE_ERR_UNSUPPORTED_FORMAT = -2
DS4MOE_ERR_DEVICE_MISMATCH = -3
DS4MOE_ERR_CAPACITY = -4
DS4MOE_ERR_OOM = -5
DS4MOE_ERR_CUDA = -6

DS4MOE_FMT_Q8_0 = 0
DS4MOE_FMT_Q2_K = 1
FORMATS = {"q8_0": DS4MOE_FMT_Q8_0, "q2_k": DS4MOE_FMT_Q2_K}

EXPORTED = ("ds4moe_create", "ds4moe_create_subset", "ds4moe_forward", "ds4moe_forward_ex", "ds4moe_forward_host",
            "ds4moe_get_route", "ds4moe_get_stats", "ds4moe_device_bytes",
            "ds4moe_launches_per_forward", "ds4moe_set_profiling", "ds4moe_get_phase_times", "ds4moe_route_noalloc",
            "ds4moe_set_test_stall",
            "ds4moe_grouped_mm", "ds4moe_grouped_mm_dx", "ds4moe_grouped_mm_dw",
            "ds4moe_linear", "ds4moe_linear_grad", "ds4moe_linear_grad_workspace",
            "ds4moe_cross_entropy", "ds4moe_cross_entropy_grad", "ds4moe_cross_entropy_workspace",
            "ds4moe_ops_status",
            "ds4moe_destroy", "ds4moe_last_error")
DS4MOE_NOALLOC_MAX_LOGITS = 262144

DS4MOE_BF16 = 0
DS4MOE_FP16 = 1
DS4MOE_FP32 = 2
DTYPES = {"bf16": DS4MOE_BF16, "fp16": DS4MOE_FP16, "fp32": DS4MOE_FP32}
DS4MOE_ACT_NONE = 0
DS4MOE_ACT_RELU = 1
DS4MOE_ACT_SILU = 2
DS4MOE_ACT_GELU = 3
ACTS = {"none": DS4MOE_ACT_NONE, "relu": DS4MOE_ACT_RELU, "silu": DS4MOE_ACT_SILU, "gelu": DS4MOE_ACT_GELU}


class ds4moe_shapes(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("f_routed", ctypes.c_int32), ("f_shared", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("fmt_gate_up", ctypes.c_int32), ("fmt_down", ctypes.c_int32), ("fmt_shared", ctypes.c_int32),
                ("has_bias", ctypes.c_int32), ("hash_vocab", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("device", ctypes.c_int32), ("reserved", ctypes.c_int32), ("workspace_limit", ctypes.c_int64)]


class ds4moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("router_w", "router_b", "gate", "up", "down", "shared_gate",
                                               "shared_up", "shared_down", "hash_table")]


class ds4moe_stats(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("distinct_experts", ctypes.c_int32),
                ("error_flags", ctypes.c_int32), ("reserved", ctypes.c_int32), ("counts", ctypes.c_int32 * 256)]


class Ds4MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"ds4moe error {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Loads the in-tree library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with quantized_moe_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.ds4moe_create.argtypes = [ctypes.POINTER(ds4moe_weights), ctypes.POINTER(ds4moe_shapes), ctypes.POINTER(vp)]
        L.ds4moe_create.restype = ctypes.c_int
        L.ds4moe_create_subset.argtypes = [ctypes.POINTER(ds4moe_weights), ctypes.POINTER(ds4moe_shapes), vp, i32,
                                           i32, ctypes.POINTER(vp)]
        L.ds4moe_create_subset.restype = ctypes.c_int
        L.ds4moe_forward.argtypes = [vp, vp, i32, vp, vp]
        L.ds4moe_forward.restype = ctypes.c_int
        L.ds4moe_forward_ex.argtypes = [vp, vp, i32, vp, i32, vp, vp]
        L.ds4moe_forward_ex.restype = ctypes.c_int
        L.ds4moe_forward_host.argtypes = [vp, vp, i32, vp, i32, vp, vp]
        L.ds4moe_forward_host.restype = ctypes.c_int
        L.ds4moe_get_route.argtypes = [vp, vp, vp, i32]
        L.ds4moe_get_route.restype = ctypes.c_int
        L.ds4moe_get_stats.argtypes = [vp, ctypes.POINTER(ds4moe_stats)]
        L.ds4moe_get_stats.restype = ctypes.c_int
        L.ds4moe_device_bytes.argtypes = [vp]
        L.ds4moe_device_bytes.restype = i64
        L.ds4moe_launches_per_forward.argtypes = [vp, i32]
        L.ds4moe_launches_per_forward.restype = i32
        L.ds4moe_set_profiling.argtypes = [vp, i32]
        L.ds4moe_set_profiling.restype = ctypes.c_int
        L.ds4moe_get_phase_times.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_char_p), i32,
                                             ctypes.POINTER(i32)]
        L.ds4moe_get_phase_times.restype = ctypes.c_int
        L.ds4moe_route_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
        L.ds4moe_route_noalloc.restype = ctypes.c_int
        L.ds4moe_set_test_stall.argtypes = [vp, i32]
        L.ds4moe_set_test_stall.restype = ctypes.c_int
        L.ds4moe_grouped_mm.argtypes = [vp] * 4 + [i32] * 5 + [i64] * 4 + [vp]
        L.ds4moe_grouped_mm_dx.argtypes = [vp] * 4 + [i32] * 5 + [i64] * 4 + [vp]
        L.ds4moe_grouped_mm_dw.argtypes = [vp] * 4 + [i32] * 7 + [i64] * 4 + [vp]
        L.ds4moe_linear.argtypes = [vp] * 6 + [i32] * 5 + [i64] * 5 + [vp]
        L.ds4moe_linear_grad.argtypes = [vp] * 7 + [i32] * 5 + [i64] * 6 + [vp, i64, vp]
        L.ds4moe_cross_entropy.argtypes = [vp] * 5 + [i32] * 5 + [i64] * 2 + [vp, i64, vp]
        L.ds4moe_cross_entropy_grad.argtypes = [vp] * 7 + [i32] * 5 + [i64] * 4 + [vp, i64, vp]
        L.ds4moe_ops_status.argtypes = [ctypes.POINTER(i32)]
        for name in ("grouped_mm", "grouped_mm_dx", "grouped_mm_dw", "linear", "linear_grad", "cross_entropy",
                     "cross_entropy_grad", "ops_status"):
            getattr(L, "ds4moe_" + name).restype = ctypes.c_int
        L.ds4moe_linear_grad_workspace.argtypes = [i32, i32, i32]
        L.ds4moe_linear_grad_workspace.restype = i64
        L.ds4moe_cross_entropy_workspace.argtypes = [i32, i32, i32]
        L.ds4moe_cross_entropy_workspace.restype = i64
        L.ds4moe_destroy.argtypes = [vp]
        L.ds4moe_destroy.restype = None
        L.ds4moe_last_error.argtypes = []
        L.ds4moe_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def ds4moe_last_error() -> str:
    return lib().ds4moe_last_error().decode()


def _check(rc: int) -> None:
    if rc != DS4MOE_OK:
        raise Ds4MoeError(rc, ds4moe_last_error())


def _ptr(a) -> Optional[int]:
    if a is None or type(a) is int:
        return a
    address = getattr(a, "data_ptr", None)
    if address is not None:
        return address()
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("arrays must be C-contiguous")
        return a.ctypes.data
    raise TypeError(f"cannot take the address of {type(a)}")


def make_shapes(d, f_routed, f_shared, n_experts, top_k, n_shared, fmt_gate_up, fmt_down, fmt_shared,
                has_bias, hash_vocab, max_tokens, device=0, workspace_limit=0) -> ds4moe_shapes:
    fm = lambda f: FORMATS[f] if isinstance(f, str) else int(f)
    return ds4moe_shapes(d, f_routed, f_shared, n_experts, top_k, n_shared, fm(fmt_gate_up), fm(fmt_down),
                         fm(fmt_shared), int(bool(has_bias)), hash_vocab, max_tokens, device, 0, workspace_limit)


def make_weights(router_w, router_b, gate, up, down, shared_gate=None, shared_up=None, shared_down=None,
                 hash_table=None) -> ds4moe_weights:
    return ds4moe_weights(*(_ptr(a) for a in (router_w, router_b, gate, up, down, shared_gate, shared_up,
                                               shared_down, hash_table)))


def ds4moe_create(weights: ds4moe_weights, shapes: ds4moe_shapes) -> int:
    h = ctypes.c_void_p()
    _check(lib().ds4moe_create(ctypes.byref(weights), ctypes.byref(shapes), ctypes.byref(h)))
    return h.value


def ds4moe_create_subset(weights: ds4moe_weights, shapes: ds4moe_shapes, owned, include_shared: bool) -> int:
    """A handle holding only the routed experts in `owned` (see the header); returns its address."""
    ids = np.ascontiguousarray(np.asarray(owned, dtype=np.int32).reshape(-1))
    buf = ids if ids.size else np.zeros(1, np.int32)  # a valid address even for an empty list
    h = ctypes.c_void_p()
    _check(lib().ds4moe_create_subset(ctypes.byref(weights), ctypes.byref(shapes), buf.ctypes.data, int(ids.size),
                                      int(bool(include_shared)), ctypes.byref(h)))
    return h.value


def ds4moe_forward(h: int, x, n_tokens: int, out, stream: int = 0) -> None:
    _check(lib().ds4moe_forward(h, _ptr(x), n_tokens, _ptr(out), stream))


def ds4moe_forward_ex(h: int, x, n_tokens: int, token_ids, n_hash: int, out, stream: int = 0) -> None:
    _check(lib().ds4moe_forward_ex(h, _ptr(x), n_tokens, _ptr(token_ids), n_hash, _ptr(out), stream))


def ds4moe_forward_host(h: int, x, n_tokens: int, token_ids, n_hash: int, out, stream: int = 0) -> None:
    _check(lib().ds4moe_forward_host(h, _ptr(x), n_tokens, _ptr(token_ids), n_hash, _ptr(out), stream))


def ds4moe_get_route(h: int, n_tokens: int, top_k: int):
    idx = np.zeros((n_tokens, top_k), np.int32)
    w = np.zeros((n_tokens, top_k), np.float32)
    _check(lib().ds4moe_get_route(h, idx.ctypes.data, w.ctypes.data, n_tokens))
    return idx, w


def ds4moe_get_stats(h: int) -> dict:
    st = ds4moe_stats()
    _check(lib().ds4moe_get_stats(h, ctypes.byref(st)))
    return dict(n_tokens=st.n_tokens, distinct_experts=st.distinct_experts, error_flags=st.error_flags,
                counts=np.array(st.counts[:], dtype=np.int32))


def ds4moe_device_bytes(h: int) -> int:
    return lib().ds4moe_device_bytes(h)


def ds4moe_launches_per_forward(h: int, n_tokens: int) -> int:
    return lib().ds4moe_launches_per_forward(h, n_tokens)


def ds4moe_set_profiling(h: int, enable: bool) -> None:
    _check(lib().ds4moe_set_profiling(h, int(bool(enable))))


def ds4moe_get_phase_times(h: int) -> list:
    """[(launch name, stream milliseconds)] of the last profiled forward."""
    cap = 16
    ms = (ctypes.c_float * cap)()
    names = (ctypes.c_char_p * cap)()
    n = ctypes.c_int32()
    _check(lib().ds4moe_get_phase_times(h, ms, names, cap, ctypes.byref(n)))
    return [(names[i].decode(), float(ms[i])) for i in range(min(n.value, cap))]


def ds4moe_route_noalloc(router_w, router_b, x, n_tokens: int, d: int, n_experts: int, top_k: int, idx, w,
                         stream: int = 0) -> None:
    """Routing without any device allocation (for callers that cannot allocate); see the header."""
    _check(lib().ds4moe_route_noalloc(_ptr(router_w), _ptr(router_b), _ptr(x), n_tokens, d, n_experts, top_k,
                                      _ptr(idx), _ptr(w), stream))


def ds4moe_set_test_stall(h: int, stage: int) -> None:
    """Test hook: the next batched forward's GEMM withholds one arrival and its waits give up (see the header)."""
    _check(lib().ds4moe_set_test_stall(h, stage))


def _enum(table: dict, v) -> int:
    n = table.get(v)
    if n is not None:
        return n
    if isinstance(v, str):
        raise ValueError(f"{v!r} is none of {sorted(table)}")
    return int(v)


# Operators on 16-bit matrices (see the header for the mathematics, layouts and limits). dtype and act
# are names ("bf16", "fp16"; "none", "relu", "silu", "gelu") or the ABI's numbers; a row distance of 0
# means that the rows lie back to back. Tensors may be views: one whose strides are not those that the call
# gives (elements of a row apart from each other, rows at another distance) is refused.


def _operand(a, ld: int = 0, step: int = 0) -> Optional[int]:
    """The address of a vector, of a matrix with rows `ld` apart or of a stack of matrices `step` apart."""
    if a is None or type(a) is int:
        return a
    try:
        if a.is_contiguous():  # (a buffer: the call alone says how it is read)
            return a.data_ptr()
    except AttributeError:
        return _ptr(a)
    strides = a.stride()
    if strides == (ld, 1):
        return a.data_ptr()
    shape = tuple(a.shape)
    want = (ld or shape[-1], 1)[-len(shape):]
    while len(want) < len(shape):
        want = (len(want) == 2 and step or shape[-len(want)] * want[0],) + want
    if any(n > 1 and have != w for n, have, w in zip(shape, strides, want)):
        raise ValueError(f"a tensor of shape {shape} has strides {strides}, the call reads it with {want}")
    return a.data_ptr()


def ds4moe_grouped_mm(x, w, offsets, y, rows: int, n: int, k: int, n_groups: int, dtype="bf16", ldx: int = 0,
                      ldw: int = 0, w_stride: int = 0, ldy: int = 0, stream: int = 0) -> None:
    """y[t] = W_g x[t] for the rows t of each group g."""
    _check(lib().ds4moe_grouped_mm(_operand(x, ldx), _operand(w, ldw, w_stride), _operand(offsets), _operand(y, ldy),
                                   rows, n, k, n_groups, _enum(DTYPES, dtype), ldx, ldw, w_stride, ldy, stream))


def ds4moe_grouped_mm_dx(dy, w, offsets, dx, rows: int, n: int, k: int, n_groups: int, dtype="bf16", lddy: int = 0,
                         ldw: int = 0, w_stride: int = 0, lddx: int = 0, stream: int = 0) -> None:
    """dx[t] = W_g^T dy[t] for the rows t of each group g."""
    _check(lib().ds4moe_grouped_mm_dx(_operand(dy, lddy), _operand(w, ldw, w_stride), _operand(offsets),
                                      _operand(dx, lddx), rows, n, k, n_groups, _enum(DTYPES, dtype), lddy, ldw,
                                      w_stride, lddx, stream))


def ds4moe_grouped_mm_dw(dy, x, offsets, dw, rows: int, n: int, k: int, n_groups: int, dtype="bf16", dw_dtype=None,
                         accumulate: bool = False, lddy: int = 0, ldx: int = 0, lddw: int = 0, dw_stride: int = 0,
                         stream: int = 0) -> None:
    """dW_g = sum over the rows t of group g of dy[t] x[t]^T (added to dw with accumulate)."""
    dt = _enum(DTYPES, dtype)
    _check(lib().ds4moe_grouped_mm_dw(_operand(dy, lddy), _operand(x, ldx), _operand(offsets),
                                      _operand(dw, lddw, dw_stride), rows, n, k, n_groups, dt,
                                      dt if dw_dtype is None else _enum(DTYPES, dw_dtype), int(bool(accumulate)),
                                      lddy, ldx, lddw, dw_stride, stream))


def ds4moe_linear(x, w, bias, residual, y, rows: int, n: int, k: int, act="none", dtype="bf16", zout=None,
                  ldx: int = 0, ldw: int = 0, ldr: int = 0, ldy: int = 0, ldz: int = 0, stream: int = 0) -> None:
    """y = act(W x + bias) + residual; zout receives W x + bias."""
    _check(lib().ds4moe_linear(_operand(x, ldx), _operand(w, ldw), _operand(bias), _operand(residual, ldr),
                               _operand(y, ldy), _operand(zout, ldz), rows, n, k, _enum(ACTS, act),
                               _enum(DTYPES, dtype), ldx, ldw, ldr, ldy, ldz, stream))


def ds4moe_linear_grad_workspace(rows: int, n: int, act="none") -> int:
    return lib().ds4moe_linear_grad_workspace(rows, n, _enum(ACTS, act))


def ds4moe_linear_grad(dy, x, w, z, dx, dw, db, rows: int, n: int, k: int, act="none", dtype="bf16",
                       workspace=None, workspace_bytes: int = 0, lddy: int = 0, ldx: int = 0, ldw: int = 0,
                       ldz: int = 0, lddx: int = 0, lddw: int = 0, stream: int = 0) -> None:
    """Gradients of ds4moe_linear: dx, dw and db (each may be None)."""
    _check(lib().ds4moe_linear_grad(_operand(dy, lddy), _operand(x, ldx), _operand(w, ldw), _operand(z, ldz),
                                    _operand(dx, lddx), _operand(dw, lddw), _operand(db), rows, n, k,
                                    _enum(ACTS, act), _enum(DTYPES, dtype), lddy, ldx, ldw, ldz, lddx, lddw,
                                    _operand(workspace), workspace_bytes, stream))


def ds4moe_cross_entropy_workspace(rows: int, vocab: int, d: int) -> int:
    return lib().ds4moe_cross_entropy_workspace(rows, vocab, d)


def ds4moe_cross_entropy(x, w, labels, loss, lse, rows: int, vocab: int, d: int, dtype="bf16",
                         ignore_index: int = -100, workspace=None, workspace_bytes: int = 0, ldx: int = 0,
                         ldw: int = 0, stream: int = 0) -> None:
    """loss[t] = lse[t] - z[t][labels[t]] of the logits z = W x, which are not stored."""
    _check(lib().ds4moe_cross_entropy(_operand(x, ldx), _operand(w, ldw), _operand(labels), _operand(loss),
                                      _operand(lse), rows, vocab, d, _enum(DTYPES, dtype), ignore_index, ldx,
                                      ldw, _operand(workspace), workspace_bytes, stream))


def ds4moe_cross_entropy_grad(x, w, labels, lse, dloss, dx, dw, rows: int, vocab: int, d: int, dtype="bf16",
                              ignore_index: int = -100, workspace=None, workspace_bytes: int = 0, ldx: int = 0,
                              ldw: int = 0, lddx: int = 0, lddw: int = 0, stream: int = 0) -> None:
    """Gradients of sum_t dloss[t] loss[t] with respect to x and w (each may be None)."""
    _check(lib().ds4moe_cross_entropy_grad(_operand(x, ldx), _operand(w, ldw), _operand(labels), _operand(lse),
                                           _operand(dloss), _operand(dx, lddx), _operand(dw, lddw), rows, vocab, d,
                                           _enum(DTYPES, dtype), ignore_index, ldx, ldw, lddx, lddw,
                                           _operand(workspace), workspace_bytes, stream))


def ds4moe_ops_status() -> int:
    """Flags that the 16-bit operators raised on the current device since the last call; clears them."""
    flags = ctypes.c_int32()
    _check(lib().ds4moe_ops_status(ctypes.byref(flags)))
    return flags.value


def ds4moe_destroy(h: Optional[int]) -> None:
    lib().ds4moe_destroy(h)

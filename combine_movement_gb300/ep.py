"""Thin Python binding of libep_gb300.so (the C ABI in include/ep.h).

Same entry-point names as the C ABI. This module only marshals arguments:
torch tensors become device pointers, the stream becomes its cudaStream_t
handle. Every step of layout, dispatch and combine runs in the library's CUDA
kernels; importing this module without the built library raises.

Convenience wrappers (``get_dispatch_layout``, ``dispatch``, ``combine`` and
those of the expert and gradient calls) allocate outputs with torch, on the
stream that the call runs on, and call the same entry points.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libep_gb300.so")

EP_OK = 0
EP_ERR_INVALID = 1
EP_ERR_UNSUPPORTED = 2
EP_ERR_CUDA = 3
EP_ERR_TIMEOUT = 4
EP_ERR_BAD_EXPERT = 5
EP_ERR_BAD_SLOT = 6
EP_ERR_WORKSPACE = 7

EP_MAX_TOPK = 32
EP_MAX_EXPERTS = 4096

# Values that share one scale in the 8-bit operands.
FP8_BLOCK = 128
_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _header_define(name: str) -> int:
    """Integer value of a #define in include/ep.h (the C ABI's own header),
    so sizes the binding checks against cannot drift from it."""
    import re
    hdr = os.path.join(os.path.dirname(_PKG), "include", "ep.h")
    with open(hdr) as f:
        m = re.search(rf"^#define\s+{name}\s+(.+?)\s*$", f.read(), re.M)
    if m is None:
        raise ImportError(f"{name} is not defined in {hdr}")
    expr = re.sub(r"(?<=\d)[uUlL]+\b", "", m.group(1))
    if not re.fullmatch(r"[\d\s()<+*x]+", expr):
        raise ImportError(f"{name} in {hdr}: unexpected expression {m.group(1)!r}")
    return int(eval(expr, {"__builtins__": {}}))  # digits, parentheses, <<, +, * only


# Size of the static scratch array behind ep_get_dispatch_layout_noalloc.
EP_NOALLOC_SCRATCH_BYTES = _header_define("EP_NOALLOC_SCRATCH_BYTES")


class EPError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {ep_status_string(code)} (code {code})")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m combine_movement_gb300.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.ep_set_num_sms.argtypes = [i32]
    lib.ep_set_num_sms.restype = i32
    lib.ep_get_num_sms.argtypes = []
    lib.ep_get_num_sms.restype = i32
    lib.ep_set_launch_overlap.argtypes = [i32]
    lib.ep_set_launch_overlap.restype = i32
    lib.ep_get_launch_overlap.argtypes = []
    lib.ep_get_launch_overlap.restype = i32
    lib.ep_set_dispatch_tail.argtypes = [i32]
    lib.ep_set_dispatch_tail.restype = i32
    lib.ep_get_dispatch_tail.argtypes = []
    lib.ep_get_dispatch_tail.restype = i32
    lib.ep_set_combine_tail.argtypes = [i32]
    lib.ep_set_combine_tail.restype = i32
    lib.ep_get_combine_tail.argtypes = []
    lib.ep_get_combine_tail.restype = i32
    lib.ep_combine_launches.argtypes = [i64, i64, i32, p]
    lib.ep_combine_launches.restype = i32
    lib.ep_num_sms_in_effect.argtypes = []
    lib.ep_num_sms_in_effect.restype = i32
    lib.ep_layout_workspace_bytes.argtypes = [i64, i32, i32]
    lib.ep_layout_workspace_bytes.restype = sz
    lib.ep_layout_launches.argtypes = [i64, i32, i32]
    lib.ep_layout_launches.restype = i32
    lib.ep_dispatch_chunk_bytes.argtypes = [i64, i64, i32]
    lib.ep_dispatch_ring_stages.argtypes = []
    lib.ep_dispatch_ring_stages.restype = i32
    lib.ep_dispatch_chunk_bytes.restype = i64
    lib.ep_dispatch_launches.argtypes = [i64, i64, i32, p]
    lib.ep_dispatch_launches.restype = i32
    lib.ep_layout_dispatch_launches.argtypes = [i64, i64, i32, i32, p]
    lib.ep_layout_dispatch_launches.restype = i32
    lib.ep_get_dispatch_layout.argtypes = [p, i64, i32, i32, p, p, p, p, sz, p, p]
    lib.ep_get_dispatch_layout.restype = i32
    lib.ep_dispatch.argtypes = [p, i64, i64, i32, p, p, i64, p, p, p, p, p]
    lib.ep_dispatch.restype = i32
    lib.ep_layout_dispatch.argtypes = [p, p, i64, i64, i32, i32, p, i64, p, p, p, p, p, p, p, p]
    lib.ep_layout_dispatch.restype = i32
    lib.ep_combine.argtypes = [p, i64, p, p, i64, i64, i32, p, p, p]
    lib.ep_combine.restype = i32
    lib.ep_get_dispatch_layout_noalloc.argtypes = [p, i64, i32, i32, p, p, p, p, p]
    lib.ep_get_dispatch_layout_noalloc.restype = i32
    lib.ep_dispatch_fp8.argtypes = [p, i64, i64, i32, p, p, i64, p, p, p, p, p, p]
    lib.ep_dispatch_fp8.restype = i32
    lib.ep_combine_grad.argtypes = [p, p, i64, p, p, i64, i64, i32, p, p, p, p]
    lib.ep_combine_grad.restype = i32
    lib.ep_dispatch_grad.argtypes = [p, i64, p, i64, i64, i32, p, p, p]
    lib.ep_dispatch_grad.restype = i32
    lib.ep_clear_unused_rows.argtypes = [p, i64, p, i64, i64, i32, p, p]
    lib.ep_clear_unused_rows.restype = i32
    lib.ep_expert_matmul_fp8.argtypes = [p, p, i64, p, i32, p, p, i64, i64, p, p, p]
    lib.ep_expert_matmul_fp8.restype = i32
    lib.ep_expert_gate_up_fp8.argtypes = [p, p, i64, p, i32, p, p, i64, i64, p, p, p, p]
    lib.ep_expert_gate_up_fp8.restype = i32
    lib.ep_sm_partition.argtypes = [i32, ctypes.POINTER(p), ctypes.POINTER(p),
                                    ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.ep_sm_partition.restype = i32
    lib.ep_selftest_wait_timeout.argtypes = [p, ctypes.c_uint64, p]
    lib.ep_selftest_wait_timeout.restype = i32
    lib.ep_get_status.argtypes = [p, p]
    lib.ep_get_status.restype = i32
    lib.ep_status_string.argtypes = [i32]
    lib.ep_status_string.restype = ctypes.c_char_p
    return lib


lib = _load()


# --------------------------------------------------------------------------
# marshalling helpers

def _ptr(t: Optional[torch.Tensor], dtype=None, what: str = "") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t.data_ptr() if t.numel() > 0 else None


# The current stream's raw handle, read without building a torch.cuda.Stream
# object (about 2 us less per call on the host). Every call passes a CUDA
# tensor first, so CUDA is initialised by the time this runs.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and _cur_device is not None:
            return _raw_stream(_cur_device()) or None
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


def _check(code: int, what: str) -> None:
    if code != EP_OK:
        raise EPError(code, what)


# --------------------------------------------------------------------------
# C ABI, same names

def ep_set_num_sms(num_sms: int) -> int:
    return lib.ep_set_num_sms(int(num_sms))


def ep_get_num_sms() -> int:
    return lib.ep_get_num_sms()


def ep_set_launch_overlap(mode: int) -> int:
    return lib.ep_set_launch_overlap(mode)


def ep_get_launch_overlap() -> int:
    return lib.ep_get_launch_overlap()


def ep_set_dispatch_tail(percent: int) -> int:
    return lib.ep_set_dispatch_tail(int(percent))


def ep_get_dispatch_tail() -> int:
    return lib.ep_get_dispatch_tail()


def ep_set_combine_tail(percent: int) -> int:
    return lib.ep_set_combine_tail(int(percent))


def ep_get_combine_tail() -> int:
    return lib.ep_get_combine_tail()


def ep_combine_launches(T: int, H: int, K: int, stream=None) -> int:
    return int(lib.ep_combine_launches(T, H, K, _stream(stream)))


def ep_num_sms_in_effect() -> int:
    return lib.ep_num_sms_in_effect()


def ep_layout_workspace_bytes(T: int, K: int, E: int) -> int:
    return int(lib.ep_layout_workspace_bytes(T, K, E))


def ep_layout_launches(T: int, K: int, E: int) -> int:
    return int(lib.ep_layout_launches(T, K, E))


def ep_dispatch_chunk_bytes(T: int, H: int, K: int) -> int:
    return int(lib.ep_dispatch_chunk_bytes(T, H, K))


def ep_dispatch_ring_stages() -> int:
    return int(lib.ep_dispatch_ring_stages())


def ep_dispatch_launches(T: int, H: int, K: int, stream=None) -> int:
    return int(lib.ep_dispatch_launches(T, H, K, _stream(stream)))


def ep_layout_dispatch_launches(T: int, H: int, K: int, E: int, stream=None) -> int:
    return int(lib.ep_layout_dispatch_launches(T, H, K, E, _stream(stream)))


def ep_status_string(code: int) -> str:
    return lib.ep_status_string(int(code)).decode()


def ep_get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int, counts: torch.Tensor,
                           offsets: torch.Tensor, slot: torch.Tensor,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None) -> None:
    T, K = topk_idx.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    code = lib.ep_get_dispatch_layout(
        _ptr(topk_idx, torch.int64, "topk_idx"), T, K, int(num_experts),
        _ptr(counts, torch.int32, "counts"), _ptr(offsets, torch.int32, "offsets"),
        _ptr(slot, torch.int32, "slot"), _ptr(workspace, None, "workspace"), ws_bytes,
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(code, "ep_get_dispatch_layout")


def ep_get_dispatch_layout_noalloc(topk_idx: torch.Tensor, num_experts: int,
                                   counts: torch.Tensor, offsets: torch.Tensor,
                                   slot: torch.Tensor, status: Optional[torch.Tensor] = None,
                                   stream=None) -> None:
    """Layout for callers that cannot allocate: the scratch is the library's
    static device array (EP_NOALLOC_SCRATCH_BYTES), shared by every call."""
    T, K = topk_idx.shape
    code = lib.ep_get_dispatch_layout_noalloc(
        _ptr(topk_idx, torch.int64, "topk_idx"), T, K, int(num_experts),
        _ptr(counts, torch.int32, "counts"), _ptr(offsets, torch.int32, "offsets"),
        _ptr(slot, torch.int32, "slot"), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(code, "ep_get_dispatch_layout_noalloc")




def ep_dispatch(x: torch.Tensor, slot: torch.Tensor, recv_x: torch.Tensor,
                topk_w: Optional[torch.Tensor] = None, recv_w: Optional[torch.Tensor] = None,
                recv_src: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                stream=None) -> None:
    T, H = x.shape
    K = slot.shape[1]
    code = lib.ep_dispatch(
        _ptr(x, torch.bfloat16, "x"), T, H, K, _ptr(slot, torch.int32, "slot"),
        _ptr(topk_w, torch.float32, "topk_w"), recv_x.shape[0],
        _ptr(recv_x, torch.bfloat16, "recv_x"), _ptr(recv_w, torch.float32, "recv_w"),
        _ptr(recv_src, torch.int32, "recv_src"), _ptr(status, torch.int32, "status"),
        _stream(stream))
    _check(code, "ep_dispatch")


def ep_layout_dispatch(topk_idx: torch.Tensor, num_experts: int, x: torch.Tensor,
                       counts: torch.Tensor, offsets: torch.Tensor, slot: torch.Tensor,
                       recv_x: torch.Tensor, topk_w: Optional[torch.Tensor] = None,
                       recv_w: Optional[torch.Tensor] = None,
                       recv_src: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> None:
    T, H = x.shape
    K = topk_idx.shape[1]
    code = lib.ep_layout_dispatch(
        _ptr(topk_idx, torch.int64, "topk_idx"), _ptr(x, torch.bfloat16, "x"), T, H, K,
        int(num_experts), _ptr(topk_w, torch.float32, "topk_w"), recv_x.shape[0],
        _ptr(counts, torch.int32, "counts"), _ptr(offsets, torch.int32, "offsets"),
        _ptr(slot, torch.int32, "slot"), _ptr(recv_x, torch.bfloat16, "recv_x"),
        _ptr(recv_w, torch.float32, "recv_w"), _ptr(recv_src, torch.int32, "recv_src"),
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(code, "ep_layout_dispatch")


def ep_combine(expert_out: torch.Tensor, slot: torch.Tensor, topk_w: torch.Tensor,
               y: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    T, H = y.shape
    K = slot.shape[1]
    code = lib.ep_combine(
        _ptr(expert_out, torch.bfloat16, "expert_out"), expert_out.shape[0],
        _ptr(slot, torch.int32, "slot"), _ptr(topk_w, torch.float32, "topk_w"), T, H, K,
        _ptr(y, torch.bfloat16, "y"), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(code, "ep_combine")


# Arguments of the expert and gradient calls: the address of a tensor of this
# type and shape, checked in one expression (the host's part of a call is
# longer than the device's of a small one). Where it lies, its caller
# checks.
def _arg(t: torch.Tensor, dtype, shape: Tuple[int, ...], what: str) -> int:
    if t.shape == shape and t.dtype is dtype and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    raise ValueError(f"{what}: expected a contiguous tensor")


def _opt(t: Optional[torch.Tensor], dtype, shape: Tuple[int, ...], what: str) -> Optional[int]:
    if t is None:
        return None
    p = _arg(t, dtype, shape, what)
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    return p


def _off_gpu(**tensors: torch.Tensor) -> ValueError:
    what = ", ".join(k for k, t in tensors.items() if not t.is_cuda)
    return ValueError(f"{what}: expected a CUDA tensor")


def ep_dispatch_fp8(x: torch.Tensor, slot: torch.Tensor, recv_q: torch.Tensor,
                    recv_scale: torch.Tensor, topk_w: Optional[torch.Tensor] = None,
                    recv_w: Optional[torch.Tensor] = None,
                    recv_src: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    T, H = x.shape
    K, R = slot.shape[1], recv_q.shape[0]
    px, ps = _arg(x, _BF16, (T, H), "x"), _arg(slot, _I32, (T, K), "slot")
    pq = _arg(recv_q, _E4M3, (R, H), "recv_q")
    pc = _arg(recv_scale, _F32, (R, -(-H // FP8_BLOCK)), "recv_scale")
    if not (x.is_cuda and slot.is_cuda and recv_q.is_cuda and recv_scale.is_cuda):
        raise _off_gpu(x=x, slot=slot, recv_q=recv_q, recv_scale=recv_scale)
    code = lib.ep_dispatch_fp8(
        px, T, H, K, ps, None if topk_w is None else _opt(topk_w, _F32, (T, K), "topk_w"), R, pq, pc,
        None if recv_w is None else _opt(recv_w, _F32, (R,), "recv_w"),
        None if recv_src is None else _opt(recv_src, _I32, (R,), "recv_src"),
        None if status is None else _ptr(status, _I32, "status"), _stream(stream))
    if code != EP_OK:
        raise EPError(code, "ep_dispatch_fp8")


def ep_combine_grad(dy: torch.Tensor, expert_out: Optional[torch.Tensor], slot: torch.Tensor,
                    topk_w: torch.Tensor, d_expert_out: Optional[torch.Tensor],
                    d_topk_w: Optional[torch.Tensor], status: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """expert_out may be None where d_topk_w is."""
    T, H = dy.shape
    if expert_out is None and d_expert_out is None:
        raise ValueError("expert_out: expected a tensor")
    K, R = slot.shape[1], (d_expert_out if expert_out is None else expert_out).shape[0]
    rows, pairs = (R, H), (T, K)
    py = _arg(dy, _BF16, (T, H), "dy")
    pe = None if expert_out is None else _arg(expert_out, _BF16, rows, "expert_out")
    ps, pw = _arg(slot, _I32, pairs, "slot"), _arg(topk_w, _F32, pairs, "topk_w")
    pde = None if d_expert_out is None else _arg(d_expert_out, _BF16, rows, "d_expert_out")
    pdw = None if d_topk_w is None else _arg(d_topk_w, _F32, pairs, "d_topk_w")
    if not (dy.is_cuda and (pe is None or expert_out.is_cuda) and slot.is_cuda and topk_w.is_cuda
            and (pde is None or d_expert_out.is_cuda) and (pdw is None or d_topk_w.is_cuda)):
        raise ValueError("ep_combine_grad: expected a CUDA tensor for every argument")
    code = lib.ep_combine_grad(
        py, pe, R, ps, pw, T, H, K, pde, pdw, None if status is None else _ptr(status, _I32, "status"),
        _stream(stream))
    if code != EP_OK:
        raise EPError(code, "ep_combine_grad")


def ep_dispatch_grad(d_recv: torch.Tensor, slot: torch.Tensor, dx: torch.Tensor,
                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    T, H = dx.shape
    K, R = slot.shape[1], d_recv.shape[0]
    pd, ps = _arg(d_recv, _BF16, (R, H), "d_recv"), _arg(slot, _I32, (T, K), "slot")
    px = _arg(dx, _BF16, (T, H), "dx")
    if not (d_recv.is_cuda and slot.is_cuda and dx.is_cuda):
        raise _off_gpu(d_recv=d_recv, slot=slot, dx=dx)
    code = lib.ep_dispatch_grad(pd, R, ps, T, H, K, px,
                                None if status is None else _ptr(status, _I32, "status"),
                                _stream(stream))
    if code != EP_OK:
        raise EPError(code, "ep_dispatch_grad")


def ep_clear_unused_rows(rows: torch.Tensor, slot: torch.Tensor,
                         status: Optional[torch.Tensor] = None, stream=None) -> None:
    (R, H), (T, K) = rows.shape, slot.shape
    pr, ps = _arg(rows, _BF16, (R, H), "rows"), _arg(slot, _I32, (T, K), "slot")
    if not (rows.is_cuda and slot.is_cuda):
        raise _off_gpu(rows=rows, slot=slot)
    code = lib.ep_clear_unused_rows(pr, R, ps, T, H, K,
                                    None if status is None else _ptr(status, _I32, "status"),
                                    _stream(stream))
    if code != EP_OK:
        raise EPError(code, "ep_clear_unused_rows")


def ep_expert_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, offsets: torch.Tensor,
                         w: torch.Tensor, w_scale: torch.Tensor, out: torch.Tensor,
                         status: Optional[torch.Tensor] = None, stream=None) -> None:
    R, K = a.shape
    E, N = w.shape[:2]
    kb = -(-K // FP8_BLOCK)
    pa, ps = _arg(a, _E4M3, (R, K), "a"), _arg(a_scale, _F32, (R, kb), "a_scale")
    po, pw = _arg(offsets, _I32, (E + 1,), "offsets"), _arg(w, _E4M3, (E, N, K), "w")
    pws = _arg(w_scale, _F32, (E, -(-N // FP8_BLOCK), kb), "w_scale")
    py = _arg(out, _BF16, (R, N), "out")
    if not (a.is_cuda and a_scale.is_cuda and offsets.is_cuda and w.is_cuda and w_scale.is_cuda
            and out.is_cuda):
        raise _off_gpu(a=a, a_scale=a_scale, offsets=offsets, w=w, w_scale=w_scale, out=out)
    code = lib.ep_expert_matmul_fp8(
        pa, ps, R, po, E, pw, pws, N, K, py, None if status is None else _ptr(status, _I32, "status"),
        _stream(stream))
    if code != EP_OK:
        raise EPError(code, "ep_expert_matmul_fp8")


def ep_expert_gate_up_fp8(a: torch.Tensor, a_scale: torch.Tensor, offsets: torch.Tensor,
                          w: torch.Tensor, w_scale: torch.Tensor, out_q: torch.Tensor,
                          out_scale: torch.Tensor, status: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    R, K = a.shape
    E, N = w.shape[:2]
    if N % 2:
        raise ValueError(f"w: expected a gate half and an up half, got {N} rows")
    kb, width = -(-K // FP8_BLOCK), N // 2
    pa, ps = _arg(a, _E4M3, (R, K), "a"), _arg(a_scale, _F32, (R, kb), "a_scale")
    po, pw = _arg(offsets, _I32, (E + 1,), "offsets"), _arg(w, _E4M3, (E, N, K), "w")
    pws = _arg(w_scale, _F32, (E, -(-N // FP8_BLOCK), kb), "w_scale")
    pq = _arg(out_q, _E4M3, (R, width), "out_q")
    pqs = _arg(out_scale, _F32, (R, -(-width // FP8_BLOCK)), "out_scale")
    if not (a.is_cuda and a_scale.is_cuda and offsets.is_cuda and w.is_cuda and w_scale.is_cuda
            and out_q.is_cuda and out_scale.is_cuda):
        raise _off_gpu(a=a, a_scale=a_scale, offsets=offsets, w=w, w_scale=w_scale, out_q=out_q,
                       out_scale=out_scale)
    code = lib.ep_expert_gate_up_fp8(
        pa, ps, R, po, E, pw, pws, width, K, pq, pqs,
        None if status is None else _ptr(status, _I32, "status"), _stream(stream))
    if code != EP_OK:
        raise EPError(code, "ep_expert_gate_up_fp8")


def ep_sm_partition(num_sms: int) -> Tuple[int, Optional[int], int, int]:
    """(stream, rest_stream, sms, rest_sms) of an SM partition of at least
    num_sms SMs on the current device; the streams are raw cudaStream_t
    handles (wrap them with torch.cuda.ExternalStream)."""
    s, r = ctypes.c_void_p(), ctypes.c_void_p()
    n, rn = ctypes.c_int(), ctypes.c_int()
    _check(lib.ep_sm_partition(int(num_sms), ctypes.byref(s), ctypes.byref(r), ctypes.byref(n),
                               ctypes.byref(rn)), "ep_sm_partition")
    return int(s.value), (int(r.value) if r.value else None), n.value, rn.value


def ep_selftest_wait_timeout(status: torch.Tensor, limit_ns: int, stream=None) -> None:
    _check(lib.ep_selftest_wait_timeout(_ptr(status, torch.int32, "status"), int(limit_ns),
                                        _stream(stream)), "ep_selftest_wait_timeout")


def ep_get_status(status: torch.Tensor, stream=None) -> int:
    return int(lib.ep_get_status(_ptr(status, torch.int32, "status"), _stream(stream)))


# --------------------------------------------------------------------------
# allocating conveniences

def _empty(shape, dtype, device, stream, keep: bool = True) -> torch.Tensor:
    """torch.empty for an output (``keep``) or a workspace of a call on `stream`.

    The memory comes from that stream's own part of the allocator: memory of
    the current stream's may still be in use by work pending there, and a
    result dropped early would go back to it while the call still runs. An
    output may be used on the current stream too, so that stream is recorded
    for it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)  # (0 names the default stream)
        stream = (torch.cuda.ExternalStream(raw, device) if raw
                  else torch.cuda.default_stream(device))
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if keep:
        t.record_stream(current)
    return t


def get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int,
                        status: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Returns (counts[E], offsets[E+1], slot[T,K]) as int32 CUDA tensors."""
    dev = topk_idx.device
    T, K = topk_idx.shape
    counts = _empty(num_experts, torch.int32, dev, stream)
    offsets = _empty(num_experts + 1, torch.int32, dev, stream)
    slot = _empty((T, K), torch.int32, dev, stream)
    nbytes = ep_layout_workspace_bytes(T, K, num_experts)
    ws = _empty(nbytes, torch.uint8, dev, stream, keep=False) if nbytes else None
    ep_get_dispatch_layout(topk_idx, num_experts, counts, offsets, slot, ws, status, stream)
    return counts, offsets, slot


def dispatch(x: torch.Tensor, slot: torch.Tensor, num_recv: int,
             topk_w: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
             stream=None):
    """Returns recv_x [num_recv, H] (and recv_w, recv_src when topk_w is given)."""
    recv_x = _empty((num_recv, x.shape[1]), x.dtype, x.device, stream)
    recv_w = recv_src = None
    if topk_w is not None:
        recv_w = _empty(num_recv, torch.float32, x.device, stream)
        recv_src = _empty(num_recv, torch.int32, x.device, stream)
    ep_dispatch(x, slot, recv_x, topk_w, recv_w, recv_src, status, stream)
    return (recv_x, recv_w, recv_src) if topk_w is not None else recv_x


def combine(expert_out: torch.Tensor, slot: torch.Tensor, topk_w: torch.Tensor,
            status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    T = slot.shape[0]
    y = _empty((T, expert_out.shape[1]), expert_out.dtype, expert_out.device, stream)
    ep_combine(expert_out, slot, topk_w, y, status, stream)
    return y


def dispatch_fp8(x: torch.Tensor, slot: torch.Tensor, num_recv: int,
                 topk_w: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream=None):
    """Returns recv_q [num_recv, H] (e4m3) and recv_scale [num_recv, ceil(H / 128)]
    (and recv_w, recv_src when topk_w is given)."""
    H, dev = x.shape[1], x.device
    recv_q = _empty((num_recv, H), _E4M3, dev, stream)
    recv_scale = _empty((num_recv, -(-H // FP8_BLOCK)), _F32, dev, stream)
    recv_w = recv_src = None
    if topk_w is not None:
        recv_w = _empty(num_recv, _F32, dev, stream)
        recv_src = _empty(num_recv, _I32, dev, stream)
    ep_dispatch_fp8(x, slot, recv_q, recv_scale, topk_w, recv_w, recv_src, status, stream)
    return (recv_q, recv_scale) if topk_w is None else (recv_q, recv_scale, recv_w, recv_src)


def combine_grad(dy: torch.Tensor, expert_out: torch.Tensor, slot: torch.Tensor,
                 topk_w: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Returns (d_expert_out [num_recv, H], d_topk_w [T, K]). Rows no entry
    maps to are left as allocated."""
    d_expert_out = _empty(expert_out.shape, expert_out.dtype, expert_out.device, stream)
    d_topk_w = _empty(topk_w.shape, topk_w.dtype, topk_w.device, stream)
    ep_combine_grad(dy, expert_out, slot, topk_w, d_expert_out, d_topk_w, status, stream)
    return d_expert_out, d_topk_w


def dispatch_grad(d_recv: torch.Tensor, slot: torch.Tensor, status: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Returns dx [T, H], each token's receive-row gradients summed."""
    dx = _empty((slot.shape[0], d_recv.shape[1]), d_recv.dtype, d_recv.device, stream)
    ep_dispatch_grad(d_recv, slot, dx, status, stream)
    return dx


def expert_matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, offsets: torch.Tensor,
                      w: torch.Tensor, w_scale: torch.Tensor,
                      status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each expert's rows times its weights: bf16 [num_recv, N]. Rows no
    expert has (from offsets[E] on) are left as allocated."""
    out = _empty((a.shape[0], w.shape[1]), _BF16, a.device, stream)
    ep_expert_matmul_fp8(a, a_scale, offsets, w, w_scale, out, status, stream)
    return out


def expert_gate_up_fp8(a: torch.Tensor, a_scale: torch.Tensor, offsets: torch.Tensor,
                       w: torch.Tensor, w_scale: torch.Tensor,
                       status: Optional[torch.Tensor] = None, stream=None
                       ) -> Tuple[torch.Tensor, torch.Tensor]:
    """silu(gate) * up of each expert's rows, quantised again: (e4m3
    [num_recv, I], fp32 scales [num_recv, I / 128]); the next product's rows."""
    R, width = a.shape[0], w.shape[1] // 2
    out_q = _empty((R, width), _E4M3, a.device, stream)
    out_scale = _empty((R, -(-width // FP8_BLOCK)), _F32, a.device, stream)
    ep_expert_gate_up_fp8(a, a_scale, offsets, w, w_scale, out_q, out_scale, status, stream)
    return out_q, out_scale

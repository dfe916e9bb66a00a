"""Python binding of the OAL C ABI (include/oal.h): argument marshalling only.

Every step of the computation runs in the CUDA library liboal.so.  PyTorch supplies device
memory and streams.  The binding raises OALError on any non-zero status and refuses to run
when the library is missing.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liboal.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "oal.h")

OAL_F32, OAL_BF16 = 0, 1
OAL_PATH_CUDA_CORE, OAL_PATH_TENSOR = 0, 1
HEAD_DIM = VALUE_DIM = 64
G_MAX = 8
FEATURES, FEATURES_PAD = 2145, 2176
STATUS = {0: "OAL_OK", -1: "OAL_ERR_NULL", -2: "OAL_ERR_SHAPE", -3: "OAL_ERR_UNSUPPORTED",
          -4: "OAL_ERR_ALIGN", -5: "OAL_ERR_GROUPS", -6: "OAL_ERR_CUDA", -7: "OAL_ERR_TIMEOUT",
          -8: "OAL_ERR_WORKSPACE", -9: "OAL_ERR_STATE", -10: "OAL_ERR_VALUE",
          -11: "OAL_ERR_OVERLAP"}


class Shape(ctypes.Structure):
    """oal_shape."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "Hq", "Hkv", "dh", "dv", "chunk",
                                               "dtype")]


class KernelStat(ctypes.Structure):
    """oal_kernel_stat."""
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_double)]


class OALError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = f"{what}: {STATUS.get(code, code)} ({status_string(code)})"
        if code == -6:
            msg += f" [{last_cuda_error()}]"
        super().__init__(msg)


_lock = threading.Lock()
_lib = None
_VP, _SZ, _PS = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Shape)


def lib() -> ctypes.CDLL:
    """The loaded liboal.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing; run "
                                   "python -m positive_quadratic_b200.build")
            L = ctypes.CDLL(LIB_PATH)
            L.oal_abi_version.restype = ctypes.c_int
            L.oal_status_string.argtypes = [ctypes.c_int]
            L.oal_status_string.restype = ctypes.c_char_p
            for name in ("oal_state_bytes", "oal_prefill_workspace_bytes",
                         "oal_decode_workspace_bytes"):
                getattr(L, name).argtypes = [_PS, ctypes.POINTER(_SZ)]
            L.oal_prefill_path.argtypes = [_PS, ctypes.POINTER(ctypes.c_int)]
            L.oal_prefill_path.restype = ctypes.c_int
            L.oal_prefill.argtypes = [_VP] * 6 + [ctypes.c_float, _VP, _VP, _VP, _SZ, _PS, _VP]
            L.oal_prefill_continue.argtypes = L.oal_prefill.argtypes
            L.oal_decode_step.argtypes = [_VP] * 6 + [_SZ, _PS, _VP]
            L.oal_dense_ref_gpu.argtypes = [_VP] * 6 + [ctypes.c_float, _VP, _PS, _VP]
            L.oal_contribution_stat.argtypes = [_VP, _VP, _VP, _PS, _VP]
            L.oal_device_error.argtypes = [ctypes.POINTER(ctypes.c_int), _VP]
            L.oal_launch_count.restype = ctypes.c_ulonglong
            L.oal_last_cuda_error.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
            L.oal_last_cuda_error.restype = ctypes.c_int
            L.oal_set_prefill_overlap.argtypes = [ctypes.c_int]
            L.oal_set_prefill_overlap.restype = ctypes.c_int
            L.oal_set_debug_skip_copies.argtypes = [ctypes.c_int]
            L.oal_set_debug_skip_copies.restype = ctypes.c_int
            L.oal_prefill_host_workspace_bytes.argtypes = [_PS, ctypes.c_int,
                                                           ctypes.POINTER(_SZ)]
            L.oal_prefill_host.argtypes = [_VP] * 6 + [ctypes.c_float, _VP, _VP, _VP, _SZ, _PS,
                                                       ctypes.c_int, _VP, _VP, _VP]
            L.oal_prefill_hadamard.argtypes = [_VP] * 7 + [_VP, _VP, _SZ, _PS, _VP]
            L.oal_dense_hadamard_gpu.argtypes = [_VP] * 7 + [_PS, _VP]
            L.oal_prefill_varlen_workspace_bytes.argtypes = [_PS, _VP, ctypes.c_int,
                                                             ctypes.c_int, ctypes.POINTER(_SZ)]
            L.oal_prefill_varlen.argtypes = [_VP] * 6 + [ctypes.c_float, _VP, _VP, _SZ, _VP,
                                                         _SZ, _PS, _VP, ctypes.c_int, _VP,
                                                         ctypes.c_int]
            L.oal_prefill_packed_workspace_bytes.argtypes = [_PS, _VP, ctypes.c_int,
                                                             ctypes.POINTER(_SZ)]
            L.oal_prefill_packed_workspace_bytes.restype = ctypes.c_int
            L.oal_prefill_packed.argtypes = [_VP] * 6 + [ctypes.c_float, _VP, _VP, _SZ, _VP,
                                                         _SZ, _PS, _VP, ctypes.c_int, _VP]
            L.oal_prefill_packed.restype = ctypes.c_int
            L.oal_state_prefix_sum.argtypes = [_VP, ctypes.c_int, _SZ, _VP, _VP]
            L.oal_state_prefix_sum.restype = ctypes.c_int
            for pre in ("oal_dense_backward", "oal_backward"):
                getattr(L, pre + "_workspace_bytes").argtypes = [_PS, ctypes.POINTER(_SZ)]
                getattr(L, pre + "_workspace_bytes").restype = ctypes.c_int
            for name in ("oal_dense_backward_gpu", "oal_backward"):
                getattr(L, name).argtypes = [_VP] * 6 + [ctypes.c_float] + [_VP] * 7 + [
                    _SZ, _PS, _VP]
                getattr(L, name).restype = ctypes.c_int
            for name in ("oal_prefill_host_workspace_bytes", "oal_prefill_host",
                         "oal_prefill_hadamard", "oal_dense_hadamard_gpu",
                         "oal_prefill_varlen_workspace_bytes", "oal_prefill_varlen"):
                getattr(L, name).restype = ctypes.c_int
            _I, _F = ctypes.c_int, ctypes.c_float
            for name, args in {
                    "oal_decay_state_bytes": [_PS, ctypes.POINTER(_SZ)],
                    "oal_decay_prefill_workspace_bytes": [_PS, ctypes.POINTER(_SZ)],
                    "oal_decay_prefill": [_VP] * 4 + [_F] + [_VP] * 4 + [_SZ, _PS, _VP],
                    "oal_decay_prefill_continue": [_VP] * 4 + [_F] + [_VP] * 4 + [_SZ, _PS, _VP],
                    "oal_decay_step": [_VP] * 4 + [_F, _VP, _I] + [_VP] * 3 + [_PS, _VP],
                    "oal_decay_backward_workspace_bytes": [_PS, ctypes.POINTER(_SZ)],
                    "oal_decay_backward": [_VP] * 4 + [_F] + [_VP] * 9 + [_SZ, _PS, _VP],
                    "oal_beam_select_workspace_bytes": [_I] * 5 + [ctypes.POINTER(_SZ)],
                    "oal_beam_select": [_VP, ctypes.c_longlong, _I, _VP, _VP] + [_I] * 5 +
                                       [_VP] * 4 + [_SZ, _VP],
                    "oal_state_reorder": [_VP, _I, _VP, _VP, _PS, _VP],
                    "oal_decay_state_reorder": [_VP, _I, _VP, _VP, _PS, _VP],
                    "oal_decode_step_beam": [_VP] * 4 + [_I] + [_VP] * 4 + [_SZ, _PS, _VP]}.items():
                getattr(L, name).argtypes = args
                getattr(L, name).restype = _I
            L.oal_profile_enable.argtypes = [ctypes.c_int]
            L.oal_profile_enable.restype = ctypes.c_int
            L.oal_profile_read.argtypes = [ctypes.POINTER(KernelStat), ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_int)]
            L.oal_profile_read.restype = ctypes.c_int
            for name in ("oal_state_bytes", "oal_prefill_workspace_bytes",
                         "oal_decode_workspace_bytes", "oal_prefill", "oal_decode_step",
                         "oal_dense_ref_gpu", "oal_device_error", "oal_contribution_stat",
                         "oal_prefill_continue"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def declared_symbols(header: str = HEADER):
    """Names of the functions include/oal.h declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:int|const char\*|unsigned long long)\s+(oal_\w+)\s*\(",
                                 text, re.M)))


def last_cuda_error() -> str:
    """Name and description of the CUDA error behind the most recent OAL_ERR_CUDA."""
    try:
        buf = ctypes.create_string_buffer(256)
        lib().oal_last_cuda_error(buf, 256)
        return buf.value.decode()
    except Exception:
        return "?"


def status_string(code: int) -> str:
    try:
        return lib().oal_status_string(int(code)).decode()
    except Exception:
        return "?"


def _check(rc: int, what: str):
    if rc != 0:
        raise OALError(rc, what)


def make_shape(B, T, Hq, Hkv, chunk=128, dtype=OAL_BF16, dh=HEAD_DIM, dv=VALUE_DIM) -> Shape:
    return Shape(int(B), int(T), int(Hq), int(Hkv), int(dh), int(dv), int(chunk), int(dtype))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return OAL_BF16
    if t.dtype == torch.float32:
        return OAL_F32
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def state_bytes(shape: Shape) -> int:
    n = _SZ()
    _check(lib().oal_state_bytes(ctypes.byref(shape), ctypes.byref(n)), "oal_state_bytes")
    return n.value


def prefill_workspace_bytes(shape: Shape) -> int:
    n = _SZ()
    _check(lib().oal_prefill_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "oal_prefill_workspace_bytes")
    return n.value


def prefill_path(shape: Shape) -> int:
    """OAL_PATH_TENSOR or OAL_PATH_CUDA_CORE: the kernels oal_prefill runs for `shape`."""
    p = ctypes.c_int()
    _check(lib().oal_prefill_path(ctypes.byref(shape), ctypes.byref(p)), "oal_prefill_path")
    return p.value


def decode_workspace_bytes(shape: Shape) -> int:
    n = _SZ()
    _check(lib().oal_decode_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "oal_decode_workspace_bytes")
    return n.value


def _shape_of(q, k, v, chunk):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, d]")
    B, Hq, T, dh = q.shape
    return make_shape(B, T, Hq, k.shape[1], chunk, _dtype_code(q), dh, v.shape[3])


def _contig_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def empty_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def prefill(q, k, v, group_id, L, G, eps: float, chunk: int = 128, out=None, state=None,
            workspace=None, stream=None):
    """oal_prefill on CUDA tensors.  Returns (out [B,Hq,T,dv] fp32, state uint8)."""
    shape = _shape_of(q, k, v, chunk)
    dev = q.device
    if out is None:
        out = torch.empty(q.shape[0], q.shape[1], q.shape[2], v.shape[3], dtype=torch.float32,
                          device=dev)
    if state is None:
        state = torch.empty(state_bytes(shape), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = empty_workspace(prefill_workspace_bytes(shape), dev)
    _contig_cuda(q, k, v, group_id, L, G, out, state, workspace)
    rc = lib().oal_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(group_id), _ptr(L), _ptr(G),
                           float(eps), _ptr(out), _ptr(state), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), ctypes.byref(shape),
                           _stream(stream))
    _check(rc, "oal_prefill")
    return out, state


def prefill_state(k, v, group_id, L, G, eps: float, Hq: int, chunk: int = 128, state=None,
                  workspace=None, stream=None):
    """oal_prefill with out = NULL: the prefix state after the T tokens of k/v (and the
    coefficient tables of Hq query heads), without computing outputs."""
    B, Hkv, T, dh = k.shape
    shape = make_shape(B, T, Hq, Hkv, chunk, _dtype_code(k), dh, v.shape[3])
    dev = k.device
    if state is None:
        state = torch.empty(state_bytes(shape), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = empty_workspace(prefill_workspace_bytes(shape), dev)
    _contig_cuda(k, v, group_id, L, G, state, workspace)
    rc = lib().oal_prefill(None, _ptr(k), _ptr(v), _ptr(group_id), _ptr(L), _ptr(G),
                           float(eps), None, _ptr(state), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), ctypes.byref(shape),
                           _stream(stream))
    _check(rc, "oal_prefill (state only)")
    return state


def state_body(state: torch.Tensor, B: int, Hq: int, Hkv: int) -> torch.Tensor:
    """fp32 view of the per-(b, kv) prefix states inside a state buffer (after the header and
    the coefficient tables): B*Hkv units of Hv[2176][64] then z[2176]."""
    off = 256 + ((Hq * FEATURES_PAD * 4 + 255) // 256) * 256
    n = B * Hkv * FEATURES_PAD * (VALUE_DIM + 1)
    return state[off:off + 4 * n].view(torch.float32)


def state_prefix_sum(parts: torch.Tensor, n_parts: int, out: torch.Tensor, stream=None):
    """oal_state_prefix_sum: out = parts[0] + ... + parts[n_parts - 1] (rows of a contiguous
    fp32 [rows, n] tensor, added in order)."""
    if parts.dim() != 2 or parts.dtype != torch.float32 or out.dtype != torch.float32:
        raise ValueError("parts [rows, n] and out [n] must be fp32")
    if not 0 <= n_parts <= parts.shape[0] or out.numel() != parts.shape[1]:
        raise ValueError("n_parts out of range or out of the wrong size")
    _contig_cuda(parts, out)
    _check(lib().oal_state_prefix_sum(_ptr(parts), int(n_parts), parts.shape[1], _ptr(out),
                                      _stream(stream)), "oal_state_prefix_sum")
    return out


def set_state_tokens(state: torch.Tensor, tokens: int) -> None:
    """Sets the token count in a state header (int64 at byte 32)."""
    state[32:40].copy_(torch.tensor([int(tokens)], dtype=torch.int64).view(torch.uint8))


def prefill_continue(q, k, v, group_id, L, G, eps: float, state, out=None, workspace=None,
                     stream=None):
    """oal_prefill_continue: appends the T tokens of q/k/v to the sequence held by `state`
    (bf16, chunk 128).  Returns out [B,Hq,T,dv] fp32; `state` is updated in place."""
    shape = _shape_of(q, k, v, 128)
    dev = q.device
    if out is None:
        out = torch.empty(q.shape[0], q.shape[1], q.shape[2], v.shape[3], dtype=torch.float32,
                          device=dev)
    if workspace is None:
        workspace = empty_workspace(prefill_workspace_bytes(shape), dev)
    _contig_cuda(q, k, v, group_id, L, G, out, state, workspace)
    rc = lib().oal_prefill_continue(_ptr(q), _ptr(k), _ptr(v), _ptr(group_id), _ptr(L),
                                    _ptr(G), float(eps), _ptr(out), _ptr(state),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    ctypes.byref(shape), _stream(stream))
    _check(rc, "oal_prefill_continue")
    return out


def decode_step(q, k, v, state, workspace, out=None, stream=None):
    """oal_decode_step on CUDA tensors q [B,Hq,1,dh], k/v [B,Hkv,1,d]; returns out."""
    shape = _shape_of(q, k, v, 128)
    shape.T = 1
    if out is None:
        out = torch.empty(q.shape[0], q.shape[1], 1, v.shape[3], dtype=torch.float32,
                          device=q.device)
    _contig_cuda(q, k, v, state, workspace, out)
    rc = lib().oal_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(state), _ptr(out),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               ctypes.byref(shape), _stream(stream))
    _check(rc, "oal_decode_step")
    return out


def decode_workspace(B, Hq, Hkv, device) -> torch.Tensor:
    """Decode workspace (zero-filled; a step writes every scratch word before reading it)."""
    n = decode_workspace_bytes(make_shape(B, 1, Hq, Hkv))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def dense_ref(q, k, v, group_id, L, G, eps: float, out=None, stream=None):
    """oal_dense_ref_gpu: the O(T^2) dense form."""
    shape = _shape_of(q, k, v, 128)
    if out is None:
        out = torch.empty(q.shape[0], q.shape[1], q.shape[2], v.shape[3], dtype=torch.float32,
                          device=q.device)
    _contig_cuda(q, k, v, group_id, L, G, out)
    rc = lib().oal_dense_ref_gpu(_ptr(q), _ptr(k), _ptr(v), _ptr(group_id), _ptr(L), _ptr(G),
                                 float(eps), _ptr(out), ctypes.byref(shape), _stream(stream))
    _check(rc, "oal_dense_ref_gpu")
    return out


def contribution_stat(q, k, out=None, stream=None):
    """oal_contribution_stat: eq. (1)'s chi per prompt (b, query head) and dimension, [B, Hq, 64]
    fp32; the page's chi_r is its mean over b."""
    if q.dim() != 4 or k.dim() != 4 or k.dtype != q.dtype:
        raise ValueError("q [B, Hq, T, d] and k [B, Hkv, T, d] of one dtype expected")
    B, Hq, T, d = q.shape
    shape = make_shape(B, T, Hq, k.shape[1], 128, _dtype_code(q), d)
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    _contig_cuda(q, k, out)
    rc = lib().oal_contribution_stat(_ptr(q), _ptr(k), _ptr(out), ctypes.byref(shape),
                                     _stream(stream))
    _check(rc, "oal_contribution_stat")
    return out


def device_error(stream=None) -> int:
    """Reads and clears the device-side error word (0 = none)."""
    code = ctypes.c_int(0)
    _check(lib().oal_device_error(ctypes.byref(code), _stream(stream)), "oal_device_error")
    return code.value


def host_prefill_buffers(q, k, v, group_id, L, G, chunk: int = 128, segments: int = 4,
                         device="cuda") -> dict:
    """Device memory and copy streams for prefill_from_host: group ids, L and G copied once,
    the state, the oal_prefill_host workspace, and two copy streams."""
    shape = _shape_of(q, k, v, chunk)
    n = _SZ(0)
    _check(lib().oal_prefill_host_workspace_bytes(ctypes.byref(shape), int(segments),
                                                  ctypes.byref(n)),
           "oal_prefill_host_workspace_bytes")
    return dict(
        g=group_id.to(device=device, dtype=torch.int32).contiguous(),
        L=L.to(device=device, dtype=torch.float32).contiguous(),
        G=G.to(device=device, dtype=torch.int32).contiguous(),
        state=torch.empty(state_bytes(shape), dtype=torch.uint8, device=device),
        ws=empty_workspace(n.value, device), chunk=int(chunk), segments=int(segments),
        copy_in=torch.cuda.Stream(device=device), copy_out=torch.cuda.Stream(device=device))


def prefill_from_host(q, k, v, eps: float, bufs: dict, out_host=None, stream=None):
    """oal_prefill_host: q/k/v in (pinned) host memory, yhat back into host memory, with the
    copies of one segment overlapped with the kernels of the next.  ``bufs`` comes from
    host_prefill_buffers; the state ends in bufs["state"].  Returns the host output tensor,
    valid once ``stream`` (default: the current stream) is synchronised."""
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous host tensors")
    shape = _shape_of(q, k, v, bufs["chunk"])
    if out_host is None:
        out_host = torch.empty(q.shape[0], q.shape[1], q.shape[2], v.shape[3],
                               dtype=torch.float32, pin_memory=True)
    ws = bufs["ws"]
    rc = lib().oal_prefill_host(_ptr(q), _ptr(k), _ptr(v), _ptr(bufs["g"]), _ptr(bufs["L"]),
                                _ptr(bufs["G"]), float(eps), _ptr(out_host),
                                _ptr(bufs["state"]), _ptr(ws), ws.numel() * ws.element_size(),
                                ctypes.byref(shape), bufs["segments"], _stream(stream),
                                ctypes.c_void_p(bufs["copy_in"].cuda_stream),
                                ctypes.c_void_p(bufs["copy_out"].cuda_stream))
    _check(rc, "oal_prefill_host")
    return out_host


def _hadamard_coefs(q, a, b, C):
    Hq = q.shape[1]
    a, b, C = (t.to(device=q.device, dtype=torch.float32).contiguous() for t in (a, b, C))
    if a.shape != (Hq,) or b.shape != (Hq, HEAD_DIM) or C.shape != (Hq, HEAD_DIM, HEAD_DIM):
        raise ValueError("a [Hq], b [Hq, 64], C [Hq, 64, 64] expected")
    return a, b, C


def prefill_hadamard(q, k, v, a, b, C, chunk: int = 128, out=None, state=None, workspace=None,
                     stream=None):
    """oal_prefill_hadamard: causal prefill with kappa = a + b.x + x^T C x, x = q*k/sqrt(64)
    (per query head a [Hq], b [Hq, 64], C [Hq, 64, 64]).  bf16 with chunk 128 (the default,
    as for prefill) runs on tensor cores.  Returns (out, state); the state continues with
    decode_step."""
    shape = _shape_of(q, k, v, chunk)
    dev = q.device
    a, b, C = _hadamard_coefs(q, a, b, C)
    if out is None:
        out = torch.empty(q.shape[0], q.shape[1], q.shape[2], v.shape[3], dtype=torch.float32,
                          device=dev)
    if state is None:
        state = torch.empty(state_bytes(shape), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = empty_workspace(prefill_workspace_bytes(shape), dev)
    _contig_cuda(q, k, v, a, b, C, out, state, workspace)
    rc = lib().oal_prefill_hadamard(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(C),
                                    _ptr(out), _ptr(state), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    ctypes.byref(shape), _stream(stream))
    _check(rc, "oal_prefill_hadamard")
    return out, state


def dense_hadamard(q, k, v, a, b, C, out=None, stream=None):
    """oal_dense_hadamard_gpu: the O(T^2) causal form of the same kernel."""
    shape = _shape_of(q, k, v, 64)
    a, b, C = _hadamard_coefs(q, a, b, C)
    if out is None:
        out = torch.empty(q.shape[0], q.shape[1], q.shape[2], v.shape[3], dtype=torch.float32,
                          device=q.device)
    _contig_cuda(q, k, v, a, b, C, out)
    rc = lib().oal_dense_hadamard_gpu(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(C),
                                      _ptr(out), ctypes.byref(shape), _stream(stream))
    _check(rc, "oal_dense_hadamard_gpu")
    return out


def prefill_varlen(qs, ks, vs, group_id, L, G, eps: float, chunk: int = 128, streams=None,
                   states=None, workspace=None):
    """oal_prefill_varlen over a list of sequences: qs[i] [Hq, T_i, 64], ks[i] / vs[i]
    [Hkv, T_i, 64] (same dtype and device).  The blocks are packed back to back into one
    buffer per tensor (the layout the call reads).  Returns (outs, states): outs[i] [Hq, T_i,
    64] fp32, states [n, stride] uint8 with row i the state of sequence i (continue it with
    decode_step).  ``streams`` (torch streams) run sequences side by side; default: the
    current stream alone."""
    n = len(qs)
    if not (len(ks) == len(vs) == n) or n == 0:
        raise ValueError("qs, ks, vs: equal, non-zero numbers of sequences")
    seq = [int(t.shape[1]) for t in qs]
    Hq, Hkv, dev = qs[0].shape[0], ks[0].shape[0], qs[0].device
    pack = lambda ts: torch.cat([t.contiguous().reshape(-1) for t in ts])  # noqa: E731
    q, k, v = pack(qs), pack(ks), pack(vs)
    shape = make_shape(1, max(seq), Hq, Hkv, chunk, _dtype_code(q), qs[0].shape[-1],
                       vs[0].shape[-1])
    lens = (ctypes.c_int32 * n)(*seq)
    if streams is None:
        streams = [torch.cuda.current_stream(dev)]
    handles = (ctypes.c_void_p * len(streams))(*[st.cuda_stream for st in streams])
    nb = _SZ(0)
    _check(lib().oal_prefill_varlen_workspace_bytes(ctypes.byref(shape), lens, n, len(streams),
                                                    ctypes.byref(nb)),
           "oal_prefill_varlen_workspace_bytes")
    stride = (state_bytes(make_shape(1, 1, Hq, Hkv, chunk, _dtype_code(q))) + 255) // 256 * 256
    out = torch.empty(Hq * sum(seq) * vs[0].shape[-1], dtype=torch.float32, device=dev)
    if states is None:
        states = torch.empty(n, stride, dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = empty_workspace(nb.value, dev)
    _contig_cuda(q, k, v, group_id, L, G, out, states, workspace)
    cur = torch.cuda.current_stream(dev)
    streams[0].wait_stream(cur)  # the packed inputs were written on the current stream
    rc = lib().oal_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(group_id), _ptr(L), _ptr(G),
                                  float(eps), _ptr(out), _ptr(states), stride, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  ctypes.byref(shape), lens, n, handles, len(streams))
    _check(rc, "oal_prefill_varlen")
    cur.wait_stream(streams[0])  # streams[0] already waits for every other stream
    outs, off = [], 0
    for t in seq:
        outs.append(out[off * Hq * 64:(off + t) * Hq * 64].view(Hq, t, 64))
        off += t
    return outs, states


def pack_sequences(qs, ks, vs):
    """The packed layout of a variable-length batch: qs[i] [Hq, T_i, 64], ks[i] / vs[i]
    [Hkv, T_i, 64] concatenated block after block into flat q, k, v; returns (q, k, v, lens)."""
    n = len(qs)
    if not (len(ks) == len(vs) == n) or n == 0:
        raise ValueError("qs, ks, vs: equal, non-zero numbers of sequences")
    pack = lambda ts: torch.cat([t.contiguous().reshape(-1) for t in ts])  # noqa: E731
    return pack(qs), pack(ks), pack(vs), [int(t.shape[1]) for t in qs]


def prefill_packed(q, k, v, lens, Hq: int, Hkv: int, group_id, L, G, eps: float, out=None,
                   states=None, workspace=None, stream=None):
    """oal_prefill_packed: the variable-length batch (packed as pack_sequences lays it out)
    in one launch per tensor-core kernel.  bf16 only (chunk 128).  Returns (out, states):
    out flat fp32 [Hq * sum(lens) * 64] (sequence i's [Hq, T_i, 64] block after the blocks
    before it), states [n, stride] uint8."""
    n = len(lens)
    dev = q.device
    shape = make_shape(1, max(lens) if n else 0, Hq, Hkv, 128, _dtype_code(q))
    c_lens = (ctypes.c_int32 * max(n, 1))(*lens)
    nb = _SZ(0)
    _check(lib().oal_prefill_packed_workspace_bytes(ctypes.byref(shape), c_lens, n,
                                                    ctypes.byref(nb)),
           "oal_prefill_packed_workspace_bytes")
    stride = (state_bytes(make_shape(1, 1, Hq, Hkv, 128, _dtype_code(q))) + 255) // 256 * 256
    if out is None:
        out = torch.empty(Hq * sum(lens) * 64, dtype=torch.float32, device=dev)
    if states is None:
        states = torch.empty(n, stride, dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = empty_workspace(nb.value, dev)
    _contig_cuda(q, k, v, group_id, L, G, out, states, workspace)
    rc = lib().oal_prefill_packed(_ptr(q), _ptr(k), _ptr(v), _ptr(group_id), _ptr(L), _ptr(G),
                                  float(eps), _ptr(out), _ptr(states), stride, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  ctypes.byref(shape), c_lens, n, _stream(stream))
    _check(rc, "oal_prefill_packed")
    return out, states


def backward(q, k, v, group_id, L, G, eps: float, dy, stream=None, workspace=None) -> dict:
    """oal_backward: the training-scale (chunked, O(T)) gradients for dy = dLoss/dyhat
    [B, Hq, T, 64] fp32.  Returns dict(dq, dk, dv, dL, deps) of fp32 device tensors."""
    return _backward("oal_backward", q, k, v, group_id, L, G, eps, dy, stream, workspace)


def dense_backward(q, k, v, group_id, L, G, eps: float, dy, stream=None) -> dict:
    """oal_dense_backward_gpu: gradients of the dense causal form for dy = dLoss/dyhat
    [B, Hq, T, 64] fp32.  Returns dict(dq, dk, dv, dL, deps) of fp32 device tensors."""
    return _backward("oal_dense_backward_gpu", q, k, v, group_id, L, G, eps, dy, stream, None)


def _backward(name, q, k, v, group_id, L, G, eps, dy, stream, ws) -> dict:
    shape = _shape_of(q, k, v, 64)
    dev = q.device
    dy = dy.to(device=dev, dtype=torch.float32).contiguous()
    dq = torch.empty(q.shape, dtype=torch.float32, device=dev)
    dk = torch.empty(k.shape, dtype=torch.float32, device=dev)
    dv_ = torch.empty(v.shape, dtype=torch.float32, device=dev)
    dL = torch.empty(L.shape, dtype=torch.float32, device=dev)
    deps = torch.empty(4, dtype=torch.float32, device=dev)
    if ws is None:
        n = _SZ(0)
        query = "oal_backward_workspace_bytes" if name == "oal_backward" else \
            "oal_dense_backward_workspace_bytes"
        _check(getattr(lib(), query)(ctypes.byref(shape), ctypes.byref(n)), query)
        ws = empty_workspace(n.value, dev)
    _contig_cuda(q, k, v, group_id, L, G, dy, dq, dk, dv_, dL, deps, ws)
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(group_id), _ptr(L), _ptr(G),
                              float(eps), _ptr(dy), _ptr(dq), _ptr(dk), _ptr(dv_), _ptr(dL),
                              _ptr(deps), _ptr(ws), ws.numel() * ws.element_size(),
                              ctypes.byref(shape), _stream(stream))
    _check(rc, name)
    return dict(dq=dq, dk=dk, dv=dv_, dL=dL, deps=deps[0])


def backward_workspace(q, k, v) -> torch.Tensor:
    """A workspace for backward() on inputs of these shapes (reusable across calls)."""
    n = _SZ(0)
    _check(lib().oal_backward_workspace_bytes(ctypes.byref(_shape_of(q, k, v, 64)),
                                              ctypes.byref(n)), "oal_backward_workspace_bytes")
    return empty_workspace(n.value, q.device)


class _There:
    """Another device or stream than the current ones, which become current inside."""

    def __init__(self, device, stream):
        self.ctx = [torch.cuda.device(device)]
        if stream is not None:
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


def _call_on_stream(f):
    """Lets the calls below run on the current stream of the device of their first argument: a
    call for another device or stream makes those current around itself, so that the tensors it
    makes belong to that stream, and their memory is not handed out again before the call's
    kernels are done with it."""
    first = f.__code__.co_varnames[0]

    @functools.wraps(f)
    def call(*args, stream=None, **kwargs):
        x = args[0] if args else kwargs[first]
        index = x.get_device()
        if index < 0:
            raise ValueError("tensors must be contiguous CUDA tensors")
        torch_c = torch._C  # (a torch without CUDA lacks the two functions)
        if stream is None and index == torch_c._cuda_getDevice():
            return f(*args, stream=torch_c._cuda_getCurrentRawStream(index), **kwargs)
        if stream is not None and stream.device != x.device:
            raise ValueError(f"the stream must be one of {x.device}, got one of {stream.device}")
        with _There(x.device, stream):
            return f(*args, stream=torch_c._cuda_getCurrentRawStream(index), **kwargs)
    return call


def _need(name, t, shape, dtype, index):
    """Pointer of a contiguous tensor of this shape and type on CUDA device `index`; refuses any
    other."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be a contiguous CUDA tensor on cuda:{index}")


def _need_ws(ws, index):
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{index}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


_CODE = {torch.bfloat16: OAL_BF16, torch.float32: OAL_F32}


_F32 = torch.float32


def _same(index, dt, *ts):
    """Whether the tensors are contiguous, of type dt and on CUDA device `index`: one pass over
    what a call's arguments have in common (a call of one token takes a few microseconds)."""
    for t in ts:
        if t.dtype is not dt or t.get_device() != index or not t.is_contiguous():
            return False
    return True


def _decay_args(q, k, v, log_decay, lens):
    """(shape, sizes, the pointers of q, k, v, log_decay, lens) of a decayed linear attention
    call; sizes: of q, of k and v, of the state."""
    qs, kv = q.shape, k.shape
    if len(qs) != 4 or len(kv) != 4:
        raise ValueError("q, k, v must be [B, H, T, 64]")
    dt, index = q.dtype, q.get_device()
    B, Hq, T, d = qs
    Hkv = kv[1]
    if not (_same(index, dt, q, k, v) and kv == v.shape and kv == (B, Hkv, T, d) and
            log_decay.shape == (Hkv,) and _same(index, _F32, log_decay)):
        kv = (B, Hkv, T, d)
        _need("q", q, qs, dt, index)
        _need("k", k, kv, dt, index)
        _need("v", v, kv, dt, index)
        _need("log_decay", log_decay, (Hkv,), _F32, index)
    shape = Shape(B, T, Hq, Hkv, d, d, 128, _CODE[dt] if dt in _CODE else _dtype_code(q))
    return shape, (qs, kv, (B, Hkv, 64, 64), dt, index), (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
        None if lens is None else _need("lens", lens, (B,), torch.int32, index))


def _bytes_of(query, shape) -> int:
    n = _SZ(0)
    _check(getattr(lib(), query)(ctypes.byref(shape), ctypes.byref(n)), query)
    return n.value


def decay_prefill_workspace(q, k, v) -> torch.Tensor:
    """A workspace for decay_prefill and decay_prefill_continue on inputs of these shapes."""
    shape = _shape_of(q, k, v, 128)
    return empty_workspace(_bytes_of("oal_decay_prefill_workspace_bytes", shape), q.device)


def decay_backward_workspace(q, k, v) -> torch.Tensor:
    """A workspace for decay_backward on inputs of these shapes."""
    shape = _shape_of(q, k, v, 128)
    return empty_workspace(_bytes_of("oal_decay_backward_workspace_bytes", shape), q.device)


def _decay_prefill(name, q, k, v, log_decay, scale, lens, out, state, want_out, workspace, stream):
    shape, (qs, _, ss, dt, index), (pq, pk, pv, pg, pl) = _decay_args(q, k, v, log_decay, lens)
    if not want_out:
        out = po = None
    else:
        if out is None:
            # rows behind a sequence's end are not written
            out = torch.empty_like(q) if lens is None else torch.zeros_like(q)
        po = _need("out", out, qs, dt, index)
    if state is None:
        state = q.new_empty(ss, dtype=_F32)
        ps = state.data_ptr()
    else:
        ps = _need("state", state, ss, _F32, index)
    if workspace is None:
        workspace = empty_workspace(_bytes_of("oal_decay_prefill_workspace_bytes", shape), q.device)
    pw, nw = _need_ws(workspace, index)
    rc = getattr(lib(), name)(pq, pk, pv, pg, scale, pl, po, ps, pw, nw, ctypes.byref(shape), stream)
    if rc:
        raise OALError(rc, name)
    return out, state


@_call_on_stream
def decay_prefill(q, k, v, log_decay, scale: float, lens=None, out=None, state=None,
                  want_out: bool = True, workspace=None, stream=None):
    """oal_decay_prefill: linear attention with decay exp(log_decay[kv head]) over prompts
    q [B, Hq, T, 64], k and v [B, Hkv, T, 64] (bf16 or fp32), scores times `scale`; lens [B]
    int32: the tokens of each sequence of a padded batch.  Returns (out like q, state
    [B, Hkv, 64, 64] fp32); want_out=False computes the state alone (out is None)."""
    return _decay_prefill("oal_decay_prefill", q, k, v, log_decay, scale, lens, out, state,
                          want_out, workspace, stream)


@_call_on_stream
def decay_prefill_continue(q, k, v, log_decay, scale: float, state, lens=None, out=None,
                           want_out: bool = True, workspace=None, stream=None):
    """oal_decay_prefill_continue: the same from `state`, which is updated; returns out."""
    if state is None:
        raise ValueError("decay_prefill_continue needs the state to continue from")
    return _decay_prefill("oal_decay_prefill_continue", q, k, v, log_decay, scale, lens, out,
                          state, want_out, workspace, stream)[0]


@_call_on_stream
def decay_step(q, k, v, log_decay, scale: float, state, src=None, parents=None, out=None,
               stream=None):
    """oal_decay_step: one token, q [B, Hq, 1, 64], k and v [B, Hkv, 1, 64]; `state` is updated
    in place, or with src [B', Hkv, 64, 64] and parents (int32, B of them) becomes the state of
    the parents one token on.  Returns out like q."""
    shape, (qs, _, ss, dt, index), (pq, pk, pv, pg, _) = _decay_args(q, k, v, log_decay, None)
    if qs[2] != 1:
        raise ValueError("decay_step takes one token: q, k, v [B, H, 1, 64]")
    ps = _need("state", state, ss, torch.float32, index)
    psrc = ppar = None
    n = 0
    if src is not None or parents is not None:
        if src is None or parents is None:
            raise ValueError("src and parents go together")
        n = src.shape[0]
        psrc = _need("src", src, (n, *ss[1:]), torch.float32, index)
        ppar = _parents(parents, qs[0], index)
    if out is None:
        out = torch.empty_like(q)
        po = out.data_ptr()
    else:
        po = _need("out", out, qs, dt, index)
    rc = lib().oal_decay_step(pq, pk, pv, pg, scale, psrc, n, ppar, ps, po, ctypes.byref(shape),
                              stream)
    if rc:
        raise OALError(rc, "oal_decay_step")
    return out


@_call_on_stream
def decay_backward(q, k, v, log_decay, scale: float, dout, lens=None, state=None, dlast=None,
                   grads=None, dstate=None, workspace=None, stream=None) -> dict:
    """oal_decay_backward: gradients of decay_prefill (state=None) or decay_prefill_continue
    (`state`: the one it started from) for dout like q and dlast = dLoss/d(last state) or None.
    `grads`: (dq, dk, dv) to write to.  Returns dict(dq, dk, dv, dstate)."""
    shape, (qs, kv, ss, dt, index), (pq, pk, pv, pg, pl) = _decay_args(q, k, v, log_decay, lens)
    f32 = torch.float32
    if grads is None:
        # rows behind a sequence's end are not written
        make = torch.empty_like if lens is None else torch.zeros_like
        grads = make(q), make(k), make(v)
    if dstate is None:
        dstate = torch.empty(ss, dtype=f32, device=q.device)
    if workspace is None:
        workspace = empty_workspace(_bytes_of("oal_decay_backward_workspace_bytes", shape), q.device)
    dq, dk, dv = grads
    pw, nw = _need_ws(workspace, index)
    rc = lib().oal_decay_backward(
        pq, pk, pv, pg, scale, pl, _need("dout", dout, qs, dt, index),
        None if state is None else _need("state", state, ss, f32, index),
        None if dlast is None else _need("dlast", dlast, ss, f32, index),
        _need("dq", dq, qs, dt, index), _need("dk", dk, kv, dt, index),
        _need("dv", dv, kv, dt, index), _need("dstate", dstate, ss, f32, index), pw, nw,
        ctypes.byref(shape), stream)
    if rc:
        raise OALError(rc, "oal_decay_backward")
    return dict(dq=dq, dk=dk, dv=dv, dstate=dstate)


def _parents(parents, B, index):
    """Pointer of `parents`, int32, B of them in any shape ([B] or [searches, beams])."""
    if parents.numel() != B:
        raise ValueError(f"parents must hold {B} indices, got {parents.numel()}")
    return _need("parents", parents, parents.shape, torch.int32, index)


def beam_select_workspace(B, beams, V, n, device) -> torch.Tensor:
    """A workspace for beam_select of these sizes, for either type of logits."""
    need = max(_select_bytes(B, beams, V, n, code) for code in (OAL_F32, OAL_BF16))
    return empty_workspace(need, device)


def _select_bytes(B, beams, V, n, code) -> int:
    nb = _SZ(0)
    _check(lib().oal_beam_select_workspace_bytes(B, beams, V, n, code, ctypes.byref(nb)),
           "oal_beam_select_workspace_bytes")
    return nb.value


@_call_on_stream
def beam_select(logits, running, n: int, ended=None, pad_token: int = 0, scores=None,
                parents=None, tokens=None, workspace=None, stream=None):
    """oal_beam_select: of logits [B, beams, V] (bf16 or fp32; rows may lie further apart than V)
    and running scores [B, beams] fp32, the n best candidates running + log_softmax of each
    search; ended [B, beams] uint8 or bool marks rows that go on with pad_token alone.  Returns
    (scores [B, n] fp32, parents [B, n] int32 rows of the B * beams, tokens [B, n] int32)."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, beams, V]")
    B, beams, V = logits.shape
    index = logits.get_device()
    if logits.is_contiguous():
        ld = V
    else:
        ld = logits.stride(1) if beams > 1 else (logits.stride(0) if B > 1 else V)
        if (V > 1 and logits.stride(2) != 1) or ld < V or (B > 1 and logits.stride(0) != beams * ld):
            raise ValueError("logits' rows must be contiguous and equally spaced")
    if ended is not None and ended.dtype is torch.bool:
        ended = ended.view(torch.uint8)
    dt = logits.dtype
    code = _CODE[dt] if dt in _CODE else _dtype_code(logits)
    rows, best, i32 = (B, beams), (B, n), torch.int32
    if scores is None and parents is None and tokens is None:
        parents, tokens, scores = running.new_empty((3, B, n), dtype=i32).unbind(0)
        scores = scores.view(_F32)
        ps, pp, pt = scores.data_ptr(), parents.data_ptr(), tokens.data_ptr()
    else:
        scores = running.new_empty(best, dtype=_F32) if scores is None else scores
        parents = running.new_empty(best, dtype=i32) if parents is None else parents
        tokens = running.new_empty(best, dtype=i32) if tokens is None else tokens
        ps, pp, pt = (_need("scores", scores, best, _F32, index),
                      _need("parents", parents, best, i32, index),
                      _need("tokens", tokens, best, i32, index))
    if workspace is None:
        workspace = empty_workspace(_select_bytes(B, beams, V, n, code), logits.device)
    pw, nw = _need_ws(workspace, index)
    rc = lib().oal_beam_select(
        logits.data_ptr(), ld, code, _need("running", running, rows, _F32, index),
        None if ended is None else _need("ended", ended, rows, torch.uint8, index), pad_token, B,
        beams, V, n, ps, pp, pt, pw, nw, stream)
    if rc:
        raise OALError(rc, "oal_beam_select")
    return scores, parents, tokens


def _state_of(name, t, B, Hq, Hkv, index):
    """(pointer, sequences) of a state buffer (uint8) with room for B sequences at least."""
    if t.dtype is not torch.uint8 or t.dim() != 1:
        raise TypeError(f"{name} must be a state buffer (uint8, one dimension)")
    if Hq < 1 or Hkv < 1:
        raise ValueError(f"Hq and Hkv must be at least 1, got {Hq} and {Hkv}")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on cuda:{index}")
    # the layout of oal_state_bytes: header and coefficient tables, then the sequences
    held = (t.numel() - 256 - Hq * FEATURES_PAD * 4) // (Hkv * FEATURES_PAD * (VALUE_DIM + 1) * 4)
    if held < B:
        raise ValueError(f"{name} holds {t.numel()} bytes, too few for its sequences")
    return t.data_ptr(), held


@_call_on_stream
def state_reorder(src, parents, dst, Hq: int, Hkv: int, stream=None):
    """oal_state_reorder: sequence i of the state buffer dst becomes sequence parents[i] (int32)
    of the state buffer src; dst has as many sequences as there are parents.  Returns dst."""
    index, B = src.get_device(), parents.numel()
    psrc, n = _state_of("src", src, 1, Hq, Hkv, index)
    pdst, _ = _state_of("dst", dst, B, Hq, Hkv, index)
    shape = Shape(B, 1, Hq, Hkv, 64, 64, 128, OAL_BF16)
    rc = lib().oal_state_reorder(psrc, n, _parents(parents, B, index), pdst, ctypes.byref(shape),
                                 stream)
    if rc:
        raise OALError(rc, "oal_state_reorder")
    return dst


@_call_on_stream
def decay_state_reorder(src, parents, dst, stream=None):
    """oal_decay_state_reorder: dst[i] = src[parents[i]] for states [B, Hkv, 64, 64] fp32."""
    index, B, Hkv = src.get_device(), parents.numel(), src.shape[1]
    psrc = _need("src", src, (src.shape[0], Hkv, 64, 64), torch.float32, index)
    pdst = _need("dst", dst, (B, Hkv, 64, 64), torch.float32, index)
    shape = Shape(B, 1, Hkv, Hkv, 64, 64, 128, OAL_BF16)
    rc = lib().oal_decay_state_reorder(psrc, src.shape[0], _parents(parents, B, index), pdst,
                                       ctypes.byref(shape), stream)
    if rc:
        raise OALError(rc, "oal_decay_state_reorder")
    return dst


@_call_on_stream
def decode_step_beam(q, k, v, src, parents, dst, workspace, out=None, stream=None):
    """oal_decode_step_beam: a decode step of sequence i from sequence parents[i] (int32) of the
    state buffer src, into the state buffer dst; returns out [B, Hq, 1, 64] fp32."""
    if q.dim() != 4 or k.dim() != 4 or q.shape[2] != 1:
        raise ValueError("decode_step_beam takes one token: q, k, v [B, H, 1, 64]")
    dt, index, qs = q.dtype, q.get_device(), q.shape
    B, Hq, _, d = qs
    kv = k.shape
    Hkv = kv[1]
    if not (_same(index, dt, q, k, v) and kv == v.shape and kv == (B, Hkv, 1, d)):
        kv = (B, Hkv, 1, d)
        _need("q", q, qs, dt, index)
        _need("k", k, kv, dt, index)
        _need("v", v, kv, dt, index)
    shape = Shape(B, 1, Hq, Hkv, d, d, 128, _CODE[dt] if dt in _CODE else _dtype_code(q))
    psrc, n = _state_of("src", src, 1, Hq, Hkv, index)
    pdst, _ = _state_of("dst", dst, B, Hq, Hkv, index)
    pw, nw = _need_ws(workspace, index)
    if out is None:
        out = q.new_empty(qs, dtype=_F32)
        po = out.data_ptr()
    else:
        po = _need("out", out, qs, _F32, index)
    rc = lib().oal_decode_step_beam(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), psrc, n, _parents(parents, B, index), pdst, po, pw,
        nw, ctypes.byref(shape), stream)
    if rc:
        raise OALError(rc, "oal_decode_step_beam")
    return out


def launch_count() -> int:
    """Kernels launched by the library since it was loaded."""
    return int(lib().oal_launch_count())


def profile_enable(on: bool = True):
    _check(lib().oal_profile_enable(1 if on else 0), "oal_profile_enable")


def profile_read() -> dict:
    """{kernel name: (launches, total device ms)} since the previous read (waits for them)."""
    arr = (KernelStat * 64)()
    n = ctypes.c_int(0)
    _check(lib().oal_profile_read(arr, 64, ctypes.byref(n)), "oal_profile_read")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms))
            for i in range(n.value)}


def set_prefill_overlap(overlap: bool) -> bool:
    """Launch the tensor-core prefill's scan and readout kernels as programmatic dependents
    (True) or in plain stream order (False); returns the previous setting."""
    return bool(lib().oal_set_prefill_overlap(1 if overlap else 0))


def set_debug_skip_copies(on: bool) -> bool:
    """Test hook: while on, the tensor-core readout issues no copies, so its bounded waits run
    out and it reports OAL_ERR_TIMEOUT (see include/oal.h); returns the previous setting."""
    return bool(lib().oal_set_debug_skip_copies(1 if on else 0))

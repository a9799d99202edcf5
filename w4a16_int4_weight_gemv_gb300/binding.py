"""ctypes binding of libw4a16.so (declared in include/w4a16.h).

Argument marshalling only: each function checks tensor dtypes, shapes and
devices, passes raw pointers and the current CUDA stream to the C ABI, and
raises W4A16Error on a non-OK status.  Every step of the computation runs in
the library's CUDA kernels; there is no CPU fallback, and importing this
module fails if the library has not been built.

bf16 tensors may be passed as torch.bfloat16 or as their int16/uint16 bit
patterns.  Packed weights are int32 (bit patterns of the uint32 words).
"""
from __future__ import annotations

import collections
import ctypes
import enum
import importlib.util
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_DEFAULT_LIB = os.path.join(_HERE, "_build", "libw4a16.so")


class Status(enum.IntEnum):
    OK = 0
    ERR_NULL = 1
    ERR_SHAPE = 2
    ERR_ALIGN = 3
    ERR_UNSUPPORTED = 4
    ERR_WORKSPACE = 5
    ERR_CUDA = 6


DEVERR_EXPERT_ID = 0x1
DEVERR_RANGE = 0x4
DEVERR_TIMEOUT = 0x2
DEVERR_SLOT = 0x8
DEVERR_BLOCKS = 0x10
OUT_BF16 = 0
OUT_F32 = 1


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = Status(status)
        super().__init__("%s: %s (%s)" % (where, status_string(status), self.status.name))


def lib_path() -> str:
    return os.environ.get("W4A16_LIB", _DEFAULT_LIB)


_lib = None


def load_library():
    """Load libw4a16.so; raises if it is missing (build it with build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError("libw4a16.so not built (expected at %s); run "
                          "w4a16_int4_weight_gemv_gb300.build_ext.build()" % path)
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.w4a16_abi_version.restype = I32
    lib.w4a16_abi_version.argtypes = []
    lib.w4a16_status_string.restype = ctypes.c_char_p
    lib.w4a16_status_string.argtypes = [I32]
    lib.int4_pack.restype = I32
    lib.int4_pack.argtypes = [P, P, I64, I64, P]
    lib.int4_dequant.restype = I32
    lib.int4_dequant.argtypes = [P, P, P, P, I32, I64, I64, I64, P]
    lib.w4a16_gemv_workspace_bytes.restype = SZ
    lib.w4a16_gemv_workspace_bytes.argtypes = [I32, I64, I64, I64]
    lib.w4a16_gemv.restype = I32
    lib.w4a16_gemv.argtypes = [P, P, P, P, P, I32, I32, I64, I64, I64, P, SZ, P]
    lib.w4a16_gemv_ex.restype = I32
    lib.w4a16_gemv_ex.argtypes = [P, P, P, P, P, I32, I32, I64, I64, I64, ctypes.c_uint, P]
    lib.w4a16_gemv_variant.restype = I32
    lib.w4a16_gemv_variant.argtypes = [P, P, P, P, P, I32, I32, I64, I64, I64, I32, I32, P]
    lib.w4a16_gemv_plan.restype = I32
    lib.w4a16_gemv_plan.argtypes = [I32, I64, I64, I64] + [ctypes.POINTER(I32)] * 5
    lib.w4a16_moe_workspace_bytes.restype = SZ
    lib.w4a16_moe_workspace_bytes.argtypes = [I32, I32, I64, I32]
    lib.w4a16_moe_gemv.restype = I32
    lib.w4a16_moe_gemv.argtypes = [P, I32, P, P, P, P, P, P, I32, I32, I32, I64, I64, I64,
                                   P, SZ, P]
    lib.w4a16_moe_ffn_workspace_bytes.restype = SZ
    lib.w4a16_moe_ffn_workspace_bytes.argtypes = [I32, I32, I64, I64]
    lib.w4a16_moe_ffn.restype = I32
    lib.w4a16_moe_ffn.argtypes = [P] * 13 + [I32, I32, I32, I64, I64, I64, P, SZ, P]
    lib.w4a16_swiglu.restype = I32
    lib.w4a16_swiglu.argtypes = [P, P, I64, P, I64, I64, I64, P]
    lib.w4a16_host_memory_mapped.restype = I32
    lib.w4a16_host_memory_mapped.argtypes = [P]
    lib.w4a16_device_error.restype = I32
    lib.w4a16_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), I32, P]
    lib.w4a16_wait_selftest.restype = I32
    lib.w4a16_wait_selftest.argtypes = [ctypes.c_uint, I32, P]
    lib.int3_pack.restype = I32
    lib.int3_pack.argtypes = [P, P, I64, I64, P]
    lib.int3_dequant.restype = I32
    lib.int3_dequant.argtypes = [P, P, P, P, I32, I64, I64, I64, P]
    lib.w3a16_moe_ffn_workspace_bytes.restype = SZ
    lib.w3a16_moe_ffn_workspace_bytes.argtypes = [I32, I32, I64, I64]
    lib.w3a16_moe_ffn.restype = I32
    lib.w3a16_moe_ffn.argtypes = [P] * 13 + [I32, I32, I32, I64, I64, I64, P, SZ, P]
    lib.w4a16_moe_gemv_variant.restype = I32
    lib.w4a16_moe_gemv_variant.argtypes = [P, I32, P, P, P, P, P, P, I32, I32, I32, I64, I64, I64,
                                           I32, P, SZ, P]
    lib.w3a16_moe_gemv.restype = I32
    lib.w3a16_moe_gemv.argtypes = [P, I32, P, P, P, P, P, P, I32, I32, I32, I64, I64, I64, P]
    lib.w4a16_paged_map.restype = I32
    lib.w4a16_paged_map.argtypes = [P, P, I32, P, I64, I32, P, I64, P, I32, I64, P, P, I64, P, P, P, P]
    lib.w4a16_rope_append.restype = I32
    lib.w4a16_rope_append.argtypes = [P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, P, I64, P, P,
                                      I32, I32, I32, ctypes.c_uint, P, P, I64, P]
    lib.w4a16_paged_attention_workspace_bytes.restype = SZ
    lib.w4a16_paged_attention_workspace_bytes.argtypes = [I32, I32, I32]
    lib.w4a16_paged_attention.restype = I32
    lib.w4a16_paged_attention.argtypes = [P, I64, I64, P, P, I64, I32, P, I32, I32, ctypes.c_float, I32, P,
                                          I64, I64, P, P, SZ, P]
    lib.w4a16_scaled_append.restype = I32
    lib.w4a16_scaled_append.argtypes = lib.w4a16_rope_append.argtypes
    lib.w4a16_scaled_read.restype = I32
    lib.w4a16_scaled_read.argtypes = [P, P, I64, I32, P, P, I32, P, I64, I64, P, I64, I64, I32, I64, P]
    lib.w4a16_scaled_attention_workspace_bytes.restype = SZ
    lib.w4a16_scaled_attention_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.w4a16_scaled_attention.restype = I32
    lib.w4a16_scaled_attention.argtypes = [P, I64, I64, I64, P, P, I64, I32, P, I32, I32, I32, ctypes.c_float, I32, P,
                                           I64, I64, I64, P, P, SZ, P]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().w4a16_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise W4A16Error(rc, where)


# The current stream's handle for a device index, without building a Stream
# object (torch.cuda.current_stream() costs a few microseconds per call,
# which a decode loop pays on every GEMV).
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int = None):
    """Stream handle (an int) for a ctypes call: `stream`, or the current
    stream of `device` (the current device if None)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_current_stream is not None and device is not None and device >= 0:
        return _raw_current_stream(device)
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream, kept: bool = True, zero: bool = False) -> torch.Tensor:
    """Memory that a call on `stream` makes itself.  Where that is not the
    current stream, it is taken on `stream`: the allocator then hands it to
    nobody else before the call's kernels are done with it.  What the caller
    gets (kept) counts as used on the current stream too."""
    make = torch.zeros if zero else torch.empty
    if stream is not None:
        here = torch.cuda.current_stream(device)
        if stream.cuda_stream != here.cuda_stream:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
            with torch.cuda.stream(stream):
                t = make(shape, dtype=dtype, device=device)
            if kept:
                t.record_stream(here)
            return t
    return make(shape, dtype=dtype, device=device)


def _ptr(t: torch.Tensor):
    return t.data_ptr()


def _need(t: torch.Tensor, name: str, dtypes, shape=None):
    # fast path: one expression over the properties a valid argument has
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous()
            and (shape is None or t.shape == tuple(shape))):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


_BF16 = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (torch.bfloat16, torch.int16)
_U8 = (torch.uint8,)
_U32 = (torch.int32,) + ((torch.uint32,) if hasattr(torch, "uint32") else ())


def int4_pack(codes: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """codes uint8 [N, K] (0..15) -> packed int32 [N, K/8] (uint32 bit patterns)."""
    _need(codes, "codes", _U8)
    N, K = codes.shape
    if out is None:
        out = _empty((N, K // 8), torch.int32, codes.device, stream)
    _need(out, "out", _U32, (N, K // 8))
    _check(load_library().int4_pack(_ptr(codes), _ptr(out), N, K, _stream(stream, codes.get_device())),
           "int4_pack")
    return out


def int4_dequant(wq, scale, zero, g: int, out_dtype=torch.bfloat16, out=None, stream=None):
    """Packed weights -> W [N, K] = (code - zero) * scale, bf16 or fp32."""
    _need(wq, "wq", _U32)
    N, K8 = wq.shape
    K = K8 * 8
    _need(scale, "scale", _BF16, (N, K // g))
    _need(zero, "zero", _U8, (N, K // g))
    if out is None:
        out = _empty((N, K), out_dtype, wq.device, stream)
    _need(out, "out", (torch.bfloat16, torch.float32), (N, K))
    kind = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check(load_library().int4_dequant(_ptr(wq), _ptr(scale), _ptr(zero), _ptr(out), kind,
                                       N, K, g, _stream(stream, wq.get_device())), "int4_dequant")
    return out


def int3_pack(codes: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """codes uint8 [N, K] (0..7, K % 128 == 0) -> INT3 words int32 [N, 3K/32]
    (uint32 bit patterns; the format is stated in include/w4a16.h)."""
    _need(codes, "codes", _U8)
    N, K = codes.shape
    if out is None:
        out = _empty((N, 3 * K // 32), torch.int32, codes.device, stream)
    _need(out, "out", _U32, (N, 3 * K // 32))
    _check(load_library().int3_pack(_ptr(codes), _ptr(out), N, K, _stream(stream, codes.get_device())),
           "int3_pack")
    return out


def int3_dequant(wq3, scale, zero, g: int, out_dtype=torch.bfloat16, out=None, stream=None):
    """INT3 words [N, 3K/32] -> W [N, K] = (code - zero) * scale, bf16 or fp32."""
    _need(wq3, "wq3", _U32)
    N, W3 = wq3.shape
    K = W3 // 3 * 32
    _need(scale, "scale", _BF16, (N, K // g))
    _need(zero, "zero", _U8, (N, K // g))
    if out is None:
        out = _empty((N, K), out_dtype, wq3.device, stream)
    _need(out, "out", (torch.bfloat16, torch.float32), (N, K))
    kind = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check(load_library().int3_dequant(_ptr(wq3), _ptr(scale), _ptr(zero), _ptr(out), kind,
                                       N, K, g, _stream(stream, wq3.get_device())), "int3_dequant")
    return out


def w4a16_gemv_workspace_bytes(M: int, N: int, K: int, g: int) -> int:
    return int(load_library().w4a16_gemv_workspace_bytes(M, N, K, g))


def gemv_plan(M: int, N: int, K: int, g: int) -> dict:
    """The launch w4a16_gemv makes for this shape (kernel id, CTAs, threads,
    K split, shared memory)."""
    vals = [ctypes.c_int(0) for _ in range(5)]
    _check(load_library().w4a16_gemv_plan(M, N, K, g, *[ctypes.byref(v) for v in vals]),
           "w4a16_gemv_plan")
    keys = ("kernel_id", "ctas", "threads", "k_split", "smem_bytes")
    return {k: v.value for k, v in zip(keys, vals)}


FLAG_WEIGHTS_STATIC = 0x1
FLAG_SWIGLU_OUTPUT = 0x2
FLAG_NO_CLUSTER = 0x4


def _host_side(x, out) -> bool:
    return (isinstance(x, torch.Tensor) and not x.is_cuda) or \
        (isinstance(out, torch.Tensor) and not out.is_cuda)


# host addresses the library has confirmed kernels can use as they are
_mapped_host = set()


def _need_pinned(t, name, dtypes, shape=None):
    if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_pinned():
        raise ValueError("%s: a page-locked host tensor is needed here (with the other of "
                         "x/out on the host)" % name)
    if t.dtype not in dtypes or not t.is_contiguous() or (shape is not None and t.shape != tuple(shape)):
        raise ValueError("%s: dtype/shape/layout not accepted" % name)
    p = t.data_ptr()
    if p not in _mapped_host:
        if not load_library().w4a16_host_memory_mapped(p):
            raise ValueError("%s: this host memory is not mapped for the device" % name)
        _mapped_host.add(p)


def w4a16_gemv(x, wq, scale, zero, g: int, out=None, out_dtype=torch.bfloat16,
               kernel_id: int = 0, k_split: int = 0, weights_static: bool = False,
               swiglu_output: bool = False, no_cluster: bool = False, stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] . dequant(wq, scale, zero)^T.

    kernel_id 0 (default) lets the library choose; 1, 2, 3 or 4 force the
    CUDA-core, bf16 warp-MMA, tensor-core (tcgen05) or fp16 warp-MMA kernel
    (measurement and tests); k_split forces the K split (for kernel 4, the
    CTAs of a cluster).  weights_static declares that no
    kernel still running on the stream writes wq/scale/zero (resident
    weights), so their loads may start before that kernel completes; it
    goes with the library's own launch choice only (ValueError with a
    forced kernel_id or k_split).  swiglu_output: the rows of wq are gate and
    up rows interleaved in blocks of 8 (interleave_gate_up) and y is the
    bf16 [M, N/2] SwiGLU of the two products, formed in the kernel's
    epilogue (same restriction on forcing).  no_cluster: plan without a
    thread-block cluster where the shape allows (a launch that follows a
    different kernel starts sooner; same restriction on forcing).

    With M == 1, x and out may both be page-locked host tensors: the kernel
    reads x and writes y there directly (over NVLink-C2C on a Grace-Blackwell
    node), with no copies around the call; y is valid on the host once the
    stream has been synchronised."""
    _need(wq, "wq", _U32)
    N = wq.shape[0]
    K = wq.shape[1] * 8
    if _host_side(x, out):
        # page-locked host x / y: read and written by the kernel in place
        # (one token: the CUDA-core kernel, plain loads and stores)
        _need_pinned(x, "x", _BF16)
        M = x.shape[0]
        if M != 1 or kernel_id not in (0, 1) or swiglu_output:
            raise ValueError("page-locked host x/out: M == 1 and the CUDA-core kernel only "
                             "(no SwiGLU input)")
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype).pin_memory()
        _need_pinned(out, "out", (torch.bfloat16, torch.float32), (M, N))
        device = wq.get_device()
    else:
        _need(x, "x", _BF16)
        M = x.shape[0]
        NO = N // 2 if swiglu_output else N
        if out is None:
            out = _empty((M, NO), torch.bfloat16 if swiglu_output else out_dtype, x.device, stream)
        _need(out, "out", (torch.bfloat16, torch.float32), (M, NO))
        device = x.get_device()
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x shape %s does not match wq %s" % (tuple(x.shape), tuple(wq.shape)))
    _need(scale, "scale", _BF16, (N, K // g))
    _need(zero, "zero", _U8, (N, K // g))
    kind = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    flags = ((FLAG_WEIGHTS_STATIC if weights_static else 0) | (FLAG_SWIGLU_OUTPUT if swiglu_output else 0) |
             (FLAG_NO_CLUSTER if no_cluster else 0))
    if flags and (kernel_id or k_split):
        raise ValueError("weights_static, swiglu_output and no_cluster apply to the library's own "
                         "launch choice; they cannot be combined with kernel_id or k_split")
    lib = load_library()
    sh = _stream(stream, device)
    if flags:
        rc = lib.w4a16_gemv_ex(_ptr(x), _ptr(wq), _ptr(scale), _ptr(zero), _ptr(out), kind,
                               M, N, K, g, flags, sh)
    elif kernel_id == 0 and k_split == 0:
        rc = lib.w4a16_gemv(_ptr(x), _ptr(wq), _ptr(scale), _ptr(zero), _ptr(out), kind,
                            M, N, K, g, None, 0, sh)
    else:
        rc = lib.w4a16_gemv_variant(_ptr(x), _ptr(wq), _ptr(scale), _ptr(zero), _ptr(out),
                                    kind, M, N, K, g, kernel_id or (1 if M == 1 else 2),
                                    k_split, sh)
    _check(rc, "w4a16_gemv")
    return out


def w4a16_moe_workspace_bytes(M: int, topk: int, N: int, route: bool) -> int:
    return int(load_library().w4a16_moe_workspace_bytes(M, topk, N, int(bool(route))))


def w4a16_moe_gemv(x, expert_ids, wq, scale, zero, g: int, route_w=None, x_per_slot=False,
                   out=None, workspace=None, stream=None, kernel_id: int = 0) -> torch.Tensor:
    """Expert-indexed GEMV.  wq int32 [E, N, K/8]; scale/zero [E, N, K/g];
    expert_ids int32 [M, topk]; x [M, K] or (x_per_slot) [M, topk, K].
    Returns bf16 [M, topk, N] (no route_w) or [M, N] (routed sum).
    kernel_id: 0 the library's choice, 2 the bf16 warp-MMA expert kernel,
    4 the fp16 warp-MMA expert kernel (no workspace)."""
    _need(expert_ids, "expert_ids", (torch.int32,))
    M, topk = expert_ids.shape
    _need(wq, "wq", _U32)
    E, N, K8 = wq.shape
    K = K8 * 8
    _need(x, "x", _BF16, (M, topk, K) if x_per_slot else (M, K))
    _need(scale, "scale", _BF16, (E, N, K // g))
    _need(zero, "zero", _U8, (E, N, K // g))
    lib = load_library()
    if route_w is not None:
        _need(route_w, "route_w", (torch.float32,), (M, topk))
        shape = (M, N)
        need = w4a16_moe_workspace_bytes(M, topk, N, True) if kernel_id != 4 else 0
        if workspace is None and need > 0:
            workspace = _empty(need // 4, torch.float32, x.device, stream, kept=False)
        if workspace is None:
            ws_ptr, ws_bytes = None, 0
        else:
            ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        rw = _ptr(route_w)
    else:
        shape = (M, topk, N)
        ws_ptr, ws_bytes, rw = None, 0, None
    if out is None:
        out = _empty(shape, torch.bfloat16, x.device, stream)
    _need(out, "out", _BF16, shape)
    if kernel_id == 0:
        _check(lib.w4a16_moe_gemv(_ptr(x), int(bool(x_per_slot)), _ptr(expert_ids), rw, _ptr(wq),
                                  _ptr(scale), _ptr(zero), _ptr(out), M, topk, E, N, K, g,
                                  ws_ptr, ws_bytes, _stream(stream, x.get_device())),
               "w4a16_moe_gemv")
    else:
        _check(lib.w4a16_moe_gemv_variant(_ptr(x), int(bool(x_per_slot)), _ptr(expert_ids), rw,
                                          _ptr(wq), _ptr(scale), _ptr(zero), _ptr(out), M, topk,
                                          E, N, K, g, int(kernel_id), ws_ptr, ws_bytes,
                                          _stream(stream, x.get_device())),
               "w4a16_moe_gemv_variant")
    return out


def interleave_gate_up(gate, up) -> torch.Tensor:
    """The row layout W4A16_FLAG_SWIGLU_OUTPUT reads: two [I, ...] tensors
    (packed weights, scales or zero points of the gate and up matrices, I a
    multiple of 8) as one [2I, ...] tensor whose 16-row blocks hold 8 gate
    rows, then the same 8 up rows.  A one-time copy at weight-load time."""
    if gate.shape != up.shape or gate.dim() < 1 or gate.shape[0] % 8 != 0:
        raise ValueError("gate and up must have the same shape, rows a multiple of 8")
    rest = tuple(gate.shape[1:])
    blocks = torch.stack((gate.reshape((-1, 8) + rest), up.reshape((-1, 8) + rest)), dim=1)
    return blocks.reshape((2 * gate.shape[0],) + rest).contiguous()


def w4a16_swiglu(gate, up, out=None, stream=None) -> torch.Tensor:
    """h = bf16(silu(gate) * up).  gate/up may be views with a row stride
    (e.g. the two halves of a stacked [rows, 2N] tensor)."""
    for t, name in ((gate, "gate"), (up, "up")):
        if not t.is_cuda or t.dtype not in _BF16 or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("%s must be a CUDA bf16 matrix with unit column stride" % name)
    if gate.shape != up.shape or gate.stride(0) != up.stride(0):
        raise ValueError("gate and up must have the same shape and row stride")
    rows, N = gate.shape
    if out is None:
        out = _empty((rows, N), torch.bfloat16, gate.device, stream)
    if out.dim() != 2 or tuple(out.shape) != (rows, N) or out.stride(1) != 1:
        raise ValueError("out must be [rows, N] with unit column stride")
    _check(load_library().w4a16_swiglu(_ptr(gate), _ptr(up), gate.stride(0), _ptr(out),
                                       out.stride(0), rows, N, _stream(stream, gate.get_device())),
           "w4a16_swiglu")
    return out


def w4a16_device_error(clear: bool = True, stream=None) -> int:
    bits = ctypes.c_uint32(0)
    _check(load_library().w4a16_device_error(ctypes.byref(bits), int(bool(clear)),
                                             _stream(stream)), "w4a16_device_error")
    return int(bits.value)


def w4a16_wait_selftest(max_iters: int, arrive: bool, stream=None) -> None:
    """One bounded mbarrier wait that completes (arrive) or expires
    (W4A16_DEVERR_TIMEOUT in the device error word)."""
    _check(load_library().w4a16_wait_selftest(int(max_iters), int(bool(arrive)), _stream(stream)),
           "w4a16_wait_selftest")


def moe_ffn(x, expert_ids, route_w, gate, up, down, g: int, stream=None,
            fused: bool = True) -> torch.Tensor:
    """Routed SwiGLU FFN for M tokens.  gate/up/down are (wq, scale, zero)
    triples with gate/up [E, F, H] and down [E, H, F].  Returns bf16 [M, H].

    fused (default): w4a16_moe_ffn -- two launches: the gate and up products
    with the SwiGLU formed in their epilogue, then the down products and the
    routed sums (older expert kernels outside the fp16 path's limits).
    fused=False: the same chain from the single-purpose calls (one
    expert-indexed GEMV each for gate and up, w4a16_swiglu, the down GEMV
    with the routed sum)."""
    M, topk = expert_ids.shape
    if fused:
        _need(x, "x", _BF16)
        _need(expert_ids, "expert_ids", (torch.int32,))
        _need(route_w, "route_w", (torch.float32,), (M, topk))
        (gw, gs, gz), (uw, us, uz), (dw, ds, dz) = gate, up, down
        E, F, H8 = gw.shape
        H = H8 * 8
        y = _empty((M, H), torch.bfloat16, x.device, stream)
        lib = load_library()
        nbytes = int(lib.w4a16_moe_ffn_workspace_bytes(M, topk, H, F))
        ws = _empty(max(nbytes, 16), torch.uint8, x.device, stream, kept=False)
        _check(lib.w4a16_moe_ffn(_ptr(x), _ptr(expert_ids), _ptr(route_w), _ptr(gw), _ptr(gs),
                                 _ptr(gz), _ptr(uw), _ptr(us), _ptr(uz), _ptr(dw), _ptr(ds),
                                 _ptr(dz), _ptr(y), M, topk, E, H, F, g, _ptr(ws), nbytes,
                                 _stream(stream, x.get_device())), "w4a16_moe_ffn")
        return y
    g_out = w4a16_moe_gemv(x, expert_ids, *gate, g, stream=stream)
    u_out = w4a16_moe_gemv(x, expert_ids, *up, g, stream=stream)
    F = g_out.shape[-1]
    h = w4a16_swiglu(g_out.view(M * topk, F), u_out.view(M * topk, F), stream=stream)
    return w4a16_moe_gemv(h.view(M, topk, F), expert_ids, *down, g, route_w=route_w,
                          x_per_slot=True, stream=stream)


def w3a16_moe_ffn(x, expert_ids, route_w, gate, up, down, g: int, stream=None) -> torch.Tensor:
    """Routed SwiGLU FFN over INT3 (~3-bit) expert banks.  gate/up/down are
    (wq3, scale, zero) triples: gate/up wq3 [E, F, 3H/32], down [E, H, 3F/32],
    scale/zero as for INT4.  Returns bf16 [M, H]."""
    M, topk = expert_ids.shape
    _need(x, "x", _BF16)
    _need(expert_ids, "expert_ids", (torch.int32,))
    _need(route_w, "route_w", (torch.float32,), (M, topk))
    (gw, gs, gz), (uw, us, uz), (dw, ds, dz) = gate, up, down
    E, F, H3 = gw.shape
    H = H3 // 3 * 32
    y = _empty((M, H), torch.bfloat16, x.device, stream)
    lib = load_library()
    nbytes = int(lib.w3a16_moe_ffn_workspace_bytes(M, topk, H, F))
    ws = _empty(max(nbytes, 16), torch.uint8, x.device, stream, kept=False)
    _check(lib.w3a16_moe_ffn(_ptr(x), _ptr(expert_ids), _ptr(route_w), _ptr(gw), _ptr(gs),
                             _ptr(gz), _ptr(uw), _ptr(us), _ptr(uz), _ptr(dw), _ptr(ds),
                             _ptr(dz), _ptr(y), M, topk, E, H, F, g, _ptr(ws), nbytes,
                             _stream(stream, x.get_device())), "w3a16_moe_ffn")
    return y


def w3a16_moe_gemv(x, expert_ids, wq3, scale, zero, g: int, route_w=None, x_per_slot=False,
                   out=None, stream=None) -> torch.Tensor:
    """Expert-indexed GEMV over an INT3 (~3-bit) expert bank.  wq3 int32
    [E, N, 3K/32]; scale/zero [E, N, K/g]; expert_ids int32 [M, topk]; x
    [M, K] or (x_per_slot) [M, topk, K].  Returns bf16 [M, topk, N] (no
    route_w) or [M, N] (routed sum).  No workspace."""
    _need(expert_ids, "expert_ids", (torch.int32,))
    M, topk = expert_ids.shape
    _need(wq3, "wq3", _U32)
    E, N, K3 = wq3.shape
    if K3 % 12 != 0:
        raise ValueError("wq3 rows must hold whole 128-code blocks (12 words each)")
    K = K3 // 12 * 128
    _need(x, "x", _BF16, (M, topk, K) if x_per_slot else (M, K))
    _need(scale, "scale", _BF16, (E, N, K // g))
    _need(zero, "zero", _U8, (E, N, K // g))
    if route_w is not None:
        _need(route_w, "route_w", (torch.float32,), (M, topk))
        shape = (M, N)
    else:
        shape = (M, topk, N)
    if out is None:
        out = _empty(shape, torch.bfloat16, x.device, stream)
    _need(out, "out", _BF16, shape)
    _check(load_library().w3a16_moe_gemv(_ptr(x), int(bool(x_per_slot)), _ptr(expert_ids),
                                         None if route_w is None else _ptr(route_w), _ptr(wq3),
                                         _ptr(scale), _ptr(zero), _ptr(out), M, topk, E, N, K, g,
                                         _stream(stream, x.get_device())), "w3a16_moe_gemv")
    return out


# --------------------------------------------------------------------------
# paged key/value cache: block map, rotary + append, one-token attention
# --------------------------------------------------------------------------
def _on_device(device: int, **tensors):
    """A call's tensors are on one device: that of its first one, and of the cache."""
    for name, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise ValueError("%s is on device %s, expected cuda:%d" % (name, t.device, device))


class _KvCache(ctypes.Structure):
    """w4a16_kv_cache of include/w4a16.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("page", ctypes.c_int32), ("blocks", ctypes.c_int64),
                ("k_block", ctypes.c_int64), ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_block", ctypes.c_int64), ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64)]


CACHE_BF16 = 0
CACHE_E4M3 = 1
ROPE_INTERLEAVED = 0x1
ROPE_INVERSE = 0x2
_I32 = (torch.int32,)
_F32 = (torch.float32,)


class PagedCache:
    """Handle of one layer's paged key/value cache.

    k, v: CUDA tensors [blocks, page, heads, dim], bfloat16 or float8_e4m3fn,
    dim contiguous, the other strides free (a cache kept as [blocks, heads,
    page, dim] is passed as its permute(0, 2, 1, 3)); k_scale, v_scale:
    float32 [heads], needed with float8 (key = code * k_scale[head]).  The
    tensors stay the caller's; the handle holds references to them, so the
    memory it points at lives as long as it does."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch.Tensor" % name)
            if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
                raise ValueError("%s must be a CUDA tensor [blocks, page, heads, dim], dim contiguous" % name)
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or v.dtype != k.dtype:
            raise TypeError("k and v must both be bfloat16 or both float8_e4m3fn")
        if v.shape != k.shape or v.device != k.device:
            raise ValueError("k and v must have the same shape and device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.blocks, self.page, self.heads, self.dim = k.shape
        e4m3 = k.dtype == torch.float8_e4m3fn
        if e4m3:
            _need(k_scale, "k_scale", _F32, (self.heads,))
            _need(v_scale, "v_scale", _F32, (self.heads,))
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        self.device = k.get_device()
        if e4m3:
            _on_device(self.device, k_scale=k_scale, v_scale=v_scale)
        self._struct = _KvCache(_ptr(k), _ptr(v), _ptr(k_scale) if e4m3 else None,
                                _ptr(v_scale) if e4m3 else None, CACHE_E4M3 if e4m3 else CACHE_BF16,
                                self.heads, self.dim, self.page, self.blocks,
                                *k.stride()[:3], *v.stride()[:3])
        self._ref = ctypes.addressof(self._struct)


PagedMap = collections.namedtuple("PagedMap", "slots positions row_start kv_len free_head")


def paged_map_buffers(requests: int, tokens: int, device) -> PagedMap:
    """Output buffers of w4a16_paged_map, to be kept from step to step."""
    return _map_buffers(requests, tokens, device, None)


def _map_buffers(requests: int, tokens: int, device, stream) -> PagedMap:
    return PagedMap(*(_empty(n, torch.int32, device, stream) for n in (tokens, tokens, requests + 1, requests, 1)))


# The paged calls run once per layer and step, next to kernels of a few
# microseconds.  So an extension module (fastcall.cpp) looks at the arguments
# and makes the call; what it does not take -- arguments left out, bit patterns
# for bf16, anything that is wrong -- goes through the functions here, which
# check what a valid argument has in one expression, and only where that fails
# look into which one it was.
_fast = None


def _load_fast():
    import importlib.machinery
    from . import build_ext
    path = build_ext.fastcall_path()
    if path is None or not os.path.exists(path) or _raw_current_stream is None or not hasattr(torch._C, "_cuda_getDevice"):
        return None
    loader = importlib.machinery.ExtensionFileLoader("_fastcall", path)
    try:
        mod = importlib.util.module_from_spec(importlib.machinery.ModuleSpec("_fastcall", loader, origin=path))
        loader.exec_module(mod)
    except ImportError:
        return None
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    mod.bind(address(_lib.w4a16_paged_map), address(_lib.w4a16_rope_append), address(_lib.w4a16_paged_attention),
             address(_lib.w4a16_scaled_append), address(_lib.w4a16_scaled_read), address(_lib.w4a16_scaled_attention),
             _raw_current_stream, torch._C._cuda_getDevice)
    return mod


_int32 = torch.int32
_bf16 = torch.bfloat16


def _vector(t, name: str, n: int) -> int:
    """Address of an int32 vector of n entries."""
    try:
        if t.dtype is _int32 and t.is_cuda and t.shape == (n,) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, _I32, (n,))
    return t.data_ptr()


def _table(t, requests: int):
    """Address, row stride and columns of a block table."""
    try:
        rows, columns = t.shape
        stride, unit = t.stride()
        if t.dtype is _int32 and t.is_cuda and rows == requests and (unit == 1 or columns == 1):
            return t.data_ptr(), stride if rows > 1 else max(stride, columns), columns
    except (AttributeError, ValueError):
        pass
    raise ValueError("block_table must be a CUDA int32 [%d, columns] with unit column stride" % requests)


def w4a16_paged_map(ctx_len, new_len, block_table, free_blocks, free_head, page: int, num_blocks: int,
                    tokens: int, out: PagedMap = None, stream=None) -> PagedMap:
    """Block tables and slot maps from the lengths of the requests.

    ctx_len, new_len int32 [B]: tokens request b has cached and adds now;
    block_table int32 [B, columns] (a row stride is allowed): the entries of
    the blocks the new tokens begin are filled in place from free_blocks
    int32 [F], from entry free_head int32 [1] on; tokens: how many places the
    slots and positions have (at least the new tokens; the rest gets -1).
    Returns PagedMap(slots [tokens], positions [tokens], row_start [B + 1],
    kv_len [B], free_head [1]), all int32."""
    if _fast is not None and out is not None:
        rc = _fast.paged_map(ctx_len, new_len, block_table, free_blocks, free_head, page, num_blocks, tokens, out,
                             None if stream is None else stream.cuda_stream)
        if rc == 0:
            return out
        if rc is not None:
            raise W4A16Error(rc, "w4a16_paged_map")
    B = len(ctx_len)
    ctx, new = _vector(ctx_len, "ctx_len", B), _vector(new_len, "new_len", B)
    F = len(free_blocks)
    free, head = _vector(free_blocks, "free_blocks", F), _vector(free_head, "free_head", 1)
    table, stride, columns = _table(block_table, B)
    if out is None:
        out = _map_buffers(B, tokens, ctx_len.device, stream)
    else:
        for t, name, n in zip(out, PagedMap._fields, (tokens, tokens, B + 1, B, 1)):
            _need(t, name, _I32, (n,))
    slots, positions, row_start, kv_len, head_out = out
    device = ctx_len.get_device()
    _on_device(device, new_len=new_len, block_table=block_table, free_blocks=free_blocks, free_head=free_head)
    _on_device(device, **out._asdict())
    rc = _lib.w4a16_paged_map(ctx, new, B, table, stride, columns, free, F, head, page, num_blocks,
                              slots.data_ptr(), positions.data_ptr(), tokens, row_start.data_ptr(),
                              kv_len.data_ptr(), head_out.data_ptr(), _stream(stream, device))
    if rc:
        raise W4A16Error(rc, "w4a16_paged_map")
    return out


def _rows(t, name: str, shape):
    """Address, row and head strides of bf16 heads [rows, heads, dim], dim contiguous."""
    try:
        rows, heads, unit = t.stride()
        if (t.dtype is _bf16 or t.dtype in _BF16) and t.is_cuda and unit == 1 and t.shape == shape:
            return t.data_ptr(), rows, heads
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda or t.dtype not in _BF16 or t.dim() != 3 or t.stride(2) != 1:
        raise ValueError("%s must be a CUDA bf16 tensor [rows, heads, dim], dim contiguous" % name)
    raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _section_array(sections):
    """The sections as a C array."""
    return (ctypes.c_int32 * len(sections))(*map(operator.index, sections))


def w4a16_rope_append(q, k, v, positions, inv_freq, slots, cache: PagedCache, sections=None,
                      interleaved: bool = False, inverse: bool = False, q_out=None, stream=None):
    """Rotary positions on q and k, and k and v into the paged cache.

    q bf16 [T, q_heads, dim], k and v bf16 [T, heads, dim] (views with token
    and head strides, e.g. of a fused QKV output); positions int32 [T] or
    [axes, T]; inv_freq float32 [rotary / 2]; sections: how many pairs go by
    each axis; slots int32 [T], -1 for a token that is not stored.
    interleaved: pairs (2i, 2i + 1) instead of (i, i + rotary / 2); inverse
    turns back (the gradient).  q, or k, v, slots and cache together, may be
    None.  Returns the rotated queries (q_out, or a new tensor; q_out=q
    rotates in place)."""
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0)
    if _fast is not None and (q is None or q_out is not None) and (cache is not None or (k is None and v is None and slots is None)):
        rc = _fast.rope_append(q, k, v, positions, inv_freq, slots, None if cache is None else cache._ref,
                               0 if cache is None else cache.heads, 0 if cache is None else cache.device, sections, flags,
                               q_out, None if stream is None else stream.cuda_stream)
        if rc == 0:
            return q_out
        if rc is not None:
            raise W4A16Error(rc, "w4a16_rope_append")
    if q is not None:
        shape = q.shape
        T, heads, dim = shape if len(shape) == 3 else (0, 0, 0)
        qa = _rows(q, "q", shape)
        device = q.get_device()
        if q_out is None:
            q_out = _empty(shape, _bf16, q.device, stream)
        qo = _rows(q_out, "q_out", shape)
    else:
        T, heads, dim = k.shape[0], 0, k.shape[2]
        qa = qo = (None, 0, 0)
        device = k.get_device()
    if cache is not None:
        shape = (T, cache.heads, cache.dim)
        ka, va, slots_at, cache_at = _rows(k, "k", shape), _rows(v, "v", shape), _vector(slots, "slots", T), cache._ref
    else:
        if k is not None or v is not None or slots is not None:
            raise ValueError("k, v and slots go with a cache")
        ka, va, slots_at, cache_at = (None, 0, 0), (None, 0, 0), None, None
    if not (inv_freq.dtype is torch.float32 and inv_freq.is_cuda and inv_freq.is_contiguous()):
        _need(inv_freq, "inv_freq", _F32)
    if positions.dim() == 1:
        axes, axis_stride = 1, 0
        positions_at = _vector(positions, "positions", T)
    else:
        axes, axis_stride = positions.shape[0], T
        if not (positions.dtype is _int32 and positions.is_cuda and positions.is_contiguous() and positions.shape == (axes, T)):
            _need(positions, "positions", _I32, (axes, T))
        positions_at = positions.data_ptr()
    sec = None
    if sections is not None:
        if len(sections) != axes:
            raise ValueError("%d sections for %d axes" % (len(sections), axes))
        sec = _section_array(sections)
    _on_device(device if cache is None else cache.device, q=q, q_out=q_out, k=k, v=v, positions=positions, inv_freq=inv_freq,
               slots=slots)
    if T == 0:
        return q_out
    rc = _lib.w4a16_rope_append(*qa, *qo, heads, *ka, *va, positions_at, axis_stride, inv_freq.data_ptr(), sec, axes,
                                2 * inv_freq.numel(), dim, flags, slots_at, cache_at, T, _stream(stream, device))
    if rc:
        raise W4A16Error(rc, "w4a16_rope_append")
    return q_out


def paged_attention_workspace(cache: PagedCache, q_heads: int) -> torch.Tensor:
    """Workspace of w4a16_paged_attention for this cache and number of query
    heads (its contents need no initialisation)."""
    return _attention_workspace(cache, q_heads, None)


def _attention_workspace(cache: PagedCache, q_heads: int, stream) -> torch.Tensor:
    n = int(load_library().w4a16_paged_attention_workspace_bytes(q_heads, cache.heads, cache.dim))
    return _empty(max(n, 16), torch.uint8, cache.k.device, stream, kept=False)


def w4a16_paged_attention(q, cache: PagedCache, block_table, kv_len, scale: float = None, window: int = 0,
                          out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per request over the paged cache.

    q bf16 [B, q_heads, dim] (request and head strides allowed); block_table
    int32 [B, columns]; kv_len int32 [B], the tokens each request sees, the
    new one among them; window > 0: only the last `window` of them.  scale
    defaults to dim ** -0.5.  Returns (out bf16 [B, q_heads, dim], lse float32
    [B, q_heads]); a request of length 0 gets zeros and -infinity.
    workspace: from paged_attention_workspace, one per stream in use (None:
    a new one for this call)."""
    if scale is None:
        scale = cache.dim ** -0.5
    if _fast is not None and workspace is not None:
        rc = _fast.paged_attention(q, cache._ref, cache.dim, cache.device, block_table, kv_len, scale, window, out, lse, workspace,
                                   None if stream is None else stream.cuda_stream)
        if rc == 0:
            return out, lse
        if rc is not None:
            raise W4A16Error(rc, "w4a16_paged_attention")
    shape = q.shape
    B, H = shape[0], shape[1]
    qa = _rows(q, "q", (B, H, cache.dim))
    table, stride, columns = _table(block_table, B)
    lengths = _vector(kv_len, "kv_len", B)
    if out is None:
        out = _empty(shape, _bf16, q.device, stream)
    oa = _rows(out, "out", shape)
    if lse is None:
        lse = _empty((B, H), torch.float32, q.device, stream)
    elif not (lse.dtype is torch.float32 and lse.is_cuda and lse.shape == (B, H) and lse.is_contiguous()):
        _need(lse, "lse", _F32, (B, H))
    if workspace is None:
        workspace = _attention_workspace(cache, H, stream)
    elif not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _on_device(cache.device, q=q, block_table=block_table, kv_len=kv_len, out=out, lse=lse, workspace=workspace)
    rc = _lib.w4a16_paged_attention(*qa, cache._ref, table, stride, columns, lengths, B, H,
                                    scale, window, *oa, lse.data_ptr(),
                                    workspace.data_ptr(), workspace.nbytes, _stream(stream, q.get_device()))
    if rc:
        raise W4A16Error(rc, "w4a16_paged_attention")
    return out, lse


# --------------------------------------------------------------------------
# Paged cache in 8 bits, a scale for each group of tokens and head
# --------------------------------------------------------------------------
CACHE_INT8 = 2


class _ScaledCache(ctypes.Structure):
    """w4a16_scaled_cache of include/w4a16.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("group", ctypes.c_int32), ("blocks", ctypes.c_int64),
                ("k_block", ctypes.c_int64), ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_block", ctypes.c_int64), ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("ks_block", ctypes.c_int64), ("ks_group", ctypes.c_int64), ("ks_head", ctypes.c_int64),
                ("vs_block", ctypes.c_int64), ("vs_group", ctypes.c_int64), ("vs_head", ctypes.c_int64)]


class ScaledCache:
    """Handle of one layer's paged key/value cache in 8 bits with a scale for
    each group of tokens and head.

    k, v: CUDA tensors [blocks, page, heads, dim], int8 or float8_e4m3fn, dim
    contiguous, the other strides free; k_scale, v_scale: float32 [blocks, page //
    group, heads], any strides: key = code * k_scale of its group and head.
    w4a16_scaled_append finds the scales and writes codes and scales; neither
    needs initialisation.  The tensors stay the caller's; the handle holds
    references to them, so the memory it points at lives as long as it does."""

    def __init__(self, k, v, k_scale, v_scale):
        for t, name in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch.Tensor" % name)
            if not t.is_cuda:
                raise ValueError("%s must be a CUDA tensor" % name)
        for t, name in ((k, "k"), (v, "v")):
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError("%s must be [blocks, page, heads, dim], dim contiguous" % name)
        if k.dtype not in (torch.int8, torch.float8_e4m3fn) or v.dtype != k.dtype:
            raise TypeError("k and v must both be int8 or both float8_e4m3fn")
        if v.shape != k.shape:
            raise ValueError("k and v must have the same shape")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.blocks, self.page, self.heads, self.dim = k.shape
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype is not torch.float32:
                raise TypeError("%s has dtype %s, expected torch.float32" % (name, t.dtype))
            if t.dim() != 3 or t.shape != k_scale.shape or t.shape[0] != self.blocks or t.shape[2] != self.heads or t.shape[1] < 1 or self.page % t.shape[1]:
                raise ValueError("%s has shape %s, expected [%d, page // group, %d] for a page of %d"
                                 % (name, tuple(t.shape), self.blocks, self.heads, self.page))
        self.group = self.page // k_scale.shape[1]
        self.device = k.get_device()
        _on_device(self.device, v=v, k_scale=k_scale, v_scale=v_scale)
        self._struct = _ScaledCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), CACHE_INT8 if k.dtype is torch.int8 else CACHE_E4M3,
                                    self.heads, self.dim, self.page, self.group, self.blocks,
                                    *k.stride()[:3], *v.stride()[:3], *k_scale.stride(), *v_scale.stride())
        self._ref = ctypes.addressof(self._struct)


def _scaled(cache) -> ScaledCache:
    if not isinstance(cache, ScaledCache):
        raise TypeError("cache must be a ScaledCache")
    return cache


def _launch(device: int, entry, *args) -> int:
    """A C call whose tensors are on `device`, made with that as the current device."""
    with torch.cuda.device(device):
        return entry(*args)


def w4a16_scaled_append(q, k, v, positions, inv_freq, slots, cache: ScaledCache, sections=None,
                        interleaved: bool = False, q_out=None, stream=None):
    """Rotary positions on q and k, and k and v into a cache whose scales are found
    as it is written.

    Arguments as in w4a16_rope_append; q may be None, k, v and slots may not.  A
    group's scale is the smallest power of two whose codes hold its values, and
    grows with them; a request fills its groups in order, and the tokens of one
    group are neighbours in the call, their slots ascending (as w4a16_paged_map
    gives them).  Tokens that are taken back (drafts) leave the scale as far as it
    grew until the group is written from its first token on again.  Returns the
    rotated queries (q_out, or a new tensor; q_out=q rotates in place)."""
    _scaled(cache)
    flags = ROPE_INTERLEAVED if interleaved else 0
    if _fast is not None and (q is None or q_out is not None):
        rc = _fast.scaled_append(q, k, v, positions, inv_freq, slots, cache._ref, cache.heads, cache.device, sections, flags,
                                 q_out, None if stream is None else stream.cuda_stream)
        if rc == 0:
            return q_out
        if rc is not None:
            raise W4A16Error(rc, "w4a16_scaled_append")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k must be a torch.Tensor [T, heads, dim]")
    T = k.shape[0]
    shape = (T, cache.heads, cache.dim)
    ka, va, slots_at = _rows(k, "k", shape), _rows(v, "v", shape), _vector(slots, "slots", T)
    heads, qa, qo = 0, (None, 0, 0), (None, 0, 0)
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != cache.dim:
            raise ValueError("q has shape %s, expected [%d, q_heads, %d]" % (tuple(q.shape), T, cache.dim))
        heads, qa = q.shape[1], _rows(q, "q", q.shape)
        if q_out is None:
            q_out = _empty(q.shape, _bf16, q.device, stream)
        qo = _rows(q_out, "q_out", q.shape)
    _need(inv_freq, "inv_freq", _F32)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must have one dimension")
    if positions.dim() == 1:
        axes, axis_stride, positions_at = 1, 0, _vector(positions, "positions", T)
    else:
        axes, axis_stride = positions.shape[0], T
        _need(positions, "positions", _I32, (axes, T))
        positions_at = positions.data_ptr()
    sec = None
    if sections is not None:
        if len(sections) != axes:
            raise ValueError("%d sections for %d axes" % (len(sections), axes))
        sec = _section_array(sections)
    _on_device(cache.device, q=q, q_out=q_out if q is not None else None, k=k, v=v, positions=positions, inv_freq=inv_freq, slots=slots)
    if T == 0:
        return q_out
    rc = _launch(cache.device, _lib.w4a16_scaled_append, *qa, *qo, heads, *ka, *va, positions_at, axis_stride, inv_freq.data_ptr(), sec, axes,
                 2 * inv_freq.numel(), cache.dim, flags, slots_at, cache._ref, T, _stream(stream, cache.device))
    if rc:
        raise W4A16Error(rc, "w4a16_scaled_append")
    return q_out


def w4a16_scaled_read(cache: ScaledCache, block_table, row_start, first=None, k_out=None, v_out=None, rows: int = None,
                      dtype=torch.bfloat16, stream=None):
    """The keys and values of requests, one request after another.

    Row row_start[b] + i of k_out and v_out [rows, heads, dim] (bfloat16 or
    float32, row and head strides allowed) is token first[b] + i of request b (first
    None: token i), for rows below row_start[b + 1]; block_table int32 [B, columns],
    row_start int32 [B + 1], first int32 [B].  Rows behind row_start[B] are left as
    they are.  Without k_out and v_out: new tensors of `rows` rows and `dtype`,
    zeros where no request has a row.  Returns (k_out, v_out)."""
    _scaled(cache)
    if _fast is not None and k_out is not None and first is None and rows is None:
        rc = _fast.scaled_read(cache._ref, cache.heads, cache.dim, cache.device, block_table, row_start, k_out, v_out,
                               None if stream is None else stream.cuda_stream)
        if rc == 0:
            return k_out, v_out
        if rc is not None:
            raise W4A16Error(rc, "w4a16_scaled_read")
    B = len(row_start) - 1
    table, stride, columns = _table(block_table, B)
    start = _vector(row_start, "row_start", B + 1)
    first_at = None if first is None else _vector(first, "first", B)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        if rows is None:
            raise ValueError("rows is needed without k_out and v_out")
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dtype must be torch.bfloat16 or torch.float32")
        k_out, v_out = (_empty((rows, cache.heads, cache.dim), dtype, cache.k.device, stream, zero=True) for _ in range(2))
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in (torch.bfloat16, torch.float32) or t.dtype != k_out.dtype:
            raise TypeError("%s must be a CUDA tensor, both bfloat16 or both float32" % name)
        if t.dim() != 3 or t.stride(2) != 1 or t.shape != k_out.shape or t.shape[1:] != (cache.heads, cache.dim):
            raise ValueError("%s has shape %s, expected [rows, %d, %d], dim contiguous" % (name, tuple(t.shape), cache.heads, cache.dim))
    if rows is not None and rows != k_out.shape[0]:
        raise ValueError("rows is %d, k_out has %d" % (rows, k_out.shape[0]))
    _on_device(cache.device, block_table=block_table, row_start=row_start, first=first, k_out=k_out, v_out=v_out)
    rc = _launch(cache.device, _lib.w4a16_scaled_read, cache._ref, table, stride, columns, start, first_at, B, k_out.data_ptr(), *k_out.stride()[:2],
                 v_out.data_ptr(), *v_out.stride()[:2], OUT_F32 if k_out.dtype is torch.float32 else OUT_BF16, k_out.shape[0],
                 _stream(stream, cache.device))
    if rc:
        raise W4A16Error(rc, "w4a16_scaled_read")
    return k_out, v_out


def scaled_attention_workspace(cache: ScaledCache, q_heads: int, new_tokens: int = 1) -> torch.Tensor:
    """Workspace of w4a16_scaled_attention for this cache, number of query heads
    and most new tokens (its contents need no initialisation)."""
    return _scaled_workspace(cache, q_heads, new_tokens, None)


def _scaled_workspace(cache: ScaledCache, q_heads: int, new_tokens: int, stream) -> torch.Tensor:
    n = int(load_library().w4a16_scaled_attention_workspace_bytes(q_heads, cache.heads, cache.dim, new_tokens))
    return _empty(max(n, 16), torch.uint8, cache.k.device, stream, kept=False)


def w4a16_scaled_attention(q, cache: ScaledCache, block_table, kv_len, scale: float = None, window: int = 0,
                           out=None, lse=None, workspace=None, stream=None):
    """Attention of the last one to sixteen tokens of each request over the cache.

    q bf16 [B, q_heads, dim], or [B, N, q_heads, dim] for N new tokens of each
    request (request, token and head strides allowed); block_table int32 [B, columns];
    kv_len int32 [B], all tokens of a request, the new ones among them: new token i
    sees kv_len - (N - 1 - i) of them, with window > 0 the last `window` of those.
    scale defaults to dim ** -0.5.  Returns (out like q, lse float32 [B, q_heads] or
    [B, N, q_heads]); a token that sees nothing gets zeros and -infinity.
    workspace: from scaled_attention_workspace, one per stream in use (None: a new
    one for this call)."""
    _scaled(cache)
    if scale is None:
        scale = cache.dim ** -0.5
    if _fast is not None and workspace is not None:
        rc = _fast.scaled_attention(q, cache._ref, cache.dim, cache.device, block_table, kv_len, scale, window, out, lse, workspace,
                                    None if stream is None else stream.cuda_stream)
        if rc == 0:
            return out, lse
        if rc is not None:
            raise W4A16Error(rc, "w4a16_scaled_attention")
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be a tensor [B, q_heads, dim] or [B, new tokens, q_heads, dim]")
    by_token = (lambda t: t) if q.dim() == 4 else (lambda t: t.unsqueeze(1))
    B, N, H = by_token(q).shape[:3]
    qa = _token_rows(by_token(q), "q", (B, N, H, cache.dim))
    table, stride, columns = _table(block_table, B)
    lengths = _vector(kv_len, "kv_len", B)
    if out is None:
        out = _empty(q.shape, _bf16, q.device, stream)
    elif not isinstance(out, torch.Tensor) or out.dim() != q.dim():
        raise ValueError("out must be a tensor of q's shape")
    oa = _token_rows(by_token(out), "out", (B, N, H, cache.dim))
    if lse is None:
        lse = _empty(q.shape[:-1], torch.float32, q.device, stream)
    else:
        _need(lse, "lse", _F32, q.shape[:-1])
    if workspace is None:
        workspace = _scaled_workspace(cache, H, N, stream)
    elif not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _on_device(cache.device, q=q, block_table=block_table, kv_len=kv_len, out=out, lse=lse, workspace=workspace)
    rc = _launch(cache.device, _lib.w4a16_scaled_attention, *qa, cache._ref, table, stride, columns, lengths, B, N, H, scale, window, *oa, lse.data_ptr(),
                 workspace.data_ptr(), workspace.nbytes, _stream(stream, cache.device))
    if rc:
        raise W4A16Error(rc, "w4a16_scaled_attention")
    return out, lse


def _token_rows(t, name: str, shape):
    """Address, request, token and head strides of bf16 heads [B, N, heads, dim], dim contiguous."""
    if not t.is_cuda or t.dtype not in _BF16 or t.stride(3) != 1:
        raise ValueError("%s must be a CUDA bf16 tensor, dim contiguous" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return (t.data_ptr(), *t.stride()[:3])


load_library()
_fast = _load_fast()

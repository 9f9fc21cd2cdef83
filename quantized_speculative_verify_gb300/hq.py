"""Python binding of libhq.so (include/hq.h): argument marshalling only.

Every step of the verify-pass linear layer runs in the library's CUDA kernels.
This module converts torch tensors to raw device pointers, passes the current
CUDA stream, and turns status codes into exceptions.  There is no fallback: if
libhq.so is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import numpy as np
import torch

from . import build as _build

HQ_OK = 0
HQ_ERR_INVALID_ARG = 1
HQ_ERR_UNSUPPORTED = 2
HQ_ERR_CUDA = 3
HQ_ERR_TIMEOUT = 4
HQ_ERR_NO_PAGES = 5
HQ_W4_ASYM = 0
HQ_W8_SYM = 1
HQ_LAUNCH_DEFAULT = 0
HQ_LAUNCH_PDL = 1
HQ_LAUNCH_DETERMINISTIC = 2
HQ_LAUNCH_EXACT_ORDER = 4
HQ_MAX_M = 128

FORMATS = {"w4": HQ_W4_ASYM, "w8": HQ_W8_SYM}

# Every symbol include/hq.h declares.
EXPORTS = ("hq_tree_accept_workspace_bytes", "hq_tree_accept", "hq_status_string", "hq_version", "hq_packed_bytes", "hq_workspace_bytes", "hq_act_operand_bytes",
           "hq_make_signs",
           "hq_pack_weights", "hq_pack_weights_at", "hq_rotate_quant_act", "hq_verify_gemm", "hq_workspace_q8_bytes",
           "hq_verify_gemm_q8", "hq_unpack_codes", "hq_workspace_status",
           "hq_selftest_wait_timeout", "hq_selftest_gemm_wait_timeout", "hq_verify_gemm_noalloc", "hq_noalloc_status",
           "hq_tree_attention_workspace_bytes",
           "hq_tree_attention", "hq_tree_commit_kv", "hq_delta_tree", "hq_delta_commit", "hq_add_norm_quant",
           "hq_lora_workspace_bytes", "hq_lora_apply", "hq_pages_scratch_bytes", "hq_pages_fork", "hq_pages_extend",
           "hq_pages_free", "hq_pages_compact", "hq_pages_copy", "hq_pages_write", "hq_pages_status",
           "hq_prefix_attention_workspace_bytes", "hq_prefix_attention", "hq_rope_freqs", "hq_rope_turns", "hq_rope_write",
           "hq_gated_norm_quant", "hq_greedy_tokens_workspace_bytes", "hq_greedy_tokens", "hq_tree_accept_batch",
           "hq_history_status")

HQ_F32, HQ_F16, HQ_BF16 = 0, 1, 2
TYPES = {torch.float32: HQ_F32, torch.float16: HQ_F16, torch.bfloat16: HQ_BF16}

ROPE_KINDS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
GATE_ACTS = {"none": 0, "sigmoid": 1, "silu": 2}

HQ_ATTN_HEAD_DIM = 128
HQ_DELTA_HEAD_DIM = 128


class HQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class hq_layer_desc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("group", ctypes.c_int32), ("format", ctypes.c_int32)]


class hq_pages(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("ref", ctypes.c_void_p), ("table", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("scratch", ctypes.c_void_p), ("plane_bytes", ctypes.c_int64),
                ("n_planes", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("row_bytes", ctypes.c_int32)]


class hq_history(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("len", ctypes.c_void_p), ("prompt", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("n_slots", ctypes.c_int32), ("cap", ctypes.c_int32)]


class hq_logit_rules(ctypes.Structure):
    _fields_ = [("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("bias_starts", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("masks", ctypes.c_void_p), ("ldmask", ctypes.c_int64), ("n_slots", ctypes.c_int32),
                ("n_bias", ctypes.c_int32), ("n_masks", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libhq.so (building it first if the sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    if not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise HQError(HQ_ERR_CUDA, f"libhq.so not found at {_build.LIB}")
    lib = ctypes.CDLL(_build.LIB)
    P, I32, U32, U64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_size_t
    I64, F32 = ctypes.c_int64, ctypes.c_float
    D, C = ctypes.POINTER(hq_layer_desc), ctypes.POINTER(hq_pages)
    HS, LR, F64 = ctypes.POINTER(hq_history), ctypes.POINTER(hq_logit_rules), ctypes.c_double
    sig = {
        "hq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hq_version": (I32, []),
        "hq_packed_bytes": (SZ, [D]),
        "hq_workspace_bytes": (SZ, [D, I32]),
        "hq_act_operand_bytes": (SZ, [D, I32]),
        "hq_make_signs": (ctypes.c_int, [U64, I32, P]),
        "hq_pack_weights": (ctypes.c_int, [D, P, P, P, P]),
        "hq_pack_weights_at": (ctypes.c_int, [D, I32, I32, P, P, P, P]),
        "hq_rotate_quant_act": (ctypes.c_int, [D, P, I32, P, P, P, P, P, U32, P]),
        "hq_verify_gemm": (ctypes.c_int, [D, P, P, P, I32, P, P, P, U32, P]),
        "hq_workspace_q8_bytes": (SZ, [D, I32]),
        "hq_verify_gemm_q8": (ctypes.c_int, [D, P, P, P, P, I32, P, P, P, U32, P]),
        "hq_unpack_codes": (ctypes.c_int, [D, P, P, P, P, P]),
        "hq_workspace_status": (ctypes.c_int, [P, P]),
        "hq_selftest_wait_timeout": (ctypes.c_int, [P, ctypes.c_int64, P]),
        "hq_selftest_gemm_wait_timeout": (ctypes.c_int, [D, P, P, P, I32, P, P, ctypes.c_int64, P]),
        "hq_verify_gemm_noalloc": (ctypes.c_int, [D, P, P, P, I32, P, P, U32, P]),
        "hq_noalloc_status": (ctypes.c_int, [P]),
        "hq_tree_accept_workspace_bytes": (SZ, [I32, I32]),
        "hq_tree_accept": (ctypes.c_int, [P, I32, I32, P, P, P, P, P, P, P, U32, P]),
        "hq_tree_attention_workspace_bytes": (SZ, [I32]),
        "hq_tree_attention": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, I32, I32, P, ctypes.c_float, P, P, U32, P]),
        "hq_tree_commit_kv": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, P, P, U32, P]),
        "hq_delta_tree": (ctypes.c_int, [P, P, P, P, P, P, P, I32, I32, I32, P, U32, P]),
        "hq_delta_commit": (ctypes.c_int, [P, P, P, P, P, P, P, I32, I32, I32, U32, P]),
        "hq_add_norm_quant": (ctypes.c_int, [D, P, I32, I64, P, P, I32, I64, P, F32, I32, P, P, I32, I64, P, P, P, P,
                                             U32, P]),
        "hq_pages_scratch_bytes": (SZ, [C]),
        "hq_pages_fork": (ctypes.c_int, [C, P, P, I32, U32, P]),
        "hq_pages_extend": (ctypes.c_int, [C, P, P, I32, U32, P]),
        "hq_pages_free": (ctypes.c_int, [C, P, I32, U32, P]),
        "hq_pages_compact": (ctypes.c_int, [C, P, P, P, I32, I32, P, I32, U32, P]),
        "hq_pages_copy": (ctypes.c_int, [C, P, P, I32, U32, P]),
        "hq_pages_write": (ctypes.c_int, [C, I32, I32, P, P, I32, I64, I64, I32, P, P, I32, I32, I32, U32, P]),
        "hq_pages_status": (ctypes.c_int, [C, P]),
        "hq_prefix_attention_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
        "hq_prefix_attention": (ctypes.c_int, [C, I32, I32, I32, P, I64, P, P, I32, I32, I32, P, I32, I32, I32, F32, P, I32,
                                               I64, P, U32, P]),
        "hq_rope_freqs": (ctypes.c_int, [I32, F64, I32, F64, F64, F64, F64, P]),
        "hq_rope_turns": (ctypes.c_int, [P, I32, P]),
        "hq_rope_write": (ctypes.c_int, [C, I32, I32, I32, P, P, P, I32, I64, I64, I64, I32, P, P, F32, P, I32, I32, F32, P, P,
                                         I32, I32, I32, P, P, P, I64, U32, P]),
        "hq_gated_norm_quant": (ctypes.c_int, [D, P, I32, I64, P, I32, I64, I32, P, I32, F32, I32, P, P, I32, I64, P, P, P, P,
                                               U32, P]),
        "hq_greedy_tokens_workspace_bytes": (SZ, [I32]),
        "hq_greedy_tokens": (ctypes.c_int, [P, I32, I64, I32, HS, LR, P, P, P, I32, I32, I32, P, P, P, I32, I64, P, P, U32, P]),
        "hq_tree_accept_batch": (ctypes.c_int, [P, P, P, P, P, I32, I32, I32, HS, P, I32, P, P, U32, P]),
        "hq_history_status": (ctypes.c_int, [HS, P]),
        "hq_lora_workspace_bytes": (SZ, [I32, I32]),
        "hq_lora_apply": (ctypes.c_int, [P, I32, I64, I32, I32, I32, P, P, I32, I32, I32, P, P, P, P, I64, P, I64, P,
                                         U32, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().hq_status_string(int(status)).decode()


def _check(rc: int, what: str) -> None:
    if rc != HQ_OK:
        raise HQError(rc, what)


_Tensor, _INT32 = torch.Tensor, torch.int32


def _ptr(t) -> int | None:
    """A device-pointer argument: None, a raw address (int), or a CUDA tensor
    (which must live on the current device: the library launches there; not
    checked per pointer, to keep eager launches cheap).  Host tensors and numpy
    arrays are refused: the kernels read and write device memory, and on a
    system whose GPU can reach host memory a host buffer would not fault but
    run silently on host memory."""
    # (isinstance with torch.Tensor runs its metaclass's check: 0.3 us)
    if type(t) is _Tensor:
        if t.is_cuda:
            return t.data_ptr()
    elif t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, torch.Tensor):
        if not t.is_cuda:
            raise TypeError("device memory expected, got a CPU tensor (move it to the GPU first)")
        return t.data_ptr()
    raise TypeError(f"device memory expected, cannot pass {type(t).__name__} as a device pointer")


# The current stream's handle without making a torch.cuda.Stream object of it:
# 0.1 us instead of 3.7 us a call (Grace host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


_cuda_ready = False  # once true it stays so


def _stream(stream) -> int | None:
    global _cuda_ready
    if stream is None:
        if _cuda_ready:
            return _raw_stream(_current_device())
        if _raw_stream is not None and _current_device is not None and torch.cuda.is_initialized():
            _cuda_ready = True
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream):
    """The stream of a call as the current one: what a call allocates, fills or
    copies for itself belongs to the stream that it launches on, in its order
    (given back, the memory goes to that stream's next allocations, not to the
    current stream's while the kernels still use it)."""
    if stream is None or _stream(stream) == _stream(None):
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _new(shape, dtype, device, stream, fill=torch.empty) -> torch.Tensor:
    """A buffer that a call makes for itself or its caller (see _on).  The
    caller may use it, and let go of it, on the current stream as well."""
    with _on(stream):
        t = fill(shape, dtype=dtype, device=device)
    if stream is not None and t.is_cuda:
        t.record_stream(torch.cuda.current_stream())
    return t


def make_desc(K: int, N: int, group: int, fmt) -> hq_layer_desc:
    return hq_layer_desc(int(K), int(N), int(group), FORMATS.get(fmt, fmt) if isinstance(fmt, str) else int(fmt))


# ------------------------------------------------------------ C-ABI calls ---
def hq_version() -> int:
    return int(load().hq_version())


def hq_packed_bytes(desc: hq_layer_desc) -> int:
    return int(load().hq_packed_bytes(ctypes.byref(desc)))


def hq_workspace_bytes(desc: hq_layer_desc, M: int) -> int:
    return int(load().hq_workspace_bytes(ctypes.byref(desc), int(M)))


def hq_act_operand_bytes(desc: hq_layer_desc, M: int) -> int:
    return int(load().hq_act_operand_bytes(ctypes.byref(desc), int(M)))


def hq_make_signs(seed: int, K: int) -> np.ndarray:
    out = np.zeros(max(K // 32, 1), dtype=np.uint32)
    _check(load().hq_make_signs(ctypes.c_uint64(seed & (2 ** 64 - 1)), int(K), out.ctypes.data), "hq_make_signs")
    return out[: K // 32]


def hq_pack_weights(desc, W, signs, blob, stream=None) -> None:
    _check(load().hq_pack_weights(ctypes.byref(desc), _ptr(W), _ptr(signs), _ptr(blob), _stream(stream)),
           "hq_pack_weights")


def hq_pack_weights_at(desc, n0: int, rows: int, W, signs, blob, stream=None) -> None:
    _check(load().hq_pack_weights_at(ctypes.byref(desc), int(n0), int(rows), _ptr(W), _ptr(signs), _ptr(blob),
                                     _stream(stream)), "hq_pack_weights_at")


def hq_rotate_quant_act(desc, X, M: int, signs, qx, gsum, qop, sx, flags: int = 0, stream=None) -> None:
    _check(load().hq_rotate_quant_act(ctypes.byref(desc), _ptr(X), int(M), _ptr(signs), _ptr(qx), _ptr(gsum),
                                      _ptr(qop), _ptr(sx), int(flags), _stream(stream)), "hq_rotate_quant_act")


def hq_verify_gemm(desc, blob, qop, sx, M: int, Y, partials, workspace, flags: int = 0, stream=None) -> None:
    _check(load().hq_verify_gemm(ctypes.byref(desc), _ptr(blob), _ptr(qop), _ptr(sx), int(M), _ptr(Y),
                                 _ptr(partials), _ptr(workspace), int(flags), _stream(stream)), "hq_verify_gemm")


def hq_workspace_q8_bytes(desc: hq_layer_desc, M: int) -> int:
    return int(load().hq_workspace_q8_bytes(ctypes.byref(desc), int(M)))


def hq_verify_gemm_q8(desc, blob, qx, sx, gsum, M: int, Y, partials, workspace, flags: int = 0, stream=None) -> None:
    _check(load().hq_verify_gemm_q8(ctypes.byref(desc), _ptr(blob), _ptr(qx), _ptr(sx), _ptr(gsum), int(M), _ptr(Y),
                                    _ptr(partials), _ptr(workspace), int(flags), _stream(stream)), "hq_verify_gemm_q8")


def hq_unpack_codes(desc, blob, codes, scales, zeros, stream=None) -> None:
    _check(load().hq_unpack_codes(ctypes.byref(desc), _ptr(blob), _ptr(codes), _ptr(scales), _ptr(zeros),
                                  _stream(stream)), "hq_unpack_codes")


def hq_workspace_status(workspace, stream=None) -> int:
    return int(load().hq_workspace_status(_ptr(workspace), _stream(stream)))


def hq_selftest_wait_timeout(workspace, limit_ns: int, stream=None) -> None:
    _check(load().hq_selftest_wait_timeout(_ptr(workspace), int(limit_ns), _stream(stream)),
           "hq_selftest_wait_timeout")


def hq_selftest_gemm_wait_timeout(desc, blob, qop, sx, M: int, Y, workspace, limit_ns: int, stream=None) -> None:
    _check(load().hq_selftest_gemm_wait_timeout(ctypes.byref(desc), _ptr(blob), _ptr(qop), _ptr(sx), int(M), _ptr(Y),
                                                _ptr(workspace), int(limit_ns), _stream(stream)),
           "hq_selftest_gemm_wait_timeout")


HQ_NOALLOC_SCRATCH_BYTES = 60 * 1024 * 1024 + 128 * 1024


def hq_verify_gemm_noalloc(desc, blob, qop, sx, M: int, Y, partials=None, flags: int = 0, stream=None) -> None:
    """hq_verify_gemm with the library's fixed device scratch array instead of a workspace."""
    rc = load().hq_verify_gemm_noalloc(ctypes.byref(desc), _ptr(blob), _ptr(qop), _ptr(sx), int(M), _ptr(Y),
                                       _ptr(partials), int(flags), _stream(stream))
    if rc == HQ_ERR_UNSUPPORTED:
        need = hq_workspace_bytes(desc, M)
        raise HQError(rc, f"hq_verify_gemm_noalloc: this call needs {need} bytes of scratch, more than the "
                          f"library's fixed {HQ_NOALLOC_SCRATCH_BYTES}-byte array")
    _check(rc, "hq_verify_gemm_noalloc")


def hq_noalloc_status(stream=None) -> int:
    """HQ_ERR_TIMEOUT if an allocation-free call on the current device timed out since the last status call."""
    return int(load().hq_noalloc_status(_stream(stream)))


# ------------------------------------------------------- tensor helpers ---
@dataclass
class PackedLayer:
    """A packed layer on the device: its descriptor, blob and device signs."""
    desc: hq_layer_desc
    blob: torch.Tensor
    signs: torch.Tensor

    @property
    def K(self) -> int:
        return self.desc.K

    @property
    def N(self) -> int:
        return self.desc.N

    @property
    def group(self) -> int:
        return self.desc.group

    @property
    def fmt(self) -> int:
        return self.desc.format


def pack_layer(W: torch.Tensor, group: int, fmt, signs_host: np.ndarray, stream=None) -> PackedLayer:
    """Rotate + quantize + pack W [N][K] (fp32, on the device)."""
    N, K = W.shape
    desc = make_desc(K, N, group, fmt)
    nbytes = hq_packed_bytes(desc)
    if nbytes == 0:
        raise HQError(HQ_ERR_INVALID_ARG, "hq_packed_bytes")
    blob = _new(nbytes, torch.uint8, W.device, stream)
    signs = torch.from_numpy(signs_host.astype(np.int32, copy=False).view(np.int32)).to(W.device)
    with _on(stream):
        hq_pack_weights(desc, W.contiguous(), signs, blob, stream)
    return PackedLayer(desc, blob, signs)


@dataclass
class FusedLayer:
    """Several layers that read the same activations, packed into one blob:
    one GEMM computes all of them; `split(Y)` gives each part's outputs as
    views of Y's columns."""
    layer: PackedLayer
    widths: list
    offsets: list

    def split(self, Y: torch.Tensor) -> list:
        return [Y[:, o:o + w] for o, w in zip(self.offsets, self.widths)]


def pack_fused(Ws: list, group: int, fmt, signs_host: np.ndarray, stream=None) -> FusedLayer:
    """Pack the parts Ws (fp32 [N_i][K] on the device, same K) into one blob;
    every part but the last must have a multiple of 128 rows."""
    K = Ws[0].shape[1]
    widths = [int(w.shape[0]) for w in Ws]
    if any(w.shape[1] != K for w in Ws) or any(n % 128 for n in widths[:-1]):
        raise HQError(HQ_ERR_INVALID_ARG, "pack_fused: parts need the same K and widths that are multiples of 128")
    offsets = [sum(widths[:i]) for i in range(len(widths))]
    desc = make_desc(K, sum(widths), group, fmt)
    nbytes = hq_packed_bytes(desc)
    if nbytes == 0:
        raise HQError(HQ_ERR_INVALID_ARG, "hq_packed_bytes")
    dev = Ws[0].device
    blob = _new(nbytes, torch.uint8, dev, stream)
    signs = torch.from_numpy(signs_host.astype(np.int32, copy=False).view(np.int32)).to(dev)
    with _on(stream):
        for W, o in zip(Ws, offsets):
            hq_pack_weights_at(desc, o, W.shape[0], W.contiguous(), signs, blob, stream)
    return FusedLayer(PackedLayer(desc, blob, signs), widths, offsets)


def act_buffers(desc: hq_layer_desc, M: int, device, int8_codes: bool = True, group_sums: bool = False) -> tuple:
    """Buffers of hq_rotate_quant_act for M rows of the activations of layers like `desc`:
    (qx int8 [M][K] or None, gsum int32 [M][K/group] or None, GEMM activation operand (opaque bytes), sx fp32 [M])."""
    K, group = desc.K, desc.group
    qx = torch.empty((M, K), dtype=torch.int8, device=device) if int8_codes else None
    gsum = torch.empty((M, K // group), dtype=torch.int32, device=device) if group_sums else None
    qop = torch.empty(hq_act_operand_bytes(desc, M), dtype=torch.uint8, device=device)
    sx = torch.empty(M, dtype=torch.float32, device=device)
    return qx, gsum, qop, sx


def workspace(desc: hq_layer_desc, M: int, device) -> torch.Tensor:
    n = hq_workspace_bytes(desc, M)
    if n == 0:
        raise HQError(HQ_ERR_INVALID_ARG, "hq_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def unpack(layer: PackedLayer, stream=None):
    N, K, G = layer.N, layer.K, layer.group
    dev = layer.blob.device
    codes = _new((N, K), torch.uint8, dev, stream)
    scales = _new((N, K // G), torch.float32, dev, stream)
    zeros = _new((N, K // G), torch.uint8, dev, stream) if layer.fmt == HQ_W4_ASYM else None
    hq_unpack_codes(layer.desc, layer.blob, codes, scales, zeros, stream)
    return codes, scales, zeros


def verify_linear(layer: PackedLayer, X: torch.Tensor, ws: torch.Tensor, Y: torch.Tensor | None = None,
                  bufs=None, flags: int = 0, partials: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = dequant(int GEMM(quant(rotate(X)), packed W)): the two kernels in sequence."""
    M, K = X.shape
    if bufs is None:
        with _on(stream):
            bufs = act_buffers(layer.desc, M, X.device, int8_codes=False)
    qx, gsum, qop, sx = bufs
    if Y is None:
        Y = _new((M, layer.N), torch.float32, X.device, stream)
    hq_rotate_quant_act(layer.desc, X, M, layer.signs, qx, gsum, qop, sx, flags & HQ_LAUNCH_PDL, stream)
    hq_verify_gemm(layer.desc, layer.blob, qop, sx, M, Y, partials, ws, flags, stream)
    return Y


def hq_tree_accept_workspace_bytes(M: int, V: int) -> int:
    return int(load().hq_tree_accept_workspace_bytes(int(M), int(V)))


def hq_tree_accept(logits, M: int, V: int, parent, tokens, greedy, path, n_accept, bonus, workspace, flags: int = 0,
                   stream=None) -> None:
    _check(load().hq_tree_accept(_ptr(logits), M, V, _ptr(parent), _ptr(tokens), _ptr(greedy), _ptr(path),
                                 _ptr(n_accept), _ptr(bonus), _ptr(workspace), flags, _stream(stream)),
           "hq_tree_accept")


def tree_accept(logits: torch.Tensor, parent: torch.Tensor, tokens: torch.Tensor, flags: int = 0, stream=None):
    """Greedy tokens, accepted path, number accepted and bonus token of a draft tree (device tensors)."""
    M, V = logits.shape
    dev = logits.device
    greedy = _new(M, torch.int32, dev, stream)
    path = _new(M, torch.int32, dev, stream)
    out = _new(2, torch.int32, dev, stream)
    ws = _new(hq_tree_accept_workspace_bytes(M, V), torch.uint8, dev, stream)
    hq_tree_accept(logits, M, V, parent, tokens, greedy, path, out[0:1], out[1:2], ws, flags, stream)
    return greedy, path, out


def hq_tree_attention_workspace_bytes(Hkv: int) -> int:
    return int(load().hq_tree_attention_workspace_bytes(int(Hkv)))


def hq_tree_attention(q, k_cache, v_cache, cap: int, L: int, M: int, Hq: int, Hkv: int, D: int, parent, scale: float,
                      out, workspace, flags: int = 0, stream=None) -> None:
    _check(load().hq_tree_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), cap, L, M, Hq, Hkv, D, _ptr(parent),
                                    float(scale), _ptr(out), _ptr(workspace), flags, _stream(stream)),
           "hq_tree_attention")


def hq_tree_commit_kv(k_cache, v_cache, cap: int, L: int, M: int, Hkv: int, D: int, path, n_accept, flags: int = 0,
                      stream=None) -> None:
    _check(load().hq_tree_commit_kv(_ptr(k_cache), _ptr(v_cache), cap, L, M, Hkv, D, _ptr(path), _ptr(n_accept),
                                    flags, _stream(stream)),
           "hq_tree_commit_kv")


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, L: int, parent: torch.Tensor,
                   scale: float, out: torch.Tensor = None, workspace: torch.Tensor = None, flags: int = 0,
                   stream=None) -> torch.Tensor:
    """Tree-masked attention of the M tree nodes.  q fp16 [M][Hq][D]; k_cache,
    v_cache fp16 [Hkv][cap][D] with the tree nodes at positions [L, L + M);
    parent int32 [M] (device).  Returns fp32 [M][Hq][D]."""
    M, Hq, D = q.shape
    Hkv, cap, _ = k_cache.shape
    if out is None:
        out = _new((M, Hq, D), torch.float32, q.device, stream)
    if workspace is None:
        workspace = _new(hq_tree_attention_workspace_bytes(Hkv), torch.uint8, q.device, stream, torch.zeros)
    hq_tree_attention(q, k_cache, v_cache, cap, L, M, Hq, Hkv, D, parent, scale, out, workspace, flags, stream)
    return out


def tree_commit_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, L: int, M: int, path: torch.Tensor,
                   n_accept: torch.Tensor, flags: int = 0, stream=None) -> None:
    """Moves the accepted path next to the root in both caches (in place)."""
    Hkv, cap, D = k_cache.shape
    hq_tree_commit_kv(k_cache, v_cache, cap, L, M, Hkv, D, path, n_accept, flags, stream)


def hq_delta_tree(state, q, k, v, alpha, beta, parent, M: int, H: int, D: int, out, flags: int = 0,
                  stream=None) -> None:
    _check(load().hq_delta_tree(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(parent), M, H,
                                D, _ptr(out), flags, _stream(stream)), "hq_delta_tree")


def hq_delta_commit(state, k, v, alpha, beta, path, n_accept, M: int, H: int, D: int, flags: int = 0,
                    stream=None) -> None:
    _check(load().hq_delta_commit(_ptr(state), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(path),
                                  _ptr(n_accept), M, H, D, flags, _stream(stream)), "hq_delta_commit")


def delta_tree(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
               beta: torch.Tensor, parent: torch.Tensor, out: torch.Tensor = None, flags: int = 0,
               stream=None) -> torch.Tensor:
    """Outputs of every tree node of a gated delta-rule layer; the committed
    state [H][D][D] is only read.  q, k, v fp32 [M][H][D]; alpha, beta [M][H]."""
    M, H, D = q.shape
    if out is None:
        out = _new((M, H, D), torch.float32, q.device, stream)
    hq_delta_tree(state, q, k, v, alpha, beta, parent, M, H, D, out, flags, stream)
    return out


def delta_commit(state: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                 path: torch.Tensor, n_accept: torch.Tensor, flags: int = 0, stream=None) -> None:
    """Advances the state (in place) along the root and the accepted path."""
    M, H, D = k.shape
    hq_delta_commit(state, k, v, alpha, beta, path, n_accept, M, H, D, flags, stream)


# ---------------------------------------------------- a batch of requests ---
# These are called once or more a layer, so their checks are written to cost a
# few microseconds: messages are formatted only when they are raised.
def _type(t) -> int:
    """The library's element type of a tensor (fp32 where there is none)."""
    if t is None:
        return HQ_F32
    ty = TYPES.get(t.dtype)
    if ty is None:
        raise TypeError(f"fp32, fp16 or bf16 expected, got {t.dtype}")
    return ty


def _rows(t, cols: int, what: str) -> int:
    """The distance in elements between the rows of a tensor whose last dimensions are `cols` contiguous elements."""
    if t is None:
        return cols
    if t.is_contiguous():
        if t.numel() != t.shape[0] * cols:
            raise ValueError(f"{what}: rows of {cols} elements expected, got shape {tuple(t.shape)}")
        return cols
    n = 1
    for d in range(t.dim() - 1, 0, -1):  # the dimensions that make up one row
        if t.shape[d] != 1 and t.stride(d) != n:
            raise ValueError(f"{what}: the elements of a row must be contiguous")
        n *= t.shape[d]
    if n != cols:
        raise ValueError(f"{what}: rows of {cols} elements expected, got shape {tuple(t.shape)}")
    return t.stride(0) if t.shape[0] > 1 else cols


def _pitch(t, cols: int, what: str) -> int:
    """_rows of a tensor whose shape [rows][cols] has been checked."""
    return cols if t is None or t.is_contiguous() else _rows(t, cols, what)


def _heads(t, dim: int, what: str) -> int:
    """The distance in elements between the rows of a tensor [rows][heads][dim] whose rows are contiguous."""
    rows, heads, _ = t.shape
    ld, of_head, one = t.stride()
    if one != 1 or (of_head != dim and heads != 1):
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    return ld if rows > 1 else heads * dim


def _dense(t, dtype, shape, what: str) -> None:
    """A contiguous tensor of the given type and shape, or None."""
    if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what}: contiguous {dtype} {shape} expected, got {t.dtype} {tuple(t.shape)}")


def _shaped(t, shape, what: str) -> None:
    if t is not None and t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")


def _room(t, need: int, what: str) -> None:
    if t.nbytes < need:
        raise ValueError(f"{what} is too small: {need} bytes needed")


def hq_add_norm_quant(desc, x, x_type: int, ldx: int, residual, residual_out, r_type: int, ldr: int, weight, eps: float,
                      M: int, signs, h, h_type: int, ldh: int, qx, gsum, qop, sx, flags: int = 0, stream=None) -> None:
    _check(load().hq_add_norm_quant(ctypes.byref(desc), _ptr(x), x_type, ldx, _ptr(residual), _ptr(residual_out),
                                    r_type, ldr, _ptr(weight), eps, M, _ptr(signs), _ptr(h), h_type, ldh, _ptr(qx),
                                    _ptr(gsum), _ptr(qop), _ptr(sx), flags, _stream(stream)), "hq_add_norm_quant")


def add_norm_quant(desc: hq_layer_desc, x: torch.Tensor, residual, weight: torch.Tensor, signs, eps: float = 1e-6,
                   residual_out=None, h=None, qx=None, gsum=None, qop=None, sx=None, flags: int = 0,
                   stream=None) -> None:
    """Residual addition, RMS norm and the quantization of the result for the
    layers like `desc` (hq_add_norm_quant), in one pass: residual_out =
    x + residual, h = the normed row, qx / gsum / qop / sx = its codes (buffers
    of act_buffers).  x, residual, residual_out and h: [M][K], fp32, fp16 or
    bf16, rows any 16-byte-aligned distance apart; residual may be None (the
    norm of x alone) and any output may be None; residual_out may be residual
    itself.  weight fp32 [K]; signs int32 [K / 32] (hq_make_signs, on the device)."""
    shape = x.shape
    M, K = shape
    x_type = TYPES.get(x.dtype)
    if x_type is None:
        raise TypeError(f"add_norm_quant: fp32, fp16 or bf16 expected, got {x.dtype}")
    if K != desc.K:
        raise ValueError(f"add_norm_quant: x has {K} features, the layer {desc.K}")
    _shaped(residual, shape, "add_norm_quant: residual")
    if residual_out is not residual:
        _shaped(residual_out, shape, "add_norm_quant: residual_out")
    _shaped(h, shape, "add_norm_quant: h")
    _dense(weight, torch.float32, (K,), "add_norm_quant: weight")
    _dense(signs, torch.int32, (K // 32,), "add_norm_quant: signs")
    _dense(qx, torch.int8, shape, "add_norm_quant: qx")
    _dense(sx, torch.float32, (M,), "add_norm_quant: sx")
    if gsum is not None:
        _dense(gsum, torch.int32, (M, K // desc.group), "add_norm_quant: gsum")
    if qop is not None:
        _room(qop, hq_act_operand_bytes(desc, M), "add_norm_quant: qop")
    r = residual if residual is not None else residual_out
    ldr = _pitch(r, K, "residual")
    if residual is not None and residual_out is not None and residual_out is not residual and (
            residual.dtype != residual_out.dtype or _pitch(residual_out, K, "residual_out") != ldr):
        raise ValueError("add_norm_quant: residual and residual_out need the same type and stride")
    ldx, ldh = _pitch(x, K, "x"), _pitch(h, K, "h")
    rc = load().hq_add_norm_quant(ctypes.byref(desc), _ptr(x), x_type, ldx, _ptr(residual), _ptr(residual_out), _type(r),
                                  ldr, _ptr(weight), eps, M, _ptr(signs), _ptr(h), _type(h), ldh, _ptr(qx), _ptr(gsum),
                                  _ptr(qop), _ptr(sx), flags, _stream(stream))
    if rc != HQ_OK:
        raise HQError(rc, "hq_add_norm_quant")


@functools.lru_cache(maxsize=1024)
def hq_lora_workspace_bytes(M: int, r_max: int) -> int:
    return int(load().hq_lora_workspace_bytes(int(M), int(r_max)))


def hq_lora_apply(x, x_type: int, ldx: int, M: int, K: int, N: int, A, B, w_type: int, n_adapters: int, r_max: int, ids,
                  ranks, scale, base, ldb: int, Y, ldy: int, workspace, flags: int = 0, stream=None) -> None:
    _check(load().hq_lora_apply(_ptr(x), x_type, ldx, M, K, N, _ptr(A), _ptr(B), w_type, n_adapters, r_max, _ptr(ids),
                                _ptr(ranks), _ptr(scale), _ptr(base), ldb, _ptr(Y), ldy, _ptr(workspace), flags,
                                _stream(stream)), "hq_lora_apply")


def lora_apply(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor, ranks=None, scale=None,
               base=None, Y=None, workspace=None, flags: int = 0, stream=None) -> torch.Tensor:
    """Y[m] = base[m] + scale[a] * B[a] (A[a] x[m]) with a = ids[m], Y = base
    where there is no such adapter (hq_lora_apply).  x [M][K]; A [n][r][K] and
    B [n][N][r], fp16 or bf16; ids int32 [M], ranks int32 [n], scale fp32 [n]
    on the device; base fp32 [M][N] may be Y itself, or None (zeros)."""
    M, K = x.shape
    n, r, _ = A.shape
    N = B.shape[1]
    _dense(A, A.dtype, (n, r, K), "lora_apply: A")
    _dense(B, A.dtype, (n, N, r), "lora_apply: B")
    _dense(ids, torch.int32, (M,), "lora_apply: ids")
    _dense(ranks, torch.int32, (n,), "lora_apply: ranks")
    _dense(scale, torch.float32, (n,), "lora_apply: scale")
    shape = (M, N)
    if Y is None:
        Y = _new(shape, torch.float32, x.device, stream)
    if base is not Y:
        _shaped(base, shape, "lora_apply: base")
    _shaped(Y, shape, "lora_apply: Y")
    if Y.dtype != torch.float32 or (base is not None and base.dtype != torch.float32):
        raise ValueError("lora_apply: base and Y must be fp32")
    need = hq_lora_workspace_bytes(M, r)
    if workspace is None:
        workspace = _new(need, torch.uint8, x.device, stream)
    _room(workspace, need, "lora_apply: the workspace")
    rc = load().hq_lora_apply(_ptr(x), _type(x), _pitch(x, K, "x"), M, K, N, _ptr(A), _ptr(B), _type(A), n, r, _ptr(ids),
                              _ptr(ranks), _ptr(scale), _ptr(base), _pitch(base, N, "base"), _ptr(Y), _pitch(Y, N, "Y"),
                              _ptr(workspace), flags, _stream(stream))
    if rc != HQ_OK:
        raise HQError(rc, "hq_lora_apply")
    return Y


class _Held:
    """Attributes whose device addresses the library holds stay the tensors they are."""
    _held = frozenset()

    def __setattr__(self, name, value):
        if name in self._held and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{type(self).__name__}.{name} is held by its address: change it in place, or make a new "
                                 f"{type(self).__name__}")
        object.__setattr__(self, name, value)


class PagedCache(_Held):
    """A paged key/value cache (hq_pages) over the caller's tensors: pool
    [planes][pages][heads][page_size][dim] (fp16 or bf16), ref int32 [pages],
    table int32 [sequences][max_pages], lens int32 [sequences].  `empty` makes
    one without sequences.  The library holds the tensors' addresses: their
    contents may be changed in place, the attributes themselves stay."""

    _held = frozenset(("pool", "ref", "table", "lens", "status", "scratch", "c"))

    def __init__(self, pool: torch.Tensor, ref: torch.Tensor, table: torch.Tensor, lens: torch.Tensor):
        planes, pages, heads, page_size, dim = pool.shape
        if pool.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"PagedCache: fp16 or bf16 expected, got {pool.dtype}")
        if not pool[0].is_contiguous():
            raise ValueError("PagedCache: the pages of a plane must be contiguous")
        if table.dim() != 2:
            raise ValueError("PagedCache: table must be [sequences][max_pages]")
        _dense(ref, torch.int32, (pages,), "PagedCache: ref")
        _dense(table, torch.int32, table.shape, "PagedCache: table")
        _dense(lens, torch.int32, (table.shape[0],), "PagedCache: lens")
        self.pool, self.ref, self.table, self.lens = pool, ref, table, lens
        self.type = TYPES[pool.dtype]
        self.status = torch.zeros(4, dtype=torch.int32, device=pool.device)
        plane_bytes = (pool.stride(0) if planes > 1 else pool[0].numel()) * 2
        self.c = hq_pages(0, 0, 0, 0, 0, 0, plane_bytes, planes, pages, table.shape[0], table.shape[1], page_size, heads,
                          dim * 2)
        need = int(load().hq_pages_scratch_bytes(ctypes.byref(self.c)))
        if need == 0:
            raise HQError(HQ_ERR_INVALID_ARG, "hq_pages_scratch_bytes")
        self.scratch = torch.empty(need, dtype=torch.uint8, device=pool.device)
        for f, t in (("pool", pool), ("ref", ref), ("table", table), ("len", lens), ("status", self.status),
                     ("scratch", self.scratch)):
            setattr(self.c, f, _ptr(t))
        self.heads, self.dim, self.n_seqs = heads, dim, table.shape[0]

    @classmethod
    def empty(cls, planes: int, pages: int, heads: int, page_size: int, dim: int, sequences: int, max_pages: int,
              dtype=torch.float16, device="cuda") -> "PagedCache":
        return cls(torch.zeros((planes, pages, heads, page_size, dim), dtype=dtype, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device),
                   torch.full((sequences, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(sequences, dtype=torch.int32, device=device))


def _list(t, n, what: str) -> int:
    """The length of an int32 list; n: the length it must have, if any."""
    shape = t.shape
    if t.dtype is not _INT32 or len(shape) != 1 or not t.is_contiguous() or (n is not None and shape[0] != n):
        raise ValueError(f"{what}: contiguous int32 [{'n' if n is None else n}] expected, got {t.dtype} {tuple(shape)}")
    return shape[0]


def pages_fork(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, flags: int = 0, stream=None) -> None:
    """Sequences dst (empty slots) take the pages of src; no data moves (hq_pages_fork)."""
    n = _list(src, None, "pages_fork: src")
    _list(dst, n, "pages_fork: dst")
    _check(load().hq_pages_fork(cache.c, _ptr(src), _ptr(dst), n, flags, _stream(stream)), "hq_pages_fork")


def pages_extend(cache: PagedCache, seqs: torch.Tensor, add: torch.Tensor, flags: int = 0, stream=None) -> None:
    """Sequences grow by add positions; a shared last page is copied first (hq_pages_extend)."""
    n = _list(seqs, None, "pages_extend: seqs")
    _list(add, n, "pages_extend: add")
    _check(load().hq_pages_extend(cache.c, _ptr(seqs), _ptr(add), n, flags, _stream(stream)), "hq_pages_extend")


def pages_free(cache: PagedCache, seqs: torch.Tensor, flags: int = 0, stream=None) -> None:
    """Sequences give up their pages and become empty slots (hq_pages_free)."""
    n = _list(seqs, None, "pages_free: seqs")
    _check(load().hq_pages_free(cache.c, _ptr(seqs), n, flags, _stream(stream)), "hq_pages_free")


def pages_compact(cache: PagedCache, seqs: torch.Tensor, base: torch.Tensor, keep: torch.Tensor, n_keep: torch.Tensor,
                  flags: int = 0, stream=None) -> None:
    """Keeps the positions base + keep[i][:n_keep[i]] after base[i], moved down,
    and gives up the rest (hq_pages_compact).  keep int32 [n][any], rows any
    distance apart."""
    n = _list(seqs, None, "pages_compact: seqs")
    _list(base, n, "pages_compact: base")
    _list(n_keep, n, "pages_compact: n_keep")
    if keep.dtype != torch.int32 or keep.dim() != 2 or keep.shape[0] != n or keep.shape[1] < 1 or (
            keep.shape[1] > 1 and keep.stride(1) != 1):
        raise ValueError(f"pages_compact: keep must be int32 [{n}][1 or more]")
    width = keep.shape[1]
    _check(load().hq_pages_compact(cache.c, _ptr(seqs), _ptr(base), _ptr(keep), keep.stride(0) if n > 1 else width, width,
                                   _ptr(n_keep), n, flags, _stream(stream)), "hq_pages_compact")


def pages_copy(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, flags: int = 0, stream=None) -> None:
    """Pages dst of every plane become copies of pages src (hq_pages_copy)."""
    n = _list(src, None, "pages_copy: src")
    _list(dst, n, "pages_copy: dst")
    _check(load().hq_pages_copy(cache.c, _ptr(src), _ptr(dst), n, flags, _stream(stream)), "hq_pages_copy")


def _batch(n_seqs, rows: int, starts, max_rows: int, seqs, what: str) -> int:
    """The number of sequences of a batch of rows (n_seqs: of the cache, None: no cache)."""
    if max_rows < 1:
        raise ValueError(f"{what}: max_rows must be at least 1, got {max_rows}")
    if starts is not None:
        B = _list(starts, None, what) - 1
        if B < 0:
            raise ValueError(f"{what}: starts is empty")
    elif seqs is not None:
        B = seqs.shape[0]
    else:
        B = rows // max_rows
    if seqs is not None:
        _list(seqs, B, what)
    elif n_seqs is not None and B > n_seqs:
        raise ValueError(f"{what}: {B} sequences, the cache has {n_seqs}")
    return B


def pages_write(cache: PagedCache, k_plane: int, v_plane: int, k: torch.Tensor, v: torch.Tensor, starts, max_rows: int,
                seqs=None, flags: int = 0, stream=None) -> None:
    """Writes the newest rows of sequences (rows starts[b] .. starts[b + 1] of k
    and v [rows][heads][dim], fp32 or the cache's type) at the end of their
    positions (hq_pages_write); starts None: max_rows rows each."""
    rows = k.shape[0]
    if v.shape[0] != rows or v.dtype != k.dtype:
        raise ValueError("pages_write: k and v need the same rows and type")
    B = _batch(cache.n_seqs, rows, starts, max_rows, seqs, "pages_write: starts and seqs")
    cols = cache.heads * cache.dim
    _check(load().hq_pages_write(cache.c, k_plane, v_plane, _ptr(k), _ptr(v), _type(k), _rows(k, cols, "k"),
                                 _rows(v, cols, "v"), cache.type, _ptr(seqs), _ptr(starts), B, rows, max_rows, flags,
                                 _stream(stream)), "hq_pages_write")


def pages_status(cache: PagedCache, stream=None) -> int:
    """Synchronizes; the first error of a page operation or of prefix_attention since the last call (HQ_OK if none), cleared."""
    return int(load().hq_pages_status(cache.c, _stream(stream)))


@functools.lru_cache(maxsize=1024)
def hq_prefix_attention_workspace_bytes(B: int, rows: int, max_rows: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load().hq_prefix_attention_workspace_bytes(B, rows, max_rows, Hq, Hkv, D))


def prefix_attention(cache: PagedCache, k_plane: int, v_plane: int, q: torch.Tensor, starts, max_rows: int, shared: int,
                     max_len: int, scale: float, parent=None, seqs=None, out=None, workspace=None, flags: int = 0,
                     stream=None) -> torch.Tensor:
    """Attention of a batch over the paged cache, its first `shared` positions
    read once for all rows (hq_prefix_attention).  q [rows][Hq][D] of the
    cache's type: sequence b's rows starts[b] .. starts[b + 1] (None: max_rows
    rows each) are its newest positions, a draft tree with `parent` (int32
    [rows]; None: a chain).  max_len: at least every sequence's length.  out
    [rows][Hq][D] of the cache's type or fp32; workspace: zeroed once.  Bad
    table entries and lengths are reported by hq_workspace_status(workspace)
    and by pages_status(cache)."""
    shape = q.shape
    rows, Hq, D = shape
    if D != cache.dim or q.dtype != cache.pool.dtype:
        raise ValueError(f"prefix_attention: q must be {cache.pool.dtype} [rows][heads][{cache.dim}]")
    B = _batch(cache.n_seqs, rows, starts, max_rows, seqs, "prefix_attention: starts and seqs")
    if parent is not None:
        _list(parent, rows, "prefix_attention: parent")
    if out is None:
        out = _new(shape, q.dtype, q.device, stream)
    _shaped(out, shape, "prefix_attention: out")
    if B == 0 and out.is_cuda:  # the library's call does nothing then, but no sequence claims these rows
        with _on(stream):
            return out.zero_()
    need = hq_prefix_attention_workspace_bytes(B, rows, max_rows, Hq, cache.heads, D)
    if workspace is None:
        workspace = _new(max(need, 16), torch.uint8, q.device, stream, torch.zeros)
    _room(workspace, need, "prefix_attention: the workspace")
    _check(load().hq_prefix_attention(cache.c, k_plane, v_plane, cache.type, _ptr(q), Hq * D if q.is_contiguous() else _rows(q, Hq * D, "q"), _ptr(seqs),
                                      _ptr(starts), B, rows, max_rows, _ptr(parent), Hq, shared, max_len, scale,
                                      _ptr(out), _type(out), Hq * D if out.is_contiguous() else _rows(out, Hq * D, "out"), _ptr(workspace), flags,
                                      _stream(stream)), "hq_prefix_attention")
    return out


# ------------------------------------------- between the calls of a step ---
def rope_freqs(rot: int, base: float = 10000.0, kind: str = "plain", factor: float = 1.0, original: float = 0.0,
               low: float | None = None, high: float | None = None) -> np.ndarray:
    """Radians a position of the rot / 2 pairs of a head (hq_rope_freqs).
    `kind` "linear", "ntk", "yarn" or "bands" scales them for contexts `factor`
    times as long as the model's own of `original` positions; low and high: the
    turns over `original` between which "yarn" (1 and 32 if not given) and
    "bands" (1 and 4) go over from divided frequencies to those as they are.
    Models with "yarn" also have a gain of rope_write, usually 0.1 ln(factor) + 1."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"rope_freqs: kind must be one of {', '.join(ROPE_KINDS)}, got {kind!r}")
    out = np.zeros(max(rot // 2, 1), dtype=np.float64)
    _check(load().hq_rope_freqs(rot, base, ROPE_KINDS[kind], factor, original, 1.0 if low is None else low,
                                (4.0 if kind == "bands" else 32.0) if high is None else high, out.ctypes.data), "hq_rope_freqs")
    return out


def rope_turns(freqs, device) -> torch.Tensor:
    """Frequencies (radians a position) as rope_write takes them: int64 [n] on the device (hq_rope_turns)."""
    f = np.ascontiguousarray(freqs, dtype=np.float64)
    out = np.zeros(f.shape, dtype=np.int64)
    if f.ndim != 1:
        raise ValueError(f"rope_turns: a list of frequencies expected, got shape {f.shape}")
    _check(load().hq_rope_turns(f.ctypes.data, f.shape[0], out.ctypes.data), "hq_rope_turns")
    return torch.from_numpy(out).to(device)


def rope_write(cache: PagedCache, k_plane: int, v_plane: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
               turns: torch.Tensor, starts, max_rows: int, layout: str = "half", gain: float = 1.0, q_weight=None, k_weight=None,
               eps: float = 1e-6, parent=None, positions=None, seqs=None, out=None, flags: int = 0, stream=None) -> torch.Tensor:
    """Rotates the newest rows' q and k by their positions and writes k and v
    into the paged cache (hq_rope_write): pages_write with the rotation, and q
    for prefix_attention.  q [rows][Hq][dim], k and v [rows][heads][dim], fp32 or
    the cache's type, rows any 16-byte-aligned distance apart (the columns of one
    projection); turns from rope_turns, 8 to dim / 2 pairs.  q_weight, k_weight
    fp32 [dim]: heads are normed first.  A row's position is positions[row]
    (int32 [rows]), or its sequence's length before these rows plus its depth in
    the tree of `parent` (None: a chain).  Returns out [rows][Hq][dim] of the
    cache's type (may be q itself); one that the call makes is zero in rows that no
    sequence claims."""
    shape, heads, dtype = q.shape, cache.heads, q.dtype
    rows, Hq, D = shape
    if D != cache.dim or k.shape != (rows, heads, D) or v.shape != k.shape:
        raise ValueError(f"rope_write: q [rows][heads][{cache.dim}], k and v [rows][{heads}][{cache.dim}] expected, got "
                         f"{tuple(shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    if k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("rope_write: q, k and v need the same type")
    if turns.dtype is not torch.int64 or len(turns.shape) != 1 or not turns.is_contiguous():
        raise ValueError(f"rope_write: turns must be contiguous int64 [pairs], got {turns.dtype} {tuple(turns.shape)}")
    side = ROPE_LAYOUTS.get(layout)
    if side is None:
        raise ValueError(f"rope_write: layout must be one of {', '.join(ROPE_LAYOUTS)}, got {layout!r}")
    B = _batch(cache.n_seqs, rows, starts, max_rows, seqs, "rope_write: starts and seqs")
    if parent is not None:
        _list(parent, rows, "rope_write: parent")
    if positions is not None:
        _list(positions, rows, "rope_write: positions")
    if q_weight is not None:
        _dense(q_weight, torch.float32, (D,), "rope_write: q_weight")
    if k_weight is not None:
        _dense(k_weight, torch.float32, (D,), "rope_write: k_weight")
    if out is None:
        out = _new(shape, cache.pool.dtype, q.device, stream, torch.zeros)  # (rows that no sequence claims)
    elif out.shape != shape or out.dtype is not cache.pool.dtype:
        raise ValueError(f"rope_write: out must be {cache.pool.dtype} {list(shape)}")
    rc = load().hq_rope_write(cache.c, k_plane, v_plane, cache.type, _ptr(q), _ptr(k), _ptr(v), _type(q), _heads(q, D, "q"),
                              _heads(k, D, "k"), _heads(v, D, "v"), Hq, _ptr(q_weight), _ptr(k_weight), eps, _ptr(turns),
                              2 * turns.shape[0], side, gain, _ptr(seqs), _ptr(starts), B, rows, max_rows, _ptr(parent),
                              _ptr(positions), _ptr(out), _heads(out, D, "out"), flags, _stream(stream))
    if rc != HQ_OK:
        raise HQError(rc, "hq_rope_write")
    return out


def gated_norm_quant(desc: hq_layer_desc, x: torch.Tensor, gate, weight, signs, dim: int, act: str = "silu", eps: float = 1e-6,
                     h=None, qx=None, gsum=None, qop=None, sx=None, flags: int = 0, stream=None) -> None:
    """The norm of every head of `dim` features with its gate, and the
    quantization of the result for the output projection `desc`
    (hq_gated_norm_quant), in one pass: y = x * weight / rms(head) * act(gate),
    h = y, qx / gsum / qop / sx = its codes (buffers of act_buffers).  x, gate
    and h: [M][K], fp32, fp16 or bf16, rows any 16-byte-aligned distance apart;
    gate may be None (no gate), weight (fp32 [dim]) None (no norm), and any
    output None; act "silu", "sigmoid" or "none" (the gate itself)."""
    shape = x.shape
    M, K = shape
    if K != desc.K:
        raise ValueError(f"gated_norm_quant: x has {K} features, the layer {desc.K}")
    if act not in GATE_ACTS:
        raise ValueError(f"gated_norm_quant: act must be one of {', '.join(GATE_ACTS)}, got {act!r}")
    _shaped(gate, shape, "gated_norm_quant: gate")
    _shaped(h, shape, "gated_norm_quant: h")
    _dense(weight, torch.float32, (dim,), "gated_norm_quant: weight")
    _dense(signs, torch.int32, (K // 32,), "gated_norm_quant: signs")
    _dense(qx, torch.int8, shape, "gated_norm_quant: qx")
    _dense(sx, torch.float32, (M,), "gated_norm_quant: sx")
    if gsum is not None:
        _dense(gsum, torch.int32, (M, K // desc.group), "gated_norm_quant: gsum")
    if qop is not None:
        _room(qop, hq_act_operand_bytes(desc, M), "gated_norm_quant: qop")
    x_type, g_type, h_type = _type(x), _type(gate), _type(h)
    ldx, ldg, ldh = _pitch(x, K, "x"), _pitch(gate, K, "gate"), _pitch(h, K, "h")
    rc = load().hq_gated_norm_quant(desc, _ptr(x), x_type, ldx, _ptr(gate), g_type, ldg, GATE_ACTS[act], _ptr(weight), dim, eps, M,
                                    _ptr(signs), _ptr(h), h_type, ldh, _ptr(qx), _ptr(gsum), _ptr(qop), _ptr(sx), flags,
                                    _stream(stream))
    if rc != HQ_OK:
        raise HQError(rc, "hq_gated_norm_quant")


class History(_Held):
    """What requests have said so far (hq_history) over the caller's tensors:
    tokens int32 [slots][cap], lens int32 [slots], prompt int32 [slots] (how many
    of them are the prompt's; None: 0).  A slot's newest token, the root of its
    next draft tree, is its last.  tree_accept_batch lets them grow."""

    _held = frozenset(("tokens", "lens", "prompt", "status", "c"))

    def __init__(self, tokens: torch.Tensor, lens: torch.Tensor, prompt=None):
        if tokens.dim() != 2:
            raise ValueError("History: tokens must be [slots][cap]")
        slots, cap = tokens.shape
        _dense(tokens, torch.int32, (slots, cap), "History: tokens")
        _dense(lens, torch.int32, (slots,), "History: lens")
        _dense(prompt, torch.int32, (slots,), "History: prompt")
        if not 1 <= slots <= 65536 or not 1 <= cap <= 1 << 24:
            raise ValueError(f"History: 1 to 65536 slots of 1 to 2^24 tokens, got {slots} of {cap}")
        self.tokens, self.lens, self.prompt, self.n_slots = tokens, lens, prompt, slots
        self.status = torch.zeros(4, dtype=torch.int32, device=tokens.device)
        self.c = hq_history(_ptr(tokens), _ptr(lens), _ptr(prompt), _ptr(self.status), slots, cap)


def history_status(history: History, stream=None) -> int:
    """Synchronizes; the first error of tree_accept_batch on this history since the last call (HQ_OK if none), cleared."""
    return int(load().hq_history_status(history.c, _stream(stream)))


class LogitRules(_Held):
    """Rules of `slots` requests on their logits (hq_logit_rules) over the
    caller's tensors, each may be None: repetition, presence and frequency fp32
    [slots]; bias = (starts int32 [slots + 1], tokens int32 [n], values fp32 [n]),
    slot s has the entries starts[s] .. starts[s + 1]; masks int32 [masks][at
    least ceil(vocabulary / 32)], bit t % 32 of word t / 32 set: token t is
    allowed."""

    _held = frozenset(("repetition", "presence", "frequency", "bias", "masks", "c"))

    def __init__(self, slots: int, repetition=None, presence=None, frequency=None, bias=None, masks=None):
        for t, what in ((repetition, "repetition"), (presence, "presence"), (frequency, "frequency")):
            _dense(t, torch.float32, (slots,), f"LogitRules: {what}")
        starts, tokens, values = bias if bias is not None else (None, None, None)
        n = 0
        if bias is not None:
            _dense(starts, torch.int32, (slots + 1,), "LogitRules: bias starts")
            n = _list(tokens, None, "LogitRules: bias tokens")
            _dense(values, torch.float32, (n,), "LogitRules: bias values")
        words = 0
        if masks is not None:
            if masks.dtype != torch.int32 or masks.dim() != 2 or (masks.shape[1] > 1 and masks.stride(1) != 1):
                raise ValueError("LogitRules: masks must be int32 [masks][words], the words of a mask contiguous")
            words = masks.shape[1]
        self.repetition, self.presence, self.frequency, self.bias, self.masks = repetition, presence, frequency, bias, masks
        self.n_slots, self.words = slots, words
        self.c = hq_logit_rules(_ptr(repetition), _ptr(presence), _ptr(frequency), _ptr(starts), _ptr(tokens), _ptr(values),
                                _ptr(masks), 0 if masks is None else masks.stride(0) if masks.shape[0] > 1 else words, slots, n,
                                0 if masks is None else masks.shape[0])


_minus_one = functools.partial(torch.full, fill_value=-1)


@functools.lru_cache(maxsize=1024)
def hq_greedy_tokens_workspace_bytes(rows: int) -> int:
    return int(load().hq_greedy_tokens_workspace_bytes(int(rows)))


def greedy_tokens(logits: torch.Tensor, starts, max_rows: int, parent=None, tokens=None, seqs=None, history: History = None,
                  rules: LogitRules = None, mask_ids=None, out=None, greedy=None, workspace=None, flags: int = 0,
                  stream=None) -> torch.Tensor:
    """Penalties, biases and masks on the logits [rows][V] (fp32, fp16 or bf16)
    of a batch's trees, and the greedy token of every row (hq_greedy_tokens), -1
    where every token is masked.  Sequence b's rows are starts[b] .. starts[b +
    1] (None: max_rows rows each); parent and tokens int32 [rows]: its draft tree
    (parent None: a chain; tokens None: nothing drafted); seqs: its slots in
    history and rules (None: b).  mask_ids int32 [rows]: the row's mask, -1 none
    (None: mask r for row r).  out [rows][V] (the logits' type or fp32, or logits
    itself): the adjusted logits.  workspace: zeroed once, of at least these
    rows' size (None: the call makes and zeroes one, up to 64 KB a row: 3 us of 20
    for 128 rows without rules).  Returns greedy int32 [rows] (one that the call makes is -1 in rows
    that no sequence claims)."""
    rows, V = logits.shape
    B = _batch(None, rows, starts, max_rows, seqs, "greedy_tokens: starts and seqs")
    ty = TYPES.get(logits.dtype)
    if ty is None:
        raise TypeError(f"greedy_tokens: fp32, fp16 or bf16 expected, got {logits.dtype}")
    if parent is not None:
        _list(parent, rows, "greedy_tokens: parent")
    if tokens is not None:
        _list(tokens, rows, "greedy_tokens: tokens")
    if mask_ids is not None:
        _list(mask_ids, rows, "greedy_tokens: mask_ids")
    if rules is not None and rules.masks is not None and rules.words * 32 < V:
        raise ValueError(f"greedy_tokens: the masks have {rules.words} words, {V} tokens need {-(-V // 32)}")
    if out is not None and out is not logits and (out.shape != logits.shape or out.dtype not in (logits.dtype, torch.float32)):
        raise ValueError(f"greedy_tokens: out must be {logits.dtype} or fp32 {[rows, V]}, got {out.dtype} {list(out.shape)}")
    if greedy is None:
        greedy = _new((rows,), _INT32, logits.device, stream, _minus_one)  # (rows that no sequence claims)
    else:
        _list(greedy, rows, "greedy_tokens: greedy")
    need = hq_greedy_tokens_workspace_bytes(rows)
    if workspace is None:
        workspace = _new(max(need, 16), torch.uint8, logits.device, stream, torch.zeros)
    _room(workspace, need, "greedy_tokens: the workspace")
    ldl, ldo = _pitch(logits, V, "logits"), _pitch(out, V, "out")
    rc = load().hq_greedy_tokens(_ptr(logits), ty, ldl, V, None if history is None else history.c,
                                 None if rules is None else rules.c, _ptr(mask_ids), _ptr(seqs), _ptr(starts), B, rows, max_rows,
                                 _ptr(parent), _ptr(tokens), _ptr(out), ty if out is None else TYPES[out.dtype], ldo,
                                 _ptr(greedy), _ptr(workspace), flags, _stream(stream))
    if rc != HQ_OK:
        raise HQError(rc, "hq_greedy_tokens")
    return greedy


def tree_accept_batch(greedy: torch.Tensor, parent, tokens: torch.Tensor, starts, max_rows: int, seqs=None,
                      history: History = None, path=None, n_accept=None, bonus=None, flags: int = 0, stream=None):
    """Accepted path, number accepted and bonus token of every draft tree of a
    batch from its greedy tokens (hq_tree_accept_batch); `history` grows by the
    accepted drafts and the bonus token.  greedy, parent (None: chains) and
    tokens int32 [rows]; starts, max_rows and seqs as in greedy_tokens.  Returns
    path int32 [B][max_rows] (-1 past the accepted nodes), n_accept and bonus
    int32 [B]: pages_compact takes path as keep and n_accept as n_keep."""
    rows = _list(greedy, None, "tree_accept_batch: greedy")
    _list(tokens, rows, "tree_accept_batch: tokens")
    if parent is not None:
        _list(parent, rows, "tree_accept_batch: parent")
    B = _batch(None, rows, starts, max_rows, seqs, "tree_accept_batch: starts and seqs")
    dev = greedy.device
    if path is None:
        path = _new((B, max_rows), _INT32, dev, stream)
    elif path.dtype is not _INT32 or path.dim() != 2 or path.shape[0] != B or path.shape[1] < max_rows or path.stride(1) != 1:
        raise ValueError(f"tree_accept_batch: path must be int32 [{B}][{max_rows} or more]")
    if n_accept is None:
        n_accept = _new(B, _INT32, dev, stream)
    else:
        _list(n_accept, B, "tree_accept_batch: n_accept")
    if bonus is None:
        bonus = _new(B, _INT32, dev, stream)
    else:
        _list(bonus, B, "tree_accept_batch: bonus")
    rc = load().hq_tree_accept_batch(_ptr(greedy), _ptr(parent), _ptr(tokens), _ptr(seqs), _ptr(starts), B, rows, max_rows,
                                     None if history is None else history.c, _ptr(path), path.stride(0) if B > 1 else path.shape[1],
                                     _ptr(n_accept), _ptr(bonus), flags, _stream(stream))
    if rc != HQ_OK:
        raise HQError(rc, "hq_tree_accept_batch")
    return path, n_accept, bonus

"""Python binding of libbinade (include/binade.h): argument marshalling only.

Every step of the path runs in the library: the table and the format 2 pack
in its host C++, the format 2 -> R4 conversion, the products and the unpack in
its HIP kernels. PyTorch provides device memory (tensors) and streams. If the
built library is missing this module raises on first use; there is no other
implementation behind it.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import threading
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libbinade.so")
CHUNK = 2048

OK, EINVAL, ECORRUPT, EUNSUPPORTED, EHIP, ENOSPACE = 0, -1, -2, -3, -4, -5
F32, BF16, E8M0 = 0, 1, 2
DEV_CORRUPT_STREAM, DEV_BAD_INDEX, DEV_CORRUPT_ESC = 0x1, 0x2, 0x4

EXPORTS = ["binade_status_str", "binade_last_hip_error", "binade_build_table",
           "binade_sizes_of", "binade_pack_rice", "binade_rice_to_r4",
           "binade_f1_sizes_of", "binade_pack_f1", "binade_f1_to_r4",
           "binade_rice_to_r4_batch", "binade_unpack", "binade_r4_gemv",
           "binade_r4_gemv_batch", "binade_bf16_gemv", "binade_bf16_gemv_batch",
           "binade_r4_gemm", "binade_bf16_gemm", "binade_gemm_workspace_bytes",
           "binade_r4_gemm_noalloc", "binade_gemm_scratch_bytes",
           "binade_r4_moe_gemv", "binade_bf16_moe_gemv", "binade_r4_gemv_rows",
           "binade_bf16_gemv_rows", "binade_moe_silu_mul", "binade_moe_combine",
           "binade_build_table_gpu", "binade_pack_gpu_workspace_bytes", "binade_pack_rice_gpu",
           "binade_huff_lengths", "binade_huff_pack", "binade_huff_workspace_bytes",
           "binade_huff_decode", "binade_rice_plan_bytes", "binade_rice_to_r4_plan",
           "binade_rice_to_r4_run", "binade_moe_combine_grad", "binade_moe_route",
           "binade_moe_route_workspace_bytes", "binade_moe_route_grad", "binade_lora_add",
           "binade_lora_workspace_bytes", "binade_lora_grad",
           "binade_lora_grad_workspace_bytes", "binade_f8_sizes_of", "binade_f8_pack",
           "binade_f8_layout", "binade_f8_gemm", "binade_f8_gemm_workspace_bytes",
           "binade_f8_gemm_grad", "binade_f8_gemm_grad_workspace_bytes", "binade_f8_moe_gemm",
           "binade_f8_moe_workspace_bytes", "binade_moe_route_scored",
           "binade_moe_route_scored_workspace_bytes", "binade_moe_route_scored_grad"]


class Table(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("exp_of_rank", ctypes.c_uint8 * 256),
                ("rank_of_exp", ctypes.c_uint16 * 256),
                ("count_of_rank", ctypes.c_uint64 * 256)]


class HuffDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("len", ctypes.c_uint8 * 256),
                ("sm", ctypes.c_void_p), ("stream", ctypes.c_void_p),
                ("stream_bytes", ctypes.c_uint64), ("stream_cap", ctypes.c_uint64),
                ("block_len", ctypes.c_void_p), ("group_off", ctypes.c_void_p)]


class Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("n_weights", "n_chunks", "unary_bits", "unary_words",
                 "rem_words", "n_esc", "nib_bytes")]


class RiceDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("k", ctypes.c_uint32), ("n", ctypes.c_uint32),
                ("exp_of_rank", ctypes.c_uint8 * 256),
                ("sm", ctypes.c_void_p), ("unary", ctypes.c_void_p),
                ("unary_bits", ctypes.c_uint64), ("unary_words", ctypes.c_uint64),
                ("rem", ctypes.c_void_p), ("rem_words", ctypes.c_uint64),
                ("anchor", ctypes.c_void_p), ("esc_pre", ctypes.c_void_p),
                ("n_esc", ctypes.c_uint64)]


class F1Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("n", ctypes.c_uint32), ("exp_of_rank", ctypes.c_uint8 * 256),
                ("sm", ctypes.c_void_p), ("width", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("code_bits", ctypes.c_uint64),
                ("code_words", ctypes.c_uint64), ("esc_rank", ctypes.c_void_p),
                ("n_f1esc", ctypes.c_uint64), ("esc_cap", ctypes.c_uint64),
                ("anchor", ctypes.c_void_p), ("f1_pre", ctypes.c_void_p),
                ("esc_pre", ctypes.c_void_p), ("n_esc", ctypes.c_uint64)]


class F1Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("n_weights", "n_tiles", "n_chunks", "code_words", "esc_cap")]


class R4Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("lut", ctypes.c_uint8 * 16),
                ("sm", ctypes.c_void_p), ("nib", ctypes.c_void_p),
                ("esc_pre", ctypes.c_void_p), ("esc", ctypes.c_void_p),
                ("n_esc", ctypes.c_uint64)]


class LoraDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("rank", ctypes.c_int32),
                ("n_adapters", ctypes.c_int32), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("scale", ctypes.c_void_p)]


class RouteRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class F8Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("count", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("values", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("values_t", ctypes.c_void_p),
                ("scales_t", ctypes.c_void_p)]


class F8Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("values_bytes", "scales_bytes", "values_t_bytes", "scales_t_bytes")]


class BinadeError(RuntimeError):
    def __init__(self, fn: str, code: int, hip: int = 0):
        lib = _lib_or_none()
        text = lib.binade_status_str(code).decode() if lib else str(code)
        super().__init__(f"{fn}: {text} ({code})" + (f", hip error {hip}" if hip else ""))
        self.code = code


_lock = threading.Lock()
_lib = None


def _lib_or_none():
    return _lib


def lib() -> ctypes.CDLL:
    global _lib
    with _lock:
        if _lib is None:
            path = os.environ.get("BINADE_LIB") or LIB_PATH   # another build of the library
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is not built; run "
                    "`python -m decode_gemv_tensor_amd.build` (hipcc, gfx950)")
            L = ctypes.CDLL(path)
            P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            L.binade_status_str.argtypes = [I32]
            L.binade_status_str.restype = ctypes.c_char_p
            L.binade_last_hip_error.restype = I32
            L.binade_gemm_workspace_bytes.argtypes = [I64, I64, I64]
            L.binade_gemm_workspace_bytes.restype = I64
            L.binade_gemm_scratch_bytes.argtypes = []
            L.binade_gemm_scratch_bytes.restype = I64
            L.binade_pack_gpu_workspace_bytes.argtypes = [I64, I64]
            L.binade_pack_gpu_workspace_bytes.restype = I64
            L.binade_huff_workspace_bytes.argtypes = []
            L.binade_huff_workspace_bytes.restype = I64
            L.binade_rice_plan_bytes.argtypes = [I32]
            L.binade_rice_plan_bytes.restype = I64
            L.binade_moe_route_workspace_bytes.argtypes = [I64, I32]
            L.binade_moe_route_workspace_bytes.restype = I64
            L.binade_lora_workspace_bytes.argtypes = [I64, I64, I64, I32]
            L.binade_lora_workspace_bytes.restype = I64
            L.binade_lora_grad_workspace_bytes.argtypes = [I64, I64, I64, I32, I32]
            L.binade_lora_grad_workspace_bytes.restype = I64
            L.binade_moe_route_scored_workspace_bytes.argtypes = [I64, I32]
            L.binade_moe_route_scored_workspace_bytes.restype = I64
            L.binade_f8_gemm_workspace_bytes.argtypes = [I64, I64, I64, I32]
            L.binade_f8_gemm_workspace_bytes.restype = I64
            L.binade_f8_gemm_grad_workspace_bytes.argtypes = [I64, I64, I64, I32, I32, I32]
            L.binade_f8_gemm_grad_workspace_bytes.restype = I64
            L.binade_f8_moe_workspace_bytes.argtypes = [I64, I32, I32, I32, I64, I64]
            L.binade_f8_moe_workspace_bytes.restype = I64
            sig = {
                "binade_build_table": [P, I64, P],
                "binade_sizes_of": [P, I64, I64, P],
                "binade_pack_rice": [P, I64, I64, P, P],
                "binade_rice_to_r4": [P, P, P, P],
                "binade_rice_to_r4_batch": [P, P, I32, P, P],
                "binade_rice_to_r4_plan": [P, P, I32, P, I64],
                "binade_rice_to_r4_run": [P, P, P, P],
                "binade_f1_sizes_of": [I64, I64, P],
                "binade_pack_f1": [P, I64, I64, P, P],
                "binade_f1_to_r4": [P, P, P, P],
                "binade_r4_gemv_batch": [P, P, P, I32, I32, P],
                "binade_bf16_gemv_batch": [P, P, P, P, P, I32, I32, P],
                "binade_unpack": [P, P, P],
                "binade_r4_gemv": [P, P, P, I32, P],
                "binade_bf16_gemv": [P, I64, I64, P, P, I32, P],
                "binade_r4_gemv_rows": [P, P, I64, I32, P, I64, I32, P],
                "binade_bf16_gemv_rows": [P, I64, I64, P, I64, I32, P, I64, I32, P],
                "binade_moe_silu_mul": [P, P, I64, P, I32, P],
                "binade_moe_combine": [P, P, I64, I32, I64, P, I32, P],
                "binade_build_table_gpu": [P, I64, P, P, P],
                "binade_huff_lengths": [P, I64, P, P],
                "binade_huff_pack": [P, P],
                "binade_huff_decode": [P, P, P, P, P],
                "binade_pack_rice_gpu": [P, I64, I64, P, P, P, P, P],
                "binade_r4_gemm": [P, P, I64, I64, P, I64, I32, P, I64, P],
                "binade_r4_gemm_noalloc": [P, P, I64, I64, P, I64, I32, P],
                "binade_bf16_gemm": [P, I64, I64, P, I64, I64, P, I64, I32, P, I64,
                                     P],
                "binade_r4_moe_gemv": [P, I32, P, I32, P, I64, I32, P, I32, P, P],
                "binade_bf16_moe_gemv": [P, I32, I64, I64, P, I32, P, I64, I32,
                                         P, I32, P, P],
                "binade_moe_combine_grad": [P, P, P, I32, I64, I32, I64, P, I32, P, P],
                "binade_moe_route": [P, I32, I64, I64, I32, I32, I32, P, P, P, P, P, P, P, I64,
                                     P],
                "binade_moe_route_grad": [P, I32, I64, I64, I32, I32, I32, P, P, P, P, P, I32,
                                          I64, P, P],
                "binade_lora_add": [P, P, I64, I64, P, P, I64, I32, P, I64, I32, P, P, I64, P,
                                    P],
                "binade_lora_grad": [P, P, I64, I64, P, P, I64, P, P, I64, P, I64, P, P, I32, P,
                                     I64, P, P],
                "binade_moe_route_scored": [P, I32, I64, I64, I32, I32, P, P, P, P, P, P, P, P,
                                            I64, P],
                "binade_moe_route_scored_grad": [P, I32, I64, I64, I32, I32, I32, I32,
                                                 ctypes.c_float, P, P, P, P, P, I32, I64, P, P],
                "binade_f8_sizes_of": [I64, I64, I32, I32, P],
                "binade_f8_pack": [P, P, P],
                "binade_f8_layout": [P, P, P, P],
                "binade_f8_gemm": [P, P, I64, I64, P, I64, I32, P, I64, P],
                "binade_f8_gemm_grad": [P, P, I64, I64, P, I64, P, I64, P, I32, P, I64, P],
                "binade_f8_moe_gemm": [P, P, I64, I32, P, I64, I32, P, I64, I32, P, I64, P, P],
            }
            for name, args in sig.items():
                if hasattr(L, name):
                    fn = getattr(L, name)
                    fn.argtypes = args
                    fn.restype = I32
            _lib = L
    return _lib


def _call(name: str, *args):
    rc = getattr(lib(), name)(*args)
    if rc != OK:
        raise BinadeError(name, rc, lib().binade_last_hip_error() if rc == EHIP else 0)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_stream(fn):
    """Run a device binding with `stream` as torch's current stream, so the
    temporaries it makes (contiguous copies, outputs, GEMM workspace) are
    allocated and filled in the same stream order as the kernel that uses
    them, and the caching allocator does not hand them to other streams while
    that kernel runs."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, stream=None, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kw)
    return wrapper


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _bits16(t: torch.Tensor) -> torch.Tensor:
    """bf16 / int16 / uint16 tensor -> contiguous view of its 16-bit patterns"""
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16, torch.float16):
        raise TypeError(f"expected 16-bit weights, got {t.dtype}")
    return t.contiguous()


# ------------------------------------------------------------------ host
def build_table(w: torch.Tensor) -> Table:
    """binade_build_table on a host bf16 tensor."""
    w = _bits16(w)
    if w.is_cuda:
        raise ValueError("build_table runs on host memory")
    t = Table()
    _call("binade_build_table", _ptr(w), w.numel(), ctypes.byref(t))
    return t


def sizes_of(table: Table, rows: int, cols: int) -> Sizes:
    s = Sizes()
    _call("binade_sizes_of", ctypes.byref(table), rows, cols, ctypes.byref(s))
    return s


@dataclass
class RicePlanes:
    """Format 2 planes of one tensor (host or device tensors) + descriptor."""
    rows: int
    cols: int
    table: Table
    sm: torch.Tensor
    unary: torch.Tensor
    rem: torch.Tensor | None
    anchor: torch.Tensor
    esc_pre: torch.Tensor
    unary_bits: int
    n_esc: int

    @property
    def k(self) -> int:
        return int(self.table.k)

    def desc(self) -> RiceDesc:
        d = RiceDesc()
        d.rows, d.cols = self.rows, self.cols
        d.k, d.n = self.table.k, self.table.n
        ctypes.memmove(d.exp_of_rank, self.table.exp_of_rank, 256)
        d.sm = self.sm.data_ptr()
        d.unary = self.unary.data_ptr()
        d.unary_bits = self.unary_bits
        d.unary_words = self.unary.numel()
        d.rem = self.rem.data_ptr() if self.rem is not None else None
        d.rem_words = self.rem.numel() if self.rem is not None else 0
        d.anchor = self.anchor.data_ptr()
        d.esc_pre = self.esc_pre.data_ptr()
        d.n_esc = self.n_esc
        return d

    def to(self, device) -> "RicePlanes":
        mv = lambda t: None if t is None else t.to(device, non_blocking=False)
        return RicePlanes(self.rows, self.cols, self.table, mv(self.sm),
                          mv(self.unary), mv(self.rem), mv(self.anchor),
                          mv(self.esc_pre), self.unary_bits, self.n_esc)

    def nbytes(self) -> dict:
        """Bytes of each plane as stored (padding words included)."""
        return {"sm": self.sm.numel(), "unary": 4 * self.unary.numel(),
                "rem": 0 if self.rem is None else 4 * self.rem.numel(),
                "anchor": 8 * self.anchor.numel(),
                "esc_pre": 4 * self.esc_pre.numel()}

    def bits_per_weight(self) -> float:
        n = self.rows * self.cols
        bits = 8 * n + self.unary_bits + self.k * n + 96 * (self.anchor.numel() - 1)
        return bits / n


def pack_rice(w: torch.Tensor, table: Table | None = None) -> RicePlanes:
    """binade_pack_rice: host bf16 [rows, cols] -> host format 2 planes."""
    w = _bits16(w)
    if w.is_cuda or w.dim() != 2:
        raise ValueError("pack_rice takes a 2-D host tensor")
    rows, cols = w.shape
    if table is None:
        table = build_table(w)
    s = sizes_of(table, rows, cols)
    sm = torch.empty(rows, cols, dtype=torch.uint8)
    unary = torch.empty(int(s.unary_words), dtype=torch.int32)
    rem = torch.empty(int(s.rem_words), dtype=torch.int32) if table.k > 0 else None
    anchor = torch.empty(int(s.n_chunks) + 1, dtype=torch.int64)
    esc_pre = torch.empty(int(s.n_chunks) + 1, dtype=torch.int32)
    planes = RicePlanes(rows, cols, table, sm, unary, rem, anchor, esc_pre, 0, 0)
    d = planes.desc()
    _call("binade_pack_rice", _ptr(w), rows, cols, ctypes.byref(table), ctypes.byref(d))
    planes.unary_bits = int(d.unary_bits)
    planes.n_esc = int(d.n_esc)
    return planes


def build_table_gpu(w: torch.Tensor, workspace: torch.Tensor | None = None,
                    stream=None) -> Table:
    """binade_build_table_gpu on a device bf16 tensor; the table is copied
    back to the host (one synchronisation)."""
    w = _bits16(w)
    if not w.is_cuda:
        raise ValueError("build_table_gpu takes a device tensor")
    if workspace is None:
        workspace = torch.empty(2048, dtype=torch.uint8, device=w.device)
    dt = torch.empty(ctypes.sizeof(Table), dtype=torch.uint8, device=w.device)
    s = torch.cuda.current_stream(w.device) if stream is None else stream
    with torch.cuda.stream(s):
        _call("binade_build_table_gpu", _ptr(w), w.numel(), _ptr(workspace), _ptr(dt),
              _stream(s))
        host = dt.cpu()
    t = Table()
    ctypes.memmove(ctypes.addressof(t), host.numpy().ctypes.data, ctypes.sizeof(Table))
    return t


def pack_rice_gpu(w: torch.Tensor, table: Table | None = None, status: torch.Tensor | None = None,
                  stream=None) -> RicePlanes:
    """binade_pack_rice_gpu: device bf16 [rows, cols] -> device format 2
    planes, byte-identical to pack_rice; the table is built on the device
    when not given."""
    w = _bits16(w)
    if not w.is_cuda or w.dim() != 2:
        raise ValueError("pack_rice_gpu takes a 2-D device tensor")
    rows, cols = w.shape
    dev = w.device
    s = torch.cuda.current_stream(dev) if stream is None else stream
    ws_bytes = int(lib().binade_pack_gpu_workspace_bytes(rows, cols))
    with torch.cuda.stream(s):
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        if table is None:
            table = build_table_gpu(w, ws, stream=s)
        sz = sizes_of(table, rows, cols)
        sm = torch.empty(rows, cols, dtype=torch.uint8, device=dev)
        unary = torch.empty(int(sz.unary_words), dtype=torch.int32, device=dev)
        rem = (torch.empty(int(sz.rem_words), dtype=torch.int32, device=dev)
               if table.k > 0 else None)
        anchor = torch.empty(int(sz.n_chunks) + 1, dtype=torch.int64, device=dev)
        esc_pre = torch.empty(int(sz.n_chunks) + 1, dtype=torch.int32, device=dev)
        planes = RicePlanes(rows, cols, table, sm, unary, rem, anchor, esc_pre, 0, 0)
        d = planes.desc()
        _call("binade_pack_rice_gpu", _ptr(w), rows, cols, ctypes.byref(table), ctypes.byref(d),
              _ptr(ws), _ptr(status), _stream(s))
        ws.record_stream(s)
    planes.unary_bits = int(d.unary_bits)
    planes.n_esc = int(d.n_esc)
    return planes


@dataclass
class HuffPlanes:
    """Huffman comparison-codec planes (host or device tensors)."""
    n: int
    len: bytes
    sm: torch.Tensor
    stream: torch.Tensor
    stream_bytes: int
    block_len: torch.Tensor
    group_off: torch.Tensor

    def desc(self) -> HuffDesc:
        d = HuffDesc()
        d.n = self.n
        ctypes.memmove(d.len, self.len, 256)
        d.sm = self.sm.data_ptr()
        d.stream = self.stream.data_ptr()
        d.stream_bytes = self.stream_bytes
        d.stream_cap = self.stream.numel()
        d.block_len = self.block_len.data_ptr()
        d.group_off = self.group_off.data_ptr()
        return d

    def to(self, device) -> "HuffPlanes":
        return HuffPlanes(self.n, self.len, self.sm.to(device), self.stream.to(device),
                          self.stream_bytes, self.block_len.to(device), self.group_off.to(device))

    def bits_per_weight(self) -> float:
        return (8 * self.n + 8 * self.stream_bytes + 8 * self.block_len.numel()
                + 64 * self.group_off.numel()) / self.n


def pack_huff(w: torch.Tensor) -> HuffPlanes:
    """binade_huff_lengths + binade_huff_pack on a host bf16 tensor."""
    w = _bits16(w).reshape(-1)
    if w.is_cuda:
        raise ValueError("pack_huff takes a host tensor")
    n = w.numel()
    ln = (ctypes.c_uint8 * 256)()
    cap = ctypes.c_uint64(0)
    _call("binade_huff_lengths", _ptr(w), n, ln, ctypes.byref(cap))
    nb = (n + 63) // 64
    planes = HuffPlanes(n, bytes(ln), torch.empty(n, dtype=torch.uint8),
                        torch.empty(int(cap.value), dtype=torch.uint8), 0,
                        torch.empty(nb, dtype=torch.uint8),
                        torch.empty((nb + 127) // 128 + 1, dtype=torch.int64))
    d = planes.desc()
    _call("binade_huff_pack", _ptr(w), ctypes.byref(d))
    planes.stream_bytes = int(d.stream_bytes)
    return planes


@_on_stream
def huff_decode(p: HuffPlanes, out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """binade_huff_decode: device planes -> bf16[n]."""
    dev = p.sm.device
    if out is None:
        out = torch.empty(p.n, dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(int(lib().binade_huff_workspace_bytes()), dtype=torch.uint8,
                                device=dev)
    d = p.desc()
    _call("binade_huff_decode", ctypes.byref(d), _ptr(out), _ptr(workspace), _ptr(status),
          _stream(stream))
    return out


@dataclass
class F1Planes:
    """Format 1 planes of one tensor (host or device tensors) + descriptor."""
    rows: int
    cols: int
    table: Table
    sm: torch.Tensor
    width: torch.Tensor
    codes: torch.Tensor
    esc_rank: torch.Tensor
    anchor: torch.Tensor
    f1_pre: torch.Tensor
    esc_pre: torch.Tensor
    code_bits: int
    n_f1esc: int
    n_esc: int

    def desc(self) -> F1Desc:
        d = F1Desc()
        d.rows, d.cols, d.n = self.rows, self.cols, self.table.n
        ctypes.memmove(d.exp_of_rank, self.table.exp_of_rank, 256)
        d.sm = self.sm.data_ptr()
        d.width = self.width.data_ptr()
        d.codes = self.codes.data_ptr()
        d.code_bits = self.code_bits
        d.code_words = self.codes.numel()
        d.esc_rank = self.esc_rank.data_ptr()
        d.n_f1esc = self.n_f1esc
        d.esc_cap = self.esc_rank.numel()
        d.anchor = self.anchor.data_ptr()
        d.f1_pre = self.f1_pre.data_ptr()
        d.esc_pre = self.esc_pre.data_ptr()
        d.n_esc = self.n_esc
        return d

    def to(self, device) -> "F1Planes":
        """The planes on `device`; the code and escape planes trimmed to what
        the tensor uses (plus a padding word)."""
        cw = (self.code_bits + 31) // 32 + 2
        mv = lambda t: t.to(device, non_blocking=False)
        return F1Planes(self.rows, self.cols, self.table, mv(self.sm), mv(self.width),
                        mv(self.codes[:cw]), mv(self.esc_rank[: max(self.n_f1esc, 1)]),
                        mv(self.anchor), mv(self.f1_pre), mv(self.esc_pre),
                        self.code_bits, self.n_f1esc, self.n_esc)

    def bits_per_weight(self) -> float:
        """Format 1 as stored: sm byte, codes, escape bytes, a width byte per
        tile and 16 index bytes per row-chunk."""
        n = self.rows * self.cols
        bits = (8 * n + self.code_bits + 8 * self.n_f1esc + 8 * self.width.numel()
                + 128 * self.anchor.numel())
        return bits / n


def pack_f1(w: torch.Tensor, table: Table | None = None) -> F1Planes:
    """binade_pack_f1: host bf16 [rows, cols] -> host format 1 planes."""
    w = _bits16(w)
    if w.is_cuda or w.dim() != 2:
        raise ValueError("pack_f1 takes a 2-D host tensor")
    rows, cols = w.shape
    if table is None:
        table = build_table(w)
    s = F1Sizes()
    _call("binade_f1_sizes_of", rows, cols, ctypes.byref(s))
    planes = F1Planes(rows, cols, table, torch.empty(rows, cols, dtype=torch.uint8),
                      torch.empty(int(s.n_tiles), dtype=torch.uint8),
                      torch.empty(int(s.code_words), dtype=torch.int32),
                      torch.empty(int(s.esc_cap), dtype=torch.uint8),
                      torch.empty(int(s.n_chunks) + 1, dtype=torch.int64),
                      torch.empty(int(s.n_chunks) + 1, dtype=torch.int32),
                      torch.empty(int(s.n_chunks) + 1, dtype=torch.int32), 0, 0, 0)
    d = planes.desc()
    _call("binade_pack_f1", _ptr(w), rows, cols, ctypes.byref(table), ctypes.byref(d))
    planes.code_bits = int(d.code_bits)
    planes.n_f1esc = int(d.n_f1esc)
    planes.n_esc = int(d.n_esc)
    return planes


# ------------------------------------------------------------------ device
@dataclass
class R4Tensor:
    """R4 weights on the device. sm and esc_pre are the format 2 planes'."""
    rows: int
    cols: int
    lut: bytes
    sm: torch.Tensor
    nib: torch.Tensor
    esc_pre: torch.Tensor
    esc: torch.Tensor
    n_esc: int
    _keep: list = field(default_factory=list, repr=False)

    def desc(self) -> R4Desc:
        """The C descriptor (built once; the tensors must not be replaced)."""
        d = getattr(self, "_desc", None)
        if d is None or d.lut[:] != list(self.lut):
            d = R4Desc()
            d.rows, d.cols = self.rows, self.cols
            ctypes.memmove(d.lut, self.lut, 16)
            d.sm = self.sm.data_ptr()
            d.nib = self.nib.data_ptr()
            d.esc_pre = self.esc_pre.data_ptr()
            d.esc = self.esc.data_ptr() if self.n_esc > 0 else None
            d.n_esc = self.n_esc
            self._desc = d
        return d

    def nbytes(self) -> int:
        return (self.sm.numel() + self.nib.numel() + 4 * self.esc_pre.numel()
                + 4 * self.n_esc)

    def bits_per_weight(self) -> float:
        return 8.0 * self.nbytes() / (self.rows * self.cols)


def r4_from_planes(rows, cols, lut, sm, nib, esc_pre, esc) -> R4Tensor:
    """Wrap R4 planes that are already on the device."""
    return R4Tensor(rows, cols, bytes(bytearray(lut)), sm, nib, esc_pre, esc,
                    int(esc.numel()))


@_on_stream
def rice_to_r4(planes: RicePlanes, status: torch.Tensor | None = None,
               stream=None, out: R4Tensor | None = None) -> R4Tensor:
    """binade_rice_to_r4 on device planes; allocates nib / esc unless `out`."""
    if not planes.sm.is_cuda:
        raise ValueError("rice_to_r4 takes device planes (RicePlanes.to('cuda'))")
    dev = planes.sm.device
    if out is None:
        nib = torch.empty(planes.rows * planes.cols // 2, dtype=torch.uint8, device=dev)
        esc = torch.empty(max(planes.n_esc, 1), dtype=torch.int32, device=dev)
    else:
        nib, esc = out.nib, out.esc
    d_in = planes.desc()
    d_out = R4Desc()
    d_out.nib = nib.data_ptr()
    d_out.esc = esc.data_ptr()
    _call("binade_rice_to_r4", ctypes.byref(d_in), ctypes.byref(d_out),
          _ptr(status), _stream(stream))
    lut = bytes(d_out.lut)
    if out is not None:
        out.lut = lut
        return out
    return R4Tensor(planes.rows, planes.cols, lut, planes.sm, nib,
                    planes.esc_pre, esc, planes.n_esc)


@_on_stream
def f1_to_r4(planes: F1Planes, status: torch.Tensor | None = None,
             stream=None, out: R4Tensor | None = None) -> R4Tensor:
    """binade_f1_to_r4 on device planes; allocates nib / esc unless `out`."""
    if not planes.sm.is_cuda:
        raise ValueError("f1_to_r4 takes device planes (F1Planes.to('cuda'))")
    dev = planes.sm.device
    if out is None:
        nib = torch.empty(planes.rows * planes.cols // 2, dtype=torch.uint8, device=dev)
        esc = torch.empty(max(planes.n_esc, 1), dtype=torch.int32, device=dev)
    else:
        nib, esc = out.nib, out.esc
    d_in = planes.desc()
    d_out = R4Desc()
    d_out.nib = nib.data_ptr()
    d_out.esc = esc.data_ptr()
    _call("binade_f1_to_r4", ctypes.byref(d_in), ctypes.byref(d_out),
          _ptr(status), _stream(stream))
    lut = bytes(d_out.lut)
    if out is not None:
        out.lut = lut
        return out
    return R4Tensor(planes.rows, planes.cols, lut, planes.sm, nib,
                    planes.esc_pre, esc, planes.n_esc)


def _r4_out(p) -> "R4Tensor":
    """Device buffers for the R4 form of format 2 tensor p."""
    dev = p.sm.device
    return R4Tensor(p.rows, p.cols, bytes(16), p.sm,
                    torch.empty(p.rows * p.cols // 2, dtype=torch.uint8, device=dev),
                    p.esc_pre,
                    torch.empty(max(p.n_esc, 1), dtype=torch.int32, device=dev),
                    p.n_esc)


@_on_stream
def rice_to_r4_batch(planes: list, status: torch.Tensor | None = None,
                     stream=None, outs: list | None = None) -> list:
    """binade_rice_to_r4_batch: decode several tensors (up to 16 per launch)."""
    n = len(planes)
    if outs is None:
        outs = [_r4_out(p) for p in planes]
    din = (RiceDesc * n)(*[p.desc() for p in planes])
    dout = (R4Desc * n)()
    for i, o in enumerate(outs):
        dout[i].nib = o.nib.data_ptr()
        dout[i].esc = o.esc.data_ptr()
    _call("binade_rice_to_r4_batch", din, dout, n, _ptr(status), _stream(stream))
    for i, o in enumerate(outs):
        o.lut = bytes(dout[i].lut)
    return outs


class RicePlan:
    """A decode plan over format 2 tensors (binade_rice_to_r4_plan): their R4
    outputs, the plan's host bytes and its copy in device memory. run()
    decodes every tensor in one launch (binade_rice_to_r4_run). The plan
    keeps references to the planes and outputs whose addresses it holds."""

    def __init__(self, planes: list, outs: list | None = None):
        n = len(planes)
        self.planes = list(planes)
        self.outs = [_r4_out(p) for p in planes] if outs is None else list(outs)
        din = (RiceDesc * n)(*[p.desc() for p in planes])
        dout = (R4Desc * n)()
        for i, o in enumerate(self.outs):
            dout[i].nib = o.nib.data_ptr()
            dout[i].esc = o.esc.data_ptr()
        nbytes = lib().binade_rice_plan_bytes(n)
        if nbytes < 0:
            raise BinadeError("binade_rice_plan_bytes", int(nbytes), 0)
        self.host = (ctypes.c_uint8 * nbytes)()
        _call("binade_rice_to_r4_plan", din, dout, n, self.host, nbytes)
        for i, o in enumerate(self.outs):
            o.lut = bytes(dout[i].lut)
        device = planes[0].sm.device if n else torch.device("cpu")   # an empty plan never launches
        self.dev = torch.frombuffer(bytearray(self.host), dtype=torch.uint8).to(device)

    @_on_stream
    def run(self, status: torch.Tensor | None = None, stream=None) -> list:
        _call("binade_rice_to_r4_run", self.host, ctypes.c_void_p(self.dev.data_ptr()),
              _ptr(status), _stream(stream))
        return self.outs


@_on_stream
def r4_gemv_batch(ws: list, xs: list, out_dtype=torch.float32,
                  ys: list | None = None, stream=None) -> list:
    """binade_r4_gemv_batch: several independent R4 GEMVs in one launch."""
    code = _dtype_code(out_dtype)
    n = len(ws)
    if ys is None:
        ys = [_y((w.rows,), code, x.device, None) for w, x in zip(ws, xs)]
    dws = (R4Desc * n)(*[w.desc() for w in ws])
    dxs = (ctypes.c_void_p * n)(*[_bits16(x).data_ptr() for x in xs])
    dys = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
    _call("binade_r4_gemv_batch", dws, dxs, dys, n, code, _stream(stream))
    return ys


@_on_stream
def bf16_gemv_batch(ws: list, xs: list, out_dtype=torch.float32,
                    ys: list | None = None, stream=None) -> list:
    """binade_bf16_gemv_batch: the batched twin."""
    code = _dtype_code(out_dtype)
    n = len(ws)
    ws = [_bits16(w) for w in ws]
    if ys is None:
        ys = [_y((w.shape[0],), code, x.device, None) for w, x in zip(ws, xs)]
    dws = (ctypes.c_void_p * n)(*[w.data_ptr() for w in ws])
    rows = (ctypes.c_int64 * n)(*[w.shape[0] for w in ws])
    cols = (ctypes.c_int64 * n)(*[w.shape[1] for w in ws])
    dxs = (ctypes.c_void_p * n)(*[_bits16(x).data_ptr() for x in xs])
    dys = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
    _call("binade_bf16_gemv_batch", dws, rows, cols, dxs, dys, n, code, _stream(stream))
    return ys


def _y(rows_shape, y_dtype, device, y):
    if y is not None:
        return y
    dt = torch.float32 if y_dtype == F32 else torch.bfloat16
    return torch.empty(rows_shape, dtype=dt, device=device)


def _dtype_code(out_dtype) -> int:
    if out_dtype in (torch.float32, F32, "f32"):
        return F32
    if out_dtype in (torch.bfloat16, BF16, "bf16"):
        return BF16
    raise ValueError(out_dtype)


@_on_stream
def r4_gemv(w: R4Tensor, x: torch.Tensor, out_dtype=torch.float32,
            y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    code = _dtype_code(out_dtype)
    x = _bits16(x)
    y = _y((w.rows,), code, x.device, y)
    d = w.desc()
    _call("binade_r4_gemv", ctypes.byref(d), _ptr(x), _ptr(y), code, _stream(stream))
    return y


@_on_stream
def bf16_gemv(w: torch.Tensor, x: torch.Tensor, out_dtype=torch.float32,
              y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    code = _dtype_code(out_dtype)
    w = _bits16(w)
    x = _bits16(x)
    rows, cols = w.shape
    y = _y((rows,), code, x.device, y)
    _call("binade_bf16_gemv", _ptr(w), rows, cols, _ptr(x), _ptr(y), code,
          _stream(stream))
    return y


@_on_stream
def r4_gemv_rows(w: R4Tensor, x: torch.Tensor, out_dtype=torch.float32,
                 y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """binade_r4_gemv_rows: Y[b] = W x[b] for the 1..8 rows of x [m, K]; each
    row bit-identical to r4_gemv of that row."""
    code = _dtype_code(out_dtype)
    x = _bits16(x)
    m = x.shape[0]
    y = _y((m, w.rows), code, x.device, y)
    d = w.desc()
    _call("binade_r4_gemv_rows", ctypes.byref(d), _ptr(x), x.shape[1], m, _ptr(y),
          y.shape[1], code, _stream(stream))
    return y


@_on_stream
def bf16_gemv_rows(w: torch.Tensor, x: torch.Tensor, out_dtype=torch.float32,
                   y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """binade_bf16_gemv_rows: the twin of r4_gemv_rows."""
    code = _dtype_code(out_dtype)
    w = _bits16(w)
    x = _bits16(x)
    rows, cols = w.shape
    m = x.shape[0]
    y = _y((m, rows), code, x.device, y)
    _call("binade_bf16_gemv_rows", _ptr(w), rows, cols, _ptr(x), x.shape[1], m, _ptr(y),
          y.shape[1], code, _stream(stream))
    return y


@_on_stream
def moe_silu_mul(gate: torch.Tensor, up: torch.Tensor, out_dtype=torch.bfloat16,
                 h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """binade_moe_silu_mul: h = silu(gate) * up (fp64 inside, one rounding)."""
    code = _dtype_code(out_dtype)
    if gate.dtype != torch.float32 or up.dtype != torch.float32 or gate.shape != up.shape:
        raise ValueError("gate and up: fp32 tensors of one shape")
    gate = gate.contiguous()
    up = up.contiguous()
    h = _y(tuple(gate.shape), code, gate.device, h)
    _call("binade_moe_silu_mul", _ptr(gate), _ptr(up), gate.numel(), _ptr(h), code,
          _stream(stream))
    return h


@_on_stream
def moe_combine(y: torch.Tensor, weights: torch.Tensor, top_k: int, out_dtype=torch.float32,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """binade_moe_combine: out[t] = sum over the token's top_k slots of
    weight * y, an fp32 fma chain in slot order."""
    code = _dtype_code(out_dtype)
    if y.dtype != torch.float32 or weights.dtype != torch.float32:
        raise ValueError("y and weights: fp32")
    y = y.contiguous()
    weights = weights.contiguous()
    pairs, n = y.shape
    if pairs % top_k or weights.numel() != pairs:
        raise ValueError("y rows and weights must be n_tokens * top_k")
    out = _y((pairs // top_k, n), code, y.device, out)
    _call("binade_moe_combine", _ptr(y), _ptr(weights), pairs // top_k, top_k, n, _ptr(out),
          code, _stream(stream))
    return out


@_on_stream
def unpack(w: R4Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.nib.device)
    d = w.desc()
    _call("binade_unpack", ctypes.byref(d), _ptr(out), _stream(stream))
    return out


def gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    """Bytes of workspace with which an M x N x K GEMM splits its slices
    over blocks (0: it never does)."""
    return int(lib().binade_gemm_workspace_bytes(m, n, k))


def _workspace(m, n, k, device, workspace):
    if workspace is None:
        nb = gemm_workspace_bytes(m, n, k)
        if nb == 0:
            return None, 0
        workspace = torch.empty(nb, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


@_on_stream
def r4_gemm(w: R4Tensor, x: torch.Tensor, out_dtype=torch.float32,
            y: torch.Tensor | None = None, stream=None,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W^T. workspace: optional device buffer (a fresh one of
    gemm_workspace_bytes is taken from torch's allocator when None)."""
    code = _dtype_code(out_dtype)
    x = _bits16(x)
    m = x.shape[0]
    y = _y((m, w.rows), code, x.device, y)
    ws, nb = _workspace(m, w.rows, w.cols, x.device, workspace)
    d = w.desc()
    _call("binade_r4_gemm", ctypes.byref(d), _ptr(x), m, x.stride(0), _ptr(y),
          y.stride(0), code, _ptr(ws), nb, _stream(stream))
    return y


@_on_stream
def r4_gemm_noalloc(w: R4Tensor, x: torch.Tensor, out_dtype=torch.float32,
                    y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W^T through binade_r4_gemm_noalloc (the library's fixed scratch,
    no workspace). With y given, nothing is allocated here either."""
    code = _dtype_code(out_dtype)
    x = _bits16(x)
    m = x.shape[0]
    y = _y((m, w.rows), code, x.device, y)
    d = w.desc()
    _call("binade_r4_gemm_noalloc", ctypes.byref(d), _ptr(x), m, x.stride(0),
          _ptr(y), y.stride(0), code, _stream(stream))
    return y


def gemm_scratch_bytes() -> int:
    return int(lib().binade_gemm_scratch_bytes())


@_on_stream
def bf16_gemm(w: torch.Tensor, x: torch.Tensor, out_dtype=torch.float32,
              y: torch.Tensor | None = None, stream=None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    code = _dtype_code(out_dtype)
    w = _bits16(w)
    x = _bits16(x)
    rows, cols = w.shape
    m = x.shape[0]
    y = _y((m, rows), code, x.device, y)
    ws, nb = _workspace(m, rows, cols, x.device, workspace)
    _call("binade_bf16_gemm", _ptr(w), rows, cols, _ptr(x), m, x.stride(0),
          _ptr(y), y.stride(0), code, _ptr(ws), nb, _stream(stream))
    return y


@_on_stream
def r4_moe_gemv(experts: R4Tensor, n_experts: int, x: torch.Tensor,
                idx: torch.Tensor, x_per_slot: bool = False,
                out_dtype=torch.float32, y: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    code = _dtype_code(out_dtype)
    x = _bits16(x)
    idx = idx.contiguous()
    n_tokens, top_k = idx.shape
    N = experts.rows // n_experts
    y = _y((n_tokens * top_k, N), code, x.device, y)
    d = experts.desc()
    _call("binade_r4_moe_gemv", ctypes.byref(d), n_experts, _ptr(x),
          1 if x_per_slot else 0, _ptr(idx), n_tokens, top_k, _ptr(y), code,
          _ptr(status), _stream(stream))
    return y


@_on_stream
def bf16_moe_gemv(experts: torch.Tensor, n_experts: int, x: torch.Tensor,
                  idx: torch.Tensor, x_per_slot: bool = False,
                  out_dtype=torch.float32, y: torch.Tensor | None = None,
                  status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    code = _dtype_code(out_dtype)
    experts = _bits16(experts)
    x = _bits16(x)
    idx = idx.contiguous()
    rows, cols = experts.shape
    N = rows // n_experts
    n_tokens, top_k = idx.shape
    y = _y((n_tokens * top_k, N), code, x.device, y)
    _call("binade_bf16_moe_gemv", _ptr(experts), n_experts, N, cols, _ptr(x),
          1 if x_per_slot else 0, _ptr(idx), n_tokens, top_k, _ptr(y), code,
          _ptr(status), _stream(stream))
    return y


# ------------------------------------------------------------------ router
_bound: dict = {}


def _entry(name: str):
    """A library function, looked up once."""
    fn = _bound.get(name)
    if fn is None:
        fn = _bound[name] = getattr(lib(), name)
    return fn


def _run(name: str, *args):
    rc = _entry(name)(*args)
    if rc != OK:
        raise BinadeError(name, rc, lib().binade_last_hip_error() if rc == EHIP else 0)


def _on_device(fn):
    """Run a device binding on the device of its first argument, with `stream`
    as a raw handle: temporaries and a default stream are that device's even
    when another one is current, and a given stream is torch's current one
    meanwhile (as in _on_stream)."""
    lead = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kw):
        first = args[0] if args else kw.get(lead)
        index = first.get_device() if isinstance(first, torch.Tensor) else -1
        if index < 0:
            raise ValueError(f"{fn.__name__} takes device tensors")
        if stream is None and index == torch._C._cuda_getDevice():
            return fn(*args, stream=torch._C._cuda_getCurrentRawStream(index), **kw)
        with torch.cuda.device(index):
            if stream is None:
                stream = torch.cuda.current_stream()
            elif not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream))
            elif stream.device_index != index:
                raise ValueError("stream of another device")
            with torch.cuda.stream(stream):
                return fn(*args, stream=stream.cuda_stream, **kw)
    return wrapper


def _arg(name: str, t: torch.Tensor, dtypes, shape, device) -> torch.Tensor:
    """t checked: one of dtypes, the shape, the device, and contiguous."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    return t.contiguous()


def _out_arg(name: str, t: torch.Tensor | None, dtype, shape, device) -> torch.Tensor:
    """An output: allocated, or the caller's, which has to fit as it is."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    return _arg(name, t, (dtype,), shape, device)


def _status_arg(status: torch.Tensor | None, device):
    """The address of a status word, or None."""
    if status is None:
        return None
    if status.device != device or status.element_size() != 4 or status.numel() < 1:
        raise ValueError("status: one 32-bit word on the device")
    return status.data_ptr()


def _scratch(nbytes: int, workspace: torch.Tensor | None, device):
    """(tensor, address, bytes) of a workspace: the caller's, or from torch's
    allocator."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


_FLOATS = (torch.bfloat16, torch.float32)
_BF16_ONLY, _F32_ONLY, _I32_ONLY = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_CODE = {torch.float32: F32, torch.bfloat16: BF16}
_TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16}


def _logits_arg(t: torch.Tensor):
    """(logits [n_tokens, n_experts], their row stride); copied if a row's
    values do not lie side by side or rows overlap. A single row's stride is
    of no matter (torch calls it contiguous whatever it is)."""
    if t.dtype not in _CODE:
        raise TypeError(f"logits: {t.dtype}, expected bf16 or fp32")
    if t.dim() != 2:
        raise ValueError("logits: [n_tokens, n_experts]")
    rows, cols = t.shape
    if t.stride(1) == 1 and rows > 1 and t.stride(0) >= cols:
        return t, t.stride(0)
    return t.contiguous(), cols


@dataclass
class MoeRoute:
    """What moe_route gives: the slots' experts and weights, and with stats
    the counts (the last entry: rows that count), the summed probabilities
    and the balance loss."""
    idx: torch.Tensor
    weights: torch.Tensor
    counts: torch.Tensor | None = None
    prob_sum: torch.Tensor | None = None
    loss: torch.Tensor | None = None


_SCORES = {"softmax": 0, "sigmoid": 1}


def _score_code(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score: {score!r}, expected 'softmax' or 'sigmoid'")
    return _SCORES[score]


@_on_device
def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True,
              valid: torch.Tensor | None = None, stats: bool = True,
              workspace: torch.Tensor | None = None, stream=None, *, score: str = "softmax",
              bias: torch.Tensor | None = None, groups: int = 1, top_groups: int = 1,
              group_best: int = 2, scale: float = 1.0) -> MoeRoute:
    """binade_moe_route: each token's top_k experts (idx int32 [T, top_k], for
    r4_moe_gemv and f8_moe_gemm) and their weights (fp32 [T, top_k], for
    moe_combine) from logits [T, E]; valid: bool or uint8 [T], False for
    padding. With another score than softmax, a bias (fp32 [E], added for the
    choice alone), groups or a scale: binade_moe_route_scored, the top_k best
    experts of the top_groups best of `groups` groups, a group's score the sum
    of its group_best best."""
    logits, ld = _logits_arg(logits)
    dev = logits.device
    T, E = logits.shape
    if valid is not None:
        valid = _arg("valid", valid, (torch.bool, torch.uint8), (T,), dev)
    if top_k < 1:
        raise BinadeError("binade_moe_route", EINVAL)
    out = MoeRoute(torch.empty((T, top_k), dtype=torch.int32, device=dev),
                   torch.empty((T, top_k), dtype=torch.float32, device=dev))
    ws, at, nb = None, None, 0
    if stats:
        out.counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
        out.prob_sum = torch.empty(E, dtype=torch.float32, device=dev)
        out.loss = torch.empty(1, dtype=torch.float32, device=dev)
    code = _score_code(score)
    if code or bias is not None or groups != 1 or top_groups != 1 or scale != 1.0:
        if bias is not None:
            bias = _arg("bias", bias, _F32_ONLY, (E,), dev)
        rule = RouteRule(code, 1 if renormalize else 0, groups, top_groups, group_best, scale,
                         _addr(bias))
        if stats:
            ws, at, nb = _scratch(_entry("binade_moe_route_scored_workspace_bytes")(T, E),
                                  workspace, dev)
        _run("binade_moe_route_scored", logits.data_ptr(), _CODE[logits.dtype], ld, T, E, top_k,
             ctypes.byref(rule), _addr(valid), out.idx.data_ptr(), out.weights.data_ptr(),
             _addr(out.counts), _addr(out.prob_sum), _addr(out.loss), at, nb, stream)
        return out
    if stats:
        ws, at, nb = _scratch(_entry("binade_moe_route_workspace_bytes")(T, E), workspace, dev)
    _run("binade_moe_route", logits.data_ptr(), _CODE[logits.dtype], ld, T, E,
         top_k, 1 if renormalize else 0, _addr(valid), out.idx.data_ptr(),
         out.weights.data_ptr(), _addr(out.counts), _addr(out.prob_sum), _addr(out.loss), at, nb,
         stream)
    return out


@_on_device
def moe_route_grad(logits: torch.Tensor, idx: torch.Tensor,
                   dweights: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                   dloss: torch.Tensor | None = None, renormalize: bool = True, out_dtype=None,
                   dlogits: torch.Tensor | None = None, status: torch.Tensor | None = None,
                   stream=None, *, score: str = "softmax", bias: torch.Tensor | None = None,
                   groups: int = 1, scale: float = 1.0) -> torch.Tensor:
    """binade_moe_route_grad: the gradient of the logits from that of the
    weights and (counts and dloss together) of the balance loss. score, bias,
    groups and scale as moe_route had them (binade_moe_route_scored_grad where
    one of them is not the default; of bias and groups no value matters, only
    that the choice went by them)."""
    logits, ld = _logits_arg(logits)
    dev = logits.device
    T, E = logits.shape
    code = _CODE[logits.dtype] if out_dtype is None else _dtype_code(out_dtype)
    if idx.dim() != 2:
        raise ValueError("idx: [n_tokens, top_k]")
    top_k = idx.shape[1]
    idx = _arg("idx", idx, _I32_ONLY, (T, top_k), dev)
    if dweights is not None:
        dweights = _arg("dweights", dweights, _F32_ONLY, (T, top_k), dev)
    if (counts is None) != (dloss is None):
        raise ValueError("counts and dloss go together")
    if counts is not None:
        counts = _arg("counts", counts, _I32_ONLY, (E + 1,), dev)
        dloss = _arg("dloss", dloss.reshape(-1), (torch.float32,), (1,), dev)
    dlogits = _out_arg("dlogits", dlogits, _TORCH_DTYPE[code], (T, E), dev)
    kind = _score_code(score)
    if kind or bias is not None or groups != 1 or scale != 1.0:
        _run("binade_moe_route_scored_grad", logits.data_ptr(), _CODE[logits.dtype], ld, T, E,
             top_k, kind, 1 if renormalize else 0, scale, idx.data_ptr(), _addr(dweights),
             _addr(counts), _addr(dloss), dlogits.data_ptr(), code, E, _status_arg(status, dev),
             stream)
        return dlogits
    _run("binade_moe_route_grad", logits.data_ptr(), _CODE[logits.dtype], ld, T, E,
         top_k, 1 if renormalize else 0, idx.data_ptr(), _addr(dweights), _addr(counts),
         _addr(dloss), dlogits.data_ptr(), code, E, _status_arg(status, dev), stream)
    return dlogits


@_on_device
def moe_combine_grad(y: torch.Tensor, weights: torch.Tensor, dout: torch.Tensor, top_k: int,
                     out_dtype=torch.float32, need_dy: bool = True, stream=None):
    """binade_moe_combine_grad: (dy [T*top_k, N] or None, dweights fp32
    [T*top_k] in the shape of weights) of moe_combine(y, weights, top_k)."""
    code = _dtype_code(out_dtype)
    dev = y.device
    if y.dim() != 2 or dout.dim() != 2:
        raise ValueError("y: [n_tokens * top_k, N], dout: [n_tokens, N]")
    T, N = dout.shape
    y = _arg("y", y, _F32_ONLY, (T * top_k, N), dev)
    dout = _arg("dout", dout, _FLOATS, (T, N), dev)
    if weights.numel() != T * top_k:
        raise ValueError("weights: n_tokens * top_k")
    w = _arg("weights", weights, _F32_ONLY, weights.shape, dev)
    dy = torch.empty_like(y, dtype=_TORCH_DTYPE[code]) if need_dy else None
    dw = torch.empty_like(w)
    _run("binade_moe_combine_grad", y.data_ptr(), w.data_ptr(), dout.data_ptr(),
         _CODE[dout.dtype], T, top_k, N, _addr(dy), code, dw.data_ptr(), stream)
    return dy, dw


# ---------------------------------------------------------------- adapters
_MAX_STRIDE = 1 << 24


def _rows16(name: str, t: torch.Tensor, cols: int, device, m: int | None = None):
    """(bf16 [m, cols] rows at a 16-byte aligned stride that the calls take,
    copied otherwise; that stride). A single row's stride is of no matter
    (torch calls it contiguous whatever it is)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: {t.dtype}, expected bf16")
    if t.dim() != 2 or t.shape[1] != cols or (m is not None and t.shape[0] != m):
        raise ValueError(f"{name}: shape {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    ld = t.stride(0)
    if t.shape[0] > 1 and t.stride(1) == 1 and cols <= ld <= _MAX_STRIDE and ld % 8 == 0 \
            and t.data_ptr() % 16 == 0:
        return t, ld
    t = t.contiguous()
    if t.data_ptr() % 16:               # a contiguous view that starts off 16 bytes
        t = t.clone()
    return t, cols


def _lora_desc(a, b, scale, device):
    """(descriptor, the tensors it points at, n, k, rank, n_adapters)."""
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a: [n_adapters, rank, K], b: [n_adapters, N, rank]")
    n_adapters, rank, k = shape = a.shape
    n = b.shape[1]
    a = _arg("a", a, _BF16_ONLY, shape, device)
    b = _arg("b", b, _BF16_ONLY, (n_adapters, n, rank), device)
    at = None
    if scale is not None:
        scale = _arg("scale", scale, _F32_ONLY, (n_adapters,), device)
        at = scale.data_ptr()
    d = LoraDesc(n, k, rank, n_adapters, a.data_ptr(), b.data_ptr(), at)
    return d, (a, b, scale), n, k, rank, n_adapters


@_on_device
def lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor | None = None,
             base: torch.Tensor | None = None, scale: torch.Tensor | None = None,
             out_dtype=torch.float32, y: torch.Tensor | None = None, keep_h: bool = False,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
             stream=None):
    """binade_lora_add: base + scale * B (A x) with row t's adapter ids[t]
    (None: adapter 0 for all; -1: none), beside r4_gemv_rows / r4_gemm of the
    same x [m, K]. y may be base. With keep_h: (y, h), h fp32 [m, rank] for
    lora_grad."""
    code = _dtype_code(out_dtype)
    dev = x.device
    d, keep, n, k, rank, _ = _lora_desc(a, b, scale, dev)
    x, ldx = _rows16("x", x, k, dev)
    m = x.shape[0]
    if ids is not None:
        ids = _arg("ids", ids, _I32_ONLY, (m,), dev)
    if base is not None:
        base = _arg("base", base, _FLOATS, (m, n), dev)
    if y is None and base is not None:
        y = torch.empty_like(base, dtype=_TORCH_DTYPE[code])
    else:
        y = _out_arg("y", y, _TORCH_DTYPE[code], (m, n), dev)
    h = torch.empty((m, rank), dtype=torch.float32, device=dev) if keep_h else None
    ws, at, nb = _scratch(_entry("binade_lora_workspace_bytes")(m, n, k, rank), workspace, dev)
    _run("binade_lora_add", ctypes.byref(d), x.data_ptr(), m, ldx, _addr(ids),
         _addr(base), n, F32 if base is None else _CODE[base.dtype], y.data_ptr(), n, code,
         _addr(h), at, nb, _status_arg(status, dev), stream)
    return (y, h) if keep_h else y


@_on_device
def lora_grad(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor | None,
              dy: torch.Tensor, h: torch.Tensor | None = None, scale: torch.Tensor | None = None,
              dx_base: torch.Tensor | None = None, grad_dtype=torch.float32,
              dx: torch.Tensor | None = None, need_dx: bool = True,
              workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
              stream=None):
    """binade_lora_grad: (dx bf16 [m, K] or None, da, db) of lora_add from dy
    bf16 [m, N]; h as lora_add(keep_h=True) gave it (None: computed again);
    dx_base: the projection's own input gradient, added; dx may be dx_base."""
    code = _dtype_code(grad_dtype)
    dev = x.device
    d, keep, n, k, rank, n_adapters = _lora_desc(a, b, scale, dev)
    x, ldx = _rows16("x", x, k, dev)
    m = x.shape[0]
    if ids is not None:
        ids = _arg("ids", ids, _I32_ONLY, (m,), dev)
    dy = _arg("dy", dy, _BF16_ONLY, (m, n), dev)
    if h is not None:
        h = _arg("h", h, _F32_ONLY, (m, rank), dev)
    ld_dx_base = 0
    if dx_base is not None:
        dx_base, ld_dx_base = _rows16("dx_base", dx_base, k, dev, m)
    dx = _out_arg("dx", dx, torch.bfloat16, (m, k), dev) if need_dx or dx is not None else None
    da, db = (torch.empty_like(t, dtype=_TORCH_DTYPE[code]) for t in keep[:2])
    ws, at, nb = _scratch(_entry("binade_lora_grad_workspace_bytes")(m, n, k, rank, n_adapters),
                          workspace, dev)
    _run("binade_lora_grad", ctypes.byref(d), x.data_ptr(), m, ldx, _addr(ids),
         dy.data_ptr(), n, _addr(h), _addr(dx_base), ld_dx_base,
         _addr(dx), k, da.data_ptr(), db.data_ptr(), code, at, nb, _status_arg(status, dev),
         stream)
    return dx, da, db


# ------------------------------------------------------------ 8-bit products
_BYTES_OF_F8 = (torch.float8_e4m3fn, torch.uint8)
_BYTES_OF_E8M0 = (torch.float8_e8m0fnu, torch.uint8)


@dataclass
class F8Weight:
    """Weights in 8 bits with a scale for each block of 128 x 128, as f8_pack
    and f8_weight lay them out: count matrices [rows, cols] (experts), and with
    train their transposed planes, which f8_gemm_grad's dx reads. The planes
    are the bytes of binade_f8_sizes_of; the tensors must not be replaced."""
    rows: int
    cols: int
    count: int
    scale_dtype: int
    values: torch.Tensor
    scales: torch.Tensor
    values_t: torch.Tensor | None = None
    scales_t: torch.Tensor | None = None

    def __post_init__(self):
        sizes = F8Sizes()
        _run("binade_f8_sizes_of", self.rows, self.cols, self.count, self.scale_dtype,
             ctypes.byref(sizes))
        if (self.values_t is None) != (self.scales_t is None):
            raise ValueError("values_t and scales_t: both or none")
        for name in ("values", "scales", "values_t", "scales_t"):
            t = getattr(self, name)
            if t is None and name.endswith("_t"):
                continue
            need = getattr(sizes, name + "_bytes")
            if t.dtype != torch.uint8 or t.numel() != need or not t.is_contiguous():
                raise ValueError(f"{name}: {need} contiguous bytes (uint8)")
            if t.device != self.values.device:
                raise ValueError(f"{name} is on {t.device}, not {self.values.device}")
        self._desc = F8Desc(self.rows, self.cols, self.count, self.scale_dtype,
                            self.values.data_ptr(), self.scales.data_ptr(), _addr(self.values_t),
                            _addr(self.scales_t))

    def desc(self) -> F8Desc:
        return self._desc


def _f8_planes(rows, cols, count, scale_dtype, train, device) -> F8Weight:
    sizes = F8Sizes()
    _run("binade_f8_sizes_of", rows, cols, count, scale_dtype, ctypes.byref(sizes))
    new = lambda n: torch.empty(n, dtype=torch.uint8, device=device)
    return F8Weight(rows, cols, count, scale_dtype, new(sizes.values_bytes),
                    new(sizes.scales_bytes), new(sizes.values_t_bytes) if train else None,
                    new(sizes.scales_t_bytes) if train else None)


def _matrices(name: str, t: torch.Tensor):
    if t.dim() not in (2, 3):
        raise ValueError(f"{name}: [N, K] or [count, N, K]")
    return (t.shape if t.dim() == 3 else (1, *t.shape))


def _whole16(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and 16-byte aligned, copied if it is not."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


@_on_device
def f8_pack(w: torch.Tensor, train: bool = False, out: F8Weight | None = None,
            stream=None) -> F8Weight:
    """binade_f8_pack: bf16 [N, K] or [count, N, K] in 8 bits with a
    power-of-two scale for each block of 128 x 128 (of a packed weight:
    f8_pack(unpack(w))). train: the transposed planes too. out: planes of an
    earlier call for the same sizes, written again (after an update)."""
    if w.dtype != torch.bfloat16:
        raise TypeError(f"w: {w.dtype}, expected bf16")
    count, rows, cols = _matrices("w", w)
    w = _whole16(w)
    if out is None:
        out = _f8_planes(rows, cols, count, E8M0, train, w.device)
    elif (out.rows, out.cols, out.count, out.scale_dtype) != (rows, cols, count, E8M0) or \
            out.values.device != w.device or train != (out.values_t is not None):
        raise ValueError("out: planes of other sizes, another type or device")
    _run("binade_f8_pack", w.data_ptr(), ctypes.byref(out.desc()), stream)
    return out


@_on_device
def f8_weight(values: torch.Tensor, scales: torch.Tensor, train: bool = False,
              stream=None) -> F8Weight:
    """binade_f8_layout: a checkpoint's e4m3 values [N, K] or [count, N, K]
    (float8_e4m3fn or their bytes) and their blocks' scales [(count,) ceil(N /
    128), ceil(K / 128)], fp32 or powers of two (float8_e8m0fnu or their
    bytes). Both are copied."""
    if values.dtype not in _BYTES_OF_F8:
        raise TypeError(f"values: {values.dtype}, expected float8_e4m3fn")
    count, rows, cols = _matrices("values", values)
    blocks = (-(-rows // 128), -(-cols // 128))
    if scales.dtype != torch.float32 and scales.dtype not in _BYTES_OF_E8M0:
        raise TypeError(f"scales: {scales.dtype}, expected fp32 or float8_e8m0fnu")
    scales = _arg("scales", scales, (scales.dtype,), (*values.shape[:-2], *blocks), values.device)
    values = _whole16(values)
    code = F32 if scales.dtype == torch.float32 else E8M0
    out = _f8_planes(rows, cols, count, code, train, values.device)
    _run("binade_f8_layout", values.data_ptr(), scales.data_ptr(), ctypes.byref(out.desc()), stream)
    return out


def _f8_arg(w: F8Weight, device):
    if not isinstance(w, F8Weight):
        raise TypeError("w: an F8Weight of f8_pack or f8_weight")
    if w.values.device != device:
        raise ValueError(f"w is on {w.values.device}, not {device}")
    return ctypes.byref(w._desc)


def _f8_one(w: F8Weight, device, expert: int | None, turned: bool = False):
    """(descriptor of w, or of one of its experts; what has to outlive the call).
    An expert's scales start at any multiple of four bytes: where that is none
    of 16 they are copied, in every call, since w may have been packed again."""
    whole = _f8_arg(w, device)
    if expert is None:
        return whole, None
    expert = operator.index(expert)
    if not 0 <= expert < w.count:
        raise ValueError(f"expert {expert} of {w.count}")

    def part(plane):
        n = plane.numel() // w.count
        t = plane[expert * n:(expert + 1) * n]
        return t.clone() if t.data_ptr() % 16 else t

    if not turned:
        values, scales = part(w.values), part(w.scales)
        return ctypes.byref(F8Desc(w.rows, w.cols, 1, w.scale_dtype, values.data_ptr(),
                                   scales.data_ptr())), (values, scales)
    values, scales = (w.values, None) if w.values_t is None else (part(w.values_t), part(w.scales_t))
    # the planes that are not turned are not read by the gradients
    return ctypes.byref(F8Desc(w.rows, w.cols, 1, w.scale_dtype, w.values.data_ptr(),
                               w.values.data_ptr(), None if scales is None else values.data_ptr(),
                               _addr(scales))), (values, scales)


@_on_device
def f8_gemm(x: torch.Tensor, w: F8Weight, out_dtype=torch.float32, y: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, stream=None, *,
            expert: int | None = None) -> torch.Tensor:
    """binade_f8_gemm: Q(x) W^T of bf16 x [m, K], x quantised in blocks of 128
    along K, summed in fp32; a bf16 result is that sum rounded once. Of weights
    of several experts, expert says which one."""
    code = _dtype_code(out_dtype)
    dev = x.device
    d, held = _f8_one(w, dev, expert)
    x, ldx = _rows16("x", x, w.cols, dev)
    m, n = x.shape[0], w.rows
    y = _out_arg("y", y, _TORCH_DTYPE[code], (m, n), dev)
    ws, at, nb = _scratch(_entry("binade_f8_gemm_workspace_bytes")(m, n, w.cols, code), workspace,
                          dev)
    _run("binade_f8_gemm", d, x.data_ptr(), m, ldx, y.data_ptr(), n, code, at, nb, stream)
    return y


@_on_device
def f8_gemm_grad(x: torch.Tensor, w: F8Weight, dy: torch.Tensor, grad_dtype=torch.float32,
                 need_dx: bool = True, need_dw: bool = True, dx: torch.Tensor | None = None,
                 dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None, *, expert: int | None = None):
    """binade_f8_gemm_grad: (dx bf16 [m, K] or None, dw [N, K] of grad_dtype or
    None) of f8_gemm from dy bf16 [m, N]; dx needs a weight made with train. Of
    f8_moe_gemm: expert by expert, with the rows of its pairs."""
    code = _dtype_code(grad_dtype)
    dev = x.device
    d, held = _f8_one(w, dev, expert, True)
    n, k = w.rows, w.cols
    x, ldx = _rows16("x", x, k, dev)
    m = x.shape[0]
    dy = _arg("dy", dy, _BF16_ONLY, (m, n), dev)
    dx = _out_arg("dx", dx, torch.bfloat16, (m, k), dev) if need_dx or dx is not None else None
    dw = _out_arg("dw", dw, _TORCH_DTYPE[code], (n, k), dev) if need_dw or dw is not None else None
    need = _entry("binade_f8_gemm_grad_workspace_bytes")(m, n, k, dx is not None, dw is not None,
                                                         code)
    ws, at, nb = _scratch(need, workspace, dev)
    _run("binade_f8_gemm_grad", d, x.data_ptr(), m, ldx, dy.data_ptr(), n, _addr(dx), k, _addr(dw),
         code, at, nb, stream)
    return dx, dw


@_on_device
def f8_moe_gemm(x: torch.Tensor, experts: F8Weight, idx: torch.Tensor, x_per_slot: bool = False,
                out_dtype=torch.float32, y: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """binade_f8_moe_gemm: [n_tokens * top_k, N], row t * top_k + s the product
    of expert idx[t, s] (moe_route's; -1: zeros) with x[t], or with
    x[t * top_k + s] where x_per_slot."""
    code = _dtype_code(out_dtype)
    dev = x.device
    d = _f8_arg(experts, dev)
    if idx.dim() != 2:
        raise ValueError("idx: [n_tokens, top_k]")
    tokens, top_k = idx.shape
    idx = _arg("idx", idx, _I32_ONLY, (tokens, top_k), dev)
    n, k = experts.rows, experts.cols
    x, ldx = _rows16("x", x, k, dev, tokens * top_k if x_per_slot else tokens)
    y = _out_arg("y", y, _TORCH_DTYPE[code], (tokens * top_k, n), dev)
    per_slot = 1 if x_per_slot else 0
    need = _entry("binade_f8_moe_workspace_bytes")(tokens, top_k, per_slot, experts.count, n, k)
    ws, at, nb = _scratch(need, workspace, dev)
    _run("binade_f8_moe_gemm", d, x.data_ptr(), ldx, per_slot, idx.data_ptr(), tokens, top_k,
         y.data_ptr(), n, code, at, nb, _status_arg(status, dev), stream)
    return y

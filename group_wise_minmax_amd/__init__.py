"""group_wise_minmax_amd -- low-bit group-wise weight quantization and the fused
dequantize-then-matmul of a frozen low-bit linear layer on AMD MI355X (gfx950).

This package is a thin binding over the C ABI of ``liblbq.so``
(``include/lbq.h``): every function below only marshals torch tensors into
pointers and sizes, allocates outputs with torch, and calls the library on the
current HIP stream.  All arithmetic runs in the library's HIP kernels; there is
no fallback.  The functions carry the C names:

    lbq_layout, lbq_quantize, lbq_dequant, lbq_linear_fwd, lbq_linear_bwd_dx,
    lbq_lora_fwd, lbq_nf4_codebook, lbq_quantize_tokens, lbq_linear_fwd_tokens

Beside them ``lbq_grad_norm``, ``lbq_clip_grad_norm_`` and ``LbqGradSet`` take a
training step's gradient tensors as Python lists.

Formats (cited by page title and section):
  * MinMax INT4 g128 / INT2 g64 -- GreenBit.AI, "只需单卡RTX 3090，低比特量化训练
    就能实现LLaMA-3 8B全参微调", section 模型量化;
  * NF4 with optional double quantization of the absmax -- "QLoRA技术在量化微调中的应用",
    section QLoRA技术原理; bitsandbytes FSDP-QLoRA guide, step 2 parameter table;
  * INT8, symmetric, one scale per output channel; its forward multiplies tokens
    quantized to 8 bits with one scale each.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
from dataclasses import dataclass, field
from typing import Optional

import torch

from ._lib import (LBQ_BF16, LBQ_F16, LBQ_F32, LBQ_INT8, LBQ_MAX_GROUP, LBQ_META_COMPACT, LBQ_META_F32,  # noqa: F401
                   LBQ_MINMAX, LBQ_NF4, LBQ_NORM_2, LBQ_NORM_INF, Desc, Grad, LbqError, QTensor, Sizes, check, lib,
                   STATUS_CODE, EXPORTED, LIB_PATH)

__all__ = [
    "QuantizedWeight", "make_desc", "lbq_layout", "lbq_quantize", "lbq_dequant",
    "lbq_linear_fwd", "lbq_linear_bwd_dx", "lbq_linear_bwd_dx_grouped", "lbq_lora_fwd", "lbq_nf4_codebook",
    "lbq_linear_workspace_bytes", "lbq_lora_workspace_bytes", "LbqError", "version",
    "lbq_quantize_tokens", "lbq_linear_fwd_tokens", "lbq_grad_norm", "lbq_clip_grad_norm_", "LbqGradSet",
]

_FMT = {"minmax": LBQ_MINMAX, "nf4": LBQ_NF4, "int8": LBQ_INT8}


def version() -> str:
    return lib.lbq_version().decode()


def make_desc(fmt: str, n: int, k: int, bits: int = 4, group: Optional[int] = None,
              double_quant: bool = True, compact: bool = False, dq_offset: bool = False) -> Desc:
    """Descriptor for W[n][k]. MinMax: bits 4/2, group 128/64 (default 128 for
    4-bit, 64 for 2-bit), ``compact`` for fp16 scales and packed zero points.
    NF4: absmax block 64, optional double quant (256), ``dq_offset`` for
    double quantization with a per-tensor offset.  INT8: one scale per row
    (``bits``, ``group`` and the other settings are not looked at)."""
    if fmt not in _FMT:
        raise ValueError(f"format must be one of {sorted(_FMT)}")
    d = Desc()
    d.format = _FMT[fmt]
    d.meta = 0
    if fmt == "minmax":
        d.bits = bits
        d.group = group if group is not None else (128 if bits == 4 else 64)
        d.double_quant = 0
        d.dq_block = 0
        d.meta = LBQ_META_COMPACT if compact else LBQ_META_F32
    elif fmt == "int8":
        d.bits = 8
        d.group = d.double_quant = d.dq_block = 0
    else:
        d.bits = 4
        d.group = 64 if group is None else group
        d.double_quant = (2 if dq_offset else 1) if double_quant else 0
        d.dq_block = 256 if double_quant else 0
    d.n = n
    d.k = k
    return d


def lbq_layout(desc: Desc) -> dict:
    s = Sizes()
    check(lib.lbq_layout(ctypes.byref(desc), ctypes.byref(s)), "lbq_layout")
    return {f: getattr(s, f) for f, _ in Sizes._fields_}


def lbq_nf4_codebook() -> list:
    buf = (ctypes.c_float * 16)()
    lib.lbq_nf4_codebook(buf)
    return list(buf)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> ctypes.c_void_p:
    index = device.index if device.index is not None else torch.cuda.current_device()
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(index))


_HERE = contextlib.nullcontext()


def _on(device: torch.device):
    """Context in which ``device`` is current: a launch needs its stream's device to be."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_out(out: torch.Tensor, m: int, qw: "QuantizedWeight", name: str = "out") -> None:
    """A forward's output: m rows, and a column for every channel unless out_rows places them."""
    if out.dtype != torch.bfloat16 or out.dim() != 2 or out.shape[0] != m or out.stride(1) != 1:
        raise ValueError(f"{name} must be bf16 [m, >=n] with unit column stride")
    if qw.out_rows is None and out.shape[1] < qw.n:
        raise ValueError(f"{name} must have at least {qw.n} columns")


@dataclass
class QuantizedWeight:
    """Device buffers of one quantized weight plus its descriptor."""
    desc: Desc
    packed: torch.Tensor
    scales: Optional[torch.Tensor] = None
    zeros: Optional[torch.Tensor] = None
    absmax: Optional[torch.Tensor] = None
    absmax_q: Optional[torch.Tensor] = None
    absmax_scale: Optional[torch.Tensor] = None
    out_rows: Optional[torch.Tensor] = field(default=None)

    @property
    def n(self) -> int:
        return self.desc.n

    @property
    def k(self) -> int:
        return self.desc.k

    @property
    def device(self) -> torch.device:
        return self.packed.device

    def _check_int8(self) -> None:
        n, k = self.desc.n, self.desc.k
        if self.packed.numel() * self.packed.element_size() != n * k or not self.packed.is_contiguous():
            raise ValueError(f"packed must hold the {n} x {k} codes, contiguous")
        s = self.scales
        if s is None or s.numel() != n or s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError(f"scales must be {n} contiguous float32 values")
        if s.device != self.packed.device or (self.out_rows is not None and self.out_rows.device != s.device):
            raise ValueError("the tensors of a weight must be on one device")
        o = self.out_rows
        if o is not None and (o.numel() != n or o.dtype != torch.int32 or not o.is_contiguous()):
            raise ValueError(f"out_rows must be {n} contiguous int32 values")

    def qtensor(self) -> QTensor:
        if self.desc.format == LBQ_INT8:
            self._check_int8()
            return QTensor(packed=self.packed.data_ptr(), scales=self.scales.data_ptr(), out_rows=_ptr(self.out_rows))
        return QTensor(_ptr(self.packed), _ptr(self.scales), _ptr(self.zeros), _ptr(self.absmax), _ptr(self.absmax_q),
                       _ptr(self.absmax_scale), _ptr(self.out_rows))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.packed, self.scales, self.zeros, self.absmax, self.absmax_q,
                    self.absmax_scale) if t is not None)

    def to_bytes(self) -> bytes:
        """The weight and its quantization state as one blob (see
        ``lbq_serialize`` in lbq.h); ``out_rows`` is not part of it."""
        nbytes = lib.lbq_serialized_bytes(ctypes.byref(self.desc))
        buf = ctypes.create_string_buffer(nbytes)
        q = self.qtensor()
        with _on(self.device):
            check(lib.lbq_serialize(ctypes.byref(self.desc), ctypes.byref(q), buf, nbytes, _stream(self.device)),
                  "lbq_serialize")
        return buf.raw

    @staticmethod
    def from_bytes(blob: bytes, device) -> "QuantizedWeight":
        """Rebuild a weight from ``to_bytes`` output into new device buffers."""
        desc = Desc()
        check(lib.lbq_blob_desc(blob, len(blob), ctypes.byref(desc)), "lbq_blob_desc")
        qw = QuantizedWeight.empty(desc, device)
        q = qw.qtensor()
        with _on(qw.device):
            check(lib.lbq_deserialize(blob, len(blob), ctypes.byref(q), _stream(qw.device)), "lbq_deserialize")
        return qw

    def storage_view(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The packed bytes reinterpreted as ``dtype`` (same bits, no copy):
        the float storage a sharding framework can hold them in."""
        return self.packed.view(dtype)

    @staticmethod
    def empty(desc: Desc, device) -> "QuantizedWeight":
        sz = lbq_layout(desc)
        dev = torch.device(device)
        n, k = desc.n, desc.k
        qw = QuantizedWeight(desc, torch.empty((n, sz["packed"] // n), dtype=torch.uint8, device=dev))
        if desc.format == LBQ_INT8:
            qw.scales = torch.empty((n, 1), dtype=torch.float32, device=dev)
        elif sz["scales"]:
            if desc.meta == LBQ_META_COMPACT:
                qw.scales = torch.empty((n, sz["scales"] // 2 // n), dtype=torch.float16, device=dev)
            else:
                qw.scales = torch.empty((n, sz["scales"] // 4 // n), dtype=torch.float32, device=dev)
            qw.zeros = torch.empty((n, sz["zeros"] // n), dtype=torch.uint8, device=dev)
        if sz["absmax"]:
            qw.absmax = torch.empty(sz["absmax"] // 4, dtype=torch.float32, device=dev)
        if sz["absmax_q"]:
            qw.absmax_q = torch.empty(sz["absmax_q"], dtype=torch.int8, device=dev)
            qw.absmax_scale = torch.empty(sz["absmax_scale"] // 4, dtype=torch.float32, device=dev)
        return qw


def lbq_quantize(W: torch.Tensor, fmt: str = "minmax", bits: int = 4, group: Optional[int] = None,
                 double_quant: bool = True, out: Optional[QuantizedWeight] = None, compact: bool = False,
                 dq_offset: bool = False) -> QuantizedWeight:
    """Quantize a device fp32 weight W[n][k] (see ``lbq_quantize`` in lbq.h)."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D [n, k]")
    _need(W, "W", torch.float32)
    desc = make_desc(fmt, W.shape[0], W.shape[1], bits, group, double_quant, compact, dq_offset)
    qw = out if out is not None else QuantizedWeight.empty(desc, W.device)
    if fmt == "int8" and (qw.desc.format, qw.n, qw.k, qw.device) != (LBQ_INT8, desc.n, desc.k, W.device):
        raise ValueError("out must be an INT8 weight of W's shape on W's device")
    q = qw.qtensor()
    with _on(W.device):
        check(lib.lbq_quantize(ctypes.byref(desc), W.data_ptr(), ctypes.byref(q), _stream(W.device)),
              "lbq_quantize")
    qw.desc = desc
    return qw


def lbq_dequant(qw: QuantizedWeight, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 W_hat[n][k] (see ``lbq_dequant`` in lbq.h)."""
    if out is None:
        out = torch.empty((qw.n, qw.k), dtype=torch.bfloat16, device=qw.device)
    _need(out, "out", torch.bfloat16, (qw.n, qw.k))
    q = qw.qtensor()
    _same_device(qw.device, out)
    with _on(qw.device):
        check(lib.lbq_dequant(ctypes.byref(qw.desc), ctypes.byref(q), out.data_ptr(), _stream(qw.device)),
              "lbq_dequant")
    return out


def lbq_linear_workspace_bytes(qw: QuantizedWeight, m: int) -> int:
    return lib.lbq_linear_workspace_bytes(ctypes.byref(qw.desc), m)


def lbq_lora_workspace_bytes(qw: QuantizedWeight, m: int, r: int) -> int:
    return lib.lbq_lora_workspace_bytes(ctypes.byref(qw.desc), m, r)


def _same_device(device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"every tensor must be on {device}, got one on {t.device}")


def _ws(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(((nbytes + 15) // 16) * 16, dtype=torch.uint8, device=device)


def lbq_linear_fwd(X: torch.Tensor, qw: QuantizedWeight, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X . deq(W)^T in bf16 (see ``lbq_linear_fwd`` in lbq.h).  With
    ``qw.out_rows`` set, ``out`` must be given and only those columns are written."""
    _need(X, "X", torch.bfloat16)
    m = X.shape[0]
    if X.dim() != 2 or X.shape[1] != qw.k:
        raise ValueError(f"X must be [m, {qw.k}]")
    if out is None:
        if qw.out_rows is not None:
            raise ValueError("out must be given when out_rows is set")
        out = X.new_empty((m, qw.n))
    else:
        _need_out(out, m, qw)
    nbytes = lbq_linear_workspace_bytes(qw, m)
    if workspace is None:
        workspace = _ws(nbytes, X.device)
    q = qw.qtensor()
    _same_device(X.device, qw.packed, out, workspace)
    with _on(X.device):
        check(lib.lbq_linear_fwd(ctypes.byref(qw.desc), ctypes.byref(q), X.data_ptr(), m, out.data_ptr(),
                                 out.stride(0), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                 _stream(X.device)), "lbq_linear_fwd")
    return out


def lbq_linear_fwd_noalloc(X: torch.Tensor, qw: QuantizedWeight, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``lbq_linear_fwd`` without a workspace (see ``lbq_linear_fwd_noalloc`` in
    lbq.h): the library's own per-device scratch array holds the partial sums."""
    _need(X, "X", torch.bfloat16)
    m = X.shape[0]
    if X.dim() != 2 or X.shape[1] != qw.k:
        raise ValueError(f"X must be [m, {qw.k}]")
    if out is None:
        if qw.out_rows is not None:
            raise ValueError("out must be given when out_rows is set")
        out = X.new_empty((m, qw.n))
    else:
        _need_out(out, m, qw)
    q = qw.qtensor()
    _same_device(X.device, qw.packed, out)
    with _on(X.device):
        check(lib.lbq_linear_fwd_noalloc(ctypes.byref(qw.desc), ctypes.byref(q), X.data_ptr(), m, out.data_ptr(),
                                         out.stride(0), _stream(X.device)), "lbq_linear_fwd_noalloc")
    return out


def lbq_linear_fwd_grouped_workspace_bytes(qws, m: int) -> int:
    descs = (Desc * len(qws))(*[q.desc for q in qws])
    return lib.lbq_linear_fwd_grouped_workspace_bytes(len(qws), descs, m)


def lbq_linear_fwd_grouped(X: torch.Tensor, qws, outs=None, workspace: Optional[torch.Tensor] = None):
    """Ys[i] = X . deq(W_i)^T for weights that share X and k (see
    ``lbq_linear_fwd_grouped`` in lbq.h).  Returns the list of outputs; an
    ``outs`` entry is required where that weight has ``out_rows`` (several
    weights may scatter into one tensor)."""
    _need(X, "X", torch.bfloat16)
    qws = list(qws)
    count = len(qws)
    if not 1 <= count <= LBQ_MAX_GROUP:
        raise ValueError(f"between 1 and {LBQ_MAX_GROUP} weights")
    m = X.shape[0]
    if X.dim() != 2 or any(q.k != X.shape[1] for q in qws):
        raise ValueError("X must be [m, k] with every weight's k")
    outs = list(outs) if outs is not None else [None] * count
    if len(outs) != count:
        raise ValueError("one output per weight")
    for i, (q, o) in enumerate(zip(qws, outs)):
        if o is None:
            if q.out_rows is not None:
                raise ValueError(f"outs[{i}] must be given when out_rows is set")
            outs[i] = torch.empty((m, q.n), dtype=torch.bfloat16, device=X.device)
        _need_out(outs[i], m, q, f"outs[{i}]")
    descs = (Desc * count)(*[q.desc for q in qws])
    qts = (QTensor * count)(*[q.qtensor() for q in qws])
    ys = (ctypes.c_void_p * count)(*[o.data_ptr() for o in outs])
    ldys = (ctypes.c_int64 * count)(*[o.stride(0) for o in outs])
    nbytes = lib.lbq_linear_fwd_grouped_workspace_bytes(count, descs, m)
    if workspace is None:
        workspace = _ws(nbytes, X.device)
    _same_device(X.device, workspace, *[q.packed for q in qws], *outs)
    with _on(X.device):
        check(lib.lbq_linear_fwd_grouped(count, descs, qts, X.data_ptr(), m, ys, ldys, _ptr(workspace),
                                         0 if workspace is None else workspace.numel(), _stream(X.device)),
              "lbq_linear_fwd_grouped")
    return outs


def lbq_linear_bwd_dx(dY: torch.Tensor, qw: QuantizedWeight, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX = dY . deq(W) in bf16 (see ``lbq_linear_bwd_dx`` in lbq.h; an INT8
    weight runs as ``lbq_linear_bwd_dx_grouped_ws``)."""
    _need(dY, "dY", torch.bfloat16)
    if dY.dim() != 2 or dY.shape[1] != qw.n:
        raise ValueError(f"dY must be [m, {qw.n}]")
    m = dY.shape[0]
    if out is None:
        out = dY.new_empty((m, qw.k))
    else:
        _need(out, "out", torch.bfloat16, (m, qw.k))
    q = qw.qtensor()
    _same_device(dY.device, qw.packed, out, workspace)
    if qw.desc.format == LBQ_INT8:
        desc, dp = ctypes.byref(qw.desc), ctypes.c_void_p(dY.data_ptr())
        if workspace is None:
            workspace = _ws(lib.lbq_linear_bwd_dx_grouped_workspace_bytes(1, desc, m), dY.device)
        with _on(dY.device):
            check(lib.lbq_linear_bwd_dx_grouped_ws(1, desc, ctypes.byref(q), ctypes.byref(dp), m, out.data_ptr(), _ptr(workspace),
                                                   0 if workspace is None else workspace.numel(), _stream(dY.device)),
                  "lbq_linear_bwd_dx_grouped_ws")
        return out
    with _on(dY.device):
        check(lib.lbq_linear_bwd_dx(ctypes.byref(qw.desc), ctypes.byref(q), dY.data_ptr(), m,
                                    out.data_ptr(), _stream(dY.device)), "lbq_linear_bwd_dx")
    return out


def lbq_linear_bwd_dx_grouped_workspace_bytes(qws, m: int) -> int:
    descs = (Desc * len(qws))(*[q.desc for q in qws])
    return lib.lbq_linear_bwd_dx_grouped_workspace_bytes(len(qws), descs, m)


def lbq_linear_bwd_dx_grouped(dYs, qws, out: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX = sum_i dYs[i] . deq(W_i) in bf16 for weights of one format that
    share X and k (see ``lbq_linear_bwd_dx_grouped_ws`` in lbq.h)."""
    qws, dYs = list(qws), list(dYs)
    count = len(qws)
    if not 1 <= count <= LBQ_MAX_GROUP or len(dYs) != count:
        raise ValueError(f"between 1 and {LBQ_MAX_GROUP} weights, one dY each")
    for i, (d, q) in enumerate(zip(dYs, qws)):
        _need(d, f"dYs[{i}]", torch.bfloat16)
        if d.dim() != 2 or d.shape[1] != q.n or d.shape[0] != dYs[0].shape[0]:
            raise ValueError(f"dYs[{i}] must be [m, {q.n}]")
        if q.k != qws[0].k:
            raise ValueError("every weight must have the same k")
    m, k = dYs[0].shape[0], qws[0].k
    if out is None:
        out = torch.empty((m, k), dtype=torch.bfloat16, device=dYs[0].device)
    _need(out, "out", torch.bfloat16, (m, k))
    descs = (Desc * count)(*[q.desc for q in qws])
    qts = (QTensor * count)(*[q.qtensor() for q in qws])
    dps = (ctypes.c_void_p * count)(*[d.data_ptr() for d in dYs])
    if workspace is None:
        workspace = _ws(lib.lbq_linear_bwd_dx_grouped_workspace_bytes(count, descs, m), dYs[0].device)
    _same_device(dYs[0].device, out, workspace, *dYs, *[q.packed for q in qws])
    with _on(dYs[0].device):
        check(lib.lbq_linear_bwd_dx_grouped_ws(count, descs, qts, dps, m, out.data_ptr(), _ptr(workspace),
                                               0 if workspace is None else workspace.numel(), _stream(dYs[0].device)),
              "lbq_linear_bwd_dx_grouped_ws")
    return out


def lbq_lora_fwd(X: torch.Tensor, qw: QuantizedWeight, A: torch.Tensor, B: torch.Tensor,
                 sigma: float, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X . deq(W)^T + sigma (X A^T) B^T (see ``lbq_lora_fwd`` in lbq.h)."""
    _need(X, "X", torch.bfloat16)
    _need(A, "A", torch.bfloat16)
    _need(B, "B", torch.bfloat16)
    m = X.shape[0]
    r = A.shape[0]
    if X.dim() != 2 or X.shape[1] != qw.k:
        raise ValueError(f"X must be [m, {qw.k}]")
    if A.shape[1] != qw.k or B.shape != (qw.n, r):
        raise ValueError("A must be [r, k] and B [n, r]")
    if out is None:
        if qw.out_rows is not None:
            raise ValueError("out must be given when out_rows is set")
        out = X.new_empty((m, qw.n))
    else:
        _need_out(out, m, qw)
    nbytes = lbq_lora_workspace_bytes(qw, m, r)
    if workspace is None:
        workspace = _ws(nbytes, X.device)
    q = qw.qtensor()
    _same_device(X.device, qw.packed, A, B, out, workspace)
    with _on(X.device):
        check(lib.lbq_lora_fwd(ctypes.byref(qw.desc), ctypes.byref(q), X.data_ptr(), m, A.data_ptr(),
                               B.data_ptr(), r, float(sigma), out.data_ptr(), out.stride(0),
                               _ptr(workspace), 0 if workspace is None else workspace.numel(),
                               _stream(X.device)), "lbq_lora_fwd")
    return out


def lbq_lora_bwd_workspace_bytes(qw: QuantizedWeight, m: int, r: int) -> int:
    return lib.lbq_lora_bwd_workspace_bytes(ctypes.byref(qw.desc), m, r)


def lbq_lora_bwd(X: torch.Tensor, dY: torch.Tensor, qw: QuantizedWeight, A: torch.Tensor,
                 B: torch.Tensor, sigma: float, dX: Optional[torch.Tensor] = None,
                 dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None):
    """(dX bf16 [m, k], dA fp32 [r, k], dB fp32 [n, r]) of ``lbq_lora_fwd`` for a
    frozen weight (see ``lbq_lora_bwd`` in lbq.h)."""
    _need(X, "X", torch.bfloat16)
    _need(dY, "dY", torch.bfloat16)
    _need(A, "A", torch.bfloat16)
    _need(B, "B", torch.bfloat16)
    m, r = X.shape[0], A.shape[0]
    if X.dim() != 2 or X.shape[1] != qw.k or dY.shape != (m, qw.n):
        raise ValueError(f"X must be [m, {qw.k}] and dY [m, {qw.n}]")
    if A.shape[1] != qw.k or B.shape != (qw.n, r):
        raise ValueError("A must be [r, k] and B [n, r]")
    dev = X.device
    if dX is None:
        dX = torch.empty((m, qw.k), dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty((r, qw.k), dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty((qw.n, r), dtype=torch.float32, device=dev)
    _need(dX, "dX", torch.bfloat16, (m, qw.k))
    _need(dA, "dA", torch.float32, (r, qw.k))
    _need(dB, "dB", torch.float32, (qw.n, r))
    nbytes = lbq_lora_bwd_workspace_bytes(qw, m, r)
    if workspace is None:
        workspace = _ws(nbytes, dev)
    q = qw.qtensor()
    _same_device(dev, qw.packed, dY, A, B, dX, dA, dB, workspace)
    with _on(dev):
        check(lib.lbq_lora_bwd(ctypes.byref(qw.desc), ctypes.byref(q), X.data_ptr(), dY.data_ptr(), m,
                               A.data_ptr(), B.data_ptr(), r, float(sigma), dX.data_ptr(), dA.data_ptr(),
                               dB.data_ptr(), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                               _stream(dev)), "lbq_lora_bwd")
    return dX, dA, dB


class _LoraLinearFn(torch.autograd.Function):
    """Y = X . deq(W)^T + sigma (X . A^T) . B^T with a frozen quantized W:
    forward through ``lbq_lora_fwd``, backward through ``lbq_lora_bwd`` (the
    gradient reaches X and the adapters, never W)."""

    @staticmethod
    def forward(ctx, X, A, B, qw, sigma):
        lead = X.shape[:-1]
        X2 = X.reshape(-1, qw.k).to(torch.bfloat16).contiguous()
        A16 = A.detach().to(torch.bfloat16).contiguous()
        B16 = B.detach().to(torch.bfloat16).contiguous()
        Y = lbq_lora_fwd(X2, qw, A16, B16, sigma)
        ctx.save_for_backward(X2, A16, B16)
        ctx.qw, ctx.sigma, ctx.x_shape, ctx.x_dtype = qw, sigma, X.shape, X.dtype
        ctx.a_dtype, ctx.b_dtype = A.dtype, B.dtype
        return Y.reshape(*lead, qw.n)

    @staticmethod
    def backward(ctx, dY):
        X2, A16, B16 = ctx.saved_tensors
        dY2 = dY.reshape(-1, ctx.qw.n).to(torch.bfloat16).contiguous()
        dX, dA, dB = lbq_lora_bwd(X2, dY2, ctx.qw, A16, B16, ctx.sigma)
        return (dX.reshape(ctx.x_shape).to(ctx.x_dtype), dA.to(ctx.a_dtype), dB.to(ctx.b_dtype), None, None)


class LbqLoraLinear(torch.nn.Module):
    """A frozen low-bit linear layer with trainable LoRA adapters (r <= 64,
    n % 64 == 0).  A [r, k] and B [n, r] are parameters (fp32 masters by
    default; the kernels see them rounded to bf16); B starts at zero, so the
    adapted layer starts equal to the frozen one."""

    def __init__(self, qw: QuantizedWeight, r: int = 16, lora_alpha: float = 16.0,
                 dtype: torch.dtype = torch.float32, generator: Optional[torch.Generator] = None):
        super().__init__()
        if not 1 <= r <= 64 or qw.n % 64 != 0:
            raise ValueError("LbqLoraLinear needs 1 <= r <= 64 and n % 64 == 0")
        self.qw = qw
        self.sigma = lora_alpha / r
        bound = 1.0 / qw.k ** 0.5
        a = torch.empty((r, qw.k), dtype=dtype, device=qw.device)
        a.uniform_(-bound, bound, generator=generator)
        self.A = torch.nn.Parameter(a)
        self.B = torch.nn.Parameter(torch.zeros((qw.n, r), dtype=dtype, device=qw.device))

    def forward(self, X: torch.Tensor) -> torch.Tensor:
        return _LoraLinearFn.apply(X, self.A, self.B, self.qw, self.sigma)


def lbq_quantize_tokens(X: torch.Tensor, out=None):
    """(codes int8 [m, k], scales fp32 [m]) of the rows of bf16 X [m, k], one
    scale a row (see ``lbq_quantize_tokens`` in lbq.h).  X may have any row
    stride that is a multiple of 8; ``out`` takes a pair of such tensors."""
    if not X.is_cuda or X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a bf16 device tensor [m, k]")
    m, k = X.shape
    if k > 1 and X.stride(1) != 1:
        raise ValueError("X must have unit column stride")
    if out is None:
        codes, scales = X.new_empty((m, k), dtype=torch.int8), X.new_empty(m, dtype=torch.float32)
    else:
        codes, scales = out
        _need(codes, "codes", torch.int8, (m, k))
        _need(scales, "scales", torch.float32, (m,))
        _same_device(X.device, codes, scales)
    ldx = X.stride(0) if m > 1 else k
    with _on(X.device):
        check(lib.lbq_quantize_tokens(X.data_ptr(), m, k, ldx, codes.data_ptr(), scales.data_ptr(), _stream(X.device)),
              "lbq_quantize_tokens")
    return codes, scales


def lbq_linear_fwd_tokens(codes: torch.Tensor, scales: torch.Tensor, qw: QuantizedWeight,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = deq(codes) . deq(W)^T in bf16 for an INT8 weight and the tokens of
    ``lbq_quantize_tokens`` (see ``lbq_linear_fwd_tokens`` in lbq.h).  ``out``
    and ``qw.out_rows`` as in ``lbq_linear_fwd``."""
    if codes.dim() != 2 or codes.shape[1] != qw.k:
        raise ValueError(f"codes must be [m, {qw.k}]")
    m, dev = codes.shape[0], codes.device
    _need(codes, "codes", torch.int8)
    _need(scales, "scales", torch.float32, (m,))
    if out is None:
        if qw.out_rows is not None:
            raise ValueError("out must be given when out_rows is set")
        out = torch.empty((m, qw.n), dtype=torch.bfloat16, device=dev)
    else:
        _need_out(out, m, qw)
    _same_device(dev, scales, out, qw.packed, workspace)
    if workspace is None:
        workspace = _ws(lib.lbq_linear_fwd_tokens_workspace_bytes(ctypes.byref(qw.desc), m), dev)
    q = qw.qtensor()
    with _on(dev):
        check(lib.lbq_linear_fwd_tokens(ctypes.byref(qw.desc), ctypes.byref(q), codes.data_ptr(), scales.data_ptr(), m,
                                        out.data_ptr(), out.stride(0), _ptr(workspace),
                                        0 if workspace is None else workspace.numel(), _stream(dev)),
              "lbq_linear_fwd_tokens")
    return out


_GRAD_DTYPE = {torch.float32: LBQ_F32, torch.bfloat16: LBQ_BF16, torch.float16: LBQ_F16}
_NORM_TYPE = {2.0: LBQ_NORM_2, float("inf"): LBQ_NORM_INF}
# What a table entry says of a tensor.
_PTR, _NUMEL, _CONTIGUOUS = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous
_DTYPE = operator.attrgetter("dtype")


class LbqGradSet:
    """The gradient tensors of one training step, for their norm and clipping
    (see ``lbq_grad_norm`` and ``lbq_clip_grads`` in lbq.h).  A program whose
    gradient buffers live as long as the training run builds it once; a tensor
    whose storage, type or layout changed is looked up (or refused) at the next call.
    The set holds the tensors themselves, not the parameters they belong to: after
    ``optimizer.zero_grad(set_to_none=True)``, torch's default, the next backward
    makes new ones and the set would go on scaling the old.  Such a loop calls
    ``lbq_clip_grad_norm_`` with the present gradients, or ``zero_grad(set_to_none=False)``.

    ``grads``: contiguous fp32, bf16 or fp16 tensors on one device.  ``outs``:
    where ``clip`` writes the scaled gradients (tensors of the same types and
    sizes); by default it scales in place."""

    def __init__(self, grads, outs=None):
        self._grads = list(grads)
        self._outs = self._grads if outs is None else list(outs)
        self._tensors = self._grads if outs is None else self._grads + self._outs
        if not self._grads:
            raise ValueError("at least one gradient")
        if len(self._outs) != len(self._grads):
            raise ValueError("one output per gradient")
        self.device = self._grads[0].device
        if self.device.type != "cuda":
            raise ValueError("gradients must be device tensors")
        self._table = (Grad * len(self._grads))()
        self._seen = None
        self._look()

    def _look(self) -> None:
        """Fill the table from the tensors, unless all are as they were: another
        view's values may begin at the same address and be as many."""
        ts = self._tensors
        seen = [*map(_PTR, ts), *map(_NUMEL, ts), *map(_DTYPE, ts), *map(_CONTIGUOUS, ts)]
        if seen == self._seen:
            return
        self._seen = None  # a refusal below leaves a table that is filled again
        for i, (g, o) in enumerate(zip(self._grads, self._outs)):
            if g.dtype not in _GRAD_DTYPE or not g.is_contiguous() or g.device != self.device:
                raise ValueError(f"grads[{i}] must be a contiguous fp32, bf16 or fp16 tensor on {self.device}")
            if o is not g and (o.dtype != g.dtype or o.numel() != g.numel() or not o.is_contiguous() or o.device != self.device):
                raise ValueError(f"outs[{i}] must be a contiguous tensor of grads[{i}]'s type and size on {self.device}")
            e = self._table[i]
            e.grad, e.out, e.numel, e.dtype, e.reserved = g.data_ptr(), o.data_ptr(), g.numel(), _GRAD_DTYPE[g.dtype], 0
        self._nbytes = lib.lbq_grad_workspace_bytes(len(self._grads), self._table)
        self._seen = seen

    def _call(self, norm_type: float, max_norm: Optional[float]) -> torch.Tensor:
        kind = _NORM_TYPE.get(norm_type)
        if kind is None:
            raise ValueError("norm_type must be 2 or inf")
        self._look()
        norm = torch.empty((), dtype=torch.float32, device=self.device)
        workspace = _ws(self._nbytes, self.device)
        with _on(self.device):
            if max_norm is None:
                check(lib.lbq_grad_norm(len(self._grads), self._table, kind, norm.data_ptr(), _ptr(workspace), self._nbytes,
                                        _stream(self.device)), "lbq_grad_norm")
            else:
                check(lib.lbq_clip_grads(len(self._grads), self._table, kind, float(max_norm), norm.data_ptr(),
                                         _ptr(workspace), self._nbytes, _stream(self.device)), "lbq_clip_grads")
        return norm

    def norm(self, norm_type: float = 2.0) -> torch.Tensor:
        """The norm over all the gradients, an fp32 device scalar."""
        return self._call(norm_type, None)

    def clip(self, max_norm: float, norm_type: float = 2.0) -> torch.Tensor:
        """Scale the gradients so that their norm is at most ``max_norm``;
        returns the norm before that, an fp32 device scalar."""
        return self._call(norm_type, max_norm)


def lbq_grad_norm(grads, norm_type: float = 2.0) -> torch.Tensor:
    """Norm over all the values of ``grads`` (a list of tensors)."""
    return LbqGradSet(grads).norm(norm_type)


def lbq_clip_grad_norm_(grads, max_norm: float, norm_type: float = 2.0) -> torch.Tensor:
    """Scale ``grads`` in place so that their norm over all the values is at
    most ``max_norm``; returns the norm before that.  The list is looked up at
    every call: the form for gradients that each step makes anew."""
    return LbqGradSet(grads).clip(max_norm, norm_type)

"""Weight-only block-32 int4/int8 qgemv/qgemm for B200 (sm_100a).

Thin Python binding over libwoq's C ABI (include/woq.h). PyTorch provides device memory
and streams only; every step of the computation runs in the library's CUDA kernels (or,
for ``qpack``, in its host C++ quantiser). There is no CPU or PyTorch fallback: if the
library is missing, every call raises.

    w = pack(W_fp32_cpu, bits=4, device="cuda")    # qpack on the host, copy to HBM
    y = qgemv(x, w)                                # decode, 1 <= m <= 64, FP32
    Y = qgemm(X, w, path="bf16_tc")                # prefill, tcgen05 tensor cores
"""

from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import (  # noqa: F401
    WOQ_GEMV_AUTO,
    WOQ_GEMV_CUDA_CORE,
    WOQ_GEMV_SPLIT_TC,
    WOQ_GEMV_SPLIT_GEMM,
    WOQ_GEMV_INT8_TC,
    WOQ_PATH_AUTO,
    WOQ_PATH_BF16_TC,
    WOQ_PATH_FP32,
    WOQ_PATH_SPLIT_TC,
    WoqError,
)

__all__ = [
    "PackedWeight",
    "qpack",
    "pack",
    "qgemv",
    "qgemv_argmax",
    "qgemv_swiglu",
    "qgemv_residual",
    "interleave_rows",
    "ChainItem",
    "chain_workspace",
    "qgemv_chain",
    "qgemm",
    "qgemm_workspace_bytes",
    "qgemm_bf16_noalloc",
    "attn_prompt",
    "attn_prompt_workspace",
    "KV4Cache",
    "kv4_append",
    "kv4_gather",
    "kv4_attn",
    "kv4_attn_workspace",
    "device_status",
    "launch_count",
    "WoqError",
]

_PATHS = {
    "auto": WOQ_PATH_AUTO,
    "fp32": WOQ_PATH_FP32,
    "bf16_tc": WOQ_PATH_BF16_TC,
    "split_tc": WOQ_PATH_SPLIT_TC,
}
_GEMV_PATHS = {
    "auto": WOQ_GEMV_AUTO,
    "cuda_core": WOQ_GEMV_CUDA_CORE,
    "split_tc": WOQ_GEMV_SPLIT_TC,
    "split_gemm": WOQ_GEMV_SPLIT_GEMM,
    "int8_tc": WOQ_GEMV_INT8_TC,
}


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class PackedWeight:
    """One packed weight in device memory, in the layout of include/woq.h."""

    packed: torch.Tensor  # uint8 [n, k*bits/8]
    scales: torch.Tensor  # int16 [n, k/32], binary16 bit patterns
    bits: int
    n: int
    k: int

    def desc(self) -> _lib.WoqWeight:
        return _lib.WoqWeight(self.bits, 32, self.n, self.k, _ptr(self.packed), _ptr(self.scales))

    @property
    def nbytes(self) -> int:
        """Packed codes plus scales: the bytes one product streams from memory."""
        return self.packed.numel() + 2 * self.scales.numel()

    def to(self, device) -> "PackedWeight":
        return PackedWeight(self.packed.to(device), self.scales.to(device), self.bits, self.n, self.k)


def qpack(W: torch.Tensor, bits: int) -> tuple[torch.Tensor, torch.Tensor]:
    """Host quantiser (C ABI ``qpack``): W float32 [n, k] on the CPU -> (packed, scales);
    bits 4, 5 or 8 (layouts in include/woq.h)."""
    if W.device.type != "cpu" or W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("qpack takes a 2-D float32 CPU tensor")
    W = W.contiguous()
    n, k = W.shape
    if bits not in (4, 5, 8) or k % 32:
        raise ValueError("bits must be 4, 5 or 8 and k a multiple of 32")
    packed = torch.empty(n, k * bits // 8, dtype=torch.uint8)
    scales = torch.empty(n, k // 32, dtype=torch.int16)
    _lib.check(_lib.lib().qpack(_ptr(W), n, k, bits, _ptr(packed), _ptr(scales)), "qpack")
    return packed, scales


def pack(W: torch.Tensor, bits: int, device="cuda") -> PackedWeight:
    """qpack on the host, then one copy of codes and scales to ``device``."""
    packed, scales = qpack(W, bits)
    n, k = W.shape
    return PackedWeight(packed.to(device), scales.to(device), bits, n, k)


def qgemv(
    x: torch.Tensor,
    w: PackedWeight,
    out: torch.Tensor | None = None,
    stream=None,
    path: str = "auto",
) -> torch.Tensor:
    """y[m, n] = x[m, k] . W_hat^T, 1 <= m <= 64, FP32 accuracy (C ABI ``qgemv_path``);
    path in {"auto", "cuda_core", "split_tc", "split_gemm", "int8_tc"}."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float32 CUDA tensor")
    m = x.shape[0]
    if out is None:
        out = torch.empty(m, w.n, dtype=torch.float32, device=x.device)
    d = w.desc()
    rc = _lib.lib().qgemv_path(_ptr(x), m, ctypes.byref(d), _ptr(out), _GEMV_PATHS[path], _stream(stream))
    _lib.check(rc, "qgemv")
    return out


def interleave_rows(W_gate: torch.Tensor, W_up: torch.Tensor) -> torch.Tensor:
    """[I, k] gate and up weights -> [2I, k] with row 2i = gate i, row 2i+1 = up i, the
    layout qgemv_swiglu expects."""
    if W_gate.shape != W_up.shape:
        raise ValueError("gate and up weights must have the same shape")
    return torch.stack([W_gate, W_up], dim=1).reshape(2 * W_gate.shape[0], W_gate.shape[1])


def qgemv_swiglu(x: torch.Tensor, w: PackedWeight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[m, n/2] = silu(gate) * up over a row-interleaved gate|up weight (C ABI ``qgemv_swiglu``)."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float32 CUDA tensor")
    m = x.shape[0]
    if out is None:
        out = torch.empty(m, w.n // 2, dtype=torch.float32, device=x.device)
    d = w.desc()
    _lib.check(_lib.lib().qgemv_swiglu(_ptr(x), m, ctypes.byref(d), _ptr(out), _stream(stream)), "qgemv_swiglu")
    return out


def qgemv_argmax(x: torch.Tensor, w: PackedWeight, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Per activation row, the index (smallest among ties) and value of the largest output of
    x . W_hat^T, without writing the outputs (C ABI ``qgemv_argmax``); 1 <= m <= 8."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float32 CUDA tensor")
    m = x.shape[0]
    idx = torch.empty(m, dtype=torch.int64, device=x.device)
    val = torch.empty(m, dtype=torch.float32, device=x.device)
    d = w.desc()
    rc = _lib.lib().qgemv_argmax(_ptr(x), m, ctypes.byref(d), _ptr(idx), _ptr(val), _stream(stream))
    _lib.check(rc, "qgemv_argmax")
    return idx, val


def qgemv_residual(x: torch.Tensor, w: PackedWeight, r: torch.Tensor, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """y = x . W_hat^T + r with the add fused (C ABI ``qgemv_residual``); ``out`` may be ``r``
    for an in-place update of the residual stream."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D float32 CUDA tensor")
    m = x.shape[0]
    if r.dtype != torch.float32 or not r.is_cuda or tuple(r.shape) != (m, w.n) or not r.is_contiguous():
        raise ValueError("r must be a contiguous float32 CUDA tensor of shape [m, n]")
    if out is None:
        out = torch.empty(m, w.n, dtype=torch.float32, device=x.device)
    d = w.desc()
    rc = _lib.lib().qgemv_residual(_ptr(x), m, ctypes.byref(d), _ptr(r), _ptr(out), _stream(stream))
    _lib.check(rc, "qgemv_residual")
    return out


_EPILOGUES = {"none": _lib.WOQ_EPI_NONE, "swiglu": _lib.WOQ_EPI_SWIGLU, "residual": _lib.WOQ_EPI_RESIDUAL}


@dataclass
class ChainItem:
    """One GEMV of a qgemv_chain launch: y = x . W_hat^T, with epilogue "none", "swiglu" (rows
    interleaved gate/up; y [m, n/2]) or "residual" (y = ... + r, r may be y)."""

    w: PackedWeight
    x: torch.Tensor
    y: torch.Tensor
    r: torch.Tensor | None = None
    epilogue: str = "none"


def chain_workspace(device="cuda") -> torch.Tensor:
    """A zeroed workspace for qgemv_chain (its counters; every successful call leaves them zero)."""
    return torch.zeros(int(_lib.lib().qgemv_chain_workspace_bytes()), dtype=torch.uint8, device=device)


def qgemv_chain(items: list[ChainItem], workspace: torch.Tensor, stream=None) -> None:
    """Run the items in order as one persistent launch (C ABI ``qgemv_chain``); item i reads
    its x only after every earlier item's outputs are complete."""
    if not items:
        raise ValueError("qgemv_chain needs at least one item")
    m = items[0].x.shape[0]
    descs = [it.w.desc() for it in items]  # kept alive for the call
    arr = (_lib.WoqChainItem * len(items))()
    for i, (it, d) in enumerate(zip(items, descs)):
        for t in (it.x, it.y) + ((it.r,) if it.r is not None else ()):
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("chain tensors must be contiguous float32 CUDA tensors")
        if it.x.shape[0] != m:
            raise ValueError("every item must have the same number of activation rows")
        arr[i].w = ctypes.pointer(d)
        arr[i].x = _ptr(it.x)
        arr[i].y = _ptr(it.y)
        arr[i].r = _ptr(it.r) if it.r is not None else None
        arr[i].epilogue = _EPILOGUES[it.epilogue]
    rc = _lib.lib().qgemv_chain(arr, len(items), m, _ptr(workspace), workspace.numel(), _stream(stream))
    _lib.check(rc, "qgemv_chain")


def qgemm_workspace_bytes(m: int, w: PackedWeight, path: str = "auto") -> int:
    d = w.desc()
    return int(_lib.lib().qgemm_workspace_bytes(m, ctypes.byref(d), _PATHS[path]))


def qgemm(
    X: torch.Tensor,
    w: PackedWeight,
    path: str = "auto",
    out: torch.Tensor | None = None,
    workspace: torch.Tensor | None = None,
    stream=None,
) -> torch.Tensor:
    """Y[m, n] = X[m, k] . W_hat^T (C ABI ``qgemm``); path in {"auto", "fp32", "bf16_tc", "split_tc"}."""
    if X.dtype != torch.float32 or not X.is_cuda or X.dim() != 2 or not X.is_contiguous():
        raise ValueError("X must be a contiguous 2-D float32 CUDA tensor")
    m = X.shape[0]
    p = _PATHS[path]
    if out is None:
        out = torch.empty(m, w.n, dtype=torch.float32, device=X.device)
    d = w.desc()
    need = int(_lib.lib().qgemm_workspace_bytes(m, ctypes.byref(d), p))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _lib.check(
        _lib.lib().qgemm(_ptr(X), m, ctypes.byref(d), _ptr(out), p, ws_ptr, ws_bytes, _stream(stream)),
        "qgemm",
    )
    return out


def qgemm_bf16_noalloc(X: torch.Tensor, w: PackedWeight, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """The bf16 tensor-core qgemm with no workspace and no device allocation in the library
    (C ABI ``qgemm_bf16_noalloc``): the bf16 copy of X goes to a fixed 32 MiB scratch array
    of the library's own, so m * k * 2 bytes must fit in it. ``out`` is allocated here by
    PyTorch when it is not given."""
    if X.dtype != torch.float32 or not X.is_cuda or X.dim() != 2 or not X.is_contiguous():
        raise ValueError("X must be a contiguous 2-D float32 CUDA tensor")
    m = X.shape[0]
    if out is None:
        out = torch.empty(m, w.n, dtype=torch.float32, device=X.device)
    d = w.desc()
    _lib.check(_lib.lib().qgemm_bf16_noalloc(_ptr(X), m, ctypes.byref(d), _ptr(out), _stream(stream)),
               "qgemm_bf16_noalloc")
    return out


# ---- attention -------------------------------------------------------------------------------

_DTYPES = {torch.float32: _lib.WOQ_F32, torch.float16: _lib.WOQ_F16, torch.bfloat16: _lib.WOQ_BF16}


def _device_of(t: torch.Tensor, what: str) -> int:
    """The current CUDA device, which has to be the tensor's."""
    d = t.get_device()
    if d < 0 or d != torch.cuda.current_device():
        raise ValueError(f"{what} must be on the current CUDA device")
    return d


# A call with a few tokens takes as long as its marshalling. Structures are made from packed bytes, half the time of
# their constructors, and handed over as they are, by reference, without a byref() for each.
_pack_rows = struct.Struct("@Piiqq").pack
_pack_kv4 = struct.Struct("@PPqiii4x").pack
_make_rows, _make_kv4 = _lib.WoqRows.from_buffer_copy, _lib.WoqKv4.from_buffer_copy


def _rows(t: torch.Tensor, what: str, device: int) -> _lib.WoqRows:
    """The [rows, heads, dim] tensor ``t`` as the C ABI takes it; dim contiguous."""
    dtype, shape, stride = _DTYPES.get(t.dtype), t.shape, t.stride()
    if dtype is None or len(shape) != 3 or t.get_device() != device or stride[2] != 1:
        raise ValueError(
            f"{what} must be a float32, float16 or bfloat16 tensor [rows, heads, dim] on the current CUDA device, "
            "contiguous along dim"
        )
    n, heads, dim = shape
    # the stride of a dimension of one element says nothing
    head = stride[1] if heads > 1 else dim
    return _make_rows(_pack_rows(t.data_ptr(), dtype, heads, stride[0] if n > 1 else heads * head, head))


def _ints(t: torch.Tensor, what: str, dims: int, device: int) -> int:
    if t.dtype is not torch.int32 or t.get_device() != device or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dims}-D int32 tensor on the current CUDA device")
    return t.data_ptr()


def _space(workspace: torch.Tensor | None, device: int) -> tuple[int | None, int]:
    if workspace is None:
        return None, 0
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
    return workspace.data_ptr(), workspace.nbytes


# The current stream's handle alone: a torch.cuda.Stream object for it costs as much as the rest of a call.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream
)


def _raw_stream(stream, device: int) -> int:
    return _current_raw_stream(device) if stream is None else stream.cuda_stream


def attn_prompt_workspace(q: torch.Tensor, k: torch.Tensor, batch: int) -> torch.Tensor | None:
    """A workspace for attn_prompt calls with rows shaped like ``q`` and ``k`` in ``batch`` sequences; None if
    they need none (16-bit types)."""
    if q.dtype not in _DTYPES or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be float32, float16 or bfloat16 tensors [tokens, heads, dim]")
    need = _lib.lib().attn_prompt_workspace_bytes(q.shape[0], batch, q.shape[1], k.shape[1], q.shape[2],
                                                  _DTYPES[q.dtype])
    return torch.empty(int(need), dtype=torch.uint8, device=q.device) if need else None


def attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, scale: float | None = None,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of packed sequences (C ABI ``attn_prompt``): q [tokens, heads, dim] over k, v
    [tokens, kv_heads, dim], sequence b in rows cu[b] .. cu[b + 1] - 1. ``scale`` defaults to dim^-1/2;
    without ``workspace`` (attn_prompt_workspace) one is made for the call. Rows of no sequence are left as they
    are in ``out`` (zeros in a new one)."""
    d = _device_of(q, "q")
    qr, kr, vr = _rows(q, "q", d), _rows(k, "k", d), _rows(v, "v", d)
    cp = _ints(cu, "cu", 1, d)
    tokens, heads, dim = q.shape
    shape = k.shape
    if shape != v.shape or shape[0] != tokens or shape[2] != dim or not qr.dtype == kr.dtype == vr.dtype:
        raise ValueError("q, k and v must have one type, as many rows and one dim, k and v one shape")
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    orow = _rows(out, "out", d)
    if out.shape != q.shape or orow.dtype != qr.dtype:
        raise ValueError("out must have q's shape and type")
    batch = cu.numel() - 1
    if workspace is None:
        # made and given back on the stream that uses it
        with torch.cuda.stream(stream):
            workspace = attn_prompt_workspace(q, k, batch)
    ws, nbytes = _space(workspace, d)
    rc = _lib.lib().attn_prompt(qr, kr, vr, tokens, cp, batch, dim,
                                dim**-0.5 if scale is None else scale, orow, ws, nbytes,
                                _raw_stream(stream, d))
    if rc:
        _lib.check(rc, "attn_prompt")
    return out


@dataclass(frozen=True)
class KV4Cache:
    """A paged cache of keys and values in int4 blocks of 32 (layout in include/woq.h).

    codes   uint8 [pages, kv_heads, 2, page, dim / 2]
    scales  float16 [pages, kv_heads, page, 2, dim / 32]
    """

    codes: torch.Tensor
    scales: torch.Tensor

    def __post_init__(self):
        c, s = self.codes, self.scales
        if c.dtype != torch.uint8 or c.dim() != 5 or c.shape[2] != 2 or not c.is_contiguous():
            raise ValueError("codes must be a contiguous uint8 tensor [pages, kv_heads, 2, page, dim / 2]")
        pages, heads, _, page, half = c.shape
        if s.dtype != torch.float16 or s.shape != (pages, heads, page, 2, half // 16) or not s.is_contiguous():
            raise ValueError("scales must be a contiguous float16 tensor [pages, kv_heads, page, 2, dim / 32]")
        if c.device != s.device:
            raise ValueError("codes and scales must be on one device")
        object.__setattr__(self, "pages", pages)
        object.__setattr__(self, "kv_heads", heads)
        object.__setattr__(self, "dim", 2 * half)
        object.__setattr__(self, "page", page)

    def desc(self) -> _lib.WoqKv4:
        return _make_kv4(
            _pack_kv4(self.codes.data_ptr(), self.scales.data_ptr(), self.pages, self.kv_heads, self.dim, self.page)
        )

    @classmethod
    def empty(cls, pages: int, kv_heads: int, dim: int, page: int = 64, device="cuda") -> "KV4Cache":
        """A cache of ``pages`` pages of ``page`` tokens, zeroed."""
        return cls(
            torch.zeros(pages, kv_heads, 2, page, dim // 2, dtype=torch.uint8, device=device),
            torch.zeros(pages, kv_heads, page, 2, dim // 32, dtype=torch.float16, device=device),
        )

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 2 * self.scales.numel()


def _step_args(cache, k, v, cu, table, start, what):
    d = _device_of(cache.codes, "the cache")
    c = cache.desc()
    kr, vr = _rows(k, "k", d), _rows(v, "v", d)
    shape = k.shape
    if shape != v.shape or shape[1] != cache.kv_heads or shape[2] != cache.dim:
        raise ValueError(f"{what}: k and v must be [tokens, {cache.kv_heads}, {cache.dim}]")
    tp = _ints(table, "table", 2, d)
    cp = _ints(cu, "cu", 1, d)
    batch, width = table.shape
    sp = None if start is None else _ints(start, "start", 1, d)
    if cu.numel() != batch + 1 or (start is not None and start.numel() != batch):
        raise ValueError(f"{what}: cu has batch + 1 entries, start and table batch")
    return d, c, kr, vr, cp, sp, batch, tp, width


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, table: torch.Tensor,
               start: torch.Tensor | None = None, stream=None) -> None:
    """Quantise packed rows of keys and values [tokens, kv_heads, dim] into the cache's pages
    (C ABI ``kv4_append``). Rows cu[b] .. cu[b + 1] - 1 become tokens start[b], start[b] + 1, ... of
    sequence b, whose pages are table[b]; ``start`` None: each sequence is new."""
    d, c, kr, vr, cp, sp, batch, tp, width = _step_args(cache, k, v, cu, table, start, "kv4_append")
    rc = _lib.lib().kv4_append(c, kr, vr, k.shape[0], cp, sp, batch, tp, width,
                               _raw_stream(stream, d))
    if rc:
        _lib.check(rc, "kv4_append")


def kv4_gather(cache: KV4Cache, cu: torch.Tensor, table: torch.Tensor, start: torch.Tensor | None = None,
               k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, tokens: int | None = None,
               dtype=torch.float32, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Read rows of the cache back (C ABI ``kv4_gather``), addressed as in kv4_append. Give ``k_out`` and
    ``v_out`` [tokens, kv_heads, dim], or ``tokens`` (cu's last entry, which is on the device) for new
    ones of ``dtype``, zero where no sequence has the row."""
    if (k_out is None) != (v_out is None) or (k_out is None and tokens is None):
        raise ValueError("kv4_gather takes k_out and v_out, or tokens")
    if k_out is None:
        shape = (tokens, cache.kv_heads, cache.dim)
        with torch.cuda.stream(stream):
            k_out, v_out = (torch.zeros(shape, dtype=dtype, device=cache.codes.device) for _ in "kv")
    d, c, kr, vr, cp, sp, batch, tp, width = _step_args(cache, k_out, v_out, cu, table, start, "kv4_gather")
    rc = _lib.lib().kv4_gather(c, cp, sp, batch, tp, width, k_out.shape[0], kr, vr,
                               _raw_stream(stream, d))
    if rc:
        _lib.check(rc, "kv4_gather")
    return k_out, v_out


def kv4_attn_workspace(cache: KV4Cache, q: torch.Tensor) -> torch.Tensor:
    """A zeroed workspace for kv4_attn calls with queries shaped like ``q``, and for smaller ones (every call
    leaves its counters zero; calls that share one must be ordered on one stream)."""
    need = _lib.lib().kv4_attn_workspace_bytes(cache.desc(), q.shape[1], q.shape[0])
    return torch.zeros(int(need), dtype=torch.uint8, device=cache.codes.device)


def kv4_attn(q: torch.Tensor, cache: KV4Cache, lens: torch.Tensor, table: torch.Tensor, scale: float | None = None,
             out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One-token attention [batch, heads, dim] over the first lens[b] cached tokens of each sequence
    (C ABI ``kv4_attn``). ``scale`` defaults to dim^-1/2; without ``workspace`` one is made for the
    call."""
    d = _device_of(cache.codes, "the cache")
    qr = _rows(q, "q", d)
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    orow = _rows(out, "out", d)
    lp, tp = _ints(lens, "lens", 1, d), _ints(table, "table", 2, d)
    batch, width = table.shape
    shape = q.shape
    if shape[0] != batch or lens.shape[0] != batch or shape[2] != cache.dim or out.shape != shape:
        raise ValueError("q and out must be [batch, heads, dim] of the cache's dim, lens [batch], table [batch, width]")
    if workspace is None:
        # made, zeroed and given back on the stream that uses it
        with torch.cuda.stream(stream):
            workspace = kv4_attn_workspace(cache, q)
    ws, nbytes = _space(workspace, d)
    rc = _lib.lib().kv4_attn(qr, cache.desc(), lp, batch, tp, width,
                             cache.dim**-0.5 if scale is None else scale, orow, ws, nbytes,
                             _raw_stream(stream, d))
    if rc:
        _lib.check(rc, "kv4_attn")
    return out


def device_status(clear: bool = True) -> int:
    """Synchronise the device and report bounded waits that gave up (C ABI woq_device_status)."""
    return int(_lib.lib().woq_device_status(1 if clear else 0))


def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(_lib.lib().woq_launch_count())

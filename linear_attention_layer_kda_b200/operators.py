"""The operators around the decode step, on torch CUDA tensors (include/kda_decode.h has the formulas).

Argument checks and output allocation only; the work is done by libkda_decode.so on torch's
current stream of the tensors' device.  Outputs and workspaces come from torch's allocator, so
the calls can be captured into CUDA graphs, and calls on different streams share nothing.  The calls
record no graph: gradients come from the *_backward functions (inside a torch.autograd.Function,
for instance), and a call that would lose one says so.
"""
from __future__ import annotations

import warnings
from array import array
from typing import NamedTuple, Optional, Sequence

import torch

from . import binding as B

_DTYPES = {torch.float32: B.KDA_DTYPE_F32, torch.bfloat16: B.KDA_DTYPE_BF16}


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _cuda(name: str, t, device, dtype=None, shape=None) -> None:
    """A contiguous tensor on `device`, of `dtype` and `shape` where given."""
    if (isinstance(t, torch.Tensor) and t.device == device and (dtype is None or t.dtype == dtype)
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _no_graph(name: str, *tensors) -> None:
    """Warns where torch's differentiation would pass over the call without a word."""
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            warnings.warn(f"{name} records no graph, and an input requires a gradient: its outputs are detached "
                          f"(call {name} under torch.no_grad(), and the function for its gradient by hand)", stacklevel=3)
            return


# The current stream's handle, without the Stream object where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


class _On:
    """The device of the call made current, and its current stream."""

    __slots__ = ("index", "before")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self) -> int:
        self.before = torch.cuda.current_device()
        if self.index != self.before:
            torch.cuda.set_device(self.index)
        return _raw_stream(self.index)

    def __exit__(self, *a):
        if self.index != self.before:
            torch.cuda.set_device(self.before)


# ------------------------------------------------------------------ the recurrence over sequences

# Descriptors of shapes seen before and the workspaces they need: (shape) -> (desc, {(ragged, backward): bytes}).
_descs: dict = {}


def _stride(name, t, rows, inner):
    """Elements between the rows of t [rows, heads(, channels)]; its rows are dense (columns of a wider projection)."""
    st, width = t.stride(), 1
    for s, n in zip(reversed(st[1:]), reversed(inner)):
        if not (s == width or n == 1 or rows == 0):
            raise ValueError(f"the rows of {name} must be dense and not overlap")
        width *= n
    if rows <= 1:
        return width
    if not (st[0] >= width):
        raise ValueError(f"the rows of {name} must be dense and not overlap")
    return st[0]


def _scan_desc(q, k, v, z, b, state0, cu_seqlens, nseq):
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 3):
        raise ValueError("q must be a CUDA tensor [rows, heads, dk]")
    dt, dev = q.dtype, q.device
    if dt not in _DTYPES:
        raise ValueError(f"q must be float32 or bfloat16, got {dt}")
    qs = q.shape
    rows, nh, dk = qs
    if not (isinstance(v, torch.Tensor) and v.dim() == 3):
        raise ValueError("v must be a CUDA tensor [rows, heads, dv]")
    vs = v.shape
    dv = vs[2]
    ld = []
    for name, t, shape in (("q", q, qs), ("k", k, qs), ("v", v, (rows, nh, dv)), ("z", z, qs), ("b", b, (rows, nh))):
        if not (isinstance(t, torch.Tensor) and t.device == dev):
            raise ValueError(f"{name} must be a CUDA tensor on {dev}")
        if t.dtype != dt:
            raise ValueError(f"{name} must be {dt} like q, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        ld.append(0 if t.is_contiguous() else _stride(name, t, rows, shape[1:]))
    if cu_seqlens is not None:
        _cuda("cu_seqlens", cu_seqlens, dev, torch.int32)
        if not (cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2):
            raise ValueError("cu_seqlens must be int32 [nseq + 1]")
        if not (nseq is None or nseq == cu_seqlens.numel() - 1):
            raise ValueError("nseq does not agree with cu_seqlens")
        nseq = cu_seqlens.numel() - 1
    elif nseq is None:
        nseq = state0.shape[0] if isinstance(state0, torch.Tensor) and state0.dim() else 1
    if not (nseq >= 1 and (cu_seqlens is not None or rows % nseq == 0)):
        raise ValueError(f"{rows} rows are not {nseq} sequences of one length: give cu_seqlens")
    if state0 is not None:
        _cuda("state0", state0, dev, torch.float32, (nseq, nh, dk, dv))
    key = (rows, nh, dk, dv, dt, nseq, *ld)
    found = _descs.get(key)
    if found is None:
        d = B.kda_scan_desc()
        d.num_heads, d.head_dk, d.head_dv, d.dtype, d.nseq, d.rows = nh, dk, dv, _DTYPES[dt], nseq, rows
        d.ld_q, d.ld_k, d.ld_v, d.ld_z, d.ld_b = ld
        if len(_descs) >= 4096:
            _descs.clear()
        found = _descs[key] = (d, {})
    return found + ((nseq, nh, dk, dv),)


def _workspace(d, sizes: dict, ragged: bool, backward: bool, device):
    n = sizes.get((ragged, backward))
    if n is None:
        n = sizes[ragged, backward] = B.kda_scan_workspace_bytes(d, ragged, backward)
    return (torch.empty(n, dtype=torch.uint8, device=device), n) if n else (None, 0)


def scan_forward(q, k, v, z, b, state0=None, cu_seqlens=None, nseq: Optional[int] = None, out=None, state_out=None):
    """Runs the recurrence over whole sequences; returns (o, states after the last tokens).

    q, k, z: [rows, heads, dk], v: [rows, heads, dv], b: [rows, heads], float32 or bfloat16, rows
    possibly strided; state0: float32 [nseq, heads, dk, dv] or None (zeros).  cu_seqlens (int32 CUDA
    tensor [nseq + 1]) gives the sequences' first rows; without it all nseq (default: state0's, or
    1) have the same length.  out and state_out may be given; state_out may be state0.  Rows of no
    sequence are not written.

    Sequences of more than 32 tokens take a workspace for the time of the call: 246 KB for 64 tokens of
    a bfloat16 head of 128 x 128 (scan_backward 410 KB, for short sequences too)."""
    d, sizes, shape = _scan_desc(q, k, v, z, b, state0, cu_seqlens, nseq)
    dev = q.device
    _no_graph("scan_forward", q, k, v, z, b, state0)
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=dev)
    else:
        _cuda("out", out, dev, q.dtype, v.shape)
    if state_out is None:
        state_out = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _cuda("state_out", state_out, dev, torch.float32, shape)
    with _On(dev) as stream:
        ws, n = _workspace(d, sizes, cu_seqlens is not None, False, dev)
        B.kda_scan_forward(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), z.data_ptr(), b.data_ptr(), _ptr(cu_seqlens),
                           _ptr(state0), out.data_ptr(), state_out.data_ptr(), _ptr(ws), n, stream)
    return out, state_out


def scan_backward(q, k, v, z, b, do, dstate=None, state0=None, cu_seqlens=None, nseq: Optional[int] = None):
    """Gradients of scan_forward for the gradients `do` of o and `dstate` (or None) of the states.

    Returns a dict with dq, dk, dv, dz, db (dense, of q's type) and, where state0 is given, dstate0.
    Rows of no sequence are zero."""
    d, sizes, shape = _scan_desc(q, k, v, z, b, state0, cu_seqlens, nseq)
    dev = q.device
    _cuda("do", do, dev, q.dtype, v.shape)
    if dstate is not None:
        _cuda("dstate", dstate, dev, torch.float32, shape)
    # a ragged batch may leave rows to no sequence, which the kernels do not write
    new = torch.empty if cu_seqlens is None else torch.zeros
    r = {"d" + n: new(t.shape, dtype=t.dtype, device=dev)
         for n, t in (("q", q), ("k", k), ("v", v), ("z", z), ("b", b))}
    if state0 is not None:
        r["dstate0"] = torch.empty(shape, dtype=torch.float32, device=dev)
    with _On(dev) as stream:
        ws, n = _workspace(d, sizes, cu_seqlens is not None, True, dev)
        B.kda_scan_backward(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), z.data_ptr(), b.data_ptr(), _ptr(cu_seqlens),
                            _ptr(state0), do.data_ptr(), _ptr(dstate), r["dq"].data_ptr(), r["dk"].data_ptr(),
                            r["dv"].data_ptr(), r["dz"].data_ptr(), r["db"].data_ptr(), _ptr(r.get("dstate0")), _ptr(ws),
                            n, stream)
    return r


# ------------------------------------------------------------------ the residual norm

class NormOut(NamedTuple):
    residual: torch.Tensor            # x + residual, in residual's type
    y: Optional[torch.Tensor]         # bfloat16
    y8: Optional[torch.Tensor]        # float8_e4m3fn: y / scale
    scale: Optional[torch.Tensor]     # float32 [rows, hidden / 128]
    rstd: torch.Tensor                # float32 [rows]


def residual_norm(x, residual, weight, eps: float = 1e-6, bf16: bool = True, fp8: bool = False, residual_out=None) -> NormOut:
    """r = x + residual, y = weight * r / sqrt(mean r^2 + eps), in bfloat16 and / or in 8 bits with a
    scale per row and 128 columns.

    x: [rows, hidden] float32 or bfloat16; residual: the same shape, float32 or bfloat16, or None (r is
    x); weight: bfloat16 [hidden].  residual_out may be residual itself."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2):
        raise ValueError("x must be a CUDA tensor [rows, hidden]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    rows, hidden = shape = x.shape
    dev = x.device
    _cuda("x", x, dev)
    like = x if residual is None else residual
    if residual is not None:
        if residual.dtype not in _DTYPES:
            raise ValueError(f"residual must be float32 or bfloat16, got {residual.dtype}")
        _cuda("residual", residual, dev, None, shape)
    _cuda("weight", weight, dev, torch.bfloat16, (hidden,))
    if residual_out is None:
        residual_out = torch.empty_like(like)
    else:
        _cuda("residual_out", residual_out, dev, like.dtype, shape)
    _no_graph("residual_norm", x, residual, weight)
    y = torch.empty_like(x, dtype=torch.bfloat16) if bf16 else None
    y8 = torch.empty_like(x, dtype=torch.float8_e4m3fn) if fp8 else None
    scale = torch.empty((rows, hidden // 128), dtype=torch.float32, device=dev) if fp8 else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    with _On(dev) as stream:
        B.kda_residual_norm(rows, hidden, x.data_ptr(), _DTYPES[x.dtype], _ptr(residual), _DTYPES[like.dtype],
                            weight.data_ptr(), eps, residual_out.data_ptr(), _ptr(y), _ptr(y8), _ptr(scale),
                            rstd.data_ptr(), stream)
    return NormOut(residual_out, y, y8, scale, rstd)


_norm_sizes: dict = {}  # (rows, hidden, device) -> workspace bytes


def residual_norm_backward(dy, residual, weight, rstd, dresidual=None):
    """Gradients of residual_norm's bfloat16 output: (gradient of x and of residual, gradient of weight).

    dy: bfloat16 [rows, hidden]; residual, rstd: the forward call's outputs; dresidual: the gradient
    that reaches the forward call's residual output from elsewhere, or None."""
    if not (isinstance(dy, torch.Tensor) and dy.is_cuda and dy.dim() == 2):
        raise ValueError("dy must be a CUDA tensor [rows, hidden]")
    rows, hidden = shape = dy.shape
    dev = dy.device
    _cuda("dy", dy, dev, torch.bfloat16)
    if not (isinstance(residual, torch.Tensor) and residual.dtype in _DTYPES):
        raise ValueError("residual must be float32 or bfloat16")
    _cuda("residual", residual, dev, None, shape)
    _cuda("weight", weight, dev, torch.bfloat16, (hidden,))
    _cuda("rstd", rstd, dev, torch.float32, (rows,))
    if dresidual is not None:
        _cuda("dresidual", dresidual, dev, residual.dtype, shape)
    out = torch.empty_like(residual)
    dweight = torch.empty(hidden, dtype=torch.float32, device=dev)
    with _On(dev) as stream:
        key = (rows, hidden, dev.index)
        n = _norm_sizes.get(key)
        if n is None:
            if len(_norm_sizes) >= 4096:
                _norm_sizes.clear()
            n = _norm_sizes[key] = B.kda_residual_norm_workspace_bytes(rows, hidden)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        B.kda_residual_norm_backward(rows, hidden, dy.data_ptr(), residual.data_ptr(), _DTYPES[residual.dtype],
                                     weight.data_ptr(), rstd.data_ptr(), _ptr(dresidual), out.data_ptr(),
                                     dweight.data_ptr(), ws.data_ptr(), n, stream)
    return out, dweight


# ------------------------------------------------------------------ rows of a state pool

def state_rows(pool, src: Sequence[int], dst: Sequence[int], source_pool=None) -> None:
    """pool[dst[i]] = source_pool[src[i]] for all i at once, in place; src[i] = -1 clears the row.

    pool: a contiguous CUDA tensor, rows along its first dimension (row size a multiple of 16 bytes);
    source_pool: pool itself (default), or another tensor of rows of the same size and type.  The
    destinations must be distinct; a source may be a destination of another move."""
    if not (isinstance(pool, torch.Tensor) and pool.is_cuda and pool.dim() >= 1):
        raise ValueError("pool must be a CUDA tensor")
    _cuda("pool", pool, pool.device)
    if source_pool is None:
        source_pool = pool
    _cuda("source_pool", source_pool, pool.device, pool.dtype)
    if not (source_pool.shape[1:] == pool.shape[1:]):
        raise ValueError("the rows of source_pool and pool must have the same shape")
    try:
        src, dst = (array("i", list(x) if isinstance(x, (bytes, bytearray)) else x) for x in (src, dst))
    except OverflowError:
        raise ValueError("row indices must fit 32 bits") from None
    if not dst and not src:
        return
    row = pool.element_size()
    for n in pool.shape[1:]:
        row *= n
    with _On(pool.device) as stream:
        B.kda_state_rows(_ptr(pool), pool.shape[0], _ptr(source_pool), source_pool.shape[0], row, dst, src, stream)

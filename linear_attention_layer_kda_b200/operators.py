"""The operators around the decode step, on torch CUDA tensors (include/kda_decode.h has the formulas).

Argument checks and output allocation only; the work is done by libkda_decode.so on torch's
current stream of the tensors' device.  Outputs and workspaces come from torch's allocator, so
the calls can be captured into CUDA graphs, and calls on different streams share nothing.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import binding as B

_DTYPES = {torch.float32: B.KDA_DTYPE_F32, torch.bfloat16: B.KDA_DTYPE_BF16}


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _cuda(name: str, t, device, dtype=None, shape=None) -> None:
    """A contiguous tensor on `device`, of `dtype` and `shape` where given."""
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.device == device, f"{name} is on {t.device}, expected {device}")
    _need(dtype is None or t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    _need(shape is None or tuple(t.shape) == tuple(shape), f"{name} must have shape {tuple(shape or ())}, got {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")


class _On:
    """The device of the call made current, and its current stream."""

    def __init__(self, device):
        self.guard = torch.cuda.device(device)
        self.device = device

    def __enter__(self) -> int:
        self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *a):
        return self.guard.__exit__(*a)


# ------------------------------------------------------------------ the recurrence over sequences

def _scan_desc(q, k, v, z, b, state0, cu_seqlens, nseq):
    _need(isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 3, "q must be a CUDA tensor [rows, heads, dk]")
    _need(q.dtype in _DTYPES, f"q must be float32 or bfloat16, got {q.dtype}")
    rows, nh, dk = q.shape
    _need(isinstance(v, torch.Tensor) and v.dim() == 3, "v must be a CUDA tensor [rows, heads, dv]")
    dv = v.shape[2]
    d = B.kda_scan_desc()
    for name, t, shape in (("q", q, (rows, nh, dk)), ("k", k, (rows, nh, dk)), ("v", v, (rows, nh, dv)),
                           ("z", z, (rows, nh, dk)), ("b", b, (rows, nh))):
        _need(isinstance(t, torch.Tensor) and t.is_cuda and t.device == q.device, f"{name} must be a CUDA tensor on {q.device}")
        _need(t.dtype == q.dtype, f"{name} must be {q.dtype} like q, got {t.dtype}")
        _need(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        inner = (t.shape[2], 1) if t.dim() == 3 else (1,)
        width = nh * inner[0] if t.dim() == 3 else nh
        # a row's heads and channels are dense; rows may be apart (columns of a wider projection)
        dense = all(s == w or n == 1 for s, w, n in zip(t.stride()[1:], inner, t.shape[1:]))
        _need(rows == 0 or (dense and (rows == 1 or t.stride(0) >= width)), f"the rows of {name} must be dense and not overlap")
        setattr(d, "ld_" + name, t.stride(0) if rows > 1 else width)
    if cu_seqlens is not None:
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2, "cu_seqlens must be int32 [nseq + 1]")
        _cuda("cu_seqlens", cu_seqlens, q.device, torch.int32)
        _need(nseq is None or nseq == cu_seqlens.numel() - 1, "nseq does not agree with cu_seqlens")
        nseq = cu_seqlens.numel() - 1
    elif nseq is None:
        nseq = 1 if state0 is None else state0.shape[0]
    _need(nseq >= 1 and (cu_seqlens is not None or rows % nseq == 0),
          f"{rows} rows are not {nseq} sequences of one length: give cu_seqlens")
    d.num_heads, d.head_dk, d.head_dv, d.dtype, d.nseq, d.rows = nh, dk, dv, _DTYPES[q.dtype], nseq, rows
    if state0 is not None:
        _cuda("state0", state0, q.device, torch.float32, (nseq, nh, dk, dv))
    return d


def _workspace(d, ragged: bool, backward: bool, device):
    n = B.kda_scan_workspace_bytes(d, ragged, backward)
    return torch.empty(n, dtype=torch.uint8, device=device), n


def scan_forward(q, k, v, z, b, state0=None, cu_seqlens=None, nseq: Optional[int] = None, out=None, state_out=None):
    """Runs the recurrence over whole sequences; returns (o, states after the last tokens).

    q, k, z: [rows, heads, dk], v: [rows, heads, dv], b: [rows, heads], float32 or bfloat16, rows
    possibly strided; state0: float32 [nseq, heads, dk, dv] or None (zeros).  cu_seqlens (int32 CUDA
    tensor [nseq + 1]) gives the sequences' first rows; without it all nseq (default: state0's, or
    1) have the same length.  out and state_out may be given; state_out may be state0.  Rows of no
    sequence are not written."""
    d = _scan_desc(q, k, v, z, b, state0, cu_seqlens, nseq)
    shape = (d.nseq, d.num_heads, d.head_dk, d.head_dv)
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=q.device)
    else:
        _cuda("out", out, q.device, q.dtype, v.shape)
    if state_out is None:
        state_out = torch.empty(shape, dtype=torch.float32, device=q.device)
    else:
        _cuda("state_out", state_out, q.device, torch.float32, shape)
    with _On(q.device) as stream:
        ws, n = _workspace(d, cu_seqlens is not None, False, q.device)
        B.kda_scan_forward(d, _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(b), _ptr(cu_seqlens), _ptr(state0), _ptr(out),
                           _ptr(state_out), _ptr(ws), n, stream)
    return out, state_out


def scan_backward(q, k, v, z, b, do, dstate=None, state0=None, cu_seqlens=None, nseq: Optional[int] = None):
    """Gradients of scan_forward for the gradients `do` of o and `dstate` (or None) of the states.

    Returns a dict with dq, dk, dv, dz, db (dense, of q's type) and, where state0 is given, dstate0.
    Rows of no sequence are zero."""
    d = _scan_desc(q, k, v, z, b, state0, cu_seqlens, nseq)
    shape = (d.nseq, d.num_heads, d.head_dk, d.head_dv)
    _cuda("do", do, q.device, q.dtype, v.shape)
    if dstate is not None:
        _cuda("dstate", dstate, q.device, torch.float32, shape)
    # a ragged batch may leave rows to no sequence, which the kernels do not write
    new = torch.empty if cu_seqlens is None else torch.zeros
    r = {"d" + n: new(t.shape, dtype=t.dtype, device=q.device)
         for n, t in (("q", q), ("k", k), ("v", v), ("z", z), ("b", b))}
    if state0 is not None:
        r["dstate0"] = torch.empty(shape, dtype=torch.float32, device=q.device)
    with _On(q.device) as stream:
        ws, n = _workspace(d, cu_seqlens is not None, True, q.device)
        B.kda_scan_backward(d, _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(b), _ptr(cu_seqlens), _ptr(state0), _ptr(do),
                            _ptr(dstate), _ptr(r["dq"]), _ptr(r["dk"]), _ptr(r["dv"]), _ptr(r["dz"]), _ptr(r["db"]),
                            _ptr(r.get("dstate0")), _ptr(ws), n, stream)
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
    _need(isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2, "x must be a CUDA tensor [rows, hidden]")
    _need(x.dtype in _DTYPES, f"x must be float32 or bfloat16, got {x.dtype}")
    rows, hidden = x.shape
    _cuda("x", x, x.device)
    like = x if residual is None else residual
    if residual is not None:
        _need(residual.dtype in _DTYPES, f"residual must be float32 or bfloat16, got {residual.dtype}")
        _cuda("residual", residual, x.device, None, x.shape)
    _cuda("weight", weight, x.device, torch.bfloat16, (hidden,))
    if residual_out is None:
        residual_out = torch.empty(x.shape, dtype=like.dtype, device=x.device)
    else:
        _cuda("residual_out", residual_out, x.device, like.dtype, x.shape)
    new = lambda dt, *s: torch.empty(s, dtype=dt, device=x.device)  # noqa: E731
    y = new(torch.bfloat16, rows, hidden) if bf16 else None
    y8 = new(torch.float8_e4m3fn, rows, hidden) if fp8 else None
    scale = new(torch.float32, rows, hidden // 128) if fp8 else None
    rstd = new(torch.float32, rows)
    with _On(x.device) as stream:
        B.kda_residual_norm(rows, hidden, _ptr(x), _DTYPES[x.dtype], _ptr(residual), _DTYPES[like.dtype], _ptr(weight),
                            eps, _ptr(residual_out), _ptr(y), _ptr(y8), _ptr(scale), _ptr(rstd), stream)
    return NormOut(residual_out, y, y8, scale, rstd)


def residual_norm_backward(dy, residual, weight, rstd, dresidual=None):
    """Gradients of residual_norm's bfloat16 output: (gradient of x and of residual, gradient of weight).

    dy: bfloat16 [rows, hidden]; residual, rstd: the forward call's outputs; dresidual: the gradient
    that reaches the forward call's residual output from elsewhere, or None."""
    _need(isinstance(dy, torch.Tensor) and dy.is_cuda and dy.dim() == 2, "dy must be a CUDA tensor [rows, hidden]")
    rows, hidden = dy.shape
    _cuda("dy", dy, dy.device, torch.bfloat16)
    _need(isinstance(residual, torch.Tensor) and residual.dtype in _DTYPES, "residual must be float32 or bfloat16")
    _cuda("residual", residual, dy.device, None, dy.shape)
    _cuda("weight", weight, dy.device, torch.bfloat16, (hidden,))
    _cuda("rstd", rstd, dy.device, torch.float32, (rows,))
    if dresidual is not None:
        _cuda("dresidual", dresidual, dy.device, residual.dtype, dy.shape)
    out = torch.empty_like(residual)
    dweight = torch.empty(hidden, dtype=torch.float32, device=dy.device)
    with _On(dy.device) as stream:
        n = B.kda_residual_norm_workspace_bytes(rows, hidden)
        ws = torch.empty(n, dtype=torch.uint8, device=dy.device)
        B.kda_residual_norm_backward(rows, hidden, _ptr(dy), _ptr(residual), _DTYPES[residual.dtype], _ptr(weight),
                                     _ptr(rstd), _ptr(dresidual), _ptr(out), _ptr(dweight), _ptr(ws), n, stream)
    return out, dweight


# ------------------------------------------------------------------ rows of a state pool

def state_rows(pool, src: Sequence[int], dst: Sequence[int], source_pool=None) -> None:
    """pool[dst[i]] = source_pool[src[i]] for all i at once, in place; src[i] = -1 clears the row.

    pool: a contiguous CUDA tensor, rows along its first dimension (row size a multiple of 16 bytes);
    source_pool: pool itself (default), or another tensor of rows of the same size and type.  The
    destinations must be distinct; a source may be a destination of another move."""
    _need(isinstance(pool, torch.Tensor) and pool.is_cuda and pool.dim() >= 1, "pool must be a CUDA tensor")
    _cuda("pool", pool, pool.device)
    if source_pool is None:
        source_pool = pool
    _cuda("source_pool", source_pool, pool.device, pool.dtype)
    _need(source_pool.shape[1:] == pool.shape[1:], "the rows of source_pool and pool must have the same shape")
    src, dst = [int(i) for i in src], [int(i) for i in dst]
    if not dst and not src:
        return
    row = pool.element_size()
    for n in pool.shape[1:]:
        row *= n
    with _On(pool.device) as stream:
        B.kda_state_rows(_ptr(pool), pool.shape[0], _ptr(source_pool), source_pool.shape[0], row, dst, src, stream)

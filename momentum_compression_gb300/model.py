"""The model-side operators for torch's autograd: dropout, the learned
relative position bias by buckets, and the attention that uses both.

Each function calls the ob_* entry points of the same name (their CUDA
kernels; there is no CPU fallback) on torch's current stream.  Random
numbers are named by (seed, offset): the backward pass draws the forward
pass's mask again instead of storing it, so calls that must be independent
(another layer, another step) take another offset.  They are values of the
host: a CUDA graph repeats the masks that it captured.  Gradients are of first
order: a graph of them (create_graph) is refused when it is differentiated."""
import torch
from torch.autograd.function import once_differentiable

from . import (ob_attn_bwd, ob_attn_fwd, ob_dropout, ob_relpos_bias, ob_relpos_bias_bwd,
               ob_relpos_init)


class RelPos:
    """Buckets of a relative position bias: one-sided (causal) or two-sided,
    one bucket a distance up to half of a side's buckets, then logarithmic
    up to max_distance."""

    def __init__(self, num_buckets=32, max_distance=128, two_sided=True):
        self.num_buckets, self.max_distance, self.two_sided = num_buckets, max_distance, two_sided
        self.plan = ob_relpos_init(num_buckets, max_distance, bool(two_sided))


def _as_rows(t):
    """t itself if it is rows that the kernels can read (the last dimension contiguous, the
    others one run of rows that do not overlap), else a contiguous copy."""
    if t.is_contiguous():
        return t
    rows, ld = 1, None
    ok = t.dim() > 0 and (t.stride(-1) == 1 or t.shape[-1] == 1)
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size > 1:
            ld = stride if ld is None else ld
            ok = ok and ld >= t.shape[-1] and stride == rows * ld
            rows *= size
    return t if ok else t.contiguous()


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
        ob_dropout(x, y, p, seed, offset, residual=residual)
        ctx.args = (p, seed, offset)
        ctx.has_residual = residual is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dx = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty(dy.shape, device=dy.device, dtype=dy.dtype)
            ob_dropout(_as_rows(dy), dx, *ctx.args)
        return dx, dy if ctx.has_residual else None, None, None, None


def dropout(x, p, seed, offset, residual=None):
    """residual + dropout(x), in one pass; the mask is never stored."""
    return _Dropout.apply(_as_rows(x), None if residual is None else _as_rows(residual), p, seed,
                          offset)


class _RelPosBias(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, plan, Lq, Lk, q_offset, dtype):
        out = torch.empty(table.shape[1], Lq, Lk, device=table.device, dtype=dtype)
        ob_relpos_bias(plan, table, out, q_offset=q_offset)
        ctx.plan, ctx.q_offset, ctx.table = plan, q_offset, (table.shape, table.dtype)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        shape, dtype = ctx.table
        dtable = torch.empty(shape, device=dout.device, dtype=dtype)
        if dout.shape[-1] > 1 and dout.stride(-1) != 1:  # the kernels read any other strides
            dout = dout.contiguous()
        ob_relpos_bias_bwd(ctx.plan, dout, dtable, q_offset=ctx.q_offset)
        return dtable, None, None, None, None, None


def relpos_bias(table, relpos, Lq, Lk, q_offset=0, dtype=None):
    """The bias [H, Lq, Lk] of table [num_buckets, H] (for use outside `attention`).
    q_offset: the position of query 0 among the keys, 0 by default; `attention`'s default
    is Lk - Lq."""
    return _RelPosBias.apply(table.contiguous(), relpos.plan, Lq, Lk, q_offset,
                             table.dtype if dtype is None else dtype)


def _inner(t):
    """t itself if the kernels can read its rows, else a contiguous copy."""
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0
    for size, stride in zip(t.shape[:3], t.stride()[:3]):
        ok = ok and (size == 1 or (stride % 8 == 0 and stride >= t.shape[3]))
    # not contiguous(): a contiguous view that starts off 16 bytes would be returned as it is
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, table, kv_len, kw):
        q, k, v = _inner(q), _inner(k), _inner(v)
        o = torch.empty(q.shape, device=q.device, dtype=q.dtype)
        B, Lq, H, _ = q.shape
        lse = torch.empty(B, H, Lq, device=q.device)
        ob_attn_fwd(q, k, v, o, lse, table=table, kv_len=kv_len, **kw)
        ctx.save_for_backward(q, k, v, o, lse, table, kv_len)
        ctx.kw = kw
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_o):
        q, k, v, o, lse, table, kv_len = ctx.saved_tensors
        dq, dk, dv = (torch.empty(t.shape, device=t.device, dtype=t.dtype) for t in (q, k, v))
        dtable = torch.empty_like(table) if ctx.needs_input_grad[3] else None
        ob_attn_bwd(_inner(grad_o), q, k, v, o, lse, dq, dk, dv, dtable=dtable, table=table,
                    kv_len=kv_len, **ctx.kw)
        return dq, dk, dv, dtable, None, None


def attention(q, k, v, table=None, relpos=None, causal=False, kv_len=None, scale=None,
              q_offset=None, p=0.0, seed=0, offset=0):
    """dropout(softmax(scale q k^T + bias)) v for q [B, Lq, H, D] and k, v
    [B, Lk, Hkv, D] in bfloat16 or float16.  table [num_buckets, H] with relpos
    (a RelPos) adds the learned bias; kv_len (int32 [B]) masks padded keys and must not
    change before the backward pass."""
    kw = dict(causal=causal, scale=scale, q_offset=q_offset, p=p, seed=seed,
              offset=offset, relpos=None if relpos is None else relpos.plan)
    return _Attention.apply(q, k, v, None if table is None else table.contiguous(), kv_len, kw)

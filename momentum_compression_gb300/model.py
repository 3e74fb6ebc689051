"""The model-side operators for torch's autograd: dropout, the learned
relative position bias by buckets, the attention that uses both, layer norm and
the dense layer with its epilogue.

Each function calls the ob_* entry points of the same name (their CUDA
kernels; there is no CPU fallback) on torch's current stream.  Random
numbers are named by (seed, offset): the backward pass draws the forward
pass's mask again instead of storing it, so calls that must be independent
(another layer, another step) take another offset.  They are values of the
host: a CUDA graph repeats the masks that it captured.  Gradients are of first
order: a graph of them (create_graph) is refused when it is differentiated.
A backward pass is captured into a CUDA graph by torch.autograd.grad, or by
.backward() while no eager graph of the same leaves lives: torch adds to a
leaf's .grad on the stream of the graph that was made first."""
import torch
from torch.autograd.function import once_differentiable

from . import (ob_attn_bwd, ob_attn_fwd, ob_dropout, ob_layernorm_bwd, ob_layernorm_fwd,
               ob_linear_bwd, ob_linear_fwd, ob_relpos_bias, ob_relpos_bias_bwd, ob_relpos_init)


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
        lse = torch.empty(B, H, Lq, device=q.device, dtype=torch.float32)
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


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, return_sum, graph):
        ctx.set_materialize_grads(False)
        train = graph and any(ctx.needs_input_grad)
        new = lambda: torch.empty(x.shape, device=x.device, dtype=x.dtype)
        y = new()
        s = new() if residual is not None and (train or return_sum) else None
        mean = rstd = None
        if train:
            rows = x.numel() // x.shape[-1] if x.shape[-1] else 0
            mean, rstd = (torch.empty(rows, device=x.device, dtype=torch.float32) for _ in range(2))
        ob_layernorm_fwd(x, y, weight=weight, bias=bias, eps=eps, residual=residual, sum=s,
                         mean=mean, rstd=rstd)
        ctx.has_residual, ctx.bias = residual is not None, bias is not None
        if train:
            ctx.save_for_backward(x if s is None else s, weight, bias, mean, rstd)
        return (y, s) if return_sum else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dw = db = None
        if dy is None:  # only the sum was used
            dx = dsum
        else:
            if need[0] or need[1]:
                dx = torch.empty(x.shape, device=x.device, dtype=x.dtype)
            if need[2]:
                dw = torch.empty_like(weight)
            if need[3]:
                db = torch.empty_like(bias)
            dsum = None if dx is None or dsum is None else _as_rows(dsum)
            ob_layernorm_bwd(_as_rows(dy), x, mean, rstd, dx, weight=weight, dweight=dw, dbias=db,
                             dsum=dsum)
        return (dx if need[0] else None, dx if ctx.has_residual and need[1] else None, dw, db, None,
                None, None)


def layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None, return_sum=False):
    """Layer norm of s = x + residual over the last dimension, times weight plus bias (both
    of one type).  With return_sum (and a residual): (y, s), s the residual stream of the
    layers after a pre-norm one; its gradient joins in the same pass."""
    if return_sum and residual is None:
        raise ValueError("layer_norm: return_sum needs a residual")
    return _LayerNorm.apply(_as_rows(x), None if residual is None else _as_rows(residual),
                            None if weight is None else weight.contiguous(),
                            None if bias is None else bias.contiguous(), eps, return_sum,
                            torch.is_grad_enabled())


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, activation, graph):
        shape = x.shape[:-1] + (w.shape[0],)
        y = torch.empty(shape, device=x.device, dtype=x.dtype)
        z = None
        if graph and activation != "none" and any(ctx.needs_input_grad[:3]):
            z = torch.empty(shape, device=x.device, dtype=x.dtype)
        ob_linear_fwd(x, w, y, bias=bias, residual=residual, z=z, activation=activation)
        ctx.save_for_backward(x, w, z)
        ctx.activation, ctx.residual_shape = activation, None if residual is None else residual.shape
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = torch.empty(x.shape, device=x.device, dtype=x.dtype) if need[0] else None
        dw = torch.empty_like(w) if need[1] else None
        db = torch.empty(w.shape[0], device=w.device, dtype=w.dtype) if need[2] else None
        if any(need[:3]):
            ob_linear_bwd(_as_rows(dy), x, w, dx=dx, dw=dw, dbias=db, z=z,
                          activation=ctx.activation)
        return dx, dw, db, dy.reshape(ctx.residual_shape) if need[3] else None, None, None


def _as_weights(w):
    """w [N, K] itself if one of its dimensions is contiguous and its rows do not overlap,
    else a contiguous copy."""
    if w.dim() == 2:
        for rows, cols in ((0, 1), (1, 0)):
            if w.stride(cols) == 1 and (w.shape[rows] <= 1 or w.stride(rows) >= w.shape[cols]):
                return w
    return w.contiguous()


def linear(x, w, bias=None, activation="none", residual=None):
    """act(x w^T + bias) + residual for x [..., K] and w [N, K] in bfloat16 or float16, the
    whole epilogue in the product's kernel.  w may be a transposed view ([K, N] in memory); its
    gradient is laid out as it is.  activation: none, relu, gelu or gelu_tanh."""
    return _Linear.apply(_as_rows(x), _as_weights(w), None if bias is None else bias.contiguous(),
                         None if residual is None else _as_rows(residual), activation,
                         torch.is_grad_enabled())

"""Calls of layer norm, the dense layer and AdamW at the edge of what they allow, without a
GPU: sizes of zero, strides of zero, arrays that are not where they seem."""
import math
import os
import subprocess
import sys

import pytest
import torch

import momentum_compression_gb300 as ob
from momentum_compression_gb300 import model as M
from test_model_binding import _zeros, library  # noqa: F401

BF16, F32 = torch.bfloat16, torch.float32
BAD = ob.OB_ERR_INVALID


@pytest.fixture(scope="module", autouse=True)
def _built():
    from momentum_compression_gb300 import _build
    _build.build()


SIZES = """
import momentum_compression_gb300 as ob
for M in (0, 1, 5, 300):
    for N in (0, 1, 5, 4096):
        for K in (0, 7, 64):
            for act in (0, 2):
                for kn in (0, 1):
                    for off in (0, 1):
                        for backward in (0, 1):
                            b = ob.ob_linear_workspace_bytes(1, act, kn, off, M, N, K, backward)
                            assert 0 <= b < 1 << 26, (M, N, K, b)
print("fine")
"""


def test_workspaces_of_sizes_of_zero():
    """In a process of its own, which a division by zero would end."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", (r.returncode, r.stderr[-2000:])


def _refused(call, name):
    with pytest.raises(ob.OBError) as e:
        call()
    assert e.value.status == BAD and name in str(e.value), str(e.value)


def test_dense_forward_refuses_strides_of_zero(library):  # noqa: F811
    """A residual that is one row for all of them is not left out, nor a z."""
    x, w, y = _zeros(4, 64), _zeros(32, 64), _zeros(4, 32)
    for row in (_zeros(32), _zeros(1, 32)):
        _refused(lambda: ob.ob_linear_fwd(x, w, y, residual=row.expand(4, 32)), "residual")
        _refused(lambda: ob.ob_linear_fwd(x, w, y, z=row.expand(4, 32)), "z")
        _refused(lambda: ob.ob_linear_fwd(x, w, row.expand(4, 32)), "y")
    _refused(lambda: ob.ob_linear_fwd(_zeros(64).expand(4, 64), w, y), "x")
    _refused(lambda: ob.ob_linear_fwd(x, _zeros(64).expand(32, 64), y), "w")
    _refused(lambda: ob.ob_linear_fwd(x, _zeros(32).expand(64, 32).t(), y), "w")
    one = _zeros(4, 1)
    _refused(lambda: ob.ob_linear_fwd(x, w[:1], one, residual=_zeros(1, 1).expand(4, 1)), "residual")
    # of one row the stride is no matter
    calls = []
    library.ob_linear_fwd = lambda *a: calls.append(a) or ob.OB_OK
    ob.ob_linear_fwd(x[:1], w, y[:1], residual=_zeros(32).expand(1, 32))
    ob.ob_linear_fwd(x, w, y)
    ob.ob_linear_fwd(x[:, :0], w[:, :0], y, z=_zeros(4, 32))
    given = [[p is not None for p in c[1:7]] for c in calls]  # x, w, bias, residual, z, y
    assert given == [[True, True, False, True, False, True], [True, True, False, False, False, True],
                     [True, True, False, False, True, True]]


@pytest.mark.parametrize("at", ["2", "3"])
def test_dense_backward_refuses_strides_of_zero(library, at):  # noqa: F811
    """One element that stands for a column of them is not read as if they lay there."""
    def column(n):
        one = _zeros(1, 1)
        return one.expand(n, 1) if at == "2" else one.view(1, 1, 1).expand(2, n // 2, 1)
    x, w, dy = _zeros(4, 64), _zeros(1, 64), _zeros(4, 1)
    x, dy = (x, dy) if at == "2" else (x.view(2, 2, 64), dy.view(2, 2, 1))
    dx, dw, act = torch.zeros_like(x), torch.zeros_like(w), dict(z=dy, activation="gelu")
    bwd = ob.ob_linear_bwd
    _refused(lambda: bwd(column(4), x, w, dx=dx), "dy")
    _refused(lambda: bwd(column(4), x, w, dbias=_zeros(1)), "dy")
    _refused(lambda: bwd(dy, x, w, dx=dx, z=column(4), activation="gelu"), "z")
    x, w = dy, _zeros(1, 1)  # one column of x
    _refused(lambda: bwd(dy, column(4), w, dw=w, **act), "x")
    _refused(lambda: bwd(dy, x, w, dx=column(4), **act), "dx")
    w, dy = _zeros(8, 1), (_zeros(4, 8) if at == "2" else _zeros(2, 2, 8))
    _refused(lambda: bwd(dy, x, _zeros(1, 1).expand(8, 1), dx=x), "w")
    _refused(lambda: bwd(dy, x, w, dw=_zeros(1, 1).expand(8, 1)), "dw")
    wide = _zeros(8)
    wide = wide.expand(4, 8) if at == "2" else wide.expand(2, 2, 8)
    _refused(lambda: bwd(wide, x, w, dx=x), "dy")
    # what is empty has no rows to be apart
    calls = []
    library.ob_linear_bwd = lambda *a: calls.append(a) or ob.OB_OK
    bwd(dy, dy[..., :0], _zeros(8, 0), dx=dy[..., :0], dw=_zeros(8, 0), dbias=_zeros(8))
    bwd(dy[..., :0], x, _zeros(0, 1), dx=x, dw=_zeros(0, 1), dbias=_zeros(0))
    assert all([p is not None for p in c[1:7]] == [True, True, True, False, True, True] for c in calls) and calls


@pytest.fixture
def recorded(library, monkeypatch):  # noqa: F811
    """The recording library for model.py: its calls by name, and tensors of torch's default type
    where none is asked for."""
    calls = {}
    for n in ("ob_layernorm_fwd", "ob_layernorm_bwd", "ob_linear_fwd", "ob_linear_bwd", "ob_adamw_step",
              "ob_adamw_moments", "ob_attn_fwd"):
        setattr(library, n, lambda *a, n=n: calls.setdefault(n, []).append(a) or ob.OB_OK)

    def empty(*shape, dtype=None, device=None):
        shape = shape[0] if shape and not isinstance(shape[0], int) else shape
        return _zeros(*shape, dtype=dtype or torch.get_default_dtype(), at=device.index)
    monkeypatch.setattr(torch, "empty", empty)
    return calls


@pytest.mark.parametrize("default", [torch.float64, BF16])
def test_statistics_are_float32_whatever_torch_makes(recorded, default):
    x, q = _zeros(4, 64).requires_grad_(), _zeros(1, 8, 2, 64).requires_grad_()
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        M.layer_norm(x)
        M.attention(q, q, q)
    finally:
        torch.set_default_dtype(before)
    assert len(recorded["ob_layernorm_fwd"]) == len(recorded["ob_attn_fwd"]) == 1


def test_gradient_of_one_row_of_weights_is_contiguous(recorded):
    """Else what lies between its elements would be written."""
    x, w, dy = _zeros(4, 64), _zeros(1, 64), _zeros(4, 1)
    _refused(lambda: ob.ob_linear_bwd(dy, x, w, dw=_zeros(1, 128)[:, ::2]), "dw")
    ob.ob_linear_bwd(dy, x, w, dw=_zeros(1, 128)[:, :64])
    ob.ob_linear_bwd(dy, x, _zeros(1, 128)[:, ::2], dw=_zeros(1, 192)[:, ::3])  # stored [K, N]: 64 rows of one
    assert len(recorded["ob_linear_bwd"]) == 2


@pytest.fixture
def adamw(recorded, monkeypatch):
    """AdamW of a tensor of 300 elements, two blocks of state."""
    real = torch.tensor

    def tensor(data, dtype=None, device=None):
        t = _zeros(len(data), dtype=dtype, at=device.index)
        t.copy_(real(data, dtype=dtype))
        return t
    monkeypatch.setattr(torch, "tensor", tensor)

    def make(bits=8, **state):
        t = F32 if bits == 32 else torch.uint8
        given = dict(m=_zeros(512, dtype=t), v=_zeros(512, dtype=t), step=0)
        if bits == 8:
            given.update(m_exp=_zeros(2, dtype=t), v_exp=_zeros(2, dtype=t))
        given.update(state)
        return ob.AdamW([_zeros(300, dtype=F32)], state_bits=bits, state={k: v for k, v in given.items() if v is not None})
    return make


@pytest.mark.parametrize("stream", [None, 77])
def test_moments_values_are_made_on_their_stream(adamw, library, recorded, monkeypatch, stream):  # noqa: F811
    """What torch's allocator hands out belongs to the stream that is current then."""
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(library.entered[-1:]) or empty(*a, **kw))
    m, v = adamw().moments(stream=stream)
    assert [t.cuda_stream for s in made for t in s] == ([] if stream is None else [77, 77])
    assert m.dtype == v.dtype == BF16 and m.shape == v.shape == (512,) and m.data_ptr() != v.data_ptr()
    assert recorded["ob_adamw_moments"][0][-1] == (0x1000 if stream is None else 77)


def test_state_waits_for_steps_on_every_stream(adamw, monkeypatch):
    """Steps may be under way on a stream that is not the current one."""
    opt = adamw(32)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: opt.counter[0].fill_(5.0))
    assert opt.state()["step"] == 5


def test_a_state_that_is_not_whole_is_refused(adamw):
    """Else moments would go on as if no step had been taken, or none had been handed over."""
    assert all(adamw(32, step=s).counter[0] == 7 for s in (7, 7.0, torch.full((), 7)))
    for missing in ("m", "v", "m_exp", "v_exp", "step"):
        _refused(lambda: adamw(8, **{missing: None}), missing)
    for step in (-1, 2.5, math.nan, "3"):
        _refused(lambda: adamw(32, step=step), "step")
    _refused(lambda: ob.AdamW([_zeros(300, dtype=F32)], state={}), "state")


def test_adamw_step_refuses_host_memory(recorded):
    """Arrays that all lie on the host are on one device, but not on one that kernels run on."""
    host = lambda n, t=F32: torch.zeros(n, dtype=t)
    p, c = host(256), host(4, torch.float64)
    table = (ob.ob_adamw_tensor * 1)(ob.ob_adamw_tensor(p.data_ptr(), 0, 256, 0.0, ob.OB_TYPE_F32, 0))
    config = ob.ob_adamw(32, ob.OB_TYPE_F32, 0.1, 0.9, 0.99, 1e-8)
    for kw in ({}, dict(at=-1)):
        _refused(lambda: ob.ob_adamw_step(config, table, [host(256)], host(256), host(256), c, **kw), "CUDA")
    assert "ob_adamw_step" not in recorded


def test_gradient_of_a_residual_has_its_shape(recorded):
    """The forward pass takes rows in any leading shape; so does the backward pass."""
    x, w, dy = _zeros(2, 2, 64), _zeros(32, 64), _zeros(2, 2, 32)
    dy.copy_(torch.arange(128).view(2, 2, 32))
    for shape in ((4, 32), (2, 2, 32), (4, 1, 32)):
        r = _zeros(*shape).requires_grad_()
        got, = torch.autograd.grad(M.linear(x, w, residual=r), r, dy)
        assert got.shape == r.shape and torch.equal(got.reshape(-1), dy.reshape(-1))
    r = _zeros(32).requires_grad_()
    got, = torch.autograd.grad(M.linear(x[0, :1], w, residual=r), r, dy[0, :1])
    assert torch.equal(got, dy[0, 0])

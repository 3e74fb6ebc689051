"""What the binding of the model-side operators does around the library's
calls, without a GPU: tensors that say they are on a device, and a library
that records its calls instead of launching."""
import contextlib
import ctypes as ct

import pytest
import torch

import momentum_compression_gb300 as ob

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from momentum_compression_gb300 import _build
    _build.build()


class _Fake(torch.Tensor):
    """A tensor in host memory that says it is on CUDA device `at`."""
    at = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.at)

    def get_device(self):
        return self.at


def _on(t, at=0):
    t = t.as_subclass(_Fake)
    t.at = at
    return t


def _zeros(*shape, dtype=BF16, at=0):
    n = 1
    for s in shape:
        n *= s
    # on a 256-byte boundary, as device memory is
    flat = torch.zeros(n + 256, dtype=dtype)
    skip = -flat.data_ptr() % 256 // flat.element_size()
    return _on(flat[skip:skip + n].view(shape), at)


class _Library:
    """The library, whose launching calls are recorded instead: (name, arguments,
    current device)."""

    def __init__(self, real):
        self.real, self.calls, self.current = real, [], 0

    def __getattr__(self, name):
        if name not in ("ob_dropout", "ob_relpos_bias", "ob_relpos_bias_bwd", "ob_attn_fwd",
                        "ob_attn_bwd"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args, self.current))
            return ob.OB_OK
        return call


class _Stream:
    def __init__(self, handle, device_index=0):
        self.cuda_stream, self.device_index = handle, device_index


@pytest.fixture
def library(monkeypatch):
    """The recording library; torch's streams and device are its own."""
    lib = _Library(ob.lib())
    lib.entered = []  # streams made current, innermost last
    lib.allocated = []  # (bytes, the stream that was current)

    @contextlib.contextmanager
    def stream(s):
        lib.entered.append(s)
        yield
        lib.entered.pop()

    @contextlib.contextmanager
    def device(d):
        before, lib.current = lib.current, d
        yield
        lib.current = before

    def empty(*shape, **kw):
        lib.allocated.append((shape, lib.entered[-1] if lib.entered else None))
        return _zeros(*shape, dtype=kw["dtype"], at=kw["device"].index)

    monkeypatch.setattr(ob, "lib", lambda: lib)
    monkeypatch.setattr(ob, "_raw_stream", lambda d: 0x1000 + d)
    monkeypatch.setattr(ob, "_current_device", lambda: lib.current)
    monkeypatch.setattr(ob, "_devices", 2)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: _Stream(h))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(_Fake, "record_stream", lambda self, s: None, raising=False)
    return lib


def _backward_calls(stream):
    """The two calls that take scratch of torch's allocator."""
    q, k = _zeros(2, 40, 4, 64), _zeros(2, 48, 2, 64)
    lse = _zeros(2, 4, 40, dtype=torch.float32)
    rp = ob.ob_relpos_init(32, 128, True)
    table = _zeros(32, 4)
    yield lambda: ob.ob_attn_bwd(q, q, k, k, q, lse, q, k, k, dtable=table, relpos=rp,
                                 table=table, stream=stream)
    dout, dtable = _zeros(3, 4, 40, 48), _zeros(32, 4, dtype=torch.float32)
    yield lambda: ob.ob_relpos_bias_bwd(rp, dout, dtable, stream=stream)


@pytest.mark.parametrize("stream", [_Stream(0x77), 0x77])
def test_scratch_belongs_to_the_stream_of_its_call(library, stream):
    """Torch's allocator hands a freed block on within the stream it was made on: scratch
    made on another one may still be in use there."""
    for call in _backward_calls(stream):
        call()
        (shape, of), = library.allocated
        assert of is not None and of.cuda_stream == 0x77
        assert library.calls[-1][1][-1] == 0x77
        library.allocated.clear()


def test_scratch_of_the_current_stream(library):
    for call in _backward_calls(None):
        call()
        assert library.allocated.pop()[1] is None
        assert library.calls[-1][1][-1] == 0x1000


# ---------------------------------------------------------------------------
# Devices
# ---------------------------------------------------------------------------

def _calls(at=0, change=None, other=None, **kw):
    """(name, call) of every entry point on tensors of device `at`; the argument called
    `change` is on device `other` instead."""
    def z(name, *shape, dtype=BF16):
        return _zeros(*shape, dtype=dtype, at=other if name == change else at)

    rp = ob.ob_relpos_init(32, 128, True)
    x = {n: z(n, 5, 24) for n in ("x", "y", "residual")}
    yield "ob_dropout", lambda: ob.ob_dropout(x["x"], x["y"], 0.5, 1, 2, residual=x["residual"], **kw)
    table, out = z("table", 32, 4), z("out", 4, 40, 48)
    yield "ob_relpos_bias", lambda: ob.ob_relpos_bias(rp, table, out, **kw)
    dout, dtable = z("dout", 3, 4, 40, 48), z("dtable", 32, 4)
    scratch = z("workspace", 1 << 20, dtype=torch.uint8)
    yield "ob_relpos_bias_bwd", lambda: ob.ob_relpos_bias_bwd(rp, dout, dtable, workspace=scratch, **kw)
    t = {n: z(n, 2, 40, 4, 64) for n in ("q", "o", "grad_o", "dq")}
    t.update({n: z(n, 2, 48, 2, 64) for n in ("k", "v", "dk", "dv")})
    t["lse"], t["kv_len"] = z("lse", 2, 4, 40, dtype=torch.float32), z("kv_len", 2, dtype=torch.int32)
    call = dict(relpos=rp, table=table, kv_len=t["kv_len"], **kw)
    yield "ob_attn_fwd", lambda: ob.ob_attn_fwd(t["q"], t["k"], t["v"], t["o"], t["lse"], **call)
    yield "ob_attn_bwd", lambda: ob.ob_attn_bwd(
        t["grad_o"], t["q"], t["k"], t["v"], t["o"], t["lse"], t["dq"], t["dk"], t["dv"],
        dtable=dtable, workspace=scratch, **call)


def test_calls_run_on_the_device_of_their_tensors(library):
    """The library launches on the current device: the binding makes the tensors' one
    current for the call, and leaves the caller's as it was."""
    for at in (0, 1):
        for name, call in _calls(at):
            call()
            got, args, current = library.calls[-1]
            assert (got, current, args[-1]) == (name, at, 0x1000 + at)
            assert library.current == 0


OPERANDS = {
    "ob_dropout": ("x", "y", "residual"),
    "ob_relpos_bias": ("table", "out"),
    "ob_relpos_bias_bwd": ("dout", "dtable"),
    "ob_attn_fwd": ("q", "k", "v", "o", "lse", "table", "kv_len"),
    "ob_attn_bwd": ("grad_o", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "dtable", "table",
                    "kv_len"),
}


@pytest.mark.parametrize("name,change", [(n, c) for n in OPERANDS for c in OPERANDS[n]])
def test_operands_of_two_devices_are_refused(library, name, change):
    call = dict(_calls(0, change, 1))[name]
    with pytest.raises(ob.OBError) as e:
        call()
    assert e.value.status == ob.OB_ERR_INVALID and not library.calls


def test_a_stream_of_another_device_is_refused(library):
    for name, call in _calls(0, stream=_Stream(0x77, 1)):
        with pytest.raises(ob.OBError) as e:
            call()
        assert e.value.status == ob.OB_ERR_INVALID and not library.calls, name
    for name, call in _calls(0, stream=_Stream(0x77, 0)):
        call()
        assert library.calls[-1][1][-1] == 0x77


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------

@pytest.fixture
def autograd(monkeypatch):
    """model.py over entry points that fill their outputs on the host."""
    from momentum_compression_gb300 import model as M
    seen = []

    def dropout(x, y, p, seed, offset, residual=None):
        seen.append(("dropout", x))
        y.copy_(x * 2 if residual is None else x * 2 + residual)

    def bias(plan, table, out, q_offset=0):
        out.copy_(table[0].view(-1, 1, 1).expand_as(out))

    def bias_bwd(plan, dout, dtable, q_offset=0):
        seen.append(("bias_bwd", dout))
        dtable.zero_()
        dtable[0] = dout.sum((1, 2))

    def fwd(q, k, v, o, lse, kv_len=None, **kw):
        seen.append(("fwd", None if kv_len is None else kv_len.tolist()))
        o.copy_(q)

    def bwd(grad_o, q, k, v, o, lse, dq, dk, dv, dtable=None, kv_len=None, **kw):
        seen.append(("bwd", None if kv_len is None else kv_len.tolist()))
        for t in (dq, dk, dv, dtable):
            if t is not None:
                t.fill_(1.0)

    for name, f in (("ob_dropout", dropout), ("ob_relpos_bias", bias),
                    ("ob_relpos_bias_bwd", bias_bwd), ("ob_attn_fwd", fwd), ("ob_attn_bwd", bwd)):
        monkeypatch.setattr(M, name, f)
    return M, seen


def _qkv(B=2):
    return [torch.zeros(B, 8, 2, 64, dtype=BF16).requires_grad_() for _ in range(3)]


def test_lengths_changed_before_the_backward_pass_are_noticed(autograd):
    M, seen = autograd
    lengths = torch.tensor([8, 4], dtype=torch.int32)
    o = M.attention(*_qkv(), kv_len=lengths)
    o.sum().backward()
    assert seen == [("fwd", [8, 4]), ("bwd", [8, 4])]
    o = M.attention(*_qkv(), kv_len=lengths)
    lengths.copy_(torch.tensor([3, 8], dtype=torch.int32))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_second_derivatives_are_refused(autograd):
    """The gradients come from kernels that autograd does not see into: a graph of them
    would be cut without a word."""
    M, _ = autograd
    x, res = torch.ones(4, 8, requires_grad=True), torch.ones(4, 8, requires_grad=True)
    table = torch.ones(32, 2, requires_grad=True)
    q, k, v = _qkv()
    for y, of in ((M.dropout(x, 0.5, 1, 2, res), x),
                  (M.relpos_bias(table, M.RelPos(), 4, 8), table),
                  (M.attention(q, k, v), q)):
        w = torch.ones_like(y).requires_grad_()
        g, = torch.autograd.grad((y * w).sum(), of, create_graph=True)
        assert g.requires_grad
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()
        # a first derivative is what it was
        y = M.dropout(x, 0.5, 1, 2, res)
        assert torch.equal(torch.autograd.grad(y.sum(), x)[0], torch.full_like(x, 2.0))


# ---------------------------------------------------------------------------
# Scratch that the caller brings
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("workspace", ["host", "other device", "strided"])
def test_scratch_that_kernels_cannot_use_is_refused(library, workspace):
    ws = {"host": torch.zeros(1 << 20, dtype=torch.uint8),
          "other device": _zeros(1 << 20, dtype=torch.uint8, at=1),
          "strided": _zeros(1 << 20, 2, dtype=torch.uint8)[:, 0]}[workspace]
    q, k = _zeros(2, 40, 4, 64), _zeros(2, 48, 2, 64)
    lse = _zeros(2, 4, 40, dtype=torch.float32)
    rp = ob.ob_relpos_init(32, 128, True)
    for call in (lambda: ob.ob_attn_bwd(q, q, k, k, q, lse, q, k, k, workspace=ws),
                 lambda: ob.ob_relpos_bias_bwd(rp, _zeros(3, 4, 40, 48), _zeros(32, 4),
                                               workspace=ws)):
        with pytest.raises(ob.OBError) as e:
            call()
        assert e.value.status == ob.OB_ERR_INVALID and not library.calls


# ---------------------------------------------------------------------------
# Views
# ---------------------------------------------------------------------------

def test_attention_of_views_that_start_anywhere(autograd):
    """q, k, v and the gradient may be contiguous and yet start off a 16-byte boundary:
    the kernels get a copy that does not."""
    M, _ = autograd

    def shifted(seed):
        g = torch.Generator()
        g.manual_seed(seed)
        flat = torch.randn(2 * 8 * 2 * 64 + 16, generator=g).to(BF16)
        skip = -flat.data_ptr() % 16 // 2 + 1
        t = flat[skip:skip + 2 * 8 * 2 * 64].view(2, 8, 2, 64)
        assert t.is_contiguous() and t.data_ptr() % 16
        return t

    for t in (shifted(1), shifted(2).transpose(1, 2), shifted(3)[:, ::2]):
        u = M._inner(t)
        assert u.data_ptr() % 16 == 0 and torch.equal(u, t)
    t = torch.zeros(2, 8, 2, 64, dtype=BF16)
    assert M._inner(t) is t or t.data_ptr() % 16


# ---------------------------------------------------------------------------
# Buckets that ob_relpos_init did not fill
# ---------------------------------------------------------------------------

def _relpos(plan=(32, 128, True), edges=(), **fields):
    rp = ob.ob_relpos.from_buffer_copy(ob.ob_relpos_init(*plan))
    for name, value in fields.items():
        setattr(rp, name, value)
    for at, value in edges:
        rp.first[at] = value
    return rp


@pytest.mark.parametrize("made", [
    dict(num_buckets=33),                        # an odd number of two sides
    dict(num_buckets=2, side=1),
    dict(plan=(128, 300, False), num_buckets=129, side=129),
    dict(edges=[(0, 1)]),
    dict(edges=[(0, -5)]),
    dict(edges=[(15, -70000)]),                  # would index in front of the staged values
    dict(edges=[(15, 60)]),                      # below the edge before it
    dict(edges=[(3, 9)]),
    dict(edges=[(15, (1 << 20) + 1)]),
    dict(edges=[(15, 1 << 30)]),                 # twice this is no int
    dict(edges=[(15, (1 << 31) - 1)]),
    dict(two_sided=0),
], ids=range(12))
def test_buckets_made_by_hand_are_checked(made):
    rp, L = _relpos(**made), ob.lib()
    n = ct.c_size_t()
    p = ct.byref(rp)
    a = ob.ob_attn(ob.OB_TYPE_BF16, 2, 4, 2, 64, 16, 24, 0.125, 0, 0, ct.pointer(rp), 0x5000, None,
                   0.1, 1, 2)
    for status in (L.ob_relpos_workspace_bytes(p, 2, 4, 8, 8, ct.byref(n)),
                   L.ob_relpos_bias(p, 0x1000, 0, 4, 8, 8, 0, 0x2000, 0, 64, 8, None),
                   L.ob_relpos_bias_bwd(p, 0x1000, 0, 2, 4, 8, 8, 256, 64, 8, 0, 0x2000, 0, 0x3000,
                                        1 << 30, None),
                   L.ob_attn_workspace_bytes(ct.byref(a), ct.byref(n))):
        assert status == ob.OB_ERR_INVALID


def test_every_plan_passes_its_check():
    n = ct.c_size_t()
    for two in (False, True):
        for nb in range(4, 257 if two else 129, 2):
            for D in (nb, 128, 1000, 1 << 20):
                if D > (nb // 4 if two else nb // 2):
                    rp = ob.ob_relpos_init(nb, D, two)
                    assert ob.lib().ob_relpos_workspace_bytes(ct.byref(rp), 1, 1, 8, 8,
                                                              ct.byref(n)) == ob.OB_OK


def test_strided_rows_reach_the_kernels_uncopied(autograd):
    """The kernels read rows at any stride: a slice of a wider buffer is not copied first,
    on the way back neither."""
    M, seen = autograd
    wide = torch.arange(6 * 20, dtype=torch.float32).view(6, 20)
    for x in (wide[:, 3:14], wide.view(3, 2, 20)[..., 3:14], wide[::2, :8], wide[1, 2:7],
              wide.view(3, 2, 20)[:, :1, :9]):
        y = M.dropout(x, 0.5, 1, 2, x)
        assert seen[-1][1].data_ptr() == x.data_ptr() and seen[-1][1].stride() == x.stride()
        assert y.is_contiguous() and torch.equal(y, 3 * x)
        leaf = torch.zeros_like(x, requires_grad=True)
        y = M.dropout(leaf, 0.5, 1, 2)
        y.backward(x)
        assert seen[-1][1].data_ptr() == x.data_ptr()
        assert torch.equal(leaf.grad, 2 * x)
    # those that are not rows are
    for x in (wide.t(), wide[:, ::2], wide[:1].expand(6, 20), wide.view(3, 2, 20)[:, :, :7].transpose(0, 1),
              wide[0, ::3]):
        y = M.dropout(x, 0.5, 1, 2, x)
        assert seen[-1][1].is_contiguous()
        assert y.is_contiguous() and torch.equal(y, 3 * x)
    table = torch.ones(32, 2, requires_grad=True)
    wide = torch.arange(2 * 4 * 12, dtype=torch.float32).view(2, 4, 12)
    for g, copied in ((wide[..., :8], False), (torch.ones(()).expand(2, 4, 8), True),
                      (torch.ones(2, 1, 8).expand(2, 4, 8), False)):
        M.relpos_bias(table, M.RelPos(), 4, 8).backward(g)
        assert (seen[-1][1].data_ptr() != g.data_ptr()) == copied


def test_the_readmes_example_draws_independent_masks(monkeypatch):
    """Its calls of several steps, one (seed, offset) each."""
    import os
    import re
    from momentum_compression_gb300 import model as M
    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(readme) as f:
        code, = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "M.attention" in c]
    drawn = []
    monkeypatch.setattr(M, "ob_attn_fwd", lambda q, k, v, o, lse, **kw: drawn.append(
        (kw["seed"], kw["offset"])))
    monkeypatch.setattr(M, "ob_dropout", lambda x, y, p, seed, offset, residual=None: drawn.append(
        (seed, offset)))
    q, k, v = _qkv()
    names = dict(q=q, k=k, v=v, lengths=torch.tensor([8, 4], dtype=torch.int32), seed=7,
                 table=torch.zeros(32, 2, dtype=BF16), w=torch.zeros(128, 16, dtype=BF16),
                 x=torch.zeros(2, 8, 16, dtype=BF16))
    for step in range(4):
        exec(code, dict(names, step=step))
    assert len(drawn) == 8 and len(set(drawn)) == 8, drawn


def test_the_first_call_may_come_from_two_threads(library, monkeypatch):
    """What a call looks up once is there in full when a second thread sees that it is."""
    monkeypatch.setattr(ob, "_raw_stream", None)
    monkeypatch.setattr(ob, "_current_device", None)
    monkeypatch.setattr(ob, "_devices", 0)
    seen = []
    monkeypatch.setattr(torch.cuda, "device_count", lambda: seen.append(ob._raw_stream) or 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x1000 + d, raising=False)
    x = _zeros(5, 24)
    ob.ob_dropout(x, x, 0.5, 1, 2)
    assert seen == [None] and ob._devices == 1 and ob._current_device is not None
    assert library.calls[-1][1][-1] == 0x1000

"""Layer norm, the dense layer and AdamW without a GPU: the refusals of every
entry point and of the binding, and the tests' own references (gradients
against central differences, codes against their definition)."""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

import layers_ref as L
import momentum_compression_gb300 as ob
from test_model_binding import _on, _zeros, library  # noqa: F401

BF16, F32 = torch.bfloat16, torch.float32
BAD, ALIGN, UNSUPPORTED = ob.OB_ERR_INVALID, ob.OB_ERR_ALIGN, ob.OB_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _built():
    from momentum_compression_gb300 import _build
    _build.build()


def _refuses(fn, ok, changes):
    """Each change (place, value, status) of the valid arguments `ok` is refused with a message."""
    for change in changes:
        args = list(ok)
        *places, status = change
        for at, value in zip(places[::2], places[1::2]):
            args[at] = value
        assert fn(*args) == status, (change, ob.ob_last_error(None))
        assert ob.ob_last_error(None)


def test_layer_norm_refuses():
    f = ob.lib().ob_layernorm_fwd
    #     x       ldx res     ldr  w       b       wt y       ldy sum     lds mean    rstd    rows cols type eps
    ok = [0x1000, 64, 0x2000, 64, 0x3000, 0x4000, 0, 0x5000, 64, 0x6000, 64, 0x7000, 0x8000, 4, 64, 0, 1e-5, None]
    _refuses(f, ok, [(0, None, BAD), (7, None, BAD), (0, 0x1002, ALIGN), (2, 0x2001, ALIGN), (7, 0x5002, ALIGN),
                     (9, 0x6001, ALIGN), (4, 0x3002, ALIGN), (5, 0x4001, ALIGN), (11, 0x7002, ALIGN),
                     (12, 0x8001, ALIGN), (1, 63, BAD), (3, 63, BAD), (8, 63, BAD), (10, 63, BAD), (15, 3, BAD),
                     (6, -1, BAD), (16, 0.0, BAD), (16, -1.0, BAD), (16, math.nan, BAD), (16, 1e-60, BAD),
                     (2, None, BAD), (9, 0x5000, BAD), (14, 1 << 24, BAD), (13, 1 << 35, BAD)])
    assert f(*ok[:13], 0, *ok[14:]) == ob.OB_OK
    f = ob.lib().ob_layernorm_bwd
    #     dy      ld  x       ld  mean    rstd    w       wt ds      ld  dx      ld  dw      db      r  c   t  ws      bytes
    ok = [0x1000, 64, 0x2000, 64, 0x3000, 0x4000, 0x5000, 0, 0x6000, 64, 0x7000, 64, 0x8000, 0x9000, 4, 64, 0,
          0xa000, 1 << 20, None]
    _refuses(f, ok, [(0, None, BAD), (2, None, BAD), (4, None, BAD), (5, None, BAD), (0, 0x1002, ALIGN),
                     (2, 0x2002, ALIGN), (4, 0x3001, ALIGN), (6, 0x5002, ALIGN), (8, 0x6001, ALIGN),
                     (10, 0x7001, ALIGN), (12, 0x8002, ALIGN), (13, 0x9002, ALIGN), (1, 63, BAD), (3, 63, BAD),
                     (9, 63, BAD), (11, 63, BAD), (16, 7, BAD), (7, 7, BAD), (17, None, BAD), (17, 0xa008, ALIGN),
                     (18, 16, BAD), (10, None, BAD), (15, 1 << 24, BAD)])
    with pytest.raises(ob.OBError):
        ob.ob_layernorm_workspace_bytes(1, 1 << 24)
    assert ob.ob_layernorm_workspace_bytes(0, 64) == ob.ob_layernorm_workspace_bytes(64, 0) == 0


def test_dense_refuses():
    def lin(**kw):
        a = dict(type=ob.OB_TYPE_BF16, act=2, w_kn=0, unaligned=0, M=16, N=32, K=64)
        a.update(kw)
        return ct.byref(ob.ob_linear(*a.values()))

    def mat(p, ld):
        return ct.byref(ob.ob_matrix(p, ld))
    f = ob.lib().ob_linear_fwd
    #     l      x                 w                 b       r                 z                 y
    ok = [lin(), mat(0x1000, 64), mat(0x2000, 64), 0x3000, mat(0x4000, 32), mat(0x5000, 32), mat(0x6000, 32),
          0x7000, 1 << 30, None]
    _refuses(f, ok, [(0, None, BAD), (0, lin(type=0), UNSUPPORTED), (0, lin(act=4), BAD), (0, lin(act=-1), BAD),
                     (0, lin(M=-1), BAD), (0, lin(N=1 << 30), BAD), (0, lin(K=1 << 30), BAD), (0, lin(M=1 << 29, N=1 << 29), BAD), (1, None, BAD),
                     (2, None, BAD), (6, None, BAD), (1, mat(0x1002, 64), ALIGN), (1, mat(0x1000, 65), ALIGN),
                     (1, mat(0x1000, 56), BAD), (2, mat(0x2000, 56), BAD), (2, mat(0x2008, 64), ALIGN),
                     (4, mat(0x4008, 32), ALIGN), (5, mat(0x5000, 33), ALIGN), (6, mat(0x6002, 32), ALIGN),
                     (6, mat(0x6000, 24), BAD), (3, 0x3001, ALIGN), (5, mat(0x6000, 32), BAD),
                     (0, lin(unaligned=1), 1, mat(0x1001, 64), ALIGN), (0, lin(w_kn=1), 2, mat(0x2000, 24), BAD)])
    f = ob.lib().ob_linear_bwd
    #     l      dy                x                w                z                dx               dw
    ok = [lin(), mat(0x1000, 32), mat(0x2000, 64), mat(0x3000, 64), mat(0x4000, 32), mat(0x5000, 64),
          mat(0x6000, 64), 0x7000, 0x8000, 1 << 30, None]
    _refuses(f, ok, [(0, None, BAD), (1, None, BAD), (2, None, BAD), (3, None, BAD), (4, None, BAD),
                     (1, mat(0x1002, 32), ALIGN), (5, mat(0x5000, 65), ALIGN), (6, mat(0x6000, 56), BAD),
                     (7, 0x7001, ALIGN), (8, None, BAD), (8, 0x8010, ALIGN), (9, 16, BAD)])
    n = ct.c_size_t()
    assert ob.lib().ob_linear_workspace_bytes(lin(type=0), 0, ct.byref(n)) == UNSUPPORTED
    assert ob.lib().ob_linear_workspace_bytes(lin(), 0, None) == BAD


def test_adamw_refuses():
    f = ob.lib().ob_adamw_step

    def conf(**kw):
        a = dict(state_bits=8, grad_type=0, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, seed=1, lr_device=None,
                 grad_scale=None, skip=None)
        a.update(kw)
        return ct.byref(ob.ob_adamw(*a.values()))

    def tensors(**kw):
        a = dict(p=0x1000, copy=0x2000, n=300, decay=0.1, p_type=0, copy_type=1)
        a.update(kw)
        return (ob.ob_adamw_tensor * 2)(ob.ob_adamw_tensor(0x9000, None, 5, 0.0, 0, 0),
                                        ob.ob_adamw_tensor(*a.values()))

    def grads(p):
        return (ct.c_void_p * 2)(0x9000, p)
    ok = [conf(), tensors(), grads(0x3000), 2, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, None]
    _refuses(f, ok, [(0, None, BAD), (0, conf(state_bits=16), BAD), (0, conf(grad_type=3), BAD),
                     (0, conf(lr=-1.0), BAD), (0, conf(lr=math.nan), BAD), (0, conf(b1=1.0), BAD),
                     (0, conf(b2=-0.1), BAD), (0, conf(eps=0.0), BAD), (0, conf(eps=2.0), BAD),
                     (0, conf(lr_device=0x11), ALIGN), (0, conf(skip=0x12), ALIGN), (0, conf(grad_scale=0x13), ALIGN),
                     (1, None, BAD), (2, None, BAD), (3, -1, BAD), (1, tensors(p=None), BAD),
                     (1, tensors(p=0x1002), ALIGN), (1, tensors(copy=0x2001), ALIGN), (1, tensors(decay=-0.1), BAD),
                     (1, tensors(decay=math.inf), BAD), (1, tensors(p_type=5), BAD), (1, tensors(copy_type=5), BAD),
                     (1, tensors(n=1 << 41), BAD), (1, tensors(n=(1 << 40)), BAD), (2, grads(0x3002), ALIGN),
                     (4, None, BAD), (5, 0x5008, ALIGN), (6, None, BAD), (7, None, BAD), (8, None, BAD),
                     (8, 0x8004, ALIGN)])
    f = ob.lib().ob_adamw_moments
    ok = [0x1000, 0x2000, 0x3000, 0x4000, 512, 0x5000, 0x6000, None]
    _refuses(f, ok, [(0, None, BAD), (1, 0x2001, ALIGN), (2, None, BAD), (3, None, BAD), (4, 500, BAD),
                     (5, None, BAD), (6, 0x6008, ALIGN)])
    assert f(*ok[:4], 0, *ok[5:]) == ob.OB_OK


def test_binding_refuses():
    """What the C calls cannot see."""
    x, w, v = _zeros(4, 64), _zeros(32, 64), _zeros(64)
    y, far = _zeros(4, 32), _zeros(4, 64, at=1)
    f = _zeros(64, dtype=F32)
    st = _zeros(4, dtype=F32)
    p, g = _zeros(300, dtype=F32), _zeros(300, dtype=F32)
    calls = [
        lambda: ob.ob_layernorm_fwd(torch.zeros(4, 64), torch.zeros(4, 64)),
        lambda: ob.ob_layernorm_fwd(x, far), lambda: ob.ob_layernorm_fwd(x, y),
        lambda: ob.ob_layernorm_fwd(x, x.float()), lambda: ob.ob_layernorm_fwd(x, x, residual=y),
        lambda: ob.ob_layernorm_fwd(x, x, sum=y, residual=x), lambda: ob.ob_layernorm_fwd(x, x, weight=v[:5]),
        lambda: ob.ob_layernorm_fwd(x, x, weight=v, bias=f), lambda: ob.ob_layernorm_fwd(x, x, mean=v),
        lambda: ob.ob_layernorm_fwd(x, x, mean=f), lambda: ob.ob_layernorm_fwd(x.double(), x.double()),
        lambda: ob.ob_layernorm_fwd(x, x, weight=_zeros(64, at=1)),
        lambda: ob.ob_layernorm_bwd(y, x, st, st, x), lambda: ob.ob_layernorm_bwd(x, x, st, None, dx=y),
        lambda: ob.ob_layernorm_bwd(x, x, st, st, dx=x, weight=v, dweight=f),
        lambda: ob.ob_linear_fwd(torch.zeros(4, 64, dtype=BF16), w, y), lambda: ob.ob_linear_fwd(x, w.t(), y),
        lambda: ob.ob_linear_fwd(x, w, x), lambda: ob.ob_linear_fwd(x, w, y, bias=v),
        lambda: ob.ob_linear_fwd(x, w, y, bias=_zeros(32, dtype=F32)), lambda: ob.ob_linear_fwd(x, w, y, residual=x),
        lambda: ob.ob_linear_fwd(x, w, y, activation="tanh"), lambda: ob.ob_linear_fwd(x, _zeros(32, 64, at=1), y),
        lambda: ob.ob_linear_fwd(x, _zeros(64, 128)[::2, ::2], y), lambda: ob.ob_linear_fwd(x, w.half(), y),
        lambda: ob.ob_linear_bwd(y, x, w, activation="gelu", dx=x), lambda: ob.ob_linear_bwd(y, x, w, dx=y),
        lambda: ob.ob_linear_bwd(y, x, w, dw=_zeros(64, 32).t()), lambda: ob.ob_linear_bwd(y, y, w),
        lambda: ob.ob_linear_bwd(y, x, w, dbias=v),
        lambda: ob.AdamW([]), lambda: ob.AdamW([torch.zeros(3)]), lambda: ob.AdamW([p], state_bits=16),
        lambda: ob.AdamW([p], weight_decay=[0.1, 0.2]), lambda: ob.AdamW([p], copies=[x]),
        lambda: ob.AdamW([p, _zeros(5, dtype=F32, at=1)]), lambda: ob.AdamW([_zeros(4, 8).t()]),
        lambda: ob.AdamW([p, p]), lambda: ob.AdamW([p], copies=[p]), lambda: ob.AdamW([p, p[:5]]),
        lambda: ob.AdamW([p], state=dict(m=p, v=p, step=1)), lambda: ob.AdamW([p], state=dict(step=1)),
    ]
    # the step's arrays: 300 elements are two blocks of state
    m, m8, e, c = _zeros(512, dtype=F32), _zeros(512, dtype=torch.uint8), _zeros(2, dtype=torch.uint8), _zeros(4, dtype=torch.float64)
    table = (ob.ob_adamw_tensor * 1)(ob.ob_adamw_tensor(256, 0, 300, 0.0, ob.OB_TYPE_F32, 0))
    config = {bits: ob.ob_adamw(bits, ob.OB_TYPE_F32, 0.1, 0.9, 0.99, 1e-8) for bits in (8, 32)}

    def step(bits=32, g=g, m=m, v=m, c=c, **exp):
        return lambda: ob.ob_adamw_step(config[bits], table, [g], m, v, c, at=0, **exp)
    calls += [
        lambda: ob.ob_adamw_step(config[32], table, [g, g], m, m, c), step(g=g[:299]), step(g=g.bfloat16()),
        step(g=_zeros(300, dtype=F32, at=1)), step(g=_zeros(600, dtype=F32)[::2]), step(m=m[:511]), step(v=m[:511]),
        step(m=m8), step(v=None), step(c=c[:3]), step(c=m), step(c=_zeros(4, dtype=torch.float64, at=1)),
        step(8, m=m, v=m8, m_exp=e, v_exp=e), step(8, m=m8, v=m8, m_exp=e), step(8, m=m8, v=m8, m_exp=e[:1], v_exp=e),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ob.OBError) as e:
            call()
        assert e.value.status in (BAD, UNSUPPORTED), i


@pytest.mark.parametrize("b", [0.0, 0.5, 0.9, 0.95, 0.999, 1 - 2 ** -40])
def test_powers_are_products(b):
    """A resumed optimizer starts from the bits that the device's products have come to."""
    want, powers = 1.0, {}
    for t in range(20001):
        powers[t] = want
        want *= b
    for t in (0, 1, 2, 4, 43, 1000, 6600, 7200, 20000):
        assert ob._power(b, t) == powers[t], t


def test_reference_gradients_against_differences():
    g = torch.Generator()
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, w, b, dy = r(3, 7), r(7), r(7), r(3, 7)
    _, _, mean, rstd = L.layer_norm(x, w, b, 1e-5)
    (dx, dw, db), _ = L.layer_norm_grad(dy, x, mean, rstd, w, None)
    f = lambda x, w, b: (L.layer_norm(x, w, b, 1e-5)[0] * dy).sum()

    def differences(f, args, k):
        out = torch.zeros_like(args[k])
        for i in range(out.numel()):
            two = []
            for s in (1e-5, -1e-5):
                a = [t.clone() for t in args]
                a[k].view(-1)[i] += s
                two.append(f(*a))
            out.view(-1)[i] = (two[0] - two[1]) / 2e-5
        return out
    for k, want in enumerate((dx, dw, db)):
        assert torch.allclose(differences(f, (x, w, b), k), want, rtol=1e-6, atol=1e-7)
    x, w, b, dy = r(3, 5), r(4, 5), r(4), r(3, 4)
    for act in ("none", "relu", "gelu", "gelu_tanh"):
        f = lambda x, w, b: (L.dense(x, w, b, None, act)[0][1] * dy).sum()
        z = L.dense(x, w, b, None, act)[0][0]
        dz = dy * L.act(z, act)[1]
        for k, want in enumerate((dz @ w, dz.t() @ x, dz.sum(0))):
            assert torch.allclose(differences(f, (x, w, b), k), want, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("bias", [7, 23])
def test_reference_codes_are_their_values(bias):
    """Every code's value is kept by every noise, and a value between two codes takes either."""
    top = 127 if bias == 7 else 255
    codes = np.zeros(256, np.uint8)
    codes[:top] = np.arange(top)
    for e in (4, 100, 127, 200, 246):
        exp = np.array([e], np.uint8)
        x = L.decode(codes, exp, bias)
        for noise in (0, 40000, 65535):
            c, u = L.encode(x, np.full(256, noise), bias)
            assert np.array_equal(c, codes) and u[0] == e
            if bias == 7:
                c, u = L.encode(-x, np.full(256, noise), bias)
                assert np.array_equal(c & 127, codes)
        order = np.sort(x[:top])
        assert (np.diff(order) > 0).all()
        mid = x.copy()
        mid[:top - 1] = (x[:top - 1].astype(float) + x[1:top]) / 2
        lo, _ = L.encode(mid, np.full(256, 0), bias)
        hi, _ = L.encode(mid, np.full(256, 65535), bias)
        first = 1 if bias == 23 else 0  # a positive v has no code 0
        assert np.array_equal(lo[first:top - 1], codes[first:top - 1])
        assert np.array_equal(hi[:top - 1], codes[1:top])


def test_fakes_reach_the_library(library):  # noqa: F811
    """The scratch of a call on a passed stream is made on it; calls go to their tensors' device."""
    names = ("ob_layernorm_fwd", "ob_layernorm_bwd", "ob_linear_fwd", "ob_linear_bwd", "ob_adamw_step")
    for n in names:
        def call(*args, n=n):
            library.calls.append((n, args, library.current))
            return ob.OB_OK
        setattr(library, n, call)
    x, w, y = _zeros(4, 64, at=1), _zeros(32, 64, at=1), _zeros(4, 32, at=1)
    st = _zeros(4, dtype=F32, at=1)
    ob.ob_layernorm_fwd(x, _zeros(4, 64, at=1), stream=77)
    ob.ob_layernorm_bwd(x, x, st, st, dweight=_zeros(64, dtype=F32, at=1), stream=77)
    ob.ob_linear_fwd(x, w, y, stream=77)
    ob.ob_linear_bwd(y, x, w, dx=x, z=y, activation="gelu", stream=77)
    assert [c[0] for c in library.calls] == list(names[:4])
    assert all(c[2] == 1 and c[1][-1] == 77 for c in library.calls)
    assert all(s is not None for _, s in library.allocated)

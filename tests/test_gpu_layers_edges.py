"""Layer norm, the dense layer and AdamW on the GPU at the edge of what they allow: GELU far
out, arrays updated in place, broadcast inputs, streams."""
import math

import pytest
import torch

import layers_ref as L
import momentum_compression_gb300 as ob
from momentum_compression_gb300 import model as M

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    from momentum_compression_gb300 import _build
    _build.build()
    yield
    assert ob.ob_layer_device_error() == 0


# ---------------------------------------------------------------------------
# GELU's tails
# ---------------------------------------------------------------------------

def _values(dtype, lo, hi):
    """Every value of a 16-bit type in [lo, hi], repeated to a multiple of 8."""
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    v = v[(v.float() >= lo) & (v.float() <= hi)]
    return v[torch.arange(-(-len(v) // 8) * 8) % len(v)].cuda()


def _act64(z, name):
    """act(z), act'(z) of doubles, the tanh form without 1 + tanh, which has no digits far out."""
    if name == "gelu":
        return L.act(z, name)
    a, b = math.sqrt(2 / math.pi), 0.044715
    s = 1 / (1 + (-2 * a * (z + b * z ** 3)).exp())
    return z * s, s + 2 * z * s * (1 - s) * a * (1 + 3 * b * z * z)


# The lowest z at which 2^126 times the tail is above 1: further out fp32 has no digits of it.
LOWEST = {"gelu": -12.5, "gelu_tanh": -9.9}


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("way", ["few rows", "tiles", "odd starts"])
def test_gelu_is_near_relative_to_itself(dtype, act, way):
    """At every z, one rounding to the type and 2^-15 of the value.  z is exact (a product by
    one).  The exponent of e^(-z^2 / 2), at most 113 in units of ln 2, is rounded three times:
    113 * 3 * 2^-24 * ln 2 = 1.4e-5; 2^-15 is 3.1e-5, and holds the rest (the fit, 5e-6, and
    some ten operations)."""
    z = _values(dtype, LOWEST[act], 20.0)
    n = len(z)
    if way == "few rows":
        x, w, y = z.new_ones(1, 1), z.view(n, 1), z.new_empty(1, n)
    elif way == "tiles":
        x, w, y = z.new_zeros(n, 8), torch.eye(8, device="cuda", dtype=dtype), z.new_empty(n, 8)
        x[:, 0] = z
    else:
        x, w, y = z.view(n, 1), z.new_ones(1, 1), z.new_empty(n, 1)
    ob.ob_linear_fwd(x, w, y, activation=act)
    got = y[0] if way == "few rows" else y[:, 0]
    want, _ = _act64(z.double(), act)
    L.within(got, want, 2.0 ** -15 * want.abs(), act)
    far = torch.linspace(LOWEST[act], -60.0, 1024, device="cuda").to(dtype)
    out = z.new_empty(1, 1024)
    ob.ob_linear_fwd(z.new_ones(1, 1), far.view(-1, 1), out, activation=act)
    assert (out <= 0).all() and (out.double().abs() <= -LOWEST[act] * 2.0 ** -110).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("cols", [8, 1])
def test_gelu_slope_is_near_relative_to_itself(dtype, act, cols):
    """As the value's, twice: for z <= -2 the slope is the difference of two terms whose sizes
    add up to 1.6 times it at most.  Nearer it passes through 0: both terms, of at most 1.2,
    are off by some 2^-21 each."""
    z = _values(dtype, LOWEST[act], 20.0)
    wide = z.view(-1, 1).expand(-1, cols).contiguous()
    w, dx = torch.eye(cols, device="cuda", dtype=dtype), torch.empty_like(wide)
    ob.ob_linear_bwd(torch.ones_like(wide), torch.zeros_like(wide), w, dx=dx, z=wide, activation=act)
    _, want = _act64(z.double(), act)
    L.within(dx[:, 0], want, 2.0 ** -14 * want.abs() + 2.0 ** -19 * (z.double() > -2), act)

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


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

# rows that share a warp, a warp's, a block's (few and many), rows read again; odd widths
ROWS = [(3, 7), (1001, 64), (1001, 100), (300, 384), (37, 768), (1300, 768), (9, 1001), (300, 1024), (65, 2050),
        (305, 4096), (3, 8192), (310, 9000), (3, 20000)]


def _rows(rows, cols, dtype, seed, shift):
    """Rows at an aligned or an odd start, away from 0."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    flat = torch.empty(rows * cols + shift, device="cuda", dtype=dtype)
    t = flat[shift:].view(rows, cols)
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda") * 1.5 + 0.7)
    return t


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("shift", [0, 1])
def test_layer_norm_statistics(dtype, rows, cols, shift):
    """mean and rstd themselves, within the errors that layers_ref derives for y from them."""
    x = _rows(rows, cols, dtype, 3, shift)
    mean, rstd = (torch.full((rows,), math.nan, device="cuda") for _ in range(2))
    ob.ob_layernorm_fwd(x, torch.empty_like(x), mean=mean, rstd=rstd)
    _, _, m, r = L.layer_norm(x, None, None, 1e-5)
    c, x = L.row_sums(cols), x.double()
    em = c * x.abs().mean(1) + L.U32 * m.abs()
    var = (x - m[:, None]).square().mean(1)
    er = 0.5 * (2 * var.sqrt() * em + em * em + (c + 4 * L.U32) * var) / (var + 1e-5) + 4 * L.U32
    assert ((mean.double() - m).abs() <= em + L.U32 * m.abs()).all()
    assert ((rstd.double() - r).abs() <= er * r).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("shift", [0, 1])
def test_layer_norm_in_place(dtype, rows, cols, shift):
    """y and sum may be x and residual: the same bits."""
    make = lambda: (_rows(rows, cols, dtype, 5, shift), _rows(rows, cols, dtype, 6, shift))
    w = _rows(1, cols, dtype, 7, 0)[0]
    x, r = make()
    y, s = torch.empty_like(x), torch.empty_like(x)
    ob.ob_layernorm_fwd(x, y, w, w, residual=r, sum=s)
    for of_y, of_s in (("x", "r"), ("r", "x"), ("x", None), (None, "x"), ("r", None), (None, "r")):
        a, b = make()
        at = dict(x=a, r=b)
        y2, s2 = at.get(of_y, torch.empty_like(a)), at.get(of_s, torch.empty_like(a))
        ob.ob_layernorm_fwd(a, y2, w, w, residual=b, sum=s2)
        assert torch.equal(y2, y) and torch.equal(s2, s), (of_y, of_s)
    x, _ = make()
    ob.ob_layernorm_fwd(x, y, w)
    ob.ob_layernorm_fwd(x, x, w)
    assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# The dense layer
# ---------------------------------------------------------------------------

# few rows (whole and cut among a cluster), tiles, tiles cut along the sum, pairs of blocks; odd sizes
SIZES = [(1, 40, 8), (8, 512, 4096), (128, 768, 768), (300, 200, 300), (257, 511, 513), (250, 768, 96),
         (300, 64, 2000), (2816, 2304, 4096), (2570, 1030, 1000)]


@pytest.mark.parametrize("Mr,N,K", SIZES)
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("keep", [False, True])
def test_dense_adds_to_its_residual_in_place(Mr, N, K, kn, shift, keep):
    """y may be residual: the same bits."""
    x, r = _rows(Mr, K, BF16, 1, shift), _rows(Mr, N, BF16, 2, shift)
    w = _rows(*((K, N) if kn else (N, K)), BF16, 3, shift).div_(K ** 0.5)
    w, b = w.t() if kn else w, _rows(1, N, BF16, 4, 0)[0]
    y, z, z2 = torch.empty_like(r), *(torch.empty_like(r) if keep else None for _ in range(2))
    ob.ob_linear_fwd(x, w, y, b, r, z, "gelu")
    ob.ob_linear_fwd(x, w, r, b, r, z2, "gelu")
    assert torch.equal(y, r)
    if keep:
        assert torch.equal(z, z2)


def test_broadcast_inputs_and_gradients():
    """model.layer_norm and model.linear take views whose elements are shared, and gradients that are;
    autograd sums them over what was broadcast."""
    mk = lambda *s: _rows(1, math.prod(s), BF16, sum(s), 0).view(*s)
    x, w, b, res = mk(64), mk(96, 64), mk(96), mk(96)
    lnw = mk(1).expand(64)
    leaves = [t.detach().requires_grad_() for t in (x, w, b, res, lnw[:1])]
    full = [x.expand(5, 7, 64).contiguous(), w, b, res.expand(5, 7, 96).contiguous(), lnw.contiguous()]
    full = [t.detach().requires_grad_() for t in full]

    def out(x, w, b, res, lnw):
        return M.linear(M.layer_norm(x, lnw), w, b, "gelu", res)
    a, c = leaves, full
    y = out(a[0].expand(5, 7, 64), a[1], a[2], a[3].expand(5, 7, 96), a[4].expand(64))
    y2 = out(*c)
    assert torch.equal(y, y2)
    dy = mk(1).expand(5, 7, 96)
    got, want = torch.autograd.grad(y, a, dy), torch.autograd.grad(y2, c, dy.contiguous())
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    for g, f, shape in ((got[0], want[0], (35, 64)), (got[3], want[3], (35, 96)), (got[4], want[4], (64, 1))):
        f = f.double().view(shape)
        # autograd's sums over the broadcast dimensions, each rounded to bf16
        assert ((g.double().view(-1) - f.sum(0)).abs() <= 3 * 2.0 ** -8 * f.abs().sum(0)).all()


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

def test_adamw_on_another_stream():
    """Steps and the moments' values on a stream that is not the current one, and state() after them."""
    def run(stream):
        p = torch.ones(1 << 22, device="cuda")
        g = torch.full_like(p, 0.5)
        opt = ob.AdamW([p], lr=1e-2, state_bits=8, seed=2)
        torch.cuda.synchronize()
        for _ in range(20):
            opt.step([g], stream=stream)
        values = opt.moments(stream=stream)
        return opt.state(), p, values
    (s, p, v), (s2, p2, v2) = run(None), run(torch.cuda.Stream())
    assert s["step"] == s2["step"] == 20 and torch.equal(p, p2)
    assert all(torch.equal(a, b) for a, b in zip(v, v2))
    assert all(torch.equal(s[n], s2[n]) for n in ("m", "v", "m_exp", "v_exp"))


# ---------------------------------------------------------------------------
# Arrays of more than 2^32 elements
# ---------------------------------------------------------------------------

LONG = 512 * 4099  # rows; of 2056 columns they hold 4.3e9 elements


def _long(cols, seed):
    """LONG rows, the same 4099 again and again."""
    return _rows(4099, cols, BF16, seed, 0).expand(512, 4099, cols).reshape(LONG, cols)


def test_layer_norm_of_long_arrays():
    """The last rows are right, and equal rows have equal bits."""
    cols, tail = 2056, slice(LONG - 300, LONG)
    x, w = _long(cols, 1), _rows(1, cols, BF16, 2, 0)[0]
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(LONG, device="cuda") for _ in range(2))
    ob.ob_layernorm_fwd(x, y, w, w, mean=mean, rstd=rstd)
    want, err, _, _ = L.layer_norm(x[tail], w, w, 1e-5)
    L.within(y[tail], want, err, "y")
    assert torch.equal(y[tail], y[4099 - 300:4099])
    dx = torch.empty_like(x)
    ob.ob_layernorm_bwd(y, x, mean, rstd, dx, w)
    (want, _, _), (err, _, _) = L.layer_norm_grad(y[tail], x[tail], mean[tail], rstd[tail], w, None)
    L.within(dx[tail], want, err, "dx")
    assert torch.equal(dx[tail], dx[4099 - 300:4099])


@pytest.mark.parametrize("kn", [False, True])
def test_dense_of_long_arrays(kn):
    N, K, tail = 2056, 64, slice(LONG - 300, LONG)
    x, b = _long(K, 3), _rows(1, N, BF16, 4, 0)[0]
    w = _rows(*((K, N) if kn else (N, K)), BF16, 5, 0).div_(8)
    w = w.t() if kn else w
    y, z = (torch.empty(LONG, N, device="cuda", dtype=BF16) for _ in range(2))
    ob.ob_linear_fwd(x, w, y, b, None, z, "gelu")
    (z64, y64), (ez, ey) = L.dense(x[tail], w, b, None, "gelu")
    L.within(y[tail], y64, ey, "y")
    L.within(z[tail], z64, ez, "z")
    dx = torch.empty_like(x)
    ob.ob_linear_bwd(y, x, w, dx=dx, z=z, activation="gelu")
    (want, _, _), (err, _, _) = L.dense_grad(y[tail], x[tail], w, z[tail], "gelu")
    L.within(dx[tail], want, err, "dx")


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_of_a_long_tensor(bits):
    """The last elements take the step that they take by themselves, the random numbers of their own place."""
    n = (1 << 32) + 1000
    p = torch.full((n,), 0.5, device="cuda", dtype=BF16)
    small = _rows(1, 5000, BF16, 6, 0)[0]
    g = torch.zeros(n, device="cuda", dtype=BF16)
    g[-5000:] = small
    opt = ob.AdamW([p], lr=1e-2, weight_decay=0.0, state_bits=bits, seed=9)
    opt.step([g])
    first = (n - 5000) // 256 * 256
    k = n - first
    pad = -k % 256
    np_ = lambda t: torch.nn.functional.pad(t[first:].float(), (0, pad)).cpu().numpy()
    zero = torch.zeros(k + pad, dtype=torch.uint8 if bits == 8 else F32).numpy()
    exps = torch.zeros((k + pad) // 256, dtype=torch.uint8).numpy()
    q, size, new = L.adamw(np_(torch.full_like(p, 0.5)), np_(g), zero, zero, 1, 9, first, 1e-2, 0.9, 0.999, 1e-8, 0.0,
                           1.0, bits, exps, exps)
    L.within(p[first:], torch.from_numpy(q[:k]).cuda(), torch.from_numpy(size[:k]).cuda() * 2.0 ** -20 + 2 * L.U32, "p")
    got = [opt.m[first:], opt.v[first:]]
    if bits == 8:
        got += [opt.m_exp[first // 256:], opt.v_exp[first // 256:]]
    for a, b in zip(got, new):
        assert torch.equal(a.cpu(), torch.from_numpy(b))
    assert (p[:first] == 0.5).all()

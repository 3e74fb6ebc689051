"""Layer norm, the dense layer and AdamW on the GPU, against the 64-bit
definitions with bounds derived from the formulas (tests/layers_ref.py); AdamW's
moments bit by bit."""
import math

import numpy as np
import pytest
import torch

import layers_ref as L
import model_ref as R
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


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, dtype=F32: torch.randn(*s, generator=g, device="cuda").to(dtype)


def _slice(mk, rows, cols, pad, shift, dtype, scale=1.0, shift_by=0.0):
    """Rows of `cols` in a buffer of NaN, `pad` elements between them, `shift` before them."""
    flat = torch.full((rows * (cols + pad) + shift,), math.nan, device="cuda", dtype=dtype)
    t = flat[shift:].view(rows, cols + pad)[:, :cols]
    t.copy_(mk(rows, cols) * scale + shift_by)
    return t


def _guarded(rows, cols, pad, shift, dtype):
    """(view to write, check that nothing around it was written)."""
    flat = torch.full((rows * (cols + pad) + shift + 16,), 7.0, device="cuda", dtype=dtype)
    t = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    def check():
        left = flat.clone()
        left[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = 7.0
        assert (left == 7.0).all(), "wrote outside the rows"
    return t, check


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 8), (3, 7), (2, 33), (5, 64), (1, 768), (37, 768), (9, 1001), (300, 1024),
          (2, 2048), (1, 2048), (65, 2050), (7, 4096), (4, 5000), (3, 8192), (2, 12345), (1, 16384),
          (2, 40000), (700, 128), (5000, 24), (1300, 520), (400, 1500),
          (305, 4096), (310, 9000), (3001, 64), (1001, 100),
          (901, 384), (1300, 300)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 1), (3, 8)])
def test_layer_norm(dtype, rows, cols, pad, shift):
    mk = _gen(rows * 7 + cols)
    wt = F32 if pad % 2 else dtype
    x = _slice(mk, rows, cols, pad, shift, dtype, 1.5, 0.7)
    r = _slice(mk, rows, cols, pad, shift, dtype)
    w, b = mk(cols, dtype=wt), mk(cols, dtype=wt)
    for residual, weight, bias in ((None, w, b), (r, w, b), (r, None, None), (None, w, None)):
        y, clean = _guarded(rows, cols, pad, shift, dtype)
        s, s_clean = _guarded(rows, cols, pad, shift, dtype)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ob.ob_layernorm_fwd(x, y, weight, bias, 1e-5, residual, s if residual is not None else None,
                            mean, rstd)
        v = x
        if residual is not None:
            v = (x.float() + r.float()).to(dtype)
            assert torch.equal(s, v)
            s_clean()
        clean()
        want, err, m64, r64 = L.layer_norm(v, weight, bias, 1e-5)
        L.within(y, want, err, "y")
        # the statistics' own bounds, as in layer_norm()
        c = L.row_sums(cols)
        assert ((mean.double() - m64).abs() <= (c + 2 * L.U32) * v.double().abs().mean(1) + 1e-30).all()
        # without the statistics and the sum: the same values
        y2, clean = _guarded(rows, cols, pad, shift, dtype)
        ob.ob_layernorm_fwd(x, y2, weight, bias, 1e-5, residual)
        clean()
        assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 1), (3, 8)])
def test_layer_norm_gradient(dtype, rows, cols, pad, shift):
    mk = _gen(rows * 5 + cols)
    wt = F32 if pad % 2 else dtype
    x = _slice(mk, rows, cols, pad, shift, dtype, 1.5, 0.7)
    dy = _slice(mk, rows, cols, pad, shift, dtype)
    ds = _slice(mk, rows, cols, pad, shift, dtype)
    w = mk(cols, dtype=wt)
    _, _, mean, rstd = L.layer_norm(x, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    for weight, dsum in ((w, None), (w, ds), (None, ds)):
        dx, clean = _guarded(rows, cols, pad, shift, dtype)
        dw, db = (torch.full((cols,), 5.0, device="cuda", dtype=wt) for _ in range(2))
        ob.ob_layernorm_bwd(dy, x, mean, rstd, dx, weight, dw, db, dsum)
        clean()
        want, err = L.layer_norm_grad(dy, x, mean, rstd, weight, dsum)
        for got, a, e, n in zip((dx, dw, db), want, err, ("dx", "dw", "db")):
            L.within(got, a, e, n)
        # each alone: the same values
        dx2, clean = _guarded(rows, cols, pad, shift, dtype)
        ob.ob_layernorm_bwd(dy, x, mean, rstd, dx2, weight, dsum=dsum)
        clean()
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        ob.ob_layernorm_bwd(dy, x, mean, rstd, None, weight, dweight=dw2)
        ob.ob_layernorm_bwd(dy, x, mean, rstd, None, weight, dbias=db2)
        for a, b in ((dx, dx2), (dw, dw2), (db, db2)):
            assert torch.equal(a, b)


def test_layer_norm_of_nothing():
    z = torch.empty(0, 16, device="cuda")
    e = torch.empty(0, device="cuda")
    dw = torch.full((16,), 3.0, device="cuda")
    ob.ob_layernorm_fwd(z, z.clone(), mean=e, rstd=e)
    ob.ob_layernorm_bwd(z, z, e, e, z.clone(), dweight=dw)
    assert (dw == 0).all()
    z = torch.empty(16, 0, device="cuda")
    ob.ob_layernorm_fwd(z, z.clone())


def test_layer_norm_of_constant_far_and_special_rows():
    """A constant row has no variance; a far one keeps its digits (a difference of squares
    would not); what is not finite stays in its row."""
    for cols in (96, 1024, 1001, 5000):
        x = torch.randn(6, cols, device="cuda")
        x[1] = 3.0
        x[2] = 4096.0 + x[2] / 64
        x[3, 5] = math.inf
        x[4, 7] = math.nan
        y, mean, rstd = torch.empty_like(x), *(torch.empty(6, device="cuda") for _ in range(2))
        ob.ob_layernorm_fwd(x, y, mean=mean, rstd=rstd)
        fine = [0, 1, 2, 5]
        want, err, _, _ = L.layer_norm(x[fine], None, None, 1e-5)
        L.within(y[fine], want, err, "y")
        assert (y[1] == 0).all()
        assert y[3].isnan().any() and y[4].isnan().all()
        dx = torch.empty_like(x)
        ob.ob_layernorm_bwd(torch.ones_like(x), x, mean, rstd, dx)
        assert dx[fine].isfinite().all() and dx[4].isnan().all()


# ---------------------------------------------------------------------------
# The dense layer
# ---------------------------------------------------------------------------

DENSE = [(1, 1, 1), (1, 64, 64), (1, 1000, 333), (2, 40, 8), (3, 129, 257), (8, 512, 1024),
         (9, 300, 70), (16, 8, 16), (17, 256, 512), (33, 65, 1), (64, 1, 100), (100, 200, 300),
         (127, 128, 129), (128, 256, 64), (129, 257, 65), (250, 768, 96), (256, 256, 256),
         (257, 511, 513), (300, 64, 2000), (513, 1024, 320), (19500, 100, 1100), (1000, 136, 1000), (777, 1301, 1001),
         (1, 300, 5003), (5, 300, 2100), (16, 1000, 5003), (30, 264, 4104), (32, 40, 8195)]


def _dense_case(Mr, N, K, dtype, kn, pad, shift, seed=0):
    mk = _gen(Mr + 3 * N + 5 * K + seed)
    x = _slice(mk, Mr, K, pad, shift, dtype)
    w = _slice(mk, *((K, N) if kn else (N, K)), pad, shift, dtype, K ** -0.5)
    r = _slice(mk, Mr, N, pad, shift, dtype)
    return mk, x, w.t() if kn else w, mk(N, dtype=dtype), r


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Mr,N,K", DENSE)
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 1)])
def test_dense(dtype, Mr, N, K, kn, pad, shift):
    mk, x, w, b, r = _dense_case(Mr, N, K, dtype, kn, pad, shift)
    for act, bias, residual, keep in (("none", None, None, False), ("gelu", b, None, True),
                                      ("relu", None, r, True), ("gelu_tanh", b, r, False)):
        y, clean = _guarded(Mr, N, pad, shift, dtype)
        z, z_clean = _guarded(Mr, N, pad, shift, dtype)
        ob.ob_linear_fwd(x, w, y, bias, residual, z if keep else None, act)
        clean()
        z_clean()
        (z64, y64), (ez, ey) = L.dense(x, w, bias, residual, act)
        L.within(y, y64, ey, f"y of {act}")
        if keep:
            L.within(z, z64, ez, f"z of {act}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Mr,N,K", DENSE)
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 1)])
def test_dense_gradient(dtype, Mr, N, K, kn, pad, shift):
    mk, x, w, b, dy = _dense_case(Mr, N, K, dtype, kn, pad, shift, 1)
    z = _slice(mk, Mr, N, pad, shift, dtype, 1.5)
    for act in ("none", "gelu", "relu", "gelu_tanh"):
        dx, x_clean = _guarded(Mr, K, pad, shift, dtype)
        dw, w_clean = _guarded(*((K, N) if kn else (N, K)), pad, shift, dtype)
        db = torch.full((N,), 5.0, device="cuda", dtype=dtype)
        kw = dict(z=None if act == "none" else z, activation=act)
        ob.ob_linear_bwd(dy, x, w, dx, dw.t() if kn else dw, db, **kw)
        x_clean()
        w_clean()
        want, err = L.dense_grad(dy, x, w, z, act)
        for got, a, e, n in zip((dx, dw.t() if kn else dw, db), want, err, ("dx", "dw", "db")):
            L.within(got, a, e, f"{n} of {act}")
    # one alone: the same values
    dx2, dw2, db2 = torch.empty(Mr, K, device="cuda", dtype=dtype), torch.empty_like(w), torch.empty_like(db)
    ob.ob_linear_bwd(dy, x, w, dx=dx2, **kw)
    ob.ob_linear_bwd(dy, x, w, dw=dw2, **kw)
    ob.ob_linear_bwd(dy, x, w, dbias=db2, **kw)
    assert torch.equal(dx, dx2) and torch.equal(dw.t() if kn else dw, dw2) and torch.equal(db, db2)


# sizes that take pairs of blocks, whole and cut along the sum, forward or backward
LARGE = [(2560, 1024, 256), (2570, 1030, 1000), (2816, 2304, 4096), (9000, 1100, 1300), (5000, 2048, 136),
         (600, 5000, 2100)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Mr,N,K", LARGE)
@pytest.mark.parametrize("kn", [False, True])
def test_dense_of_large_sizes(dtype, Mr, N, K, kn):
    mk, x, w, b, r = _dense_case(Mr, N, K, dtype, kn, 0, 0, 3)
    y, clean = _guarded(Mr, N, 0, 0, dtype)
    z, z_clean = _guarded(Mr, N, 0, 0, dtype)
    ob.ob_linear_fwd(x, w, y, b, r, z, "gelu")
    clean()
    z_clean()
    (z64, y64), (ez, ey) = L.dense(x, w, b, r, "gelu")
    L.within(y, y64, ey, "y")
    L.within(z, z64, ez, "z")
    for got, want in ((y, y64), (z, z64)):
        assert (got.double() - want).norm() <= 1.02 * (want.to(dtype).double() - want).norm()
    dx, x_clean = _guarded(Mr, K, 0, 0, dtype)
    dw, w_clean = _guarded(*((K, N) if kn else (N, K)), 0, 0, dtype)
    dwt, db = dw.t() if kn else dw, torch.empty_like(b)
    ob.ob_linear_bwd(r, x, w, dx, dwt, db, z=z, activation="gelu")
    x_clean()
    w_clean()
    want, err = L.dense_grad(r, x, w, z, "gelu")
    for got, a, e, n in zip((dx, dwt, db), want, err, ("dx", "dw", "db")):
        L.within(got, a, e, n)
        once = (a.to(dtype).double() - a).norm()
        assert (got.double() - a).norm() <= math.sqrt(1 + 1.1 ** 2) * once, n


@pytest.mark.parametrize("Mr,N,K", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0), (130, 9, 0)])
def test_dense_of_nothing(Mr, N, K):
    x, w = torch.ones(Mr, K, device="cuda", dtype=BF16), torch.ones(N, K, device="cuda", dtype=BF16)
    b, r = torch.ones(N, device="cuda", dtype=BF16), torch.ones(Mr, N, device="cuda", dtype=BF16)
    y, z = torch.zeros(Mr, N, device="cuda", dtype=BF16), torch.zeros(Mr, N, device="cuda", dtype=BF16)
    ob.ob_linear_fwd(x, w, y, b, r, z, "relu")
    assert (y == 2).all() and (z == 1).all()
    dx, dw, db = torch.full_like(x, 9), torch.full_like(w, 9), torch.full_like(b, 9)
    ob.ob_linear_bwd(r, x, w, dx, dw, db, z=z, activation="relu")
    assert (dx == N).all() and (dw == Mr).all() and (db == Mr).all()


@pytest.mark.parametrize("Mr,N,K", [(1, 2048, 4096), (640, 768, 2048), (2048, 1024, 1024)])
def test_dense_is_as_near_as_one_rounding(Mr, N, K):
    """By norm: y is the exact one rounded once, a gradient the exact one rounded once of
    operands that were rounded once (1.1 times: the rounding's spread over a binade)."""
    for dtype in (BF16, F16):
        mk, x, w, b, dy = _dense_case(Mr, N, K, dtype, False, 0, 0, 2)
        y, z = (torch.empty(Mr, N, device="cuda", dtype=dtype) for _ in range(2))
        ob.ob_linear_fwd(x, w, y, b, None, z, "gelu")
        (z64, y64), _ = L.dense(x, w, b, None, "gelu")
        for got, want in ((y, y64), (z, z64)):
            assert (got.double() - want).norm() <= 1.02 * (want.to(dtype).double() - want).norm()
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        ob.ob_linear_bwd(dy, x, w, dx, dw, db, z=z, activation="gelu")
        want, _ = L.dense_grad(dy, x, w, z, "gelu")
        for got, a in zip((dx, dw, db), want):
            once = (a.to(dtype).double() - a).norm()
            assert (got.double() - a).norm() <= math.sqrt(1 + 1.1 ** 2) * once


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

TYPES = {F32: np.float32, BF16: None, F16: np.float16}


def _adam_tensors(mk, sizes, p_type, g_type, shift):
    ps, gs = [], []
    for i, n in enumerate(sizes):
        whole = torch.full((n + shift + 8,), 7.0, device="cuda", dtype=p_type)
        whole[shift:shift + n] = mk(n).mul(0.1).to(p_type)
        ps.append((whole, whole[shift:shift + n]))
        g = torch.zeros(n + shift, device="cuda", dtype=g_type)
        g[shift:] = (mk(n) * 10.0 ** (-(i % 5))).to(g_type)
        gs.append(g[shift:])
    return ps, gs


def _padded(x, blocks):
    out = np.zeros(blocks * 256, np.float32)
    out[:x.numel()] = x.float().cpu().numpy()
    return out


SIZES = [1, 255, 256, 257, 2048, 5, 1000, 0, 4096, 777, 8, 3000]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("p_type", [F32, BF16, F16])
@pytest.mark.parametrize("g_type", [F32, BF16, F16])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_adamw(bits, p_type, g_type, shift):
    """Three steps: m and v bit by bit, p within its roundings."""
    mk = _gen(bits + shift)
    ps, gs = _adam_tensors(mk, SIZES, p_type, g_type, shift)
    copies = [torch.zeros(n, device="cuda", dtype=BF16) if i % 2 else None for i, n in enumerate(SIZES)]
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    seed, lr, (b1, b2), eps = 0xABCDEF0123456789, 1e-2, (0.9, 0.99), 1e-8
    opt = ob.AdamW([p for _, p in ps], lr=lr, betas=(b1, b2), eps=eps, weight_decay=decay, seed=seed,
                   state_bits=bits, copies=copies)
    scale = torch.tensor([0.5], device="cuda")
    blocks = [-(-n // 256) for n in SIZES]
    first = np.cumsum([0] + blocks)
    kind = np.uint8 if bits == 8 else np.float32
    state = [[np.zeros(k * 256, kind), np.zeros(k * 256, kind), np.zeros(k, np.uint8), np.zeros(k, np.uint8)]
             for k in blocks]
    for step in range(1, 4):
        before = [p.clone() for _, p in ps]
        skipped = 3 if step == 2 else None  # no gradient: nothing of it changes
        grads = [None if i == skipped else g * step for i, g in enumerate(gs)]
        opt.step(grads, grad_scale=scale)
        for i, n in enumerate(SIZES):
            whole, p = ps[i]
            assert (whole[:shift] == 7.0).all() and (whole[shift + n:] == 7.0).all()
            at, end = first[i] * 256, first[i + 1] * 256
            got = [opt.m[at:end], opt.v[at:end]]
            if bits == 8:
                got += [opt.m_exp[first[i]:first[i + 1]], opt.v_exp[first[i]:first[i + 1]]]
            if i != skipped and n:
                m, v, me, ve = state[i]
                q, size, new = L.adamw(_padded(before[i], blocks[i]), _padded(grads[i], blocks[i]), m, v,
                                       step, seed, int(at), lr, b1, b2, eps, decay[i], 0.5, bits, me, ve)
                state[i][:len(new)] = new
                # the update: a square root, a product, a sum, a quotient, each a few ulp
                err = torch.from_numpy(size[:n]).cuda() * 2.0 ** -20
                want = torch.from_numpy(q[:n]).cuda()
                err += 3 * L.U32 * (want.abs() + before[i].double().abs())
                L.within(p, want, err, f"p of {i} at step {step}")
                if copies[i] is not None:
                    L.within(copies[i], want, err, f"copy of {i} at step {step}")
            elif n:
                assert torch.equal(p, before[i])
            for a, b, name in zip(got, state[i], ("m", "v", "m_exp", "v_exp")):
                assert np.array_equal(a.cpu().numpy().view(np.uint8), np.asarray(b).view(np.uint8)), (i, step, name)
    if bits == 8:
        mv = opt.moments()
        for got, k, bias in zip(mv, (0, 1), (7, 23)):
            want = np.concatenate([L.decode(s[k], s[k + 2], bias) for s in state])
            assert torch.equal(got.float().cpu(), torch.from_numpy(want))
    assert opt.state()["step"] == 3


def _codes(opt):
    return [t for t in (opt.m, opt.v, opt.m_exp, opt.v_exp) if t is not None]


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_with_values_that_are_not_finite_or_tiny(bits):
    """They stay with their element: the block's others go on; units at both ends."""
    n = 256 * 6
    g = torch.randn(n, device="cuda")
    g[3], g[300], g[301] = math.nan, math.inf, -math.inf
    g[512:768] = 0.0
    g[768:1024] *= 1e-30
    g[1024:1280] *= 1e18
    p = torch.zeros(n, device="cuda")
    opt = ob.AdamW([p], lr=1e-2, weight_decay=0.0, state_bits=bits, seed=3)
    z = np.zeros(n, np.uint8 if bits == 8 else np.float32)
    state = [z, z, np.zeros(6, np.uint8), np.zeros(6, np.uint8)]
    for step in (1, 2):
        q, size, new = L.adamw(p.cpu().numpy(), g.cpu().numpy(), state[0], state[1], step, 3, 0, 1e-2, 0.9,
                               0.999, 1e-8, 0.0, 1.0, bits, state[2], state[3])
        state[:len(new)] = new
        opt.step([g])
        bad = np.isin(np.arange(n), (3, 300, 301))
        got = p.cpu().numpy()
        assert np.isnan(got[bad]).all()
        lim = 2.0 ** -20 * size + 4 * L.U32 * np.abs(q)
        assert (np.abs(got - q) <= lim)[~bad].all()
        for a, b in zip(_codes(opt), state):
            a = a.cpu().numpy()
            if bits == 8:
                if len(a) == n:  # the sign of a NaN is free
                    a, b = np.where(bad, a & 127, a), np.where(bad, b & 127, b)
                assert np.array_equal(a, b)
            else:
                assert np.array_equal(np.where(bad, 0, a), np.where(bad, 0, b))


def test_adamw_rounding_is_even_handed():
    """8 bits: a value between two codes takes the upper one as often as its place says (five
    deviations of the binomial's), and v falls under gradients of zero."""
    n = 1 << 20
    g = torch.full((n,), 1.07, device="cuda")
    g[::256] = 1.5  # the unit of every block
    opt = ob.AdamW([torch.zeros(n, device="cuda")], betas=(0.0, 0.0), state_bits=8, seed=11)
    opt.step([g])
    m, v = (t.float().view(-1, 256)[:, 1:].double() for t in opt.moments())
    for got, x in ((m, float(g[1])), (v, float(g[1]) ** 2)):
        lo, hi = got.min().item(), got.max().item()
        assert lo < x < hi and ((got == lo) | (got == hi)).all()
        place = (x - lo) / (hi - lo)
        share = (got == hi).double().mean().item()
        assert abs(share - place) <= 5 * math.sqrt(place * (1 - place) / got.numel()) + 2.0 ** -16
    opt = ob.AdamW([torch.zeros(n, device="cuda")], betas=(0.9, 0.999), state_bits=8, seed=12)
    opt.step([g])
    before = opt.moments()[1].double().mean()
    for _ in range(100):
        opt.step([torch.zeros_like(g)])
    after = opt.moments()[1].double().mean()
    # each code's step is at most 1/8 of its value: 100 steps' deviations, five times
    assert abs(after / before - 0.999 ** 100) <= 5 * 0.125 * math.sqrt(100 / n) + 1e-4


def test_adamw_skip_and_device_rate():
    mk = _gen(9)
    g = mk(1000)
    runs = []
    for device_lr in (False, True):
        p = mk(1000) * 0 + 1
        opt = ob.AdamW([p], lr=0.25, state_bits=8, seed=1)
        lr = torch.tensor([0.25], device="cuda") if device_lr else None
        opt.step([g], lr=lr)
        kept = [t.clone() for t in [p, *_codes(opt), opt.counter]]
        opt.step([g], lr=lr, skip=torch.ones(1, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(kept, [p, *_codes(opt), opt.counter]))
        opt.step([g], lr=lr, skip=torch.zeros(1, device="cuda"))
        assert opt.state()["step"] == 2
        runs.append(p)
    assert torch.equal(*runs)


def test_adamw_of_many_tensors():
    """More than one launch holds; the same bits as one after another."""
    mk = _gen(4)
    sizes = [(i * 37) % 700 for i in range(1100)]
    ps, gs = [mk(n) for n in sizes], [mk(n) for n in sizes]
    whole = [p.clone() for p in ps]
    opt = ob.AdamW(whole, lr=1e-2)
    opt.step(gs)
    opt.step(gs)
    for k in (0, 1, 18, 19, 511, 512, 513, 1023, 1024, 1025, 1099):
        p = ps[k].clone()
        one = ob.AdamW([p], lr=1e-2)
        one.step([gs[k]])
        one.step([gs[k]])
        assert torch.equal(p, whole[k])
    assert opt.state()["step"] == 2


def test_adamw_state_goes_on_and_graphs_step():
    """A state handed over continues bit for bit; replays of a captured step are further steps."""
    mk = _gen(6)
    g = [mk(3000, dtype=BF16), mk(70, dtype=BF16)]
    for bits in (8, 32):
        def make(state=None, ps=None):
            ps = ps or [torch.ones(3000, device="cuda"), torch.ones(70, device="cuda")]
            return ps, ob.AdamW(ps, lr=1e-2, state_bits=bits, seed=5, state=state)
        ps, a = make()
        for _ in range(5):
            a.step(g)
        qs, b = make()
        b.step(g)
        b.step(g)
        _, b = make(b.state(), qs)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.step(g)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert b.state()["step"] == 5
        assert all(torch.equal(x, y) for x, y in zip(ps, qs))
        for x, y in zip(_codes(a), _codes(b)):
            assert torch.equal(x, y)
        # powers of b1 and b2 by products: five roundings of 2^-53
        assert torch.allclose(a.counter, b.counter, rtol=1e-15, atol=0)


def test_adamw_of_a_late_state_and_of_replaced_memory():
    """A state of some steps goes on with the counter's own bits; a parameter that got other
    memory keeps it, and the step goes to the memory it was made with."""
    g = [_gen(8)(700, dtype=BF16)]
    ps, qs = [torch.ones(700, device="cuda")], [torch.ones(700, device="cuda")]
    a, b = ob.AdamW(ps, lr=1e-2), ob.AdamW(qs, lr=1e-2)
    for t in range(50):
        if t == 43:
            b = ob.AdamW(qs, lr=1e-2, state=b.state())
        a.step(g)
        b.step(g)
    assert torch.equal(a.counter, b.counter) and torch.equal(ps[0], qs[0])
    old, new = qs[0].detach(), torch.full((700,), 3.0, device="cuda")
    at = old.data_ptr()
    qs[0].data = new
    del old
    a.step(g)
    b.step(g)
    assert b._kept[0].data_ptr() == at and torch.equal(b._kept[0], ps[0])
    assert (qs[0] == 3.0).all()


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------

def _pass(seed, dtype=BF16, rows=520, d=320, f=768):
    """(inputs, a function that runs layer norm and a dense layer both ways, into new tensors)"""
    mk = _gen(seed)
    x, r, ds, w1, b1 = mk(rows, d, dtype=dtype), mk(rows, d, dtype=dtype), mk(rows, d, dtype=dtype), mk(d), mk(d)
    w, b, dy = mk(f, d, dtype=dtype), mk(f, dtype=dtype), mk(rows, f, dtype=dtype)
    E = lambda *s, dt=dtype: torch.empty(*s, device="cuda", dtype=dt)
    h, s, mean, rstd = E(rows, d), E(rows, d), E(rows, dt=F32), E(rows, dt=F32)
    y, z, dh, dw, db = E(rows, f), E(rows, f), E(rows, d), E(f, d), E(f)
    dx, dw1, db1 = E(rows, d), E(d, dt=F32), E(d, dt=F32)

    def run(stream=None):
        kw = dict(stream=stream)
        ob.ob_layernorm_fwd(x, h, w1, b1, 1e-5, r, s, mean, rstd, **kw)
        ob.ob_linear_fwd(h, w, y, b, None, z, "gelu", **kw)
        ob.ob_linear_bwd(dy, h, w, dh, dw, db, z, "gelu", **kw)
        ob.ob_layernorm_bwd(dh, s, mean, rstd, dx, w1, dw1, db1, ds, **kw)
        return (y, z, s, dw, db, dx, dw1, db1)
    return run


@pytest.mark.parametrize("handle", [False, True])
def test_layers_on_two_streams(handle):
    """In turn on two streams and without waiting: the same bits as one after another."""
    runs = [_pass(1), _pass(2, rows=3000)]
    want = []
    for r in runs:
        want.append([t.clone() for t in r()])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = [runs[0](), runs[1](side.cuda_stream if handle else side)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_layers_in_a_graph():
    """Captured and replayed on new inputs: the same bits as called."""
    mk = _gen(31)
    x, w1 = mk(300, 256, dtype=BF16), mk(256, dtype=BF16)
    up, down = mk(512, 256, dtype=BF16), mk(256, 512, dtype=BF16)
    dy = mk(300, 256, dtype=BF16)

    def step(x):
        leaves = [t.detach().requires_grad_() for t in (x, w1, up, down)]
        y, s = M.layer_norm(leaves[0], leaves[1], residual=leaves[0], return_sum=True)
        h = M.linear(y, leaves[2], activation="gelu")
        out = M.linear(h, leaves[3], residual=s)
        return [out.detach(), *torch.autograd.grad(out, leaves, dy)]

    held = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    for k in range(3):
        held.copy_(mk(300, 256, dtype=BF16))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step(held)))


FIRST = """
import torch, momentum_compression_gb300 as ob
mk = lambda *s: torch.ones(*s, device="cuda", dtype=torch.bfloat16)
x, w, y, z, dx, dw, db = mk(300, 64), mk(96, 64), mk(300, 96), mk(300, 96), mk(300, 64), mk(96, 64), mk(96)
m, d, p = torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda"), torch.ones(500, device="cuda")
g, opt = torch.ones_like(p), ob.AdamW([p], state_bits=8)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ob.ob_layernorm_fwd(x, dx, mean=m, rstd=d)
    ob.ob_layernorm_bwd(x, x, m, d, dx, dweight=db[:64])
    ob.ob_linear_fwd(x, w, y, db, None, z, "gelu")
    ob.ob_linear_bwd(y, x, w, dx, dw, db, z, "gelu")
    opt.step([g])
graph.replay()
torch.cuda.synchronize()
assert (y[0, 95] - 65).abs() < 1 and ob.ob_layer_device_error() == 0
print("fine")
"""


@pytest.mark.parametrize("kn", [False, True])
def test_few_rows_in_a_graph_and_on_two_streams(kn):
    """Products whose blocks share a sum: replays and calls side by side give the call's bits."""
    mk = _gen(12)
    x, w, b = mk(5, 4096, dtype=BF16), mk(4096, 1024, dtype=BF16), mk(1024, dtype=BF16)
    w = w if kn else w.t().contiguous().t()
    want = torch.empty(5, 1024, device="cuda", dtype=BF16)
    ob.ob_linear_fwd(x, w.t(), want, b, activation="gelu")
    y = [torch.zeros_like(want) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ob.ob_linear_fwd(x, w.t(), y[0], b, activation="gelu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        graph.replay()
        for s, out in zip(streams, y[1:]):
            ob.ob_linear_fwd(x, w.t(), out, b, activation="gelu", stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in y)
    assert ob.ob_layer_device_error() == 0


@pytest.mark.parametrize("what", ["dense", "attention"])
def test_first_call_of_a_thread(what):
    """A thread that has done nothing on the GPU yet, as autograd's."""
    import threading
    mk = _gen(12)
    x, w, y = mk(300, 64, dtype=BF16), mk(96, 64, dtype=BF16), torch.zeros(300, 96, device="cuda", dtype=BF16)
    q, o = mk(1, 70, 2, 64, dtype=BF16), torch.zeros(1, 70, 2, 64, device="cuda", dtype=BF16)
    call = (lambda out: ob.ob_linear_fwd(x, w, out)) if what == "dense" else \
        (lambda out: ob.ob_attn_fwd(q, q, q, out))
    out = y if what == "dense" else o
    got, errors = torch.zeros_like(out), []

    def body():
        try:
            call(got)
        except Exception as e:
            errors.append(e)
    t = threading.Thread(target=body)
    t.start()
    t.join()
    call(out)
    torch.cuda.synchronize()
    assert not errors and torch.equal(got, out)


def test_first_calls_are_in_a_capture():
    """A process whose first calls are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


def test_model_functions_are_the_entry_points():
    """Views that kernels cannot read are copied; without gradients nothing is kept."""
    mk = _gen(41)
    x, w, b = mk(6, 40, 2 * 96, dtype=BF16)[..., ::2], mk(96, 200, dtype=BF16), mk(200, dtype=BF16)
    assert torch.equal(M.linear(x, w.t(), b, "gelu"), M.linear(x.contiguous(), w.t().contiguous(), b, "gelu"))
    res = mk(6, 200, 40, dtype=BF16).transpose(1, 2)
    got = M.linear(x, w.t(), b, "relu", res)
    assert torch.equal(got, M.linear(x, w.t(), b, "relu", res.contiguous()))
    weight = mk(192)[::2]
    assert torch.equal(M.layer_norm(x, weight), M.layer_norm(x.contiguous(), weight.contiguous()))
    a, r = (mk(50, 96, dtype=BF16).requires_grad_() for _ in range(2))
    y, s = M.layer_norm(a, residual=r, return_sum=True)
    dy, ds = mk(50, 96, dtype=BF16), mk(50, 96, dtype=BF16)
    both = torch.autograd.grad((y, s), (a, r), (dy, ds), retain_graph=True)
    assert torch.equal(*both)
    only_y, = torch.autograd.grad(y, a, dy, retain_graph=True)
    only_s, = torch.autograd.grad(s, a, ds)
    assert torch.equal(only_s, ds)
    near = (both[0].double() - only_y.double() - ds.double()).abs()
    assert (near <= 2.0 ** -8 * (both[0].double().abs() + only_y.double().abs())).all()
    with pytest.raises(ValueError):
        M.layer_norm(a, return_sum=True)
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(M.layer_norm(a).sum(), a, create_graph=True)
        g.sum().backward()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

def _block(p, x, M_, exact):
    """A pre-norm feed-forward layer of a residual stream x (+ r): its output and the stream."""
    def ln(s, w, b):
        if not exact:
            return M.layer_norm(s, w, b)
        d = s - s.mean(-1, keepdim=True)
        return d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def lin(x, w, b, act="none", residual=None):
        if not exact:
            return M.linear(x, w, b, act, residual)
        y = L.act(x @ w.t() + b, act)[0]
        return y if residual is None else y + residual
    h = lin(ln(x, p["w1"], p["b1"]), p["up"], p["up_b"], "gelu")
    return lin(h, p["down"].t(), p["down_b"], residual=x)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_layer_and_its_step(bits):
    """Norm, two dense layers and AdamW as a model uses them: outputs, every gradient and the
    parameters after three steps near those of the same in 64 bits."""
    mk = _gen(77)
    d, f = 96, 200
    shapes = dict(w1=(d,), b1=(d,), up=(f, d), up_b=(f,), down=(f, d), down_b=(d,))
    master = {n: (torch.ones(s, device="cuda") if n == "w1" else mk(*s) * 0.1) for n, s in shapes.items()}
    work = {n: t.to(BF16) for n, t in master.items()}
    opt = ob.AdamW(list(master.values()), lr=1e-2, weight_decay=0.0, state_bits=bits,
                   copies=list(work.values()))
    exact = {n: t.double() for n, t in master.items()}
    m = {n: torch.zeros_like(t) for n, t in exact.items()}
    v = {n: torch.zeros_like(t) for n, t in exact.items()}
    for step in range(1, 4):
        x, dy = mk(7, 40, d, dtype=BF16), mk(7, 40, d, dtype=BF16)
        leaves = {n: t.detach().requires_grad_() for n, t in work.items()}
        xr = x.detach().requires_grad_()
        y = _block(leaves, xr, M, False)
        grads = torch.autograd.grad(y, [*leaves.values(), xr], dy)
        ref = {n: t.double().detach().requires_grad_() for n, t in work.items()}
        x64 = x.double().requires_grad_()
        y64 = _block(ref, x64, M, True)
        want = torch.autograd.grad(y64, [*ref.values(), x64], dy.double())
        # a few roundings to bf16 on the way of each, whose errors are independent
        near = lambda a, b: (a.double() - b).norm() / b.norm()
        assert near(y, y64) < 4 * 2.0 ** -9
        for n, a, b in zip([*leaves, "x"], grads, want):
            assert near(a, b) < 8 * 2.0 ** -9, n
        opt.step(list(grads[:-1]))
        for n, g in zip(leaves, grads):
            g = g.double()
            m[n] = 0.9 * m[n] + 0.1 * g
            v[n] = 0.999 * v[n] + 0.001 * g * g
            exact[n] = exact[n] - 1e-2 * (m[n] / (1 - 0.9 ** step)) / ((v[n] / (1 - 0.999 ** step)).sqrt() + 1e-8)
            # 8 bits: m and v were off by at most one code (1/8 of themselves) after each step
            lim = 1e-2 * (step if bits == 8 else 1e-4)
            assert (master[n].double() - exact[n]).abs().max() < lim, n
            assert torch.equal(work[n], master[n].to(BF16))

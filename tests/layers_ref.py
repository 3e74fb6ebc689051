"""Plain forms of layer norm, the dense layer and AdamW for the tests: layer norm
and the dense layer in 64 bits with elementwise error bounds, AdamW's moments bit
by bit in fp32.  CPU or CUDA torch tensors."""
import math

import numpy as np
import torch

import model_ref as R

U32 = 2.0 ** -24
BLOCK = 256


def _unit(t):
    return R.UNIT[t], R.TINY[t]


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

def row_sums(cols):
    """Relative error of a fp32 sum over a row, of the sum of magnitudes: at least 32 threads
    share a row, and their sums are joined in at most ten steps."""
    return (min(cols, -(-cols // 32) + 10) + 2) * U32


def layer_norm(x, weight, bias, eps):
    """(y, its bound but for the last rounding, mean, rstd) for rows x."""
    x = x.double()
    n, c = x.shape[1], row_sums(x.shape[1])
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    # the mean is off by em; that moves the variance by em^2 only in exact sums, and the
    # centred values, each rounded, by U32 of themselves
    em = c * x.abs().mean(1, keepdim=True) + U32 * mean.abs()
    evar = 2 * var.sqrt() * em + em * em + (c + 4 * U32) * var
    er = 0.5 * evar / (var + eps) + 4 * U32
    xhat = d * rstd
    y = xhat * w + b
    err = w.abs() * (rstd * em + xhat.abs() * (er + 4 * U32)) + U32 * (y.abs() + (xhat * w).abs())
    return y, err, mean[:, 0], rstd[:, 0]


def layer_norm_grad(dy, x, mean, rstd, weight, dsum):
    """dx, dw, db and their bounds (but for the last rounding), of fp32 mean and rstd."""
    rows, n = x.shape
    c = row_sums(n)
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    xhat = (x - mean) * rstd
    ex = 3 * U32 * xhat.abs()
    h = dy * w
    m1, m2 = h.mean(1, keepdim=True), (h * xhat).mean(1, keepdim=True)
    e1 = (c + 2 * U32) * h.abs().mean(1, keepdim=True)
    e2 = (c + 6 * U32) * (h * xhat).abs().mean(1, keepdim=True)
    dx = rstd * (h - m1 - xhat * m2)
    mag = h.abs() + m1.abs() + (xhat * m2).abs()
    edx = rstd * (e1 + xhat.abs() * e2 + ex * m2.abs() + 5 * U32 * mag)
    if dsum is not None:
        dx = dx + dsum.double()
        edx = edx + 2 * U32 * (dx.abs() + dsum.double().abs())
    # down a column: no chain is longer than the rows, and with many rows at least 32 share them
    k = (min(rows, rows // 32 + 1300) + 6) * U32
    dw, edw = (dy * xhat).sum(0), k * (dy * xhat).abs().sum(0)
    db, edb = dy.sum(0), k * dy.abs().sum(0)
    return (dx, dw, db), (edx, edw, edb)


# ---------------------------------------------------------------------------
# The dense layer
# ---------------------------------------------------------------------------

# |act''| and the error of act and act' in fp32 (CUDA's erf, exp and tanh: 2 ulp each)
CURVE = {"none": 0.0, "relu": 0.0, "gelu": 0.8, "gelu_tanh": 0.9}
EACT = 2.0 ** -20


def act(z, name):
    """act(z), act'(z) of doubles."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * (-0.5 * z * z).exp() / math.sqrt(2 * math.pi)
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)


def product(a, b):
    """a b and the bound of a product accumulated in fp32 in any order, cut or rounded."""
    a, b = a.double(), b.double()
    return a @ b, (a.shape[1] + 4) * 2 * U32 * (a.abs() @ b.abs())


def dense(x, w, bias, residual, name):
    """(z, y) and their bounds but for the last rounding."""
    z, e = product(x, w.t())
    if bias is not None:
        z = z + bias.double()
        e = e + U32 * z.abs()
    y, _ = act(z, name)
    ey = 1.2 * e + EACT * z.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + U32 * (y.abs() + residual.double().abs())
    return (z, y), (e, ey)


def dense_grad(dy, x, w, z, name):
    """dx, dw, db and their bounds but for the last rounding, of the z that is stored."""
    t = dy.dtype
    u, tiny = _unit(t)
    dy = dy.double()
    dz, e = dy, torch.zeros_like(dy)
    if name != "none":
        dz = dy * act(z.double(), name)[1]
        if name != "relu":
            e = dy.abs() * EACT * (1 + z.double().abs()) + U32 * dz.abs()
    k = (min(dy.shape[0], dy.shape[0] // 32 + 1300) + 4) * U32
    db, edb = dz.sum(0), e.sum(0) + k * dz.abs().sum(0)
    if name != "none":  # as an operand
        e = e + u * (dz.abs() + e) + tiny
    x, w = x.double(), w.double()
    (dx, edx), (dw, edw) = product(dz, w), product(dz.t(), x)
    return (dx, dw, db), (edx + e @ w.abs(), edw + e.t() @ x.abs(), edb)


def within(got, want, err, name, t=None):
    """|got - want| <= err plus one rounding to got's type."""
    t = got.dtype if t is None else t
    u, tiny = _unit(t)
    top = torch.finfo(t).max
    lim = err + u * (want.abs() + err) + tiny
    got = got.double()
    over = want.abs() + lim > top  # may have become infinite
    bad = ((got - want).abs() > lim) & ~(over & got.isinf())
    bad |= got.isnan()
    assert not bad.any(), (name, int(bad.sum()), ((got - want).abs() / lim).nan_to_num(1e9).max().item())


# ---------------------------------------------------------------------------
# AdamW: moments bit by bit, in numpy's fp32
# ---------------------------------------------------------------------------

F = np.float32


def decode(codes, exp, bias):
    """fp32 values of codes [n] with units of exp [n / 256]."""
    k = codes.astype(np.int64)
    size = k & 127 if bias == 7 else k
    e, f = size >> 3, size & 7
    v = np.where(e > 0, np.ldexp(8.0 + f, e - bias - 3), np.ldexp(f.astype(float), -bias - 2))
    v = np.where((k > 127) & (bias == 7), -v, v)
    unit = np.where(exp > 0, np.ldexp(1.0, exp.astype(np.int64) - 127), 0.0)
    out = (v.reshape(-1, BLOCK) * unit[:, None]).reshape(-1)
    out[size == (127 if bias == 7 else 255)] = np.nan
    return out.astype(F)


def encode(x, noise, bias):
    """(codes, exp) of fp32 x [n] by the definition, one block at a time, in doubles and whole numbers."""
    n = len(x)
    codes, exps = np.zeros(n, np.uint8), np.zeros(n // BLOCK, np.uint8)
    top_code, least = (126, 1) if bias == 7 else (254, 3)
    for b in range(n // BLOCK):
        s = slice(b * BLOCK, (b + 1) * BLOCK)
        a = np.abs(x[s].astype(np.float64))
        fine = np.isfinite(a)
        top = a[fine].max(initial=0.0)
        if top > 0:
            f, e = math.frexp(top)  # top = 2 f 2^(e - 1)
            biased = max(e - 1 + 127, 0)
            exps[b] = min(max(biased - 8 + (2 * f > 1.75 and biased > 0), least), 246)
        y = np.where(fine, a, 0.0) * (2.0 ** (127 - int(exps[b])) if exps[b] else 0.0)
        f, e = np.frexp(np.where(y > 0, y, 2.0 ** -200))
        q = np.maximum(e - 1, 1 - bias) - 3  # log2 of the codes' step at y
        k = np.ldexp(y, -q)                  # in steps
        k = np.floor(np.floor(np.ldexp(k, 16)) / 65536 + noise[s] / 65536).astype(np.int64)
        c = k + ((q + 3 + bias - 1) << 3)    # a step up from 15 is the next binade's first code
        c = np.minimum(c, top_code)
        if bias == 23:
            c = np.where(a > 0, np.maximum(c, 1), c)
        c = np.where(fine, c, top_code + 1)
        if bias == 7:
            c = c + 128 * np.signbit(x[s])
        codes[s] = c
    return codes, exps


def adamw(p, g, m, v, step, seed, first, lr, b1, b2, eps, decay, scale=1.0, bits=32, m_exp=None,
          v_exp=None):
    """One tensor's step (fp32 numpy arrays of whole blocks; `first`: its first element in the
    state).  Returns p in 64 bits, the update's magnitude, and the new state."""
    g = (g.astype(F) * F(scale)).astype(F)
    with np.errstate(all="ignore"):
        if bits == 8:
            m, v = decode(m, m_exp, 7), decode(v, v_exp, 23)
        m = (m * F(b1)) + (g * F(1 - b1))
        v = (v * F(b2)) + ((g * F(1 - b2)) * g)
        assert m.dtype == F and v.dtype == F
        den = np.sqrt(v.astype(np.float64)) / math.sqrt(1 - b2 ** step) + eps
        update = lr / (1 - b1 ** step) * m.astype(np.float64) / den
        q = p.astype(np.float64) * (1 - lr * decay) - update
    if bits == 32:
        return q, np.abs(update), (m, v)
    i = np.arange(first, first + len(g))
    words = R.philox(np.arange(first // 4, (first + len(g)) // 4), seed, step)[np.arange(len(g)) // 4, i % 4]
    mo, me = encode(m, (words & np.uint64(0xFFFF)).astype(np.int64), 7)
    vo, ve = encode(v, (words >> np.uint64(16)).astype(np.int64), 23)
    return q, np.abs(update), (mo, vo, me, ve)

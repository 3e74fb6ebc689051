"""Workloads of three more operators of a training step: layer norm, the matrix
product of a dense layer with bias, activation and residual in its epilogue,
and the AdamW step over many tensors at once with moments in 32 or 8 bits.

Each workload has a plain form in elementary torch operations (32 bits,
rounded once at the end) and the call a user of the library makes.

The formulas
------------
Layer norm, over the last dimension, with s = x + residual (rounded to the type):
    y = (s - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
    xhat = (s - mean) rstd,  h = dy w
    ds = rstd (h - mean(h) - xhat mean(h xhat)) + dsum
    dw = sum over rows of dy xhat,  db = sum over rows of dy
dsum is the gradient of s itself, where a program uses it (a pre-norm layer).
Dense layer, x [M, K] and w [N, K]:
    z = x w^T + b,  y = act(z) + residual
    dz = dy act'(z),  dx = dz w,  dw = dz^T x,  db = sum over rows of dz
AdamW at step t, with a decay of each tensor's own and g scaled by a device scalar:
    m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g
    p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
m and v are rounded after each of their operations.  In 8 bits they are held in
blocks of 256 elements of a tensor, each with a power of two as its unit: one
byte E a block, unit 2^(E - 127), 0 for a block of zeros.  With `a` the block's
largest finite value, E = (a's biased exponent) - 8, plus 1 if a's significand
is over 1.75, at least 1 (v: 3), at most 246.  In that unit m is a float of 1 + 4 + 3 bits
(sign, exponent with bias 7, significand; 127 = not a number) and v one of
5 + 3 bits (exponent with bias 23; 255 = not a number).  A value between two
codes takes the upper one with the probability of its place between them: the
value's bits plus 16 random ones, cut off.  Those are the low (m) and high (v)
half of word i % 4 of Philox4x32-10 at counter (i / 4, t) under the key `seed`, i the
element's place in the state.  A positive v takes no code below the smallest.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MASK = 0xFFFFFFFF
BLOCK = 256
LN_EPS = 1e-5
LR, B1, B2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.01


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of the GPT-1.3B configuration between two layers: latency
        dict(name="ln_token", op="layernorm", rows=1, cols=2048, pad=0, dtype="bf16", w32=False,
             residual=True, train=False),
        # a BERT-large batch, 32 sequences of 512: the sum with the residual stream normalised,
        # forward and backward
        dict(name="ln_bert", op="layernorm", rows=16384, cols=1024, pad=0, dtype="bf16", w32=True,
             residual=True, train=True),
        # an odd slice of a wider buffer, rows that start at any alignment
        dict(name="ln_odd", op="layernorm", rows=4099, cols=1001, pad=7, dtype="f16", w32=False,
             residual=False, train=True),
        # 32 sequences of 2048 tokens of the GPT-1.3B configuration, forward and backward
        dict(name="ln_gpt", op="layernorm", rows=65536, cols=2048, pad=0, dtype="bf16", w32=False,
             residual=False, train=True),
        # one new token through the first product of a GPT-1.3B feed-forward layer: the
        # weights' way through the memory
        dict(name="dense_token", op="dense", M=1, N=8192, K=2048, pad=0, dtype="bf16", act="gelu",
             residual=False, train=False, kn=False),
        # the same layer's second product with the residual stream, 8 sequences of 2048, evaluation
        dict(name="dense_gpt", op="dense", M=16384, N=2048, K=8192, pad=0, dtype="bf16",
             act="none", residual=True, train=False, kn=False),
        # a training step of BERT-large's first feed-forward product, 32 sequences of 512
        dict(name="dense_bert", op="dense", M=16384, N=4096, K=1024, pad=0, dtype="bf16",
             act="gelu", residual=False, train=True, kn=False),
        # odd sizes: rows off every alignment, the weights stored [K, N]
        dict(name="dense_odd", op="dense", M=777, N=1301, K=1001, pad=3, dtype="f16",
             act="gelu_tanh", residual=True, train=True, kn=True),
        # the layer norms of the GPT-1.3B configuration, which stay uncompressed: 98 small
        # tensors, where the launch is all that counts
        dict(name="adamw_norms", op="adamw", layers=24, hidden=2048, vocab=0, norms=True, odd=0,
             p="f32", g="f32", copy=False, bits=32, shift=0, clip=False),
        # six layers of that configuration in 32 bits
        dict(name="adamw_gpt6", op="adamw", layers=6, hidden=2048, vocab=0, norms=False, odd=0,
             p="f32", g="f32", copy=False, bits=32, shift=0, clip=True),
        # all of it, bf16 gradients, moments in 8 bits, the bf16 copy that the next pass computes with
        dict(name="adamw8_gpt", op="adamw", layers=24, hidden=2048, vocab=50257, norms=False,
             odd=0, p="f32", g="bf16", copy=True, bits=8, shift=0, clip=True),
        # odd tensors that start one element off, 16-bit parameters
        dict(name="adamw8_odd", op="adamw", layers=3, hidden=1001, vocab=777, norms=False, odd=1,
             p="bf16", g="bf16", copy=False, bits=8, shift=1, clip=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layernorm", "dense", "dense", "adamw"])
    if op == "layernorm":
        cols = _log(rng, 16, 8192)
        return dict(op=op, rows=_log(rng, 1, min(65536, (1 << 27) // cols)), cols=cols,
                    pad=rng.choice([0, 0, 1, 8]), dtype=rng.choice(sorted(TYPES)),
                    w32=rng.random() < 0.5, residual=rng.random() < 0.5, train=rng.random() < 0.6)
    if op == "dense":
        c = dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 1, 8192), K=_log(rng, 1, 8192),
                 pad=rng.choice([0, 0, 1, 8]), dtype=rng.choice(["bf16", "f16"]),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh"]),
                 residual=rng.random() < 0.5, train=rng.random() < 0.6, kn=rng.random() < 0.4)
        if rng.random() < 0.5:  # a model's sizes: whole tiles
            c.update(N=-(-c["N"] // 64) * 64, K=-(-c["K"] // 64) * 64, pad=0)
        while c["M"] * c["N"] * c["K"] * (3 if c["train"] else 1) > 1 << 38:
            c["M"] = (c["M"] + 1) // 2
        return c
    return dict(op=op, layers=rng.randint(1, 6), hidden=_log(rng, 16, 2048),
                vocab=rng.choice([0, _log(rng, 1, 50257)]), norms=rng.random() < 0.2,
                odd=rng.choice([0, 1]), p=rng.choice(sorted(TYPES)), g=rng.choice(sorted(TYPES)),
                copy=rng.random() < 0.4, bits=rng.choice([8, 32]), shift=rng.choice([0, 0, 1]),
                clip=rng.random() < 0.5)


def _tensors(c):
    """(elements, whether it decays) of each tensor: a transformer's, or its layer norms alone."""
    h = c["hidden"]
    norm = [(h, False), (h, False)]
    t = [] if c["norms"] or not c["vocab"] else [(c["vocab"] * h, True)]
    for _ in range(c["layers"]):
        t += norm + norm
        if not c["norms"]:
            t += [(3 * h * h, True), (3 * h, False), (h * h, True), (h, False),
                  (4 * h * h, True), (4 * h, False), (4 * h * h, True), (h, False)]
    t += norm
    return [(max(1, n - c["odd"] * (i % 5)), decays) for i, (n, decays) in enumerate(t)]


def _places(c):
    """(first element of each tensor in the state, elements of the state)."""
    at, end = [], 0
    for n, _ in _tensors(c):
        at.append(end)
        end += -(-n // BLOCK) * BLOCK
    return at, end


def work(case):
    c = case
    if c["op"] == "layernorm":
        n, s, w = c["rows"] * c["cols"], TYPES[c["dtype"]].itemsize, c["cols"] * 4
        arrays = (4 if c["residual"] else 2) + ((4 if c["residual"] else 3) if c["train"] else 0)
        return {"bytes": n * s * arrays + w * 2, "flops": n * (22 if c["train"] else 8)}
    if c["op"] == "dense":
        M, N, K = c["M"], c["N"], c["K"]
        b = M * K + N * K + M * N * (2 if c["residual"] else 1) + N
        if c["train"]:
            b += M * N + M * K + N * K + N
        return {"bytes": 2 * b, "flops": 2 * M * N * K * (3 if c["train"] else 1)}
    n, p, g = sum(n for n, _ in _tensors(c)), TYPES[c["p"]].itemsize, TYPES[c["g"]].itemsize
    # in 8 bits the moments are read back as values too
    state = 16 if c["bits"] == 32 else 4 + 6
    return {"bytes": n * (2 * p + g + (2 if c["copy"] else 0) + state), "flops": n * 14}


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0, shift=0.0):
        x = torch.randn(*shape, generator=gen, device=DEV)
        return (x if scale == 1.0 and shift == 0.0 else x.mul_(scale).add_(shift)).to(dtype)

    st = {"case": c}
    if c["op"] == "layernorm":
        t, wide = TYPES[c["dtype"]], c["cols"] + c["pad"]
        wt = torch.float32 if c["w32"] else t

        def rows(**kw):  # a slice of rows of a wider buffer where pad > 0
            return normal(c["rows"], wide, dtype=t, **kw)[:, :c["cols"]]

        def empty():
            return torch.empty(c["rows"], c["cols"], device=DEV, dtype=t)

        st["x"] = rows(shift=0.5)
        st["residual"] = rows(scale=2.0) if c["residual"] else None
        st["w"], st["b"] = normal(c["cols"], dtype=wt, scale=0.2, shift=1.0), normal(c["cols"], dtype=wt)
        st["y"], st["sum"] = empty(), empty() if c["residual"] else None
        if c["train"]:
            st["dy"], st["dsum"] = rows(), rows() if c["residual"] else None
            st["dx"], st["dw"], st["db"] = empty(), torch.empty_like(st["w"]), torch.empty_like(st["b"])
            st["mean"], st["rstd"] = (torch.empty(c["rows"], device=DEV) for _ in range(2))
    elif c["op"] == "dense":
        t, (M, N, K, pad) = TYPES[c["dtype"]], (c[n] for n in ("M", "N", "K", "pad"))

        def rows(n):
            return normal(M, n + pad, dtype=t)[:, :n]

        st["x"] = rows(K)
        w = normal(*((K, N) if c["kn"] else (N, K)), dtype=t, scale=K ** -0.5)
        st["w"] = w.t() if c["kn"] else w
        st["b"] = normal(N, dtype=t)
        st["residual"] = rows(N) if c["residual"] else None
        st["y"], st["z"] = torch.empty(M, N, device=DEV, dtype=t), None
        if c["train"]:
            st["dy"] = rows(N)
            st["z"] = torch.empty_like(st["y"]) if c["act"] != "none" else None
            st["dx"], st["db"] = torch.empty(M, K, device=DEV, dtype=t), torch.empty_like(st["b"])
            dw = torch.empty_like(w)
            st["dw"] = dw.t() if c["kn"] else dw
    else:
        sizes, (at, total) = _tensors(c), _places(c)
        n = torch.tensor([k for k, _ in sizes], device=DEV)
        real = torch.zeros(total + 1, dtype=torch.int8, device=DEV)  # 1 on what the tensors cover
        first = torch.tensor(at, device=DEV)
        real[first] += 1
        real.index_add_(0, first + n, torch.full((len(at),), -1, dtype=torch.int8, device=DEV))
        real = real.cumsum(0)[:total].to(torch.uint8)

        def flat(dtype, scale):  # one buffer of all tensors, which are views of it
            whole = torch.zeros(total + c["shift"], device=DEV, dtype=dtype)
            whole[c["shift"]:] = normal(total, dtype=dtype, scale=scale) * real
            return whole[c["shift"]:]

        st["p"] = flat(TYPES[c["p"]], 0.02)
        # gradients of tensors and of elements differ in size by orders of magnitude
        size = torch.exp(2.0 * torch.randn(len(at), generator=gen, device=DEV) - 7.0)
        spans = torch.tensor(at[1:] + [total], device=DEV) - first
        st["g"] = flat(TYPES[c["g"]], 1.0)
        st["g"].mul_(torch.repeat_interleave(size, spans, output_size=total).to(st["g"].dtype))
        st["copy"] = torch.zeros(total, device=DEV, dtype=torch.bfloat16) if c["copy"] else None
        st["scale"] = torch.rand(1, generator=gen, device=DEV) if c["clip"] else None
        st["sizes"], st["at"], st["spans"] = sizes, at, spans
        st["decay"] = [DECAY if d else 0.0 for _, d in sizes]
        st["keep"] = torch.tensor([1 - LR * d for d in st["decay"]], device=DEV)
        st["seed"], st["step"] = 0x5851F42D00000000 + seed, 3 + seed % 1000
        if c["bits"] == 32:
            st["m"] = st["g"].float() * 0.3
            st["v"] = torch.square(st["g"].float()) * (0.1 + torch.rand(total, generator=gen, device=DEV))
        else:
            # as a step leaves them: codes of all sizes, units near the tensor's own
            st["m"] = torch.randint(0, 127, (total,), generator=gen, device=DEV, dtype=torch.uint8) * real
            st["m"] += 128 * torch.randint(0, 2, (total,), generator=gen, device=DEV, dtype=torch.uint8) * real
            st["v"] = torch.randint(208, 255, (total,), generator=gen, device=DEV, dtype=torch.uint8) * real
            unit = (127 + torch.log2(size).round() - 8)
            unit = torch.repeat_interleave(unit, spans // BLOCK, output_size=total // BLOCK)
            st["m_exp"] = unit.to(torch.uint8)
            st["v_exp"] = (2 * unit - 127 + 8).to(torch.uint8)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return _library(state) if own else _plain(state)


def _views(s, name):
    return [s[name][a:a + n] for a, (n, _) in zip(s["at"], s["sizes"])]


def _library(s):
    """The calls a user of the library makes."""
    import momentum_compression_gb300 as ob
    c = s["case"]
    if c["op"] == "layernorm":
        kw = dict(mean=s["mean"], rstd=s["rstd"]) if c["train"] else {}
        ob.ob_layernorm_fwd(s["x"], s["y"], weight=s["w"], bias=s["b"], eps=LN_EPS,
                            residual=s["residual"], sum=s["sum"], **kw)
        out = [s["y"]] + ([s["sum"]] if c["residual"] else [])
        if c["train"]:
            ob.ob_layernorm_bwd(s["dy"], s["sum"] if c["residual"] else s["x"], s["mean"],
                                s["rstd"], s["dx"], weight=s["w"], dweight=s["dw"], dbias=s["db"],
                                dsum=s["dsum"])
            out += [s["dx"], s["dw"], s["db"]]
        return out
    if c["op"] == "dense":
        ob.ob_linear_fwd(s["x"], s["w"], s["y"], bias=s["b"], residual=s["residual"], z=s["z"],
                         activation=c["act"])
        if not c["train"]:
            return [s["y"]]
        ob.ob_linear_bwd(s["dy"], s["x"], s["w"], dx=s["dx"], dw=s["dw"], dbias=s["db"], z=s["z"],
                         activation=c["act"])
        return [s["y"], s["dx"], s["dw"], s["db"]]
    if "opt" not in s:  # what a program makes once, with its parameters
        state = {n: s[n] for n in ("m", "v", "m_exp", "v_exp") if n in s}
        s["opt"] = ob.AdamW(_views(s, "p"), lr=LR, betas=(B1, B2), eps=EPS, weight_decay=s["decay"],
                            state_bits=c["bits"], seed=s["seed"], state=dict(state, step=s["step"]),
                            copies=_views(s, "copy") if c["copy"] else None)
        s["grads"] = _views(s, "g")
    s["opt"].step(s["grads"], grad_scale=s["scale"])
    return [s["p"], *s["opt"].moments()] + ([s["copy"]] if c["copy"] else [])


def _act(z, act):
    """(act(z), act'(z))"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z * (z > 0), (z > 0).to(z.dtype)
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _mulhilo(m, x):
    """High and low word of m * x for 32-bit words held in int64 (the product wraps, its bits hold)."""
    t = m * x
    return (t >> 32) & MASK, t & MASK


def _words(n, seed, step):
    """The random words of elements 0..n-1 at a step; n a multiple of 4."""
    call = torch.arange(n // 4, device=DEV, dtype=torch.int64)
    c = [call & MASK, call >> 32, torch.full_like(call, step & MASK), torch.full_like(call, step >> 32)]
    del call
    k0, k1 = seed & MASK, seed >> 32
    for _ in range(10):  # the generator's ten rounds
        h0, l0 = _mulhilo(0xD2511F53, c[0])
        h1, l1 = _mulhilo(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return torch.stack(c, 1).reshape(-1)


def _unpack(codes, exp, bias):
    """The values of codes: exponent fields with `bias`, 3 bits of significand, of m (bias 7) signed."""
    k = torch.arange(256, device=DEV)
    size = k & 127 if bias == 7 else k
    e, f = size >> 3, (size & 7).float()
    binade = ((e + (124 - bias)) << 23).int().view(torch.float32)  # 2^(e - bias - 3)
    value = torch.where(e > 0, (8 + f) * binade, f * math.ldexp(1.0, -bias - 2))
    value = torch.where(size == (127 if bias == 7 else 255), math.nan, value)
    value = torch.where((k > 127) & (bias == 7), -value, value)
    return (value[codes.int()].view(-1, BLOCK) * _unit(exp)).view(-1)


def _unit(exp):
    return (exp.int() << 23).view(torch.float32)[:, None]


def _pack(x, noise, bias):
    """(codes, units) of x, rounded by the 16 random bits of each element."""
    blocks = x.view(-1, BLOCK)
    size = blocks.abs()
    top = torch.where(size < math.inf, size, 0).amax(1).view(torch.int32)
    e = (top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000).int()
    exp = torch.where(top > 0, e.clamp(min=1 if bias == 7 else 3, max=246), 0)
    y = size * torch.where(exp > 0, (254 - exp) << 23, 0).view(torch.float32)[:, None]
    bits = y.view(torch.int32)
    noise = noise.view(-1, BLOCK)
    code = ((bits + (noise << 4)) >> 20) - ((127 - bias) << 3)
    low = ((y * 2.0 ** (18 + bias)).int() + noise) >> 16
    code = torch.where(y < 2.0 ** (1 - bias), low, code)
    code = code.clamp(max=126 if bias == 7 else 254)
    if bias == 7:
        code = torch.where(size < math.inf, code, 127) + 128 * torch.signbit(blocks)
    else:
        code = torch.maximum(code, (size > 0).int())
        code = torch.where(size < math.inf, code, 255)
    return code.to(torch.uint8).view(-1), exp.to(torch.uint8)


def _plain(s):
    c = s["case"]
    if c["op"] == "layernorm":
        x, t = s["x"].float(), s["x"].dtype
        if c["residual"]:
            x = (x + s["residual"].float()).to(t)
        out = [x] if c["residual"] else []
        x = x.float()
        w, b = s["w"].float(), s["b"].float()
        mean = x.mean(1, keepdim=True)
        xhat = x - mean
        rstd = 1 / torch.sqrt(xhat.square().mean(1, keepdim=True) + LN_EPS)
        xhat = xhat * rstd
        out = [(xhat * w + b).to(t)] + out
        if c["train"]:
            dy = s["dy"].float()
            h = dy * w
            dx = rstd * (h - h.mean(1, keepdim=True) - xhat * (h * xhat).mean(1, keepdim=True))
            if c["residual"]:
                dx = dx + s["dsum"].float()
            out += [dx.to(t), (dy * xhat).sum(0).to(s["w"].dtype), dy.sum(0).to(s["w"].dtype)]
        return out
    if c["op"] == "dense":
        t, x, w = s["x"].dtype, s["x"].float(), s["w"].float()
        y, slope = _act(x @ w.t() + s["b"].float(), c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        if not c["train"]:
            return [y.to(t)]
        dz = s["dy"].float() * slope
        dw = dz.t() @ x
        return [y.to(t), (dz @ w).to(t), dw.to(t), dz.sum(0).to(t)]

    g = s["g"].float()
    if c["clip"]:
        g = g * s["scale"]
    s["step"] += 1
    t, total = s["step"], g.numel()
    eight = c["bits"] == 8
    m = _unpack(s["m"], s["m_exp"], 7) if eight else s["m"]
    v = _unpack(s["v"], s["v_exp"], 23) if eight else s["v"]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * (1 - B2) * g
    del g
    if eight:
        words = _words(total, s["seed"], t)
        s["m"], s["m_exp"] = _pack(m, (words & 0xFFFF).int(), 7)
        s["v"], s["v_exp"] = _pack(v, (words >> 16).int(), 23)
        del words
    else:
        s["m"], s["v"] = m, v
    p = s["p"].float()
    p = p * torch.repeat_interleave(s["keep"], s["spans"], output_size=total)
    p -= LR / (1 - B1 ** t) * m / (torch.sqrt(v) * (1 - B2 ** t) ** -0.5 + EPS)
    del m, v
    s["p"].copy_(p)
    out = [s["p"], s["m"], s["v"]]
    if eight:
        out[1] = _unpack(s["m"], s["m_exp"], 7).to(torch.bfloat16)
        out[2] = _unpack(s["v"], s["v_exp"], 23).to(torch.bfloat16)
    if c["copy"]:
        s["copy"].copy_(p)
        out.append(s["copy"])
    return out


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _words64(first, count, seed, step):
    """The random words of elements first .. first + count - 1 (both multiples of 4); products by 16-bit limbs."""
    e = torch.arange(first // 4, (first + count) // 4, device=DEV)
    x = torch.empty(4, count // 4, device=DEV, dtype=torch.int64)
    x[0], x[1], x[2], x[3] = e % 2**32, e // 2**32, step % 2**32, step // 2**32

    def product(m, a):
        low, high = a % 65536 * m, a // 65536 * m       # a m = low + 65536 high, each < 2**48
        mid = low // 65536 + high
        return mid // 65536, mid % 65536 * 65536 + low % 65536

    for r in range(10):
        key = [(seed + r * 0x9E3779B9) % 2**32, (seed // 2**32 + r * 0xBB67AE85) % 2**32]
        (a, b), (y, z) = product(0xD2511F53, x[0]), product(0xCD9E8D57, x[2])
        x = torch.stack([y ^ x[1] ^ key[0], z, a ^ x[3] ^ key[1], b])
    return x.t().reshape(-1)


def _value64(code, exp, least):
    """Values of codes (sign, exponent, significand from a whole number), `least` the exponent of code 8."""
    e, f = code // 8, (code % 8).double()
    size = torch.where(e > 0, torch.ldexp(1 + f / 8, e - 1 + least), torch.ldexp(f / 8, e + least))
    return torch.ldexp(size.view(-1, BLOCK), exp.long()[:, None] - 127).view(-1)


def _rounded64(x, u, least, lowest):
    """x in 8 bits: multiples of the step of its own binade in its block's unit, u of a step added, cut off."""
    a = x.abs().view(-1, BLOCK)
    top = a.amax(1, keepdim=True)
    f, e = torch.frexp(top)                             # top = f 2^e, f in [0.5, 1)
    unit = (e - 1 - 8 + (f > 0.875).int()).clamp(min=lowest - 127)
    y = torch.ldexp(a, -unit)
    step = torch.frexp(y)[1].clamp(min=least + 1) - 4
    k = torch.floor(torch.ldexp(y, -step) + u.view(-1, BLOCK))
    if lowest == 3:
        k = torch.maximum(k, (y > 0).double())
    size = torch.ldexp(torch.ldexp(k, step).clamp(max=448.0), unit)
    return (torch.sign(x).view(-1, BLOCK) * size).view(-1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "layernorm":
        x = s["x"].double()
        if c["residual"]:
            x = x + s["residual"].double()
        total = [x] if c["residual"] else []
        if c["residual"]:  # what follows is of the sum as it is kept
            x = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
        n, w, b = c["cols"], s["w"].double(), s["b"].double()
        centred = x - x.sum(1, True) / n
        sigma = torch.sqrt((centred * centred).sum(1, True) / n + LN_EPS)
        out = [centred / sigma * w + b] + total
        if c["train"]:
            dy, q = s["dy"].double(), centred / sigma
            h = dy * w
            ds = (h - h.sum(1, True) / n - q * (h * q).sum(1, True) / n) / sigma
            if c["residual"]:
                ds = ds + s["dsum"].double()
            out += [ds, torch.einsum("rc,rc->c", dy, q), dy.sum(0)]
        return out
    if c["op"] == "dense":
        x, w = s["x"].double(), s["w"].double()
        z = torch.einsum("mk,nk->mn", x, w) + s["b"].double()
        a, r2 = 0.7978845608028654, 0.7071067811865476
        if c["act"] == "gelu":
            y, slope = z * torch.special.erfc(-z * r2) / 2, \
                torch.special.erfc(-z * r2) / 2 + z * (-z * z / 2).exp() * 0.3989422804014327
        elif c["act"] == "gelu_tanh":
            q = a * (z + 0.044715 * z ** 3)
            sig = 1 / (1 + (-2 * q).exp())
            y, slope = z * sig, sig + z * sig * (1 - sig) * 2 * a * (1 + 0.134145 * z ** 2)
        elif c["act"] == "relu":
            y, slope = z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).double()
        else:
            y, slope = z, torch.ones_like(z)
        if c["residual"]:
            y = y + s["residual"].double()
        if not c["train"]:
            return [y]
        dz = s["dy"].double() * slope
        return [y, torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x), dz.sum(0)]

    total, t, eight = s["p"].numel(), s["step"] + 1, c["bits"] == 8
    up = float(s["scale"]) if c["clip"] else 1.0
    p, m, v = (torch.empty(total, device=DEV, dtype=torch.float64) for _ in range(3))
    for a, (n, decays), span in zip(s["at"], s["sizes"], s["spans"].tolist()):
        for lo in range(a, a + span, 1 << 26):
            hi = min(a + span, lo + (1 << 26))
            g = s["g"][lo:hi].double() * up
            if eight:
                code, be = s["m"][lo:hi].long(), slice(lo // BLOCK, hi // BLOCK)
                m0 = _value64(code % 128, s["m_exp"][be], -6) * (1 - 2 * (code // 128))
                v0 = _value64(s["v"][lo:hi].long(), s["v_exp"][be], -22)
            else:
                m0, v0 = s["m"][lo:hi].double(), s["v"][lo:hi].double()
            m1, v1 = m0 + (g - m0) * (1 - B1), v0 + (g * g - v0) * (1 - B2)
            size = (m1 / (1 - B1 ** t)) / ((v1 / (1 - B2 ** t)).sqrt() + EPS)
            p0 = s["p"][lo:hi].double()
            p[lo:hi] = p0 - LR * (size + (DECAY if decays else 0.0) * p0)
            if eight:
                words = _words64(lo, hi - lo, s["seed"], t)
                m1 = _rounded64(m1, (words % 65536) / 65536.0, -6, 1)
                v1 = _rounded64(v1, (words // 65536) / 65536.0, -22, 3)
            m[lo:hi], v[lo:hi] = m1, v1
    return [p, m, v] + ([p] if c["copy"] else [])

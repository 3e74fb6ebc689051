"""Workloads of the model-side operators: dropout from a counter-based
generator, the learned relative position bias by buckets with its gradient,
and the attention that uses both, forward and backward.

Each workload has a plain form in elementary torch operations (32 bits,
rounded once at the end) and the call a user of the library makes.

The formulas
------------
Keep bits.  Element e of an array (its index in row-major order) belongs to
Philox4x32-10 call e // 8: key = seed (low, high word), counter = (e // 8 low,
high word; offset low, high word).  Halfword e % 8 of the call (low half of
word 0 first), its lowest 15 bits: u.  With T = round(32768 p) the element is
dropped iff u < T, and a kept one is scaled by 32768 / (32768 - T).
    dropout    y = residual + keep * x / (1 - p)
Buckets.  For the distance d = key - query of a pair, two-sided: half of the
buckets for d <= 0, half for d > 0, n = |d|; one-sided: n = max(-d, 0).  With
nb buckets a side, E = nb // 2 and D = max_distance: bucket n for n < E, then
E + floor((nb - E) log(n / E) / log(D / E)), at most nb - 1.
    bias       out[h, i, j] = table[bucket(j - i - q_offset), h]
    gradient   dtable[b, h] = sum of dout[n, h, i, j] over n and the pairs of b
Attention, for query i of head h and the key j of its batch entry and group,
on the pairs with j < kv_len and, if causal, j <= i + q_offset:
    S = scale q.k + bias,  P = softmax(S),  Z = keep * P / (1 - p),  o = Z v
    dv = Z^T do,  dP = keep * (do v^T) / (1 - p),  dS = P (dP - rowsum(dP P))
    dq = scale dS k,  dk = scale dS^T q,  dtable = dS summed by buckets
A row without keys gives o = 0 and no gradient.  The keep bits are those of
an array [batch, head, query, keys rounded up to a multiple of 8].
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MASK = 0xFFFFFFFF


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # dropout: one token's hidden state between two layers of BERT-base
        # (a call whose latency is all that counts)
        dict(name="drop_token", op="dropout", rows=1, cols=768, pad=0, dtype="f32",
             residual=True, p=0.1),
        # the hidden states of a BERT-large batch, 32 sequences of 512, added to the residual stream
        dict(name="drop_bert", op="dropout", rows=16384, cols=1024, pad=0, dtype="bf16",
             residual=True, p=0.1),
        # its backward pass on an odd slice of a wider buffer: rows that start at any alignment
        dict(name="drop_odd", op="dropout", rows=4099, cols=1001, pad=7, dtype="f16",
             residual=False, p=0.25),
        # the hidden states of 32 sequences of 2048 tokens of the GPT-1.3B configuration
        dict(name="drop_gpt", op="dropout", rows=65536, cols=2048, pad=0, dtype="bf16",
             residual=True, p=0.1),
        # bias of one new token against all earlier positions
        dict(name="bias_token", op="bias", H=16, Lq=1, Lk=2047, q_offset=2046, dtype="f32",
             num_buckets=32, max_distance=128, two_sided=False),
        # the whole bias of a 2048-token encoder, 16 heads
        dict(name="bias_2048", op="bias", H=16, Lq=2048, Lk=2048, q_offset=0, dtype="bf16",
             num_buckets=32, max_distance=128, two_sided=True),
        # gradient of BERT-base's 12 heads over a batch of 32 sequences of 512
        dict(name="bias_grad_bert", op="bias_grad", N=32, H=12, Lq=512, Lk=512, q_offset=0,
             dtype="bf16", num_buckets=32, max_distance=128, two_sided=True),
        # odd lengths, one-sided, fp32 gradient (rows at any alignment)
        dict(name="bias_grad_odd", op="bias_grad", N=3, H=5, Lq=777, Lk=1301, q_offset=524,
             dtype="f32", num_buckets=32, max_distance=128, two_sided=False),
        # attention of one short BERT-base sequence, forward (latency)
        dict(name="attn_short", op="attn", train=False, B=1, H=12, Hkv=12, D=64, Lq=128, Lk=128,
             causal=False, p=0.1, bias=True, num_buckets=32, max_distance=128, shortest=128,
             dtype="bf16"),
        # forward over 8 sequences of the GPT-1.3B configuration (16 heads of 128), evaluation
        dict(name="attn_eval_gpt", op="attn", train=False, B=8, H=16, Hkv=16, D=128, Lq=2048,
             Lk=2048, causal=True, p=0.0, bias=False, num_buckets=32, max_distance=128,
             shortest=2048, dtype="bf16"),
        # a training step's attention in BERT-base: 32 padded sequences of 128..512 tokens,
        # dropout and the learned bias, forward and backward
        dict(name="attn_train_bert", op="attn", train=True, B=32, H=12, Hkv=12, D=64, Lq=512,
             Lk=512, causal=False, p=0.1, bias=True, num_buckets=32, max_distance=128,
             shortest=128, dtype="bf16"),
        # odd lengths, shared key/value heads of 80, more keys than queries, causal
        dict(name="attn_train_odd", op="attn", train=True, B=3, H=8, Hkv=2, D=80, Lq=333, Lk=517,
             causal=True, p=0.1, bias=True, num_buckets=32, max_distance=128, shortest=301,
             dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dropout", "bias", "bias_grad", "attn", "attn"])
    if op == "dropout":
        cols = _log(rng, 1, 4096)
        return dict(op=op, rows=_log(rng, 1, min(65536, (1 << 27) // cols)), cols=cols,
                    pad=rng.choice([0, 0, 1, 8]), dtype=rng.choice(sorted(TYPES)),
                    residual=rng.random() < 0.5, p=rng.choice([0.0, 0.1, 0.25, 0.5]))
    buckets = dict(num_buckets=rng.choice([16, 32, 64]), max_distance=rng.choice([64, 128, 300]))
    if op in ("bias", "bias_grad"):
        H, Lq, Lk = rng.randint(1, 32), _log(rng, 1, 2048), _log(rng, 1, 2048)
        c = dict(op=op, H=H, Lq=Lq, Lk=Lk, q_offset=rng.choice([0, Lk - Lq]),
                 dtype=rng.choice(sorted(TYPES)), two_sided=rng.random() < 0.5, **buckets)
        if op == "bias":
            while c["H"] * Lq * Lk > 1 << 26:
                c["H"] //= 2
        else:
            c["N"] = max(1, min(rng.randint(1, 32), 100_000_000 // (H * Lq * Lk)))
            while c["H"] * Lq * Lk > 50_000_000:
                c["H"] //= 2
        return c
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 4])
    Lk = _log(rng, 16, 2048)
    Lq = Lk if rng.random() < 0.5 else _log(rng, 16, 2048)
    B = max(1, min(rng.randint(1, 16), 50_000_000 // (H * Lq * Lk)))
    return dict(op="attn", train=rng.random() < 0.6, B=B, H=H, Hkv=Hkv,
                D=rng.choice([32, 64, 80, 128]), Lq=Lq, Lk=Lk, causal=rng.random() < 0.5,
                p=rng.choice([0.0, 0.1, 0.2]), bias=rng.random() < 0.6,
                shortest=rng.randint(max(1, Lk // 4), Lk), dtype=rng.choice(["bf16", "f16"]),
                **buckets)


def _lens(c):
    """Key lengths of the batch: from `shortest` to Lk in even steps, the longest first."""
    B, lo, hi = c["B"], c["shortest"], c["Lk"]
    return [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]


def _pairs(c):
    """Pairs of queries and keys that the masks leave, over the batch, for one head."""
    total = 0
    for n in _lens(c):
        if not c["causal"]:
            total += c["Lq"] * n
        else:
            off = c["Lk"] - c["Lq"]
            total += sum(min(n, max(0, i + off + 1)) for i in range(c["Lq"]))
    return total


def work(case):
    c, s = case, TYPES[case["dtype"]].itemsize
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return {"bytes": n * s * (3 if c["residual"] else 2), "flops": n * (2 if c["residual"] else 1)}
    if c["op"] == "bias":
        return {"bytes": c["H"] * (c["Lq"] * c["Lk"] + c["num_buckets"]) * s, "flops": 0}
    if c["op"] == "bias_grad":
        n = c["N"] * c["H"] * c["Lq"] * c["Lk"]
        return {"bytes": n * s + c["H"] * c["num_buckets"] * 4, "flops": n}
    q, k = c["B"] * c["Lq"] * c["H"] * c["D"], sum(_lens(c)) * c["Hkv"] * c["D"]
    flops = 4 * c["D"] * _pairs(c) * c["H"]
    if not c["train"]:  # q, k, v -> o
        return {"bytes": s * (2 * q + 2 * k), "flops": flops}
    # and back: do in, dq, dk, dv out
    return {"bytes": s * (4 * q + 4 * k), "flops": flops + 10 * c["D"] * _pairs(c) * c["H"]}


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, dtype=t):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    st = {"case": c, "seed": 0x5851F42D00000000 + seed, "offset": 3 + seed % 1000}
    if c["op"] == "dropout":
        wide = c["cols"] + c["pad"]  # a slice of rows of a wider buffer where pad > 0
        st["x"] = normal(c["rows"], wide)[:, :c["cols"]]
        st["residual"] = normal(c["rows"], wide)[:, :c["cols"]] if c["residual"] else None
        st["y"] = torch.empty(c["rows"], c["cols"], device=DEV, dtype=t)
    elif c["op"] == "bias":
        st["table"] = normal(c["num_buckets"], c["H"], dtype=torch.float32)
        st["out"] = torch.empty(c["H"], c["Lq"], c["Lk"], device=DEV, dtype=t)
    elif c["op"] == "bias_grad":
        st["dout"] = normal(c["N"], c["H"], c["Lq"], c["Lk"])
        st["dtable"] = torch.empty(c["num_buckets"], c["H"], device=DEV)
    else:
        B, H, K, D = c["B"], c["H"], c["Hkv"], c["D"]
        st["q"] = normal(B, c["Lq"], H, D)
        st["k"], st["v"] = normal(B, c["Lk"], K, D), normal(B, c["Lk"], K, D)
        st["kv_len"] = None
        if c["shortest"] < c["Lk"]:
            st["kv_len"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
        st["table"] = normal(c["num_buckets"], H) if c["bias"] else None
        st["o"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(B, H, c["Lq"], device=DEV)
        if c["train"]:
            st["do"] = normal(B, c["Lq"], H, D)
            for n in ("q", "k", "v", "table"):
                st["d" + n] = None if st[n] is None else torch.empty_like(st[n])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return _library(state) if own else _plain(state)


def _library(s):
    """The calls a user of the library makes."""
    import momentum_compression_gb300 as ob
    c = s["case"]
    if c["op"] == "dropout":
        ob.ob_dropout(s["x"], s["y"], c["p"], s["seed"], s["offset"], residual=s["residual"])
        return [s["y"]]
    relpos = None
    if c["op"] != "attn" or c["bias"]:
        two = c["two_sided"] if c["op"] != "attn" else not c["causal"]
        relpos = ob.ob_relpos_init(c["num_buckets"], c["max_distance"], two)
    if c["op"] == "bias":
        ob.ob_relpos_bias(relpos, s["table"], s["out"], q_offset=c["q_offset"])
        return [s["out"]]
    if c["op"] == "bias_grad":
        ob.ob_relpos_bias_bwd(relpos, s["dout"], s["dtable"], q_offset=c["q_offset"])
        return [s["dtable"]]
    kw = dict(causal=c["causal"], kv_len=s["kv_len"], relpos=relpos, table=s["table"], p=c["p"],
              seed=s["seed"], offset=s["offset"])
    ob.ob_attn_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], **kw)
    if not c["train"]:
        return [s["o"]]
    ob.ob_attn_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dq"], s["dk"], s["dv"],
                   dtable=s["dtable"], **kw)
    return [s["o"], s["dq"], s["dk"], s["dv"]] + ([s["dtable"]] if c["bias"] else [])


def _mulhilo(m, x):
    """High and low word of m * x for 32-bit words held in int64 (the product wraps, its bits hold)."""
    t = m * x
    return (t >> 32) & MASK, t & MASK


def _keep(n, p, seed, offset):
    """(keep of elements 0..n-1, scale of a kept one); n a multiple of 8."""
    T = round(32768 * p)
    call = torch.arange(n // 8, device=DEV, dtype=torch.int64)
    c = [call & MASK, call >> 32, torch.full_like(call, offset & MASK),
         torch.full_like(call, offset >> 32)]
    del call
    k0, k1 = seed & MASK, seed >> 32
    for _ in range(10):  # the generator's ten rounds
        h0, l0 = _mulhilo(0xD2511F53, c[0])
        h1, l1 = _mulhilo(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    u = torch.stack([w >> s for w in c for s in (0, 16)], 1).to(torch.int16) & 0x7FFF
    return (u >= T).reshape(-1), 32768 / (32768 - T)


def _edges(nb, D):
    """First distance of each of a side's buckets, in whole numbers: bucket E + k begins at the
    first n with (n / E) ** (nb - E) >= (D / E) ** k (neighbours may share it: the upper one holds)."""
    E = nb // 2
    K, first = nb - E, list(range(E))
    for k in range(K):
        n = first[-1] if k else E
        while n ** K < D ** k * E ** (K - k):
            n += 1
        first.append(n)
    return first


def _bucket_of(Lq, Lk, off, num_buckets, D, two_sided):
    """[Lq, Lk] buckets."""
    side = num_buckets // 2 if two_sided else num_buckets
    first = torch.tensor(_edges(side, D), device=DEV)
    i, j = torch.arange(Lq, device=DEV), torch.arange(Lk, device=DEV)
    d = j[None, :] - (i[:, None] + off)
    n = d.abs() if two_sided else (-d).clamp(min=0)
    b = torch.bucketize(n, first, right=True) - 1
    return b + side * (d > 0) if two_sided else b


def _by_bucket(x, bucket, num_buckets):
    """[num_buckets, H] sums of x [N, H, Lq, Lk]."""
    which = (bucket.reshape(-1, 1) == torch.arange(num_buckets, device=DEV)).to(x.dtype)
    return (x.sum(0).flatten(1) @ which).t().contiguous()


def _plain(s):
    c = s["case"]
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        keep, scale = _keep(-(-n // 8) * 8, c["p"], s["seed"], s["offset"])
        y = s["x"].float() * scale * keep[:n].reshape(c["rows"], c["cols"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(s["x"].dtype)]
    if c["op"] == "bias":
        b = _bucket_of(c["Lq"], c["Lk"], c["q_offset"], c["num_buckets"], c["max_distance"],
                       c["two_sided"])
        return [s["table"].t()[:, b].to(TYPES[c["dtype"]])]
    if c["op"] == "bias_grad":
        b = _bucket_of(c["Lq"], c["Lk"], c["q_offset"], c["num_buckets"], c["max_distance"],
                       c["two_sided"])
        return [_by_bucket(s["dout"].float(), b, c["num_buckets"])]

    B, H, K, D, Lq, Lk = (c[n] for n in ("B", "H", "Hkv", "D", "Lq", "Lk"))
    t, off, scale = s["q"].dtype, Lk - Lq, 1 / math.sqrt(D)
    q = s["q"].float().transpose(1, 2)                                      # [B, H, Lq, D]
    k, v = (s[n].float().transpose(1, 2).repeat_interleave(H // K, 1) for n in "kv")
    S = q @ k.transpose(2, 3) * scale
    if c["bias"]:
        bucket = _bucket_of(Lq, Lk, off, c["num_buckets"], c["max_distance"], not c["causal"])
        S += s["table"].float().t()[:, bucket]
    j = torch.arange(Lk, device=DEV)
    if c["causal"]:
        S.masked_fill_(j[None, :] > torch.arange(Lq, device=DEV)[:, None] + off, -math.inf)
    if s["kv_len"] is not None:
        S.masked_fill_((j[None, :] >= s["kv_len"][:, None])[:, None, None, :], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = (S - m.masked_fill(m == -math.inf, 0)).exp_()
    del S
    P /= P.sum(-1, keepdim=True).clamp(min=1e-30)
    keep, up = None, 1.0
    if c["p"] > 0:
        keep, up = _keep(B * H * Lq * (-(-Lk // 8) * 8), c["p"], s["seed"], s["offset"])
        keep = keep.reshape(B, H, Lq, -1)[..., :Lk]
    Z = P if keep is None else P * keep * up
    o = Z @ v
    out = [o.transpose(1, 2).to(t)]
    if not c["train"]:
        return out
    do = s["do"].float().transpose(1, 2)
    dv = Z.transpose(2, 3) @ do
    del Z
    dP = do @ v.transpose(2, 3)
    if keep is not None:
        dP *= keep * up
    dS = P * (dP - (dP * P).sum(-1, keepdim=True))
    del dP, P
    dq = dS @ k * scale
    dk = dS.transpose(2, 3) @ q * scale
    dk, dv = (x.reshape(B, K, H // K, Lk, D).sum(2) for x in (dk, dv))
    out += [x.transpose(1, 2).to(t) for x in (dq, dk, dv)]
    if c["bias"]:
        out.append(_by_bucket(dS, bucket, c["num_buckets"]).to(t))
    return out


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _uniform64(first, count, seed, offset):
    """u of elements first .. first + count - 1 (both multiples of 8); the products by 16-bit limbs."""
    e = torch.arange(first // 8, (first + count) // 8, device=DEV)
    x = torch.empty(4, count // 8, device=DEV, dtype=torch.int64)
    x[0], x[1], x[2], x[3] = e % 2**32, e // 2**32, offset % 2**32, offset // 2**32

    def product(m, a):
        low, high = a % 65536 * m, a // 65536 * m       # a m = low + 65536 high, each < 2**48
        mid = low // 65536 + high
        return mid // 65536, mid % 65536 * 65536 + low % 65536

    for r in range(10):
        key = [(seed + r * 0x9E3779B9) % 2**32, (seed // 2**32 + r * 0xBB67AE85) % 2**32]
        (a, b), (y, z) = product(0xD2511F53, x[0]), product(0xCD9E8D57, x[2])
        x = torch.stack([y ^ x[1] ^ key[0], z, a ^ x[3] ^ key[1], b])
    return torch.stack([x % 32768, x // 65536 % 32768], 1).reshape(8, -1).t().reshape(-1)


def _bucket64(d, c, two_sided):
    """Bucket of each distance in `d` (a list of whole numbers), one by one."""
    nb = c["num_buckets"] // 2 if two_sided else c["num_buckets"]
    E, D = nb // 2, c["max_distance"]
    out = []
    for x in d:
        n, base = (abs(x), nb * (x > 0)) if two_sided else (max(-x, 0), 0)
        b = n
        if n >= E:
            b = E
            while b < nb - 1 and n ** (nb - E) >= D ** (b + 1 - E) * E ** (nb - 1 - b):
                b += 1
        out.append(base + b)
    return out


def _toeplitz64(c, Lq, Lk, off, two_sided):
    """(buckets of the distances -(Lq - 1) - off .. Lk - 1 - off, index of each pair's)."""
    b = torch.tensor(_bucket64(range(-(Lq - 1) - off, Lk - off), c, two_sided), device=DEV)
    at = torch.arange(Lk, device=DEV)[None, :] - torch.arange(Lq, device=DEV)[:, None] + Lq - 1
    return b, at


def exact(case, seed):
    c, s = case, prepare(case, seed)
    T = round(32768 * c.get("p", 0.0))
    up = 32768 / (32768 - T)
    if c["op"] == "dropout":
        n, x = c["rows"] * c["cols"], s["x"].double().reshape(-1)
        y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double().reshape(-1).clone()
        step = 1 << 25
        for at in range(0, n, step):
            m = min(step, n - at)
            u = _uniform64(at, -(-m // 8) * 8, s["seed"], s["offset"])[:m]
            y[at:at + m] += torch.where(u < T, 0.0, x[at:at + m] * up)
        return [y.reshape(c["rows"], c["cols"])]
    if c["op"] == "bias":
        b, at = _toeplitz64(c, c["Lq"], c["Lk"], c["q_offset"], c["two_sided"])
        return [s["table"].double()[b].t()[:, at]]
    if c["op"] == "bias_grad":
        b, at = _toeplitz64(c, c["Lq"], c["Lk"], c["q_offset"], c["two_sided"])
        out = torch.zeros(c["num_buckets"], c["H"], device=DEV, dtype=torch.float64)
        which = torch.nn.functional.one_hot(b, c["num_buckets"]).double()
        for h in range(c["H"]):
            x = s["dout"][:, h].double().sum(0)
            by_d = torch.zeros(len(b), device=DEV, dtype=torch.float64)
            by_d.index_add_(0, at.reshape(-1), x.reshape(-1))
            out[:, h] = which.t() @ by_d
        return [out]

    B, H, D, Lq, Lk = (c[n] for n in ("B", "H", "D", "Lq", "Lk"))
    group, off, width, lens = H // c["Hkv"], Lk - Lq, -(-Lk // 8) * 8, _lens(c)
    o = torch.zeros(B, Lq, H, D, device=DEV, dtype=torch.float64)
    dq, (dk, dv) = torch.zeros_like(o), torch.zeros(2, *s["k"].shape, device=DEV, dtype=torch.float64)
    if c["bias"]:
        b, at = _toeplitz64(c, Lq, Lk, off, not c["causal"])
        dtable = torch.zeros(c["num_buckets"], H, device=DEV, dtype=torch.float64)
    for n in range(B):
        for h in range(H):
            q, k, v = s["q"][n, :, h].double(), s["k"][n, :, h // group].double(), s["v"][n, :, h // group].double()
            live = (torch.arange(Lk, device=DEV) < lens[n]).expand(Lq, Lk)
            if c["causal"]:
                live = live.tril(off)
            x = torch.einsum("id,jd->ij", q, k) / math.sqrt(D)
            if c["bias"]:
                x = x + s["table"][:, h].double()[b][at]
            w = torch.where(live, x - torch.where(live, x, -1e300).amax(1, True), -torch.inf).exp()
            w = torch.where(live.any(1, True), w / w.sum(1, True), 0.0)
            g = torch.ones_like(w)
            if c["p"] > 0:
                u = _uniform64((n * H + h) * Lq * width, Lq * width, s["seed"], s["offset"])
                g = torch.where(u.reshape(Lq, width)[:, :Lk] < T, 0.0, up)
            o[n, :, h] = (w * g) @ v
            if not c["train"]:
                continue
            do = s["do"][n, :, h].double()
            dv[n, :, h // group] += (w * g).t() @ do
            ds = w * (g * (do @ v.t()) - (do * o[n, :, h]).sum(1, True))
            dq[n, :, h] = ds @ k / math.sqrt(D)
            dk[n, :, h // group] += ds.t() @ q / math.sqrt(D)
            if c["bias"]:
                by_d = torch.zeros(len(b), device=DEV, dtype=torch.float64)
                by_d.index_add_(0, at.reshape(-1), ds.reshape(-1))
                dtable[:, h].index_add_(0, b, by_d)
    return [o] if not c["train"] else [o, dq, dk, dv] + ([dtable] if c["bias"] else [])

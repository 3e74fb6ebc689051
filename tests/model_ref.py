"""Plain 64-bit forms of the model-side operators for the tests: keep bits,
buckets, dropout, relative position bias, attention with its gradients, and
the magnitudes that error bounds are made of.  CPU or CUDA torch tensors."""
import math

import numpy as np
import torch

# |fl(x) - x| <= UNIT |x| for normal x; below TINY[...] the spacing is fixed
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def philox(call, seed, offset):
    """[n, 4] words of Philox4x32-10 (uint64 holding 32 bits) for 64-bit call numbers."""
    m = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    call = np.asarray(call, np.uint64)
    c = [call & m, call >> s32, np.full_like(call, offset & 0xFFFFFFFF),
         np.full_like(call, offset >> 32)]
    k = [np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s32) ^ c[1] ^ k[0], b & m, (a >> s32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + np.uint64(0x9E3779B9)) & m, (k[1] + np.uint64(0xBB67AE85)) & m]
    return np.stack(c, 1)


def keep(first, count, p, seed, offset):
    """(bool keep of elements first .. first + count - 1, scale) -- first a multiple of 8."""
    T = round(p * 32768)
    calls = np.arange(first // 8, first // 8 + -(-count // 8))
    w = philox(calls, seed, offset)
    half = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:count]
    kept = (half & np.uint64(0x7FFF)) >= np.uint64(T)
    return kept, (32768 / (32768 - T) if T < 32768 else 0.0)


def bucket(d, num_buckets, max_distance, two_sided):
    """Bucket of one distance, in whole numbers."""
    side = num_buckets // 2 if two_sided else num_buckets
    E = side // 2
    n = abs(d) if two_sided else max(-d, 0)
    b = n
    if n >= E:
        b = E
        while (b < side - 1 and
               n ** (side - E) >= max_distance ** (b + 1 - E) * E ** (side - 1 - b)):
            b += 1
    return b + (side if two_sided and d > 0 else 0)


def buckets(Lq, Lk, off, num_buckets, max_distance, two_sided):
    """[Lq, Lk] int64 numpy array."""
    by_d = np.array([bucket(d, num_buckets, max_distance, two_sided)
                     for d in range(-(Lq - 1) - off, Lk - off)], np.int64)
    return by_d[np.arange(Lk)[None, :] - np.arange(Lq)[:, None] + Lq - 1]


def bucket_sums(x, b, num_buckets):
    """[num_buckets] float64 sums of x (any shape of b)."""
    out = torch.zeros(num_buckets, dtype=torch.float64, device=x.device)
    return out.index_add_(0, b.reshape(-1), x.reshape(-1))


def attention(q, k, v, do=None, table=None, relpos=None, causal=False, q_offset=None,
              kv_len=None, scale=None, p=0.0, seed=0, offset=0, bounds=False):
    """o, lse (and dq, dk, dv, dtable) in 64 bits; q [B, Lq, H, D], k, v [B, Lk, Hkv, D].
    relpos: (num_buckets, max_distance, two_sided).  With bounds: also the elementwise
    error bounds of an implementation that rounds P, dS, o and its outputs to q's type
    and works in fp32 otherwise."""
    B, Lq, H, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    dev, t = q.device, q.dtype
    off = Lk - Lq if q_offset is None else q_offset
    scale = D ** -0.5 if scale is None else scale
    u, tiny = UNIT.get(t, 0.0), TINY.get(t, 0.0)
    out = {"o": torch.zeros(B, Lq, H, D, dtype=torch.float64, device=dev),
           "lse": torch.full((B, H, Lq), -math.inf, dtype=torch.float64, device=dev)}
    names = ["o"]
    if do is not None:
        names += ["dq", "dk", "dv"]
        out.update(dq=torch.zeros_like(out["o"]), dk=torch.zeros_like(k, dtype=torch.float64),
                   dv=torch.zeros_like(k, dtype=torch.float64))
        if table is not None:
            names.append("dtable")
            out["dtable"] = torch.zeros(table.shape, dtype=torch.float64, device=dev)
    err = {n: torch.zeros_like(out[n]) for n in names}
    if table is not None:
        bk = torch.from_numpy(buckets(Lq, Lk, off, *relpos)).to(dev)
    live0 = torch.ones(Lq, Lk, dtype=torch.bool, device=dev)
    if causal:
        live0 = torch.arange(Lk, device=dev)[None, :] <= torch.arange(Lq, device=dev)[:, None] + off
    width = -(-Lk // 8) * 8
    for b in range(B):
        n = Lk if kv_len is None else max(0, min(Lk, int(kv_len[b])))
        live = live0 & (torch.arange(Lk, device=dev) < n)[None, :]
        some = live.any(1, keepdim=True)
        for h in range(H):
            kh = h // (H // Hkv)
            Q = q[b, :, h].double()
            K, V = (torch.where((torch.arange(Lk, device=dev) < n)[:, None], x[b, :, kh].double(), 0.0)
                    for x in (k, v))
            S = Q @ K.T * scale
            if table is not None:
                S = S + table[:, h].double()[bk]
            S = torch.where(live, S, -math.inf)
            m = torch.where(some, S.amax(1, keepdim=True) if Lk else 0.0, 0.0)
            E = torch.where(live, (S - m).exp(), 0.0)
            l = E.sum(1, keepdim=True)
            P = torch.where(some, E / l, 0.0)
            kb, up = keep((b * H + h) * Lq * width, Lq * width, p, seed, offset)
            g = torch.from_numpy(kb).to(dev).reshape(Lq, width)[:, :Lk].double() * up
            Z = P * g
            out["o"][b, :, h] = Z @ V
            out["lse"][b, h] = torch.where(some, m + l.log(), -math.inf)[:, 0]
            # relative error of P in fp32: its exponent's absolute error (D + 8
            # roundings of terms of the magnitude of |q||k|, bias and lse), doubled
            # for the normalisation, and 2^-20 for exp2, sums and divisions
            mag = (Q.abs() @ K.abs().T * scale).amax(1, keepdim=True) if Lk else 0.0
            if table is not None:
                mag = mag + table[:, h].double().abs().max()
            eP = 2 * (D + 8) * 2.0 ** -24 * (mag + m.abs() + 1) + 2.0 ** -20
            if bounds:
                e = ((u + eP) * Z) @ V.abs() + Lk * tiny
                err["o"][b, :, h] = e + u * (out["o"][b, :, h].abs() + e)
            if do is None:
                continue
            G = do[b, :, h].double()
            Oh = out["o"][b, :, h]
            dP = (G @ V.T) * g
            delta = (G * Oh).sum(1, keepdim=True)
            dS = P * (dP - delta)
            out["dv"][b, :, kh] += Z.T @ G
            out["dq"][b, :, h] = dS @ K * scale
            out["dk"][b, :, kh] += dS.T @ Q * scale
            if table is not None:
                out["dtable"][:, h] += bucket_sums(dS, bk, table.shape[0])
            if bounds:
                # dS: P off by eP; do.v and rowsum(do o) off by D roundings of their
                # magnitudes; o itself off by its own bound
                ga = (G.abs() @ V.abs().T) * g
                da = (G.abs() * Oh.abs()).sum(1, keepdim=True)
                do_err = (G.abs() * err["o"][b, :, h]).sum(1, keepdim=True)
                eS = P * ((eP + D * 2.0 ** -23) * (ga + da) + do_err)
                if table is not None:
                    err["dtable"][:, h] += bucket_sums(eS + 2.0 ** -14 * dS.abs(), bk, table.shape[0])
                eS = eS + u * (dS.abs() + eS)
                err["dq"][b, :, h] = (eS + 2.0 ** -18 * dS.abs()) @ K.abs() * scale + Lk * tiny
                err["dk"][b, :, kh] += (eS + 2.0 ** -18 * dS.abs()).T @ Q.abs() * scale + Lq * tiny
                err["dv"][b, :, kh] += ((u + eP) * Z).T @ G.abs() + Lq * tiny
    if bounds:
        for x in names[1:]:
            err[x] = err[x] + u * (out[x].abs() + err[x]) + tiny
        return out, err
    return out

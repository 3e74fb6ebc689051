"""The model-side operators without a GPU: bucket edges, the refusals of every
entry point, and the tests' own 64-bit reference (its gradients against
central differences, its generator against the oracle's)."""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

import model_ref as R
import momentum_compression_gb300 as ob
import oracle as O


@pytest.fixture(scope="module", autouse=True)
def _built():
    from momentum_compression_gb300 import _build
    _build.build()


@pytest.mark.parametrize("two", [False, True])
def test_bucket_edges_are_exact(two):
    """first[b] of every width and distance is the first n whose bucket, by the
    definition in whole numbers, is b or above."""
    for nb in list(range(2, 41)) + [64, 100, 128] + ([200, 256] if two else []):
        side = nb // 2 if two else nb
        for D in (3, 17, 64, 128, 300, 1000):
            if side < 2 or (two and nb % 2) or D <= side // 2:
                continue
            rp = ob.ob_relpos_init(nb, D, two)
            got = [max(b for b in range(side) if rp.first[b] <= n) for n in range(D + 2)]
            assert got == [R.bucket(-n, nb, D, two) for n in range(D + 2)], (nb, D)
            if two:
                assert R.bucket(1, nb, D, True) == side + (1 if rp.first[1] == 1 else 0)


@pytest.mark.parametrize("args", [(1, 128, False), (129, 1000, False), (2, 128, True),
                                  (33, 128, True), (258, 1000, True), (32, 16, False),
                                  (32, 8, True), (32, (1 << 20) + 1, True), (0, 5, False)])
def test_relpos_init_refuses(args):
    with pytest.raises(ob.OBError) as e:
        ob.ob_relpos_init(*args)
    assert e.value.status == ob.OB_ERR_INVALID


def _refused(status, fn, *args):
    assert fn(*args) == status, ob.ob_last_error(None)
    assert ob.ob_last_error(None)


def test_dropout_refuses():
    f = ob.lib().ob_dropout
    ok = [0x1000, 64, None, 0, 0x2000, 64, 4, 64, ob.OB_TYPE_F32, 0.5, 1, 2, None]
    for at, value, status in ((0, None, ob.OB_ERR_INVALID), (4, None, ob.OB_ERR_INVALID),
                              (0, 0x1002, ob.OB_ERR_ALIGN), (4, 0x2001, ob.OB_ERR_ALIGN),
                              (2, 0x3002, ob.OB_ERR_ALIGN), (1, 63, ob.OB_ERR_INVALID),
                              (5, 63, ob.OB_ERR_INVALID), (8, 3, ob.OB_ERR_INVALID),
                              (9, -0.1, ob.OB_ERR_INVALID), (9, 1.1, ob.OB_ERR_INVALID),
                              (9, math.nan, ob.OB_ERR_INVALID), (6, 1 << 35, ob.OB_ERR_INVALID)):
        a = list(ok)
        a[at] = value
        _refused(status, f, *a)
    a = list(ok)
    a[2], a[3] = 0x3000, 63
    _refused(ob.OB_ERR_INVALID, f, *a)
    a = list(ok)
    a[6] = 0
    assert f(*a) == ob.OB_OK


def test_relpos_calls_refuse():
    L = ob.lib()
    rp = ob.ob_relpos_init(32, 128, True)
    r = ct.byref(rp)
    ok = [r, 0x1000, 0, 4, 8, 8, 0, 0x2000, 0, 64, 8, None]
    for at, value, status in ((0, None, ob.OB_ERR_INVALID), (1, None, ob.OB_ERR_INVALID),
                              (1, 0x1002, ob.OB_ERR_ALIGN), (7, 0x2001, ob.OB_ERR_ALIGN),
                              (2, 9, ob.OB_ERR_INVALID), (3, -1, ob.OB_ERR_INVALID),
                              (4, -1, ob.OB_ERR_INVALID), (5, 1 << 30, ob.OB_ERR_INVALID),
                              (6, 1 << 30, ob.OB_ERR_INVALID), (10, 7, ob.OB_ERR_INVALID),
                              (9, 7, ob.OB_ERR_INVALID), (0, ct.byref(ob.ob_relpos()),
                                                          ob.OB_ERR_INVALID)):
        a = list(ok)
        a[at] = value
        _refused(status, L.ob_relpos_bias, *a)
    need = ob.ob_relpos_workspace_bytes(rp, 2, 4, 8, 8)
    ok = [r, 0x1000, 0, 2, 4, 8, 8, 256, 64, 8, 0, 0x2000, 0, 0x3000, need, None]
    for at, value, status in ((1, None, ob.OB_ERR_INVALID), (1, 0x1001, ob.OB_ERR_ALIGN),
                              (11, None, ob.OB_ERR_INVALID), (13, None, ob.OB_ERR_INVALID),
                              (13, 0x3004, ob.OB_ERR_ALIGN), (14, 0, ob.OB_ERR_INVALID),
                              (3, -1, ob.OB_ERR_INVALID), (2, 7, ob.OB_ERR_INVALID),
                              (12, 7, ob.OB_ERR_INVALID)):
        a = list(ok)
        a[at] = value
        _refused(status, L.ob_relpos_bias_bwd, *a)


def _attn(**over):
    a = ob.ob_attn(ob.OB_TYPE_BF16, 2, 4, 2, 64, 16, 24, 0.125, 0, 0, None, None, None, 0.1, 1, 2)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_attention_refuses():
    L = ob.lib()
    rp = ob.ob_relpos_init(32, 128, True)
    far = ob.ob_relpos_init(32, 800, True)
    q = ob.ob_heads(0x1000, 4096, 256, 64)
    kv = ob.ob_heads(0x2000, 4096, 128, 64)
    o = ob.ob_heads(0x3000, 4096, 256, 64)
    b = ct.byref

    def fwd(a, q=q, k=kv, v=kv, o=o, lse=0x4000):
        return L.ob_attn_fwd(b(a), q and b(q), k and b(k), v and b(v), o and b(o), lse, None)

    P = ct.pointer
    for over, status in ((dict(type=ob.OB_TYPE_F32), ob.OB_ERR_UNSUPPORTED),
                         (dict(D=63), ob.OB_ERR_UNSUPPORTED), (dict(D=136), ob.OB_ERR_UNSUPPORTED),
                         (dict(D=0), ob.OB_ERR_UNSUPPORTED), (dict(H=3), ob.OB_ERR_INVALID),
                         (dict(Hkv=0), ob.OB_ERR_INVALID), (dict(B=-1), ob.OB_ERR_INVALID),
                         (dict(B=20000), ob.OB_ERR_INVALID), (dict(Lq=-1), ob.OB_ERR_INVALID),
                         (dict(Lk=1 << 24), ob.OB_ERR_INVALID), (dict(scale=0.0), ob.OB_ERR_INVALID),
                         (dict(scale=-1.0), ob.OB_ERR_INVALID),
                         (dict(scale=math.nan), ob.OB_ERR_INVALID),
                         (dict(scale=math.inf), ob.OB_ERR_INVALID),
                         (dict(p=1.0), ob.OB_ERR_INVALID), (dict(p=math.nan), ob.OB_ERR_INVALID),
                         (dict(q_offset=1 << 24), ob.OB_ERR_INVALID),
                         (dict(relpos=P(rp)), ob.OB_ERR_INVALID),
                         (dict(table=0x5000), ob.OB_ERR_INVALID),
                         (dict(relpos=P(rp), table=0x5001), ob.OB_ERR_ALIGN),
                         (dict(relpos=P(far), table=0x5000), ob.OB_ERR_UNSUPPORTED),
                         (dict(kv_len=0x5002), ob.OB_ERR_ALIGN)):
        _refused(status, fwd, _attn(**over))
    a = _attn()
    for bad, status in ((None, ob.OB_ERR_INVALID), (ob.ob_heads(0x1008, 4096, 256, 64), ob.OB_ERR_ALIGN),
                        (ob.ob_heads(None, 4096, 256, 64), ob.OB_ERR_INVALID),
                        (ob.ob_heads(0x1000, 4096, 257, 64), ob.OB_ERR_ALIGN),
                        (ob.ob_heads(0x1000, 4096, 0, 64), ob.OB_ERR_INVALID),
                        (ob.ob_heads(0x1000, -4096, 256, 64), ob.OB_ERR_INVALID),
                        (ob.ob_heads(0x1000, 4096, 256, 56), ob.OB_ERR_INVALID)):
        for name in "qkvo":
            _refused(status, lambda: fwd(a, **{name: bad}))
    _refused(ob.OB_ERR_ALIGN, lambda: fwd(a, lse=0x4002))
    assert fwd(_attn(B=0), q=None, k=None, v=None, o=None) == ob.OB_OK
    n = ct.c_size_t()
    ab = _attn(relpos=P(rp), table=0x5000)
    assert L.ob_attn_workspace_bytes(b(ab), b(n)) == ob.OB_OK

    def bwd(a, dtable=0x7000, ws=0x10000, nbytes=n.value, dk=kv, lse=0x4000):
        return L.ob_attn_bwd(b(a), b(o), b(q), b(kv), b(kv), b(o), lse, b(q), dk and b(dk), b(kv),
                             dtable, ws, nbytes, None)

    _refused(ob.OB_ERR_INVALID, lambda: bwd(a))  # dtable without a bias
    _refused(ob.OB_ERR_ALIGN, lambda: bwd(ab, dtable=0x7001))
    _refused(ob.OB_ERR_INVALID, lambda: bwd(ab, ws=None))
    _refused(ob.OB_ERR_ALIGN, lambda: bwd(ab, ws=0x10010))
    _refused(ob.OB_ERR_INVALID, lambda: bwd(ab, nbytes=n.value - 1))
    _refused(ob.OB_ERR_INVALID, lambda: bwd(ab, dk=None))
    _refused(ob.OB_ERR_INVALID, lambda: bwd(ab, lse=None))


def test_binding_refuses():
    """The binding refuses what the C call could not see: CPU tensors, types and
    shapes that do not go together."""
    x = torch.zeros(4, 8)
    for call in (lambda: ob.ob_dropout(x, x, 0.5, 1, 2, stream=0),
                 lambda: ob.ob_dropout(x.double(), x, 0.5, 1, 2, stream=0),
                 lambda: ob.ob_relpos_bias(ob.ob_relpos_init(32, 128, True), x, x, stream=0)):
        with pytest.raises(ob.OBError) as e:
            call()
        assert e.value.status == ob.OB_ERR_INVALID
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ob.OBError):
        ob.ob_attn_fwd(q, q, q[:, :2], q, stream=0)


def test_reference_generator_is_the_oracles():
    calls = [0, 1, 5, (1 << 32) - 1, 1 << 32, (7 << 40) + 3]
    seed, offset = 0x0123456789ABCDEF, (9 << 32) + 4
    got = R.philox(calls, seed, offset)
    for c, row in zip(calls, got):
        ctr = np.array([c & 0xFFFFFFFF, c >> 32, offset & 0xFFFFFFFF, offset >> 32], np.uint32)
        key = np.array([seed & 0xFFFFFFFF, seed >> 32], np.uint32)
        assert np.array_equal(row.astype(np.uint32), O.philox4x32_10(ctr, key))


def test_reference_gradients_against_differences():
    g = torch.Generator()
    g.manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    q, k, v, do, table = r(2, 5, 4, 8), r(2, 7, 2, 8), r(2, 7, 2, 8), r(2, 5, 4, 8), r(8, 4)
    kw = dict(relpos=(8, 6, True), causal=True, kv_len=[7, 3], p=0.25, seed=5, offset=6)
    out = R.attention(q, k, v, do, table=table, **kw)
    base = dict(q=q, k=k, v=v, table=table)
    for name in base:
        e, f = r(*base[name].shape), []
        for s in (1, -1):
            x = dict(base)
            x[name] = base[name] + s * 1e-5 * e
            f.append((R.attention(x["q"], x["k"], x["v"], table=x["table"], **kw)["o"] * do).sum())
        slope = (f[0] - f[1]) / 2e-5
        assert abs(slope - (out["d" + name] * e).sum()) < 1e-7 * (1 + abs(slope))

"""The model-side operators on the GPU against their 64-bit definitions
(tests/model_ref.py): dropout, the bucketed relative position bias and its
gradient, the attention forward and backward.  Every tolerance is an error
bound computed from the inputs: roundings to the type where the operator
says it rounds, fp32 everywhere else."""
import math

import numpy as np
import pytest
import torch

import model_ref as R
import momentum_compression_gb300 as ob

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    from momentum_compression_gb300 import _build
    _build.build()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, dtype=F32: torch.randn(*s, generator=g, device="cuda").to(dtype)


def _within(got, want, bound, what):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{got[i].item()} against {want[i].item()}, bound {bound[i].item()}")


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

def _dropout_ref(x, res, p, seed, offset):
    kb, up = R.keep(0, x.numel(), p, seed, offset)
    k = torch.from_numpy(kb).cuda().reshape(x.shape)
    y = torch.where(k, x.double() * up, 0.0)
    bound = 2.0 ** -23 * y.abs()
    if res is not None:
        y = y + res.double()
    u, tiny = R.UNIT[x.dtype], R.TINY[x.dtype]
    return y, bound + u * (y.abs() + bound) + tiny


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 7, 0), (1, 8, 0), (1, 4097, 0),
                                           (3, 1001, 0), (37, 64, 0), (37, 64, 8), (5, 33, 3),
                                           (300, 1, 4), (1000, 260, 12), (129, 4096, 8)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(dtype, rows, cols, pad, residual):
    mk = _gen(rows * 7 + cols)
    x = mk(rows, cols + pad, dtype=dtype)[:, :cols]
    res = mk(rows, cols + pad, dtype=dtype)[:, :cols] if residual else None
    whole = torch.full((rows, cols + pad + 5), 7.0, device="cuda", dtype=dtype)
    for y in (torch.empty(rows, cols, device="cuda", dtype=dtype), whole[:, :cols]):
        ob.ob_dropout(x, y, 0.3, 0x123456789ABCDEF0, (5 << 32) + 9, residual=res)
        want, bound = _dropout_ref(x, res, 0.3, 0x123456789ABCDEF0, (5 << 32) + 9)
        _within(y, want, bound, "y")
    assert (whole[:, cols:] == 7.0).all(), "wrote past a row"


@pytest.mark.parametrize("shift", range(1, 9))
def test_dropout_at_any_alignment(shift):
    x = _gen(1)(5000, dtype=BF16)[shift:]
    y = torch.zeros(5003, device="cuda", dtype=BF16)[3:][:x.numel()]
    ob.ob_dropout(x, y, 0.5, 1, 2)
    want, bound = _dropout_ref(x, None, 0.5, 1, 2)
    _within(y, want, bound, "y")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift", range(8))
def test_dropout_of_rows_at_any_alignment_into_an_aligned_run(dtype, shift):
    """x and the residual at their own offsets and strides; the last eight is short."""
    mk = _gen(40 + shift)
    for rows, cols, pad in ((37, 8, 1), (91, 9, 8), (53, 131, 3), (1, 1003, 0)):
        n = rows * (cols + pad)
        x = mk(n + shift, dtype=dtype)[shift:].view(rows, cols + pad)[:, :cols]
        res = mk(n + 7 - shift, dtype=dtype)[7 - shift:].view(rows, cols + pad)[:, :cols]
        y = torch.full((rows * cols + 8,), 7.0, device="cuda", dtype=dtype)
        for r in (res, None):
            ob.ob_dropout(x, y[:rows * cols].view(rows, cols), 0.3, 5, 6, residual=r)
            want, bound = _dropout_ref(x, r, 0.3, 5, 6)
            _within(y[:rows * cols].view(rows, cols), want, bound, "y")
            assert (y[rows * cols:] == 7.0).all(), "wrote past the end"


def test_dropout_probabilities_and_values_that_are_dropped():
    x = torch.full((64, 1024), math.nan, device="cuda")
    kb, up = R.keep(0, x.numel(), 0.75, 3, 4)
    k = torch.from_numpy(kb).cuda().reshape(x.shape)
    x[k] = 1.0
    x[0, (~k)[0].nonzero()[0]] = math.inf
    y = torch.empty_like(x)
    ob.ob_dropout(x, y, 0.75, 3, 4)
    assert torch.equal(y, k * 4.0), "a dropped value reached the output"
    share = float((y == 0).double().mean())
    assert abs(share - 0.75) < 5 * math.sqrt(0.75 * 0.25 / x.numel())
    x.fill_(2.0)
    ob.ob_dropout(x, y, 0.0, 3, 4)
    assert (y == 2.0).all()
    ob.ob_dropout(x, y, 1.0, 3, 4, residual=x)
    assert (y == 2.0).all()
    ob.ob_dropout(x, y, 1.0, 3, 4)
    assert (y == 0.0).all()


def test_dropout_in_place_and_backward():
    """y may be x or the residual; the backward pass is the call on dy."""
    mk = _gen(3)
    x, r, dy = mk(333, 77), mk(333, 77), mk(333, 77)
    want = torch.empty_like(x)
    ob.ob_dropout(x, want, 0.2, 8, 1, residual=r)
    for y in (x.clone(), r.clone()):
        a, b = (y, r) if torch.equal(y, x) else (x, y)
        ob.ob_dropout(a, y, 0.2, 8, 1, residual=b)
        assert torch.equal(y, want)
    dx = torch.empty_like(x)
    ob.ob_dropout(dy, dx, 0.2, 8, 1)
    # the operator is linear in x: its gradient against differences
    e = mk(333, 77)
    plus, zero = torch.empty_like(x), torch.empty_like(x)
    ob.ob_dropout(e, plus, 0.2, 8, 1)
    ob.ob_dropout(torch.zeros_like(e), zero, 0.2, 8, 1)
    lhs, rhs = ((plus - zero).double() * dy.double()).sum(), (dx.double() * e.double()).sum()
    assert abs(lhs - rhs) <= 2.0 ** -22 * (dx.double() * e.double()).abs().sum()


def test_dropout_past_32_bits_of_elements():
    """Element numbers over 2^32: the last rows of 2^32 + 2^21 bf16 elements."""
    n = (1 << 32) + (1 << 21) + 5
    x = torch.ones(n, device="cuda", dtype=BF16)
    ob.ob_dropout(x, x, 0.5, 11, 12)
    at = (1 << 32) - 4096
    kb, _ = R.keep(at, n - at, 0.5, 11, 12)
    assert np.array_equal((x[at:] == 2).cpu().numpy(), kb)


# ---------------------------------------------------------------------------
# relative position bias
# ---------------------------------------------------------------------------

RELPOS = [(32, 128, True), (32, 128, False), (64, 64, False), (4, 3, True), (16, 300, True)]


@pytest.mark.parametrize("rp", RELPOS)
@pytest.mark.parametrize("H,Lq,Lk,off", [(1, 1, 1, 0), (3, 1, 333, 332), (2, 70, 64, 0),
                                         (5, 129, 2056, 1000), (2, 200, 131, -69), (1, 65, 8, -500)])
def test_relpos_bias(rp, H, Lq, Lk, off):
    p = ob.ob_relpos_init(*rp)
    b = torch.from_numpy(R.buckets(Lq, Lk, off, *rp)).cuda()
    for table_type, out_type in ((F32, F32), (F32, BF16), (BF16, F16), (F16, F32)):
        table = _gen(H)(rp[0], H, dtype=table_type)
        want = table.float().t()[:, b].to(out_type)
        for ld in (Lk, Lk + 3, -(-Lk // 8) * 8 + 8):
            whole = torch.full((H, Lq, ld), 7.0, device="cuda", dtype=out_type)
            ob.ob_relpos_bias(p, table, whole[..., :Lk], q_offset=off)
            assert torch.equal(whole[..., :Lk], want), (table_type, out_type, ld)
            assert (whole[..., Lk:] == 7.0).all(), "wrote past a row"


@pytest.mark.parametrize("rp", RELPOS)
@pytest.mark.parametrize("N,H,Lq,Lk,off", [(1, 1, 1, 1, 0), (2, 3, 1, 333, 332), (3, 2, 70, 64, 0),
                                           (1, 5, 129, 2056, 1000), (7, 2, 200, 131, -69),
                                           (33, 1, 65, 8, -500), (40, 2, 64, 256, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_relpos_bias_gradient(rp, N, H, Lq, Lk, off, dtype):
    p = ob.ob_relpos_init(*rp)
    b = torch.from_numpy(R.buckets(Lq, Lk, off, *rp)).cuda()
    for ld in (Lk, Lk + 3):
        dout = _gen(N)(N, H, Lq, ld, dtype=dtype)[..., :Lk]
        table_type = BF16 if dtype == F16 else F32
        dt = torch.full((rp[0], H), 9.0, device="cuda", dtype=table_type)
        ob.ob_relpos_bias_bwd(p, dout, dt, q_offset=off)
        again = torch.empty_like(dt)
        ob.ob_relpos_bias_bwd(p, dout, again, q_offset=off)
        assert torch.equal(dt, again)
        for h in range(H):
            x = dout[:, h].double()
            want = R.bucket_sums(x.sum(0), b, rp[0])
            # the longest chain of additions: 32 rows of N entries down a diagonal, 16
            # distances and a butterfly, 8 warps, at most 32 parts in a row, 32 sums
            u = 2.0 ** -24
            bound = (32 * N + 120) * u * R.bucket_sums(x.abs().sum(0), b, rp[0])
            bound = bound + R.UNIT[table_type] * (want.abs() + bound)
            _within(dt[:, h], want, bound, f"dtable of head {h}")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift", [0, 1, 5])
@pytest.mark.parametrize("N,H,Lq,Lk", [(3, 2, 70, 251), (2, 3, 37, 509), (1, 2, 33, 1003),
                                       (2, 1, 100, 77), (5, 1, 34, 255)])
def test_relpos_bias_gradient_of_odd_rows(N, H, Lq, Lk, shift, dtype):
    """Rows at every alignment, with NaN before, between and after them."""
    p = ob.ob_relpos_init(32, 128, True)
    b = torch.from_numpy(R.buckets(Lq, Lk, 3, 32, 128, True)).cuda()
    for pad in (0, 3):
        ld = Lk + pad
        whole = torch.full((N * H * Lq * ld + shift + 9,), math.nan, device="cuda", dtype=dtype)
        dout = whole[shift:shift + N * H * Lq * ld].view(N, H, Lq, ld)[..., :Lk]
        dout.copy_(_gen(N)(N, H, Lq, Lk))
        dt = torch.full((32, H), 9.0, device="cuda")
        ob.ob_relpos_bias_bwd(p, dout, dt, q_offset=3)
        for h in range(H):
            x = dout[:, h].double()
            want = R.bucket_sums(x.sum(0), b, 32)
            # as in test_relpos_bias_gradient
            bound = (32 * N + 120) * 2.0 ** -24 * R.bucket_sums(x.abs().sum(0), b, 32)
            bound = bound + R.UNIT[F32] * (want.abs() + bound)
            _within(dt[:, h], want, bound, f"dtable of head {h}")


def test_relpos_gradient_of_nothing_is_zero():
    p = ob.ob_relpos_init(32, 128, True)
    dt = torch.full((32, 4), 9.0, device="cuda")
    ob.ob_relpos_bias_bwd(p, torch.empty(0, 4, 8, 8, device="cuda"), dt)
    assert (dt == 0).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _attn_case(B=1, H=2, Hkv=None, D=64, Lq=64, Lk=64, dtype=BF16, bias=None, causal=False,
               kv_len=None, p=0.0, q_offset=None, scale=None, seed=1, spread=1.0):
    Hkv = H if Hkv is None else Hkv
    mk = _gen(seed)
    q, do = mk(B, Lq, H, D, dtype=dtype) * spread, mk(B, Lq, H, D, dtype=dtype)
    k, v = mk(B, Lk, Hkv, D, dtype=dtype), mk(B, Lk, Hkv, D, dtype=dtype)
    kw = dict(causal=causal, q_offset=q_offset, scale=scale, p=p, seed=0x9876543210 + seed,
              offset=(3 << 32) + 5)
    ref = dict(kw, kv_len=kv_len)
    if bias is not None:
        kw["table"] = ref["table"] = mk(bias[0], H, dtype=dtype)
        kw["relpos"], ref["relpos"] = ob.ob_relpos_init(*bias), bias
    if kv_len is not None:
        kw["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    return q, k, v, do, kw, ref


def _attn_run(q, k, v, do, kw):
    B, Lq, H, D = q.shape
    nan = lambda t: torch.full_like(t, math.nan)
    got = {"o": nan(q), "lse": torch.full((B, H, Lq), math.nan, device="cuda")}
    ob.ob_attn_fwd(q, k, v, got["o"], got["lse"], **kw)
    if do is not None:
        got.update(dq=nan(q), dk=nan(k), dv=nan(v))
        if kw.get("table") is not None:
            got["dtable"] = nan(kw["table"])
        ob.ob_attn_bwd(do, q, k, v, got["o"], got["lse"], got["dq"], got["dk"], got["dv"],
                       dtable=got.get("dtable"), **kw)
    assert ob.ob_attn_device_error() == 0
    return got


def _attn_check(q, k, v, do, kw, ref):
    got = _attn_run(q, k, v, do, kw)
    want, err = R.attention(q, k, v, do, bounds=True, **ref)
    for name in err:
        _within(got[name], want[name], err[name], name)
    lse, w = got["lse"].double(), want["lse"]
    assert torch.equal(lse == -math.inf, w == -math.inf)
    fin = w > -math.inf
    assert ((lse - w)[fin].abs() <= 2.0 ** -24 * 200 * (w[fin].abs() + 8)).all()
    return got


T5 = (32, 128, True)
ONE = (32, 128, False)

CASES = {
    "one": dict(Lq=1, Lk=1),
    "one_token": dict(B=2, H=4, Hkv=2, Lq=1, Lk=777, bias=ONE, causal=True),
    "one_key": dict(B=2, Lq=100, Lk=1, p=0.3),
    "tile": dict(Lq=128, Lk=128),
    "tile_d128": dict(Lq=128, Lk=128, D=128),
    "drop": dict(Lq=128, Lk=128, p=0.1),
    "drop_half": dict(Lq=200, Lk=136, p=0.5, D=128, dtype=F16),
    "drop_most": dict(Lq=64, Lk=300, p=0.98),
    "bias": dict(Lq=128, Lk=128, bias=T5),
    "bias_far": dict(H=1, Lq=600, Lk=700, bias=T5, q_offset=0),
    "bias_16": dict(H=3, Lq=257, Lk=257, bias=(16, 64, True), D=80, dtype=F16),
    "bias_wide": dict(H=1, Lq=300, Lk=2100, bias=(64, 520, False), q_offset=1800),
    "bias_wide_two": dict(H=1, Lq=900, Lk=1100, bias=(128, 260, True), q_offset=100),
    "drop_almost_all": dict(Lq=40, Lk=600, p=255 / 256, dtype=F16),
    "causal": dict(Lq=300, Lk=300, causal=True, D=128),
    "causal_more_keys": dict(Lq=65, Lk=400, causal=True, p=0.2, bias=ONE),
    "causal_fewer_keys": dict(Lq=400, Lk=65, causal=True, p=0.2, bias=ONE),
    "causal_offset": dict(Lq=150, Lk=150, causal=True, q_offset=-20),
    "lens": dict(B=6, Lq=130, Lk=260, kv_len=[260, 0, 1, 129, 128, 64], p=0.1, bias=T5),
    "lens_out_of_range": dict(B=3, Lq=20, Lk=30, kv_len=[-5, 31, 1 << 30]),
    "lens_causal": dict(B=4, Lq=190, Lk=190, kv_len=[190, 0, 100, 7], causal=True, D=128, p=0.1),
    "shared_heads": dict(B=2, H=8, Hkv=2, Lq=150, Lk=170, p=0.1, bias=T5, D=40),
    "one_kv_head": dict(B=2, H=6, Hkv=1, Lq=77, Lk=91, D=128, dtype=F16, causal=True),
    "d8": dict(Lq=70, Lk=70, D=8, bias=T5),
    "d72": dict(Lq=140, Lk=140, D=72, p=0.1),
    "d120": dict(Lq=66, Lk=195, D=120, p=0.1, dtype=F16),
    "odd": dict(B=3, H=3, Lq=333, Lk=517, p=0.1, bias=T5),
    "peaked": dict(Lq=200, Lk=200, spread=8.0, p=0.1),
    "scale": dict(Lq=100, Lk=100, scale=0.5, bias=T5),
    "many_blocks": dict(B=8, H=16, Lq=700, Lk=700, D=128),
    "many_blocks_causal": dict(B=8, H=16, Hkv=4, Lq=520, Lk=700, D=72, causal=True, p=0.1, bias=ONE),
    "long": dict(H=1, Lq=1111, Lk=1300, D=128, causal=True, p=0.1, bias=ONE),
    "long_64": dict(H=2, Lq=1025, Lk=1025, p=0.1, bias=T5),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    _attn_check(*_attn_case(**CASES[name]))


# Few queries: two, four or eight blocks share the keys of the same ones, some
# of them without any.
SHARED_KEYS = {
    "token": dict(H=2, Lq=1, Lk=3500, D=64, causal=True, bias=ONE),
    "token_d128": dict(B=2, H=2, Hkv=1, Lq=1, Lk=3333, D=128, kv_len=[3333, 65]),
    "lens": dict(B=3, H=2, Hkv=1, Lq=40, Lk=1700, D=128, p=0.1, bias=ONE, causal=True,
                 kv_len=[1700, 100, 0]),
    "causal_offset": dict(H=2, Lq=200, Lk=1600, D=40, causal=True, q_offset=-64, p=0.1),
    "four": dict(B=2, H=8, Lq=300, Lk=900, D=72, p=0.1, bias=T5, kv_len=[900, 333]),
    "two": dict(H=4, Lq=1000, Lk=800, D=64),
    "peaked": dict(H=2, Lq=130, Lk=1600, spread=8.0, p=0.1),
}


@pytest.mark.parametrize("name", SHARED_KEYS)
def test_attention_of_few_queries(name):
    _attn_check(*_attn_case(**SHARED_KEYS[name]))


def test_attention_repeats_bit_for_bit():
    c = _attn_case(B=3, H=4, Hkv=2, Lq=300, Lk=300, p=0.1, bias=T5, kv_len=[300, 17, 200])
    a = _attn_run(*c[:5])
    for _ in range(3):
        b = _attn_run(*c[:5])
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_attention_ignores_what_lies_past_the_lengths():
    """NaN and infinities in K and V past kv_len, and in the memory around the
    arrays, reach nothing."""
    q, k, v, do, kw, ref = _attn_case(B=3, H=2, Lq=100, Lk=200, kv_len=[0, 77, 130], p=0.1,
                                      bias=T5, D=80)
    clean = _attn_run(q, k, v, do, kw)
    pad = lambda t: torch.full((t.shape[0], t.shape[1] + 140, t.shape[2] + 1, t.shape[3] + 8),
                               math.nan, device="cuda", dtype=t.dtype)
    ins = []
    for t in (q, k, v, do):
        w = pad(t)
        s = w[:, :t.shape[1], :t.shape[2], :t.shape[3]]
        s.copy_(t)
        ins.append(s)
    for b, n in enumerate(ref["kv_len"]):
        ins[1][b, n:] = math.inf
        ins[2][b, n:] = math.nan
    dirty = _attn_run(*ins, kw)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    assert (dirty["o"][0] == 0).all() and (dirty["lse"][0] == -math.inf).all()
    assert (dirty["dk"][1, 77:] == 0).all() and (dirty["dv"][2, 130:] == 0).all()


def test_attention_strides():
    """[B, H, L, D] memory, slices of a fused projection, and outputs in wider
    buffers whose margins stay untouched."""
    q, k, v, do, kw, ref = _attn_case(B=2, H=4, Lq=90, Lk=90, p=0.1, D=64)
    want = _attn_run(q, k, v, do, kw)
    turned = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, do)]
    got = _attn_run(*turned, kw)
    assert all(torch.equal(want[n], got[n]) for n in want)
    fused = torch.stack([q, k, v], 2)  # [B, L, 3, H, D]
    wide = {n: torch.full((2, 95, 5, 72), 7.0, device="cuda", dtype=BF16)
            for n in ("o", "dq", "dk", "dv")}
    cut = {n: t[:, :90, :4, :64] for n, t in wide.items()}
    lse = torch.empty(2, 4, 90, device="cuda")
    qkv = fused.unbind(2)
    ob.ob_attn_fwd(*qkv, cut["o"], lse, **kw)
    ob.ob_attn_bwd(do, *qkv, cut["o"], lse, cut["dq"], cut["dk"], cut["dv"], **kw)
    for n in cut:
        assert torch.equal(cut[n], want[n]), n
        whole = wide[n].clone()
        whole[:, :90, :4, :64] = 7.0
        assert (whole == 7.0).all(), f"{n}: wrote outside"


def test_attention_nan_and_infinities_that_count():
    q, k, v, do, kw, _ = _attn_case(Lq=130, Lk=130, causal=True, D=64, H=1)
    q[0, 5, 0, 0] = math.nan
    got = _attn_run(q, k, v, do, kw)
    assert got["o"][0, 5].isnan().all()
    assert not got["o"][0, :5].isnan().any() and not got["o"][0, 6:].isnan().any()


def test_attention_extremes_of_the_scores():
    """Scores near the type's largest value: the softmax still sums to one."""
    q, k, v, do, kw, ref = _attn_case(Lq=64, Lk=96, D=64, H=1)
    q = q * 200
    k = k * 200
    got = _attn_run(q, k, torch.ones_like(v), None, kw)
    assert ((got["o"].double() - 1).abs() <= 2.0 ** -8).all()
    assert got["lse"].isfinite().all()


def test_attention_of_nothing():
    q, k, v, do, kw, _ = _attn_case(B=2, Lq=40, Lk=8, bias=T5, p=0.1)
    k, v = k[:, :0], v[:, :0]
    got = _attn_run(q, k, v, do, kw)
    assert (got["o"] == 0).all() and (got["lse"] == -math.inf).all()
    assert (got["dq"] == 0).all() and (got["dtable"] == 0).all()
    q, k, v, do, kw, _ = _attn_case(B=2, Lq=8, Lk=40, bias=T5, p=0.1)
    got = _attn_run(q[:, :0], k, v, do[:, :0], kw)
    assert (got["dk"] == 0).all() and (got["dv"] == 0).all() and (got["dtable"] == 0).all()


def test_attention_gradients_against_differences():
    """Directional derivatives: central differences of the 64-bit forward
    against the kernels' gradients, within the gradients' own bounds."""
    c = _attn_case(B=2, H=4, Hkv=2, Lq=70, Lk=90, D=64, dtype=F16, p=0.2, bias=T5,
                   kv_len=[90, 31])
    q, k, v, do, kw, ref = c
    got = _attn_run(q, k, v, do, kw)
    _, err = R.attention(q, k, v, do, bounds=True, **ref)
    mk = _gen(77)
    table = ref.pop("table")
    base = dict(q=q.double(), k=k.double(), v=v.double(), table=table.double())
    for name, eps in (("q", 1e-4), ("k", 1e-4), ("v", 1e-4), ("table", 1e-4)):
        e = mk(*base[name].shape).double()
        f = []
        for s in (1, -1):
            x = dict(base)
            x[name] = base[name] + s * eps * e
            f.append((R.attention(x["q"], x["k"], x["v"], table=x["table"], **ref)["o"]
                      * do.double()).sum())
        slope = (f[0] - f[1]) / (2 * eps)
        mine = (got["d" + name].double() * e).sum()
        slack = (err["d" + name] * e.abs()).sum() + 1e-5 * (1 + slope.abs())
        assert (slope - mine).abs() <= slack, (name, slope.item(), mine.item(), slack.item())


def test_operators_on_another_stream():
    """Everything runs on the stream it is given and on torch's current one."""
    q, k, v, do, kw, _ = _attn_case(B=2, H=4, Lq=200, Lk=200, p=0.1, bias=T5)
    want = _attn_run(q, k, v, do, kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _attn_run(q, k, v, do, kw)
    s.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in want)
    o = torch.empty_like(q)
    ob.ob_attn_fwd(q, k, v, o, stream=s, **kw)
    s.synchronize()
    assert torch.equal(o, want["o"])


def test_operators_in_a_graph():
    q, k, v, do, kw, _ = _attn_case(B=2, H=4, Lq=200, Lk=200, p=0.1, bias=T5)
    want = _attn_run(q, k, v, do, kw)
    got = {n: torch.zeros_like(t) for n, t in want.items()}
    ws = torch.empty(ob.ob_attn_workspace_bytes(q, k, relpos=kw["relpos"], table=kw["table"]),
                     dtype=torch.uint8, device="cuda")
    x, y = torch.ones(1000, device="cuda"), torch.zeros(1000, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ob.ob_attn_fwd(q, k, v, got["o"], got["lse"], **kw)
        ob.ob_attn_bwd(do, q, k, v, got["o"], got["lse"], got["dq"], got["dk"], got["dv"],
                       dtable=got["dtable"], workspace=ws, **kw)
        ob.ob_dropout(x, y, 0.5, 1, 2)
    for _ in range(2):
        for t in got.values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], got[n]) for n in want)
    assert set(y.unique().tolist()) == {0.0, 2.0}

"""The model-side operators on the GPU where their arguments are unusual:
streams, masked values, misaligned views, wide plans.  Against the 64-bit
definitions (tests/model_ref.py), or against calls whose results must be the
same bits."""
import math

import pytest
import torch

import model_ref as R
import momentum_compression_gb300 as ob
import test_gpu_model_ops as G

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


@pytest.mark.parametrize("handle", [False, True])
def test_backward_calls_on_two_streams(handle):
    """Both calls with scratch, on torch's current stream and on one that is passed, in
    turn and without waiting, each on its own inputs: the same bits as one after another."""
    rp = ob.ob_relpos_init(32, 128, True)
    cases = []
    for seed in range(2):
        mk = _gen(50 + seed)
        q, do = mk(4, 300, 8, 64, dtype=BF16), mk(4, 300, 8, 64, dtype=BF16)
        k, v = mk(4, 300, 2, 64, dtype=BF16), mk(4, 300, 2, 64, dtype=BF16)
        kw = dict(relpos=rp, table=mk(32, 8, dtype=BF16), p=0.1, seed=seed, offset=7)
        o, lse = torch.empty_like(q), torch.empty(4, 8, 300, device="cuda")
        ob.ob_attn_fwd(q, k, v, o, lse, **kw)
        cases.append((do, q, k, v, o, lse, kw, mk(8, 6, 300, 300, dtype=BF16)))

    def run(case, stream=None):
        do, q, k, v, o, lse, kw, dout = case
        out = [torch.empty_like(t) for t in (q, k, v, kw["table"])]
        out.append(torch.empty(32, 6, device="cuda"))
        return out, lambda: (
            ob.ob_attn_bwd(do, q, k, v, o, lse, *out[:3], dtable=out[3], stream=stream, **kw),
            ob.ob_relpos_bias_bwd(rp, dout, out[4], stream=stream))

    want = []
    for c in cases:
        out, call = run(c)
        call()
        torch.cuda.synchronize()
        want.append(out)
    side = torch.cuda.Stream()
    work = [[run(cases[0]), run(cases[1], side.cuda_stream if handle else side)]
            for _ in range(6)]
    torch.cuda.synchronize()
    for pair in work:
        for _, call in pair:
            call()
    torch.cuda.synchronize()
    assert ob.ob_attn_device_error() == 0
    for pair in work:
        for (out, _), w in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


# ---------------------------------------------------------------------------
# Masked places
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,Lk,off,lens", [(3, 200, 50, None), (1, 1600, 700, None),
                                            (1, 1500, 1000, [1500, 600, 0]), (300, 500, 100, None),
                                            (150, 333, -20, [333, 100, 50]), (40, 90, -60, None)])
def test_attention_ignores_keys_behind_the_last_query(D, Lq, Lk, off, lens):
    """Causal: a cache longer than what is filled.  Keys that no query sees may hold
    anything, and get no gradient."""
    B = len(lens) if lens else 2
    q, k, v, do, kw, _ = G._attn_case(B=B, H=4, Hkv=2, Lq=Lq, Lk=Lk, D=D, causal=True, q_offset=off,
                                      kv_len=lens, p=0.1, bias=G.ONE)
    clean = G._attn_run(q, k, v, do, kw)
    end = max(0, Lq + off)
    for t, junk in ((k, math.nan), (v, math.inf), (k, -math.inf), (v, math.nan)):
        t[:, end:] = junk
        dirty = G._attn_run(q, k, v, do, kw)
        for n in clean:
            assert torch.equal(clean[n], dirty[n]), n
    assert (dirty["dk"][:, end:] == 0).all() and (dirty["dv"][:, end:] == 0).all()


def _masked_table(table, rows, value):
    t = table.clone()
    t[list(rows)] = value
    return t


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,Lq,Lk", [(64, 130, 200), (128, 130, 200), (64, 1, 1500)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_attention_where_every_bias_is_the_types_extreme(dtype, D, Lq, Lk, sign):
    """A bias that is the same for all keys of a row changes nothing, be it the type's
    lowest or highest value."""
    case = dict(B=2, H=2, D=D, Lq=Lq, Lk=Lk, dtype=dtype, bias=G.T5, p=0.1, q_offset=Lk + 300,
                kv_len=[Lk, Lk // 3])
    q, k, v, do, kw, ref = G._attn_case(**case)
    far = 15  # the bucket of every distance here
    extreme = sign * torch.finfo(dtype).max
    kw["table"] = _masked_table(kw["table"], [far], extreme)
    got = G._attn_run(q, k, v, do, kw)
    ref["table"] = _masked_table(ref["table"].double(), [far], 0.0)
    want, err = R.attention(q, k, v, do, bounds=True, **ref)
    # The forward's weights are taken relative to a row's reference, whose difference from
    # the bias is exact: o's bound is that without a bias.  The backward's go by lse, near
    # 2^16: its rounding (2^-8) and that of its product with log2 e (2^-8), and the two
    # constants' own errors (2^-25 each, of 94548), make one factor of a row's weights of
    # 1 + 0.0105 at most.  The bounds hold `unit` times the magnitudes that it multiplies.
    G._within(got["o"], want["o"], err["o"], "o")
    for n in ("dq", "dk", "dv"):
        G._within(got[n], want[n], err[n] * (1 + 0.0105 / R.UNIT[dtype]), n)
    # every row's dS sums to zero: the factor multiplies what is left of that
    G._within(got["dtable"], want["dtable"], err["dtable"] * 1.02, "dtable")
    base = max(-65536.0, min(65536.0, extreme))
    assert ((got["lse"].double() - base - want["lse"]).abs() <= 0.02).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("low", ["lowest", "infinite"])
def test_attention_where_the_bias_masks(dtype, D, low):
    """Far buckets of the type's lowest value, or of -inf: their keys get no weight."""
    q, k, v, do, kw, ref = G._attn_case(B=2, H=3, D=D, Lq=230, Lk=260, dtype=dtype, bias=G.T5, p=0.1,
                                        kv_len=[260, 200])
    value = torch.finfo(dtype).min if low == "lowest" else -math.inf
    kw["table"] = _masked_table(kw["table"], [15, 31], value)
    # exp(-200) is no weight either, and keeps the bounds' magnitudes small
    ref["table"] = _masked_table(ref["table"].double(), [15, 31], -200.0)
    got = G._attn_run(q, k, v, do, kw)
    want, err = R.attention(q, k, v, do, bounds=True, **ref)
    for n in err:
        G._within(got[n], want[n], err[n], n)


def test_attention_where_every_bias_is_minus_infinity():
    """As a row without keys."""
    for D in (64, 128):
        q, k, v, do, kw, _ = G._attn_case(B=2, H=2, D=D, Lq=130, Lk=200, bias=G.T5, p=0.1,
                                          q_offset=500)
        kw["table"] = _masked_table(kw["table"], [15], -math.inf)
        got = G._attn_run(q, k, v, do, kw)
        assert (got["lse"] == -math.inf).all()
        for n in ("o", "dq", "dk", "dv", "dtable"):
            assert (got[n] == 0).all(), n


def test_dropout_of_strided_rows_through_autograd():
    """The same bits as of a contiguous copy, forward and backward."""
    from momentum_compression_gb300 import model as M
    for dtype in (F32, BF16):
        wide = _gen(21)(9, 4, 150, dtype=dtype)
        for cut in (lambda t: t[..., 5:138], lambda t: t[..., :128], lambda t: t[:, 1, 3:8],
                    lambda t: t.transpose(0, 1), lambda t: t[..., ::2]):
            x, res, dy = cut(wide), cut(wide * 2), cut(wide * 3)
            runs = []
            for make in (lambda t: t, lambda t: t.contiguous()):
                a, r = make(x).detach().requires_grad_(), make(res).detach().requires_grad_()
                y = M.dropout(a, 0.3, 5, 6, r)
                runs.append((y, *torch.autograd.grad(y, (a, r), make(dy))))
            assert all(torch.equal(a, b) for a, b in zip(*runs))
            assert runs[0][0].is_contiguous()


# ---------------------------------------------------------------------------
# Wide plans of the bias
# ---------------------------------------------------------------------------

def _plan_of_span(span, two):
    """A plan whose outermost buckets are `span` distances apart."""
    last = span // 2 if two else span
    nb = 64 if two else 32
    for D in range(last, 4 * last):
        if ob.ob_relpos_init(nb, D, two).first[31] == last:
            return nb, D, two
    raise AssertionError("no such plan")


# the forward looks buckets up in a map up to a span of 2048, and searches beyond
WIDE = [(32, 5000, False), (64, 3000, True), (256, 1 << 20, True), (2048, False), (2049, False),
        (2048, True), (2050, True)]


def _plan(p):
    return p if len(p) == 3 else _plan_of_span(*p)


@pytest.mark.parametrize("plan", WIDE)
@pytest.mark.parametrize("Lq,Lk,off", [(3, 9000, 6000), (70, 4100, 2000), (1, 2056, 5000), (40, 31, 2040)])
def test_wide_relpos_bias(plan, Lq, Lk, off):
    plan = _plan(plan)
    p = ob.ob_relpos_init(*plan)
    b = torch.from_numpy(R.buckets(Lq, Lk, off, *plan)).cuda()
    for out_type in (F32, BF16):
        table = _gen(9)(plan[0], 2)
        want = table.t()[:, b].to(out_type)
        for ld in (Lk, Lk + 3):
            whole = torch.full((2, Lq, ld), 7.0, device="cuda", dtype=out_type)
            ob.ob_relpos_bias(p, table, whole[..., :Lk], q_offset=off)
            assert torch.equal(whole[..., :Lk], want), (out_type, ld)
            assert (whole[..., Lk:] == 7.0).all(), "wrote past a row"


@pytest.mark.parametrize("plan", WIDE)
@pytest.mark.parametrize("Lq,Lk,off", [(3, 9000, 6000), (70, 4100, 2000), (40, 31, 2040)])
def test_wide_relpos_bias_gradient(plan, Lq, Lk, off):
    plan, N, H = _plan(plan), 3, 2
    p = ob.ob_relpos_init(*plan)
    b = torch.from_numpy(R.buckets(Lq, Lk, off, *plan)).cuda()
    for dtype, ld in ((F32, Lk), (F32, Lk + 3), (BF16, Lk), (BF16, Lk + 3)):
        dout = _gen(N)(N, H, Lq, ld, dtype=dtype)[..., :Lk]
        dt = torch.full((plan[0], H), 9.0, device="cuda")
        ob.ob_relpos_bias_bwd(p, dout, dt, q_offset=off)
        for h in range(H):
            x = dout[:, h].double()
            want = R.bucket_sums(x.sum(0), b, plan[0])
            # the longest chain of additions: 32 rows of N entries down a diagonal, a bucket's
            # 287 distances in a tile, 8 warps, at most 5 parts in a row, 32 sums
            bound = (32 * N + 332) * 2.0 ** -24 * R.bucket_sums(x.abs().sum(0), b, plan[0])
            bound = bound + R.UNIT[F32] * (want.abs() + bound)
            G._within(dt[:, h], want, bound, f"dtable of head {h}")


# ---------------------------------------------------------------------------
# How near the gradients are
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("case", [
    dict(B=8, H=4, Lq=27, Lk=27, D=64, causal=True), dict(B=8, H=4, Lq=200, Lk=27, D=80, causal=True, p=0.2),
    dict(B=6, H=4, Lq=139, Lk=139, D=32), dict(B=6, H=4, Hkv=2, Lq=90, Lk=16, D=128, p=0.1),
    dict(B=4, H=4, Lq=900, Lk=900, D=128, causal=True, p=0.1), dict(B=4, H=2, Hkv=1, Lq=300, Lk=256, D=64),
    dict(B=6, H=4, Lq=150, Lk=700, D=64, kv_len=[700, 200, 20, 64, 0, 130], p=0.1),
    dict(B=4, H=4, Lq=500, Lk=600, D=80, causal=True, q_offset=-60, kv_len=[600, 500, 70, 301]),
    dict(B=4, H=4, Lq=400, Lk=1000, D=32, causal=True, q_offset=100),
])
@pytest.mark.parametrize("bias", [False, True])
def test_gradients_are_as_near_as_two_roundings(dtype, case, bias):
    """An output is rounded to the type, and so is dS, the operand of its product.  By norm
    each is the error of rounding the exact gradient once (dS up to 1.1 times: its spread
    over a binade is another), so both are under sqrt(1 + 1.1^2) < 1.5 times it: no third
    error of that size, as rowsum(do o) of a rounded o would be where keys are few.  The
    table's gradient is summed from dS before it is rounded."""
    case = dict(case, dtype=dtype)
    if bias:
        case["bias"] = G.ONE if case.get("causal") else G.T5
    q, k, v, do, kw, ref = G._attn_case(**case)
    got = G._attn_run(q, k, v, do, kw)
    want = R.attention(q, k, v, do, **ref)
    for n in ("dq", "dk", "dv") + (("dtable",) if bias else ()):
        once = (want[n].to(dtype).double() - want[n]).norm()
        assert (got[n].double() - want[n]).norm() <= 1.5 * once, n

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

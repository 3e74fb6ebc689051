"""The model-side operators through torch's autograd, and the example that
trains an encoder with them and the 1-bit Adam step."""
import math
import os
import sys

import pytest
import torch

import model_ref as R
import momentum_compression_gb300 as ob
from momentum_compression_gb300 import model as M

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    from momentum_compression_gb300 import _build
    _build.build()


def test_autograd_functions_are_the_entry_points():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16).requires_grad_()
    q, k, v, table = r(2, 50, 4, 64), r(2, 60, 2, 64), r(2, 60, 2, 64), r(32, 4)
    rp = M.RelPos()
    o = M.attention(q, k, v, table=table, relpos=rp, p=0.1, seed=3, offset=4)
    do = torch.randn(o.shape, generator=g, device="cuda").to(o.dtype)
    # a transposed gradient, as a permuted consumer hands it back
    got = torch.autograd.grad(o, (q, k, v, table), do.transpose(1, 3).contiguous().transpose(1, 3))
    with torch.no_grad():
        o2, lse = torch.empty_like(o), torch.empty(2, 4, 50, device="cuda")
        want = [torch.empty_like(t) for t in (q, k, v, table)]
        kw = dict(relpos=rp.plan, table=table, p=0.1, seed=3, offset=4)
        ob.ob_attn_fwd(q, k, v, o2, lse, **kw)
        ob.ob_attn_bwd(do, q, k, v, o2, lse, *want[:3], dtable=want[3], **kw)
    assert torch.equal(o, o2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_dropout_and_bias():
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x, res, dy = (torch.randn(40, 72, generator=g, device="cuda") for _ in range(3))
    x.requires_grad_()
    res.requires_grad_()
    y = M.dropout(x, 0.25, 9, 10, res)
    dx, dres = torch.autograd.grad(y, (x, res), dy)
    kb, up = R.keep(0, x.numel(), 0.25, 9, 10)
    keep = torch.from_numpy(kb).cuda().view(40, 72)
    assert torch.equal(dres, dy)
    assert torch.equal(dx == 0, ~keep | (dy == 0))
    assert torch.allclose(dx, dy * keep * up, rtol=2 ** -22, atol=0)
    table = torch.randn(32, 3, generator=g, device="cuda").requires_grad_()
    rp = M.RelPos(32, 128, two_sided=False)
    b = M.relpos_bias(table, rp, 20, 30, q_offset=10)
    db = torch.randn(b.shape, generator=g, device="cuda")
    dt, = torch.autograd.grad(b, table, db)
    bk = torch.from_numpy(R.buckets(20, 30, 10, 32, 128, False)).cuda()
    assert torch.equal(b, table.detach().t()[:, bk])
    want = torch.stack([R.bucket_sums(db[h].double(), bk, 32) for h in range(3)], 1)
    assert (dt.double() - want).abs().max() <= 1e-6 * db.abs().sum()


def test_example_learns():
    """The loss falls from that of a uniform guess (log 64) through the warmup and
    the compressed steps."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_encoder
    finally:
        sys.path.pop(0)
    losses = train_encoder.train(steps=60, warmup=60, log=lambda s: None)
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(64)) < 1.0
    assert sum(losses[-10:]) / 10 < sum(losses[50:60]) / 10 < losses[0] - 0.5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,causal,lens,p", [(64, False, [90, 0, 33], 0.1), (128, True, None, 0.2),
                                             (128, False, [17, 90, 90], 0.0), (72, True, [90, 5, 64], 0.1)])
def test_autograd_of_attention_in_its_forms(dtype, D, causal, lens, p):
    """Lengths, causality, both types, every head size's kernels, views that start anywhere:
    within the bounds of the 64-bit definition."""
    g = torch.Generator(device="cuda")
    g.manual_seed(D)

    def make(L, H):
        flat = torch.randn(3 * L * (3 * H) * D + 1, generator=g, device="cuda").to(dtype)
        wide = flat[1:].view(3, L, 3 * H, D)  # off a 16-byte boundary
        return wide, wide[:, :, H:2 * H]

    views = [make(70, 4)[1], make(90, 2)[1], make(90, 2)[1]]
    q, k, v = (t.detach().requires_grad_() for t in views)
    plan = (32, 128, not causal)
    table = torch.randn(32, 4, generator=g, device="cuda").to(dtype).requires_grad_()
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(causal=causal, p=p, seed=77, offset=(1 << 32) + 3)
    o = M.attention(q, k, v, table=table, relpos=M.RelPos(*plan), kv_len=lengths, **kw)
    do = make(70, 4)[1]
    got = (o.detach(), *torch.autograd.grad(o, (q, k, v, table), do))
    assert ob.ob_attn_device_error() == 0
    want, err = R.attention(q.detach(), k.detach(), v.detach(), do, table=table.detach(), relpos=plan,
                            kv_len=lens, bounds=True, **kw)
    for x, n in zip(got, ("o", "dq", "dk", "dv", "dtable")):
        d = (x.double() - want[n]).abs()
        assert (d <= err[n]).all(), (n, (d - err[n]).max().item())

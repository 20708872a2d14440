"""GPU tests of latent attention rows whose every visible score is minus infinity:
softmax has no value there, so o is NaN (and with it what the gradients say), the log
sum of exp is -inf.  A query that sees nothing, for padding, missing pages or no tokens, keeps
its o of 0."""
import pytest
import torch

from test_latent_prompt import inputs, run
from test_latent_step import places

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WAYS = [("simt", F32), ("simt", BF), ("tc", BF)]
INF = float("inf")


@pytest.mark.parametrize("impl,dtype", WAYS)
@pytest.mark.parametrize("T", [1, 150, 300])
def test_prompt(impl, dtype, T):
    """The first token of a run sees itself alone; the others see it and themselves."""
    gen = torch.Generator().manual_seed(T)
    B, H, K, R, V = 2, 2, 64, 32, 64
    x, _ = inputs(B, T, H, K, R, V, dtype, gen, strided=False)
    d_o = torch.randn(B, T, H, V, generator=gen).to(dtype).cuda()
    seg = torch.ones(B, T, dtype=torch.int32)
    first = T // 2
    seg[0, :first] = 0
    seg[1] = 0
    x["q"][0, :, 0, 5] = 1.0
    x["q"][0, :, 1, 5] = 0.25
    clean = run(x, seg.cuda(), impl)
    x["k"][0, first, 0, 5] = -INF
    got = run(x, seg.cuda(), impl, d_o)
    assert got["o"][0, first, 0].isnan().all() and float(got["lse"][0, 0, first]) == -INF
    # the others give it a weight of 0
    assert torch.isfinite(got["o"][0, first + 1:]).all() and torch.isfinite(got["o"][0, :, 1]).all()
    assert torch.equal(got["o"][0, :, 1], clean["o"][0, :, 1])
    assert not got["o"][0, :first].any() and not got["o"][1].any()
    assert bool((got["lse"][1] == -INF).all()) and bool((got["lse"][0, :, :first] == -INF).all())
    assert got["dq"][0, first, 0].isnan().all() and got["dv"][0, first, 0].isnan().all()
    for n in ("dq", "dk", "dv", "dq_rope", "dk_rope"):
        assert not got[n][0, :first].any() and not got[n][1].any(), n
    assert torch.isfinite(got["dv"][0, :, 1]).all() and torch.isfinite(got["dq"][0, :, 1]).all()


@pytest.mark.parametrize("impl,dtype", WAYS)
@pytest.mark.parametrize("B,T,n", [(1, 1, 1), (1, 1, 40), (1, 1, 5000), (9, 1, 700), (1, 3, 700),
                                   (200, 2, 90), (1, 2, 3000)])
def test_step(impl, dtype, B, T, n):
    """All of a sequence's tokens at an infinity of the other sign for one head, in
    parts of many CTAs and of one; another sequence has no pages, another no tokens."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(B + T + n)
    H, C, R, page = 5, 128, 32, 16
    lengths = torch.full((B,), n, dtype=torch.int32)
    table, n_pages = places(lengths, page, -(-n // page), gen)
    new = torch.full((B,), T, dtype=torch.int32)
    if B > 2:
        table[1] = n_pages
        new[2], lengths[2] = 0, 0
    cache = torch.randn(n_pages, page, C + R, generator=gen).to(dtype).cuda()
    cache[..., 7] = -INF
    q = torch.randn(B, T, H, C, generator=gen).to(dtype)
    q[..., 7] = 0.0
    q[:, :, 2, 7] = 1.0
    # (a 0 times the infinity is not a number: the other heads' scores)
    r = torch.randn(B, T, H, R, generator=gen).to(dtype)
    o, lse = kda.latent_step(q.cuda(), r.cuda(), cache, table.cuda(), lengths.cuda(), scale=0.1,
                             new=new.cuda(), return_lse=True, impl=impl)
    some = [b for b in range(B) if B <= 2 or b not in (1, 2)]
    assert o[some][:, :, 2].isnan().all()
    assert bool((lse[some][:, 2] == -INF).all())
    if B > 2:
        assert not o[1:3].any() and bool((lse[1:3] == -INF).all())


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_step_where_the_last_pages_alone_are_there(impl, dtype):
    """A query whose only tokens with a page have scores of minus infinity, beside one whose
    tokens have none."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(3)
    C, page, n = 256, 16, 640
    for there in (True, False):
        table = torch.full((1, 40), -1, dtype=torch.int32)
        if there:
            table[0, 39] = 1
        cache = torch.randn(2, page, C, generator=gen).to(dtype).cuda()
        cache[..., 0] = INF
        q = torch.randn(1, 2, 3, C, generator=gen).to(dtype).cuda()
        q[..., 0] = -1.0
        lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
        o, lse = kda.latent_step(q, None, cache, table.cuda(), lengths, scale=1.0,
                                 return_lse=True, impl=impl)
        assert bool((lse == -INF).all())
        assert o.isnan().all() if there else not o.any()

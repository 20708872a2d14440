"""GPU tests of what the latent attention's documentation allows and the other tests do
not call: the largest and smallest sizes, shared pages, odd lengths and scales,
broadcast inputs, long packed rows, calls at once.  Tolerances as in latent64.py."""
import pytest
import torch

import latent64
from test_latent_prompt import compare, inputs, run
from test_latent_step import expect, places

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WAYS = [("simt", F32), ("simt", BF), ("tc", BF)]


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_many_sequences(impl, dtype):
    """More sequences than a CTA has threads, most of a few tokens, many idle."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(1)
    B, H, C, R, page = 701, 3, 128, 32, 16
    lengths = torch.randint(0, 40, (B,), generator=gen).int()
    lengths[::97] = 400
    new = torch.randint(0, 2, (B,), generator=gen).int()
    new[::97] = 1
    table, n_pages = places(lengths, page, 26, gen)
    cache = torch.randn(n_pages, page, C + R, generator=gen).to(dtype)
    q = torch.randn(B, 1, H, C, generator=gen).to(dtype)
    r = torch.randn(B, 1, H, R, generator=gen).to(dtype)
    got, lse = kda.latent_step(q.cuda(), r.cuda(), cache.cuda(), table.cuda(), lengths.cuda(),
                               scale=0.1, new=new.cuda(), return_lse=True, impl=impl)
    o, want = expect(q, r, cache, table, lengths, new, 0.1, impl, dtype)
    latent64.check(got, o, "o")
    latent64.check(lse, want, "lse")


@pytest.mark.parametrize("impl,dtype", WAYS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-20, 3.0])
def test_scales(impl, dtype, scale):
    """0 weighs all tokens alike; a negative scale turns the order round."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(2)
    C, H, page, n = 128, 5, 8, 150
    cache = torch.randn(19, page, C, generator=gen).to(dtype)
    table, lengths = torch.randperm(19, generator=gen).int()[None], torch.tensor([n]).int()
    q = (torch.randn(1, 2, H, C, generator=gen) / 4).to(dtype)
    got = kda.latent_step(q.cuda(), None, cache.cuda(), table.cuda(), lengths.cuda(), scale=scale,
                          impl=impl)
    o, _ = expect(q, None, cache, table, lengths, None, scale, impl, dtype)
    latent64.check(got, o, "step")
    x, x64 = inputs(1, 130, 2, 64, 32, 64, dtype, gen, strided=False)
    for n in ("q", "q_rope"):
        x[n].div_(4)
        x64[n] = x[n].double()
    d_o = torch.randn(1, 130, 2, 64, generator=gen).to(dtype).cuda()
    way = impl if scale > 0 or impl == "simt" else "auto"
    compare(run(x, None, way, d_o, scale=scale),
            latent64.prompt(x64, scale, None, impl, dtype, d_o.double()))


def test_tensor_cores_refuse_a_negative_scale():
    import gated_delta_rule_21_gb300 as kda
    x, _ = inputs(1, 20, 1, 64, 32, 64, BF, torch.Generator().manual_seed(3), strided=False)
    with pytest.raises(kda.KdaError):
        run(x, None, "tc", scale=-1.0)


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_shared_pages_and_odd_counts(impl, dtype):
    """Two sequences that share their first pages; counts beyond T, below 0; lengths
    below 0 and below the new tokens; pages far outside the cache."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(4)
    C, R, H, T, page = 128, 64, 3, 4, 16
    table = torch.tensor([[0, 1, 2, 3], [0, 1, 4, 5], [6, 7, 8, 9], [6, 7, 8, 9], [6, 7, 8, 9],
                          [2 ** 31 - 1, -2 ** 31, 6, 10]], dtype=torch.int32)
    lengths = torch.tensor([60, 50, 2, -5, 40, 64], dtype=torch.int32)
    new = torch.tensor([9, 4, 4, 4, -3, 2], dtype=torch.int32)
    cache = torch.randn(10, page, C + R, generator=gen).to(dtype)
    q = torch.randn(6, T, H, C, generator=gen).to(dtype)
    r = torch.randn(6, T, H, R, generator=gen).to(dtype)
    got, lse = kda.latent_step(q.cuda(), r.cuda(), cache.cuda(), table.cuda(), lengths.cuda(),
                               scale=0.1, new=new.cuda(), return_lse=True, impl=impl)
    o, want = expect(q, r, cache, table, lengths, new, 0.1, impl, dtype)
    latent64.check(got, o, "o")
    latent64.check(lse, want, "lse")
    assert not got[2, :2].any() and not got[3].any() and not got[4].any()


@pytest.mark.parametrize("page,stride", [(1, 0), (7, 0), (8, 0), (128, 64), (512, 8), (48, 0)])
def test_pages_of_any_size(page, stride):
    """bf16, whichever way serves them; tokens apart from each other."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(5)
    C, R, H, n = 256, 32, 9, 700
    wide = -(-n // page)
    whole = torch.randn(wide, page, C + R + stride, generator=gen).to(BF).cuda()
    cache = whole[..., :C + R]
    table, lengths = torch.randperm(wide, generator=gen).int()[None], torch.tensor([n]).int()
    q = torch.randn(1, 1, H, C, generator=gen).to(BF)
    r = torch.randn(1, 1, H, R, generator=gen).to(BF)
    got = kda.latent_step(q.cuda(), r.cuda(), cache, table.cuda(), lengths.cuda(), scale=0.08)
    tc = page & (page - 1) == 0 and page >= 8
    o, _ = expect(q, r, cache.cpu(), table, lengths, None, 0.08, "tc" if tc else "simt", BF)
    latent64.check(got, o, "o")
    if not tc:
        with pytest.raises(kda.KdaError):
            kda.latent_step(q.cuda(), r.cuda(), cache, table.cuda(), lengths.cuda(), scale=0.08,
                            impl="tc")


@pytest.mark.parametrize("impl,dtype", [("simt", F32), ("tc", BF)])
def test_queries_that_are_not_aligned_or_broadcast(impl, dtype):
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(6)
    C, R, H, page, n = 128, 64, 6, 16, 333
    cache = torch.randn(21, page, C + R, generator=gen).to(dtype)
    table, lengths = torch.randperm(21, generator=gen).int()[None], torch.tensor([n]).int()
    odd = torch.randn(1, 2, H, C + R + 1, generator=gen).to(dtype)
    one = torch.randn(1, 2, 1, C, generator=gen).to(dtype)
    for q, r in ((odd[..., 1:C + 1], odd[..., C + 1:]),
                 (one.expand(1, 2, H, C), odd[..., :1, C:C + R].expand(1, 2, H, R))):
        dq, dr = (t.cuda() if t.is_contiguous() else t for t in (q, r))
        base = odd.cuda()
        if q.stride(2) == 0:
            dq, dr = one.cuda().expand(1, 2, H, C), base[..., :1, C:C + R].expand(1, 2, H, R)
        else:
            dq, dr = base[..., 1:C + 1], base[..., C + 1:]
        got = kda.latent_step(dq, dr, cache.cuda(), table.cuda(), lengths.cuda(), scale=0.1,
                              impl=impl)
        o, _ = expect(q, r, cache, table, lengths, None, 0.1, impl, dtype)
        latent64.check(got, o, "o")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_keys_and_values_broadcast_over_heads(dtype):
    gen = torch.Generator().manual_seed(7)
    x, x64 = inputs(2, 77, 3, 64, 32, 64, dtype, gen, strided=False)
    for n in ("k", "v"):
        x[n] = x[n][:, :, :1].expand(-1, -1, 3, -1)
        x64[n] = x[n].double()
    d_o = torch.randn(2, 77, 3, 64, generator=gen).to(dtype).cuda()
    compare(run(x, None, "auto", d_o),
            latent64.prompt(x64, 96 ** -0.5, None, "simt", dtype, d_o.double()))


@pytest.mark.parametrize("impl,dtype", [("simt", F32), ("tc", BF)])
def test_long_packed_rows(impl, dtype):
    """Runs across the chunks that the table of runs is made in, one of them longer than
    a chunk: the packed row gives what the runs give by themselves."""
    gen = torch.Generator().manual_seed(8)
    T, H, K, R, V = 20011, 1, 32, 32, 32
    edges = [0, 5, 8190, 8193, 8200, 19000, 19003, 20000]
    x, _ = inputs(1, T, H, K, R, V, dtype, gen, strided=False)
    d_o = torch.randn(1, T, H, V, generator=gen).to(dtype).cuda()
    seg = torch.zeros(1, T, dtype=torch.int32)
    for i, (a, z) in enumerate(zip(edges, edges[1:])):
        seg[0, a:z] = 1 + i % 2
    seg[0, 8193:8195] = 0
    got = run(x, seg.cuda(), impl, d_o)
    for a, z in zip(edges, edges[1:]):
        a = 8195 if a == 8193 else a
        part = {n: None if t is None else t[:, a:z].contiguous() for n, t in x.items()}
        want = run(part, None, impl, d_o[:, a:z].contiguous())
        for n in want:
            w, g = want[n], got[n][:, :, a:z] if n == "lse" else got[n][:, a:z]
            # the tiles fall elsewhere: weights and outputs are rounded at other maxima
            tol = (4e-2 if dtype == BF else 1e-4) * float(w.abs().amax()) + 1e-4
            assert float((g - w).abs().max()) <= tol, (n, a, z)
    for n in got:
        if n != "lse":
            assert not got[n][:, 20000:].any() and not got[n][:, 8193:8195].any(), n


def test_a_long_row_of_many_heads():
    """8192 tokens of 32 heads: a few heads and rows against the plain form."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    T, H, K, R, V = 8192, 32, 128, 64, 128
    q = torch.randn(1, T, H, K + R, generator=gen, device="cuda").to(BF)
    kv = torch.randn(1, T, H, K + V, generator=gen, device="cuda").to(BF)
    x = {"q": q[..., :K], "q_rope": q[..., K:], "k": kv[..., :K], "v": kv[..., K:],
         "k_rope": torch.randn(1, T, R, generator=gen, device="cuda").to(BF)}
    d_o = torch.randn(1, T, H, V, generator=gen, device="cuda").to(BF)
    got = run(x, None, "tc", d_o)
    for h in (0, 13, 31):
        part = {n: (t if n == "k_rope" else t[:, :, h:h + 1]).double() for n, t in x.items()}
        want = latent64.prompt(part, (K + R) ** -0.5, None, "tc", BF, d_o[:, :, h:h + 1].double())
        for n, pair in want.items():
            if n == "dk_rope":
                continue               # the sum over all heads
            have = got[n][:, h:h + 1] if n == "lse" else got[n][:, :, h:h + 1]
            latent64.check(have, pair, f"{n} of head {h}")


@pytest.mark.parametrize("impl,dtype", [("simt", F32), ("tc", BF)])
def test_every_row_made_again(impl, dtype):
    """An infinite value at the first token: every row comes out not finite and is made
    again key by key, no wait of the others runs out, and the other columns are right."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(11)
    B, T, H, K, R, V = 1, 3000, 2, 64, 32, 64
    x, _ = inputs(B, T, H, K, R, V, dtype, gen, strided=False)
    clean = run(x, None, impl)
    x["v"][0, 0, :, 7] = float("inf")
    ws = kda.alloc_latent_workspace(B, T, H, R)
    got = run(x, None, impl, workspace=ws)
    assert kda.read_device_status(ws) == 0
    assert not torch.isfinite(got["o"][..., 7]).any()
    rest = [c for c in range(V) if c != 7]
    a, b = got["o"][..., rest].double(), clean["o"][..., rest].double()
    # weights rounded to bf16 or not, and the output's own rounding
    assert float((a - b).abs().max()) <= (3e-2 if dtype == BF else 1e-4) * float(b.abs().max())
    assert float((got["lse"] - clean["lse"]).abs().max()) <= 1e-3


def test_calls_at_once():
    """Two streams, each with its own workspace, while a third appends."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(10)
    made = []
    for s in range(2):
        lengths = torch.full((5,), 1000 + 300 * s, dtype=torch.int32)
        table, n_pages = places(lengths, 64, 24, gen)
        a = [torch.randn(5, 1, 32, 512, generator=gen).to(BF).cuda(),
             torch.randn(5, 1, 32, 64, generator=gen).to(BF).cuda(),
             torch.randn(n_pages, 64, 576, generator=gen).to(BF).cuda(), table.cuda(),
             lengths.cuda()]
        x, _ = inputs(1, 700, 4, 128, 64, 128, BF, gen, strided=False)
        d_o = torch.randn(1, 700, 4, 128, generator=gen).to(BF).cuda()
        made.append((a, x, d_o, kda.latent_step(*a, scale=0.07), run(x, None, "auto", d_o)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, (a, x, d_o, _, _) in zip(streams, made):
        got.append(([], []))
        for _ in range(4):
            got[-1][0].append(kda.latent_step(*a, scale=0.07, stream=s))
            got[-1][1].append(run(x, None, "auto", d_o, stream=s))
    torch.cuda.synchronize()
    for (steps, prompts), (_, _, _, o, want) in zip(got, made):
        for y in steps:
            assert torch.equal(y, o)
        for y in prompts:
            for n in want:
                assert torch.equal(y[n], want[n]), n


def test_refusals_with_tensors():
    import gated_delta_rule_21_gb300 as kda
    q = torch.zeros(2, 1, 4, 128, device="cuda")
    cache = torch.zeros(3, 16, 160, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="q_rope"):
        kda.latent_step(q, None, cache, table, n, scale=1.0)
    r = torch.zeros(2, 1, 4, 32, device="cuda")
    with pytest.raises(TypeError):
        kda.latent_step(q, r, cache, table.long(), n, scale=1.0)
    with pytest.raises(TypeError):
        kda.latent_step(q, r, cache.bfloat16(), table, n, scale=1.0)
    with pytest.raises(ValueError):
        kda.latent_step(q, r, cache, table, n[:1], scale=1.0)
    with pytest.raises(ValueError, match="contiguous"):
        kda.latent_step(q, r, cache.transpose(1, 2).contiguous().transpose(1, 2), table, n,
                        scale=1.0)
    with pytest.raises(ValueError, match="workspace"):
        kda.latent_step(q, r, cache, table, n, scale=1.0, workspace=torch.zeros(1 << 20))
    with pytest.raises(kda.KdaError):
        kda.latent_step(q, r, cache, table, n, scale=1.0,
                        workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="less than"):
        kda.latent_step(q, r, cache[..., :100], table, n, scale=1.0)
    with pytest.raises(ValueError, match="even"):
        kda.rotate(torch.zeros(1, 2, 5, device="cuda"), torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="empty"):
        kda.rotate(torch.zeros(0, 2, 4, device="cuda"), torch.zeros(2, device="cuda"))
    x = torch.zeros(1, 8, 2, 64, device="cuda")
    with pytest.raises(ValueError, match="together"):
        kda.latent_fwd(x, x, x, q_rope=x[..., :32])
    with pytest.raises(kda.KdaError):
        kda.latent_fwd(x[..., :48], x[..., :48], x)
    with pytest.raises(TypeError):
        kda.latent_fwd(x.half(), x.half(), x.half())
    with pytest.raises(kda.KdaError):
        kda.latent_fwd(x[:0], x[:0], x[:0])

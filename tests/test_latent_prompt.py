"""GPU tests of the expanded latent attention and its gradients against the
plain 64-bit form; the tolerances are derived in latent64.py."""
import pytest
import torch

import latent64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WAYS = [("simt", F32), ("simt", BF), ("tc", BF)]


def ids_of(kind, B, T, gen):
    """None, or segment ids with padding in front, between and behind."""
    if kind == "full":
        return None
    ids = torch.zeros(B, T, dtype=torch.int32)
    for b in range(B):
        t, run = (b * 3) % 5 if T > 8 else 0, 1
        while t < T:
            n = int(torch.randint(1, max(2, T // 3) + 1, (1,), generator=gen))
            ids[b, t:t + n] = run
            t += n + (int(torch.randint(0, 4, (1,), generator=gen)) if run % 2 else 0)
            run += 1
    if T > 2:
        ids[0, -(T // 8 + 1):] = 0
    if B > 1:
        ids[1] = 0                     # a row without a token
    return ids


def inputs(B, T, H, K, R, V, dtype, gen, strided=True):
    """Slices of projections, as a layer has them, and their 64-bit values."""
    def made(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(dtype).cuda()
    q = made(B, T, H, K + R, std=1.5)
    kv = made(B, T, H, K + V)
    x = {"q": q[..., :K], "k": kv[..., :K], "v": kv[..., K:],
         "q_rope": q[..., K:] if R else None, "k_rope": made(B, T, R) if R else None}
    if not strided:
        x = {n: None if t is None else t.contiguous() for n, t in x.items()}
    return x, {n: None if t is None else t.double() for n, t in x.items()}


def run(x, seg, impl, d_o=None, **kw):
    import gated_delta_rule_21_gb300 as kda
    rope = dict(q_rope=x["q_rope"], k_rope=x["k_rope"], segment_ids=seg, impl=impl, **kw)
    o, lse = kda.latent_fwd(x["q"], x["k"], x["v"], save_lse=True, **rope)
    got = {"o": o, "lse": lse}
    if d_o is not None:
        g = kda.latent_bwd(x["q"], x["k"], x["v"], o, lse, d_o, **rope)
        got.update(zip(("dq", "dk", "dv", "dq_rope", "dk_rope"), g))
    return got


def compare(got, want, what=""):
    for n, pair in want.items():
        latent64.check(got[n], pair, f"{what}{n}")


SHAPES = [(1, 1, 1, 128, 64, 128), (2, 2, 3, 128, 64, 128), (1, 63, 2, 128, 64, 128),
          (2, 128, 1, 128, 64, 128), (1, 129, 3, 128, 64, 128), (3, 200, 2, 128, 64, 128),
          (1, 257, 1, 128, 64, 128), (2, 513, 2, 128, 64, 128), (1, 70, 2, 32, 0, 32),
          (2, 150, 2, 64, 32, 64), (2, 190, 3, 32, 64, 128), (1, 300, 2, 128, 0, 64),
          (2, 100, 2, 64, 64, 32), (1, 257, 2, 128, 32, 128)]


@pytest.mark.parametrize("kind", ["full", "packed"])
@pytest.mark.parametrize("B,T,H,K,R,V", SHAPES)
@pytest.mark.parametrize("impl,dtype", WAYS)
def test_prompt(impl, dtype, B, T, H, K, R, V, kind):
    gen = torch.Generator().manual_seed(T * 7 + H)
    x, x64 = inputs(B, T, H, K, R, V, dtype, gen)
    seg = ids_of(kind, B, T, gen)
    d_o = torch.randn(B, T, H, V, generator=gen).to(dtype).cuda()
    got = run(x, None if seg is None else seg.cuda(), impl, d_o)
    want = latent64.prompt(x64, (K + R) ** -0.5, seg, impl, dtype, d_o.double())
    compare(got, want)


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_strides_and_scale(impl, dtype):
    """Heads before tokens, contiguous parts, a scale of the caller's; tensors whose
    rows are not aligned go to the CUDA cores by themselves."""
    gen = torch.Generator().manual_seed(3)
    B, T, H, K, R, V = 2, 140, 3, 64, 32, 64
    x, x64 = inputs(B, T, H, K, R, V, dtype, gen, strided=False)
    d_o = torch.randn(B, T, H, V, generator=gen).to(dtype).cuda()
    want = latent64.prompt(x64, 0.3, None, impl, dtype, d_o.double())
    compare(run(x, None, impl, d_o, scale=0.3), want, "contiguous ")
    turned = {n: None if t is None else t if n == "k_rope" else
              t.transpose(1, 2).contiguous().transpose(1, 2) for n, t in x.items()}
    compare(run(turned, None, impl, d_o, scale=0.3), want, "heads first ")
    odd = {}
    for n, t in x.items():
        w = torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=dtype, device="cuda")
        w[..., 1:] = t
        odd[n] = w[..., 1:]
    compare(run(odd, None, "simt" if impl == "simt" else "auto", d_o, scale=0.3), want, "odd ")


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_values_that_are_not_finite_stay_where_they_are_seen(impl, dtype):
    """NaN and infinities in padding reach nothing; in a token they reach those
    that see it, in its own run, and the gradients of what those see."""
    gen = torch.Generator().manual_seed(8)
    B, T, H, K, R, V = 1, 300, 2, 128, 64, 128
    x, _ = inputs(B, T, H, K, R, V, dtype, gen, strided=False)
    d_o = torch.randn(B, T, H, V, generator=gen).to(dtype).cuda()
    seg = torch.ones(B, T, dtype=torch.int32)
    seg[0, 90:100], seg[0, 100:230], seg[0, 230:] = 0, 2, 3
    clean = run(x, seg.cuda(), impl, d_o)
    for n, t in list(x.items()) + [("d_o", d_o)]:
        t[0, 90:100] = float("nan")
        t[0, 95] = float("inf")
    got = run(x, seg.cuda(), impl, d_o)
    for n in got:
        a, b = got[n], clean[n]
        on = torch.isfinite(b)
        same = bool((on == torch.isfinite(a)).all()) and (n == "lse" or bool(on.all()))
        near = bool(((a - b)[on].abs() <= 1e-2 * b[on].abs().amax()).all())
        assert same and near, n
    # a value in the middle of the second run
    x["v"][0, 150, 1, 5] = float("inf")
    got = run(x, seg.cuda(), impl, d_o)
    bad = ~torch.isfinite(got["o"])
    assert bad[0, 150:230, 1, 5].all() and int(bad.sum()) == 80
    for n in ("dq", "dq_rope"):          # of the tokens that see it
        bad = ~torch.isfinite(got[n])
        assert bad[0, 150:230, 1].all() and not bad[0, :150].any() and not bad[0, 230:].any()
        assert not bad[:, :, 0].any()
    bad = ~torch.isfinite(got["dk"])     # of what those see: the run up to the last
    assert bad[0, 100:230, 1].all() and not bad[0, :100].any() and not bad[0, 230:].any()
    bad = ~torch.isfinite(got["dv"])     # weights and d_o are finite
    assert not bad.any()


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_far_apart_scores(impl, dtype):
    """Scores that grow along the row (the running maximum moves at every tile)
    and fall along it; weights that underflow."""
    gen = torch.Generator().manual_seed(9)
    B, T, H, K, R, V = 1, 400, 2, 64, 0, 64
    x, _ = inputs(B, T, H, K, R, V, dtype, gen, strided=False)
    for sign in (1.0, -1.0):
        x["q"].zero_()
        x["k"].zero_()
        x["q"][..., 0] = 8.0
        x["k"][..., 0] = (sign * torch.arange(T, device="cuda") / 2).to(dtype)[None, :, None]
        x64 = {n: None if t is None else t.double() for n, t in x.items()}
        d_o = torch.randn(B, T, H, V, generator=gen).to(dtype).cuda()
        got = run(x, None, impl, d_o)
        # scores of up to 200 take 2^-24 of that in fp32 (twice in the difference to lse)
        want = latent64.prompt(x64, K ** -0.5, None, impl, dtype, d_o.double())
        for n, (ref, tol) in want.items():
            extra = 1e-4 if n == "lse" else 1e-4 * (ref.abs().amax() + 1)
            latent64.check(got[n], (ref, tol + extra), n)


def test_gradients_against_differences():
    """fp32: the directional difference quotient of <o, d_o>, made in 64 bits from
    the plain form, against the kernels' gradients."""
    gen = torch.Generator().manual_seed(4)
    B, T, H, K, R, V = 1, 90, 2, 32, 32, 32
    x, x64 = inputs(B, T, H, K, R, V, F32, gen, strided=False)
    d_o = torch.randn(B, T, H, V, generator=gen).cuda()
    seg = ids_of("packed", B, T, gen)
    got = run(x, seg.cuda(), "simt", d_o)
    e = 1e-5

    def loss(y):
        return float((latent64.prompt(y, (K + R) ** -0.5, seg)["o"][0] * d_o.double()).sum())

    for n in ("q", "k", "v", "q_rope", "k_rope"):
        u = torch.randn(x[n].shape, generator=gen, dtype=torch.float64).cuda()
        up, down = (loss({**x64, n: x64[n] + s * e * u}) for s in (1, -1))
        g = got["d" + n].double()
        # the quotient is off by e^2 of a third derivative and 1e-16 / e of the sum's terms
        assert abs((up - down) / (2 * e) - float((g * u).sum())) <= 1e-5 * float((g * u).abs().sum())


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_calls_agree_bit_for_bit_and_in_a_graph(impl, dtype):
    """Repeated, on another stream, captured and replayed on new values."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(12)
    B, T, H, K, R, V = 2, 333, 2, 128, 64, 128
    x, _ = inputs(B, T, H, K, R, V, dtype, gen, strided=False)
    d_o = torch.randn(B, T, H, V, generator=gen).to(dtype).cuda()
    seg = ids_of("packed", B, T, gen).cuda()
    ws = kda.alloc_latent_workspace(B, T, H, R, backward=True)
    first = run(x, seg, impl, d_o, workspace=ws)
    again = run(x, seg, impl, d_o, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(x, seg, impl, d_o, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(x, seg, impl, d_o, workspace=ws)
    second = {n: None if t is None else torch.randn_like(t) for n, t in x.items()}
    want = run(second, seg, impl, d_o)
    graph.replay()
    torch.cuda.synchronize()
    for n in first:
        assert torch.equal(first[n], again[n]) and torch.equal(first[n], other[n]), n
        assert torch.equal(first[n], held[n]), n
    for n, t in x.items():
        t.copy_(second[n])
    graph.replay()
    torch.cuda.synchronize()
    for n in first:
        assert torch.equal(want[n], held[n]), n
    assert kda.read_device_status(ws) == 0


def test_out_and_no_lse():
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(1)
    x, _ = inputs(1, 50, 2, 64, 32, 64, BF, gen)
    o, _ = kda.latent_fwd(x["q"], x["k"], x["v"], q_rope=x["q_rope"], k_rope=x["k_rope"],
                          save_lse=True)
    out = torch.empty_like(o)
    got = kda.latent_fwd(x["q"], x["k"], x["v"], q_rope=x["q_rope"], k_rope=x["k_rope"], out=out)
    assert got is out and torch.equal(out, o)

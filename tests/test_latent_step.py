"""GPU tests of the absorbed latent attention over the paged cache against the
plain 64-bit form; the tolerances are derived in latent64.py."""
import pytest
import torch

import latent64
from test_latent_rotate import frequencies

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WAYS = [("simt", F32), ("simt", BF), ("tc", BF)]


def places(lengths, page, wide, gen, spare=3):
    """A page table over shuffled pages, -1 behind each sequence's last."""
    n_pages = sum(-(-int(n) // page) for n in lengths) + spare
    order = torch.randperm(n_pages, generator=gen)
    table, k = torch.full((len(lengths), wide), -1, dtype=torch.int32), 0
    for b, n in enumerate(lengths):
        m = min(-(-int(n) // page), wide)
        table[b, :m] = order[k:k + m].int()
        k += m
    return table, n_pages


def gathered(cache, table, b, length):
    """The tokens of a sequence in 64 bits, and whether their pages exist."""
    page = cache.shape[1]
    n = min(max(length, 0), table.shape[1] * page)
    at = torch.arange(n)
    pg = table[b].long()[at // page]
    there = (pg >= 0) & (pg < cache.shape[0])
    tokens = cache[torch.where(there, pg, 0), at % page].double()
    return torch.where(there[:, None], tokens, 0.0), there


def expect(q, q_rope, cache, table, lengths, new, scale, impl, dtype):
    B, T, H, C = q.shape
    o, lse = [torch.zeros(B, T, H, C, dtype=torch.float64) for _ in range(2)], \
        [torch.full((B, H, T), v, dtype=torch.float64) for v in (-torch.inf, 0.0)]
    for b in range(B):
        n = T if new is None else min(max(int(new[b]), 0), T)
        if n == 0:
            continue
        tokens, there = gathered(cache, table, b, int(lengths[b]))
        if len(tokens) == 0:
            continue
        seen = (int(lengths[b]) - n + 1 + torch.arange(T)).clamp(max=tokens.shape[0])
        seen[n:] = 0
        got = latent64.step(q[b].double(), None if q_rope is None else q_rope[b].double(), tokens,
                            there, seen, scale, impl, dtype)
        o[0][b], o[1][b] = got[0]
        lse[0][b], lse[1][b] = got[1][0].t(), got[1][1].t()
    return o, lse


CASES = [  # B, T, H, C, R, page, longest
    (1, 1, 32, 512, 64, 64, 1000), (1, 1, 1, 128, 0, 16, 1), (3, 1, 5, 512, 64, 64, 300),
    (2, 4, 6, 128, 32, 16, 200), (4, 3, 33, 256, 64, 32, 150), (9, 1, 32, 512, 64, 64, 700),
    (200, 1, 8, 512, 64, 64, 90), (2, 2, 64, 512, 64, 128, 2000), (1, 1, 16, 512, 32, 8, 129),
    (2, 6, 3, 256, 0, 256, 400), (1, 130, 2, 128, 64, 16, 260), (1, 1, 20, 512, 64, 64, 40000)]


@pytest.mark.parametrize("impl,dtype", WAYS)
@pytest.mark.parametrize("B,T,H,C,R,page,most", CASES)
def test_step(B, T, H, C, R, page, most, impl, dtype):
    """Ragged lengths, idle sequences, pages that are not there, a length beyond
    the table; the unused places of the cache hold NaN."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(B * 17 + T * 3 + H)
    lengths = torch.randint(1, most + 1, (B,), generator=gen).int()
    lengths[0] = most
    new = torch.randint(0, T + 1, (B,), generator=gen).int() if B > 1 else None
    if B > 1:
        new[0], lengths[1], new[1] = T, min(most, 1), min(T, 1)
    if B > 2:
        lengths[2], new[2] = 0, 0
    wide = -(-most // page) + 1
    table, n_pages = places(lengths, page, wide, gen)
    cache = torch.full((n_pages, page, C + R), float("nan"))
    for b in range(B):
        for k in range(-(-int(lengths[b]) // page)):
            m = min(page, int(lengths[b]) - k * page)
            cache[table[b, k], :m] = torch.randn(m, C + R, generator=gen)
    if B > 3:
        table[3, 0] = -1 if B % 2 else n_pages      # its first tokens are nowhere
        lengths[4 % B] = wide * page + 5 if B > 4 else lengths[3]
    cache = cache.to(dtype)
    if B > 4:     # a length beyond the table: all its pages are there
        for k in range(wide):
            if table[4, k] < 0:
                table[4, k] = table[0, 0]
        cache[table[4].long()] = torch.randn(wide, page, C + R, generator=gen).to(dtype)
    std = 2.0 * (192 / (C + R)) ** 0.5
    wide_q = (torch.randn(B, T, H, C + R, generator=gen) * std).to(dtype)
    q, q_rope = wide_q[..., :C], (wide_q[..., C:] if R else None)
    dev = wide_q.cuda()
    ws = kda.alloc_latent_step_workspace(B, T, H, C)
    got, lse = kda.latent_step(dev[..., :C], dev[..., C:] if R else None, cache.cuda(),
                               table.cuda(), lengths.cuda(), scale=192 ** -0.5,
                               new=None if new is None else new.cuda(), return_lse=True,
                               workspace=ws, impl=impl)
    o, want_lse = expect(q, q_rope, cache, table, lengths, new, 192 ** -0.5, impl, dtype)
    assert kda.read_device_status(ws) == 0
    latent64.check(got, o, "o")
    latent64.check(lse, want_lse, "lse")


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_scores_that_move_the_maximum(impl, dtype):
    """Scores that rise and fall by much along the cache, and a few large ones."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(5)
    n, C, H, page = 1500, 128, 40, 64
    cache = torch.randn(-(-n // page), page, C, generator=gen)
    flat = cache.view(-1, C)
    flat[:, 0] = torch.arange(flat.shape[0]) / 16
    flat[700, 1] = 60.0
    q = torch.zeros(1, 1, H, C)
    q[..., 0] = torch.linspace(-2, 2, H)
    q[..., 1] = 1.0
    q, cache = q.to(dtype), cache.to(dtype)
    table = torch.arange(cache.shape[0]).int()[None]
    lengths = torch.tensor([n], dtype=torch.int32)
    got, lse = kda.latent_step(q.cuda(), None, cache.cuda(), table.cuda(), lengths.cuda(),
                               scale=1.0, return_lse=True, impl=impl)
    o, want = expect(q, None, cache, table, lengths, None, 1.0, impl, dtype)
    # scores of up to 190: 2^-24 of that a rounding, in the products with log2 e too
    latent64.check(got, (o[0], o[1] + 2e-4 * o[0].abs().amax()), "o")
    latent64.check(lse, (want[0], want[1] + 1e-4), "lse")


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_values_that_are_not_finite_reach_the_tokens_that_see_them(impl, dtype):
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(6)
    C, R, H, T, page = 256, 64, 7, 4, 32
    lengths = torch.tensor([300, 90], dtype=torch.int32)
    table, n_pages = places(lengths, page, 12, gen)
    cache = torch.randn(n_pages, page, C + R, generator=gen).to(dtype)
    q = torch.randn(2, T, H, C, generator=gen).to(dtype).cuda()
    r = torch.randn(2, T, H, R, generator=gen).to(dtype).cuda()

    def go():
        return kda.latent_step(q, r, cache.cuda(), table.cuda(), lengths.cuda(), scale=0.05,
                               impl=impl)
    clean = go()
    at = 298                                    # the third of the four new tokens
    cache[table[0, at // page], at % page, 5] = float("inf")
    got = go()
    assert torch.equal(got[1], clean[1])
    assert bool((got[0, :2] - clean[0, :2]).abs().max() <= 1e-2)
    assert not torch.isfinite(got[0, 2:, :, 5]).any()
    q[1, 1, 2] = float("nan")                   # a query of its own
    got = go()
    assert got[1, 1, 2].isnan().all() and torch.equal(got[1, 2:], clean[1, 2:])
    assert torch.equal(got[1, 1, 3:], clean[1, 1, 3:])


@pytest.mark.parametrize("impl", ["simt", "tc"])
def test_cache_with_strides_and_past_32_bits(impl):
    """Pages of a cache that holds several layers, behind 2^31 values."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(7)
    C, R, page, layers = 512, 64, 64, 4
    n_pages = 2 ** 31 // (page * (C + R) * layers) + 8
    whole = torch.full((n_pages, layers, page, C + R), float("nan"), dtype=BF, device="cuda")
    cache = whole[:, 2]
    lengths = torch.tensor([200], dtype=torch.int32)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2, n_pages - 5]], dtype=torch.int32)
    for k in range(4):
        m = min(page, 200 - k * page)
        cache[int(table[0, k]), :m] = torch.randn(m, C + R, generator=gen).to(BF).cuda()
    q = torch.randn(1, 8, 1, C, generator=gen).to(BF).transpose(1, 2)     # [1, 1, 8, C]
    r = torch.randn(1, 1, 8, R, generator=gen).to(BF)
    got = kda.latent_step(q.cuda(), r.cuda(), cache, table.cuda(), lengths.cuda(), scale=0.1,
                          impl=impl)
    few = torch.stack([cache[int(p)].cpu() for p in table[0]])
    o, _ = expect(q, r, few, torch.arange(4).int()[None], lengths, None, 0.1, impl, BF)
    latent64.check(got, o, "o")


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_a_captured_call_follows_the_lengths(impl, dtype):
    """Append and step captured together and replayed while the texts grow; the
    same on another stream; repeated calls agree bit for bit."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(8)
    B, H, C, R, page, wide = 3, 6, 128, 64, 16, 24
    lengths = torch.tensor([1, 130, 255], dtype=torch.int32)
    table = torch.randperm(B * wide, generator=gen).view(B, wide).int()
    freq = frequencies(R).cuda()
    cache = torch.randn(B * wide, page, C + R, generator=gen).to(dtype).cuda()
    first = cache.clone()
    ws = kda.alloc_latent_step_workspace(B, 1, H, C)
    t = {n: torch.randn(*s, generator=gen).to(dtype).cuda() for n, s in dict(
        latent=(B, 1, C), k=(B, 1, R), q=(B, 1, H, C), r=(B, 1, H, R)).items()}
    dev_table, dev_lengths = table.cuda(), lengths.cuda()

    def go(cache, lengths, **kw):
        r = kda.latent_append(t["latent"], t["k"], cache, dev_table, lengths, inv_freq=freq,
                              q_rope=t["r"], stream=kw.get("stream"))
        return kda.latent_step(t["q"], r, cache, dev_table, lengths, scale=0.1, impl=impl, **kw)

    want, grown = [], first.clone()
    for i in range(4):
        want.append(go(grown, (lengths + 40 * i).cuda()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = first.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = go(other, dev_lengths, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = go(cache, dev_lengths, workspace=ws)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want[i]), i
        dev_lengths += 40
    assert torch.equal(cache, grown) and kda.read_device_status(ws) == 0


def test_two_captured_graphs_share_a_workspace():
    """One workspace serves graphs that run one after another."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(10)
    C, R, page = 512, 64, 64
    ws = kda.alloc_latent_step_workspace(4, 1, 32, C)
    made = []
    for B, n in ((1, 3000), (4, 500)):
        lengths = torch.full((B,), n, dtype=torch.int32)
        table, n_pages = places(lengths, page, -(-n // page), gen)
        a = [torch.randn(B, 1, 32, C, generator=gen).to(BF).cuda(),
             torch.randn(B, 1, 32, R, generator=gen).to(BF).cuda(),
             torch.randn(n_pages, page, C + R, generator=gen).to(BF).cuda(), table.cuda(),
             lengths.cuda()]
        want = kda.latent_step(*a, scale=0.07)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = kda.latent_step(*a, scale=0.07, workspace=ws)
        made.append((graph, held, want, a))
    for _ in range(3):
        for graph, held, want, _ in made:
            graph.replay()
    torch.cuda.synchronize()
    for _, held, want, _ in made:
        assert torch.equal(held, want)


def test_the_absorbed_form_is_the_expanded_one():
    """A prompt through latent_fwd with expanded keys and values, and its last
    tokens through append and step on the latents: the same layer, fp32."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(11)
    B, T, n, H, K, R, V, C, page = 2, 90, 5, 3, 64, 32, 64, 128, 16
    latent = torch.randn(B, T, C, generator=gen).cuda()
    k_up, v_up = (torch.randn(H, C, d, generator=gen).cuda() * C ** -0.5 for d in (K, V))
    q, q_rope = torch.randn(B, T, H, K, generator=gen).cuda(), torch.randn(
        B, T, H, R, generator=gen).cuda()
    k_rope, freq = torch.randn(B, T, R, generator=gen).cuda(), frequencies(R).cuda()
    k, v = (torch.einsum("btc,hcd->bthd", latent.double(), u.double()).float() for u in (k_up, v_up))
    whole = kda.latent_fwd(q, k, v, q_rope=kda.rotate(q_rope, freq), k_rope=kda.rotate(k_rope, freq))
    table, n_pages = places([T] * B, page, -(-T // page), gen)
    table = table.cuda()
    cache = torch.full((n_pages, page, C + R), float("nan"), device="cuda")

    def some(lo, hi):
        at = torch.full((B,), hi, dtype=torch.int32, device="cuda")
        r = kda.latent_append(latent[:, lo:hi], k_rope[:, lo:hi], cache, table, at,
                              inv_freq=freq, q_rope=q_rope[:, lo:hi])
        absorbed = torch.einsum("bthd,hcd->bthc", q[:, lo:hi].double(), k_up.double()).float()
        o = kda.latent_step(absorbed, r, cache, table, at, scale=(K + R) ** -0.5)
        return torch.einsum("bthc,hcd->bthd", o.double(), v_up.double()).float()

    got = torch.cat([some(0, T - n)] + [some(T - n + i, T - n + i + 1) for i in range(n)], 1)
    # scores 2e-5 off either way (latent64.py), the products around them in 64 bits
    assert float((got - whole).abs().max()) <= 1e-4 * float(whole.abs().max())

"""GPU tests of the position rotation and of appending to the paged cache.

Tolerance of a rotated value: the reduced angle is rounded to fp32 once (2^-24 of
at most pi), cos and sin are a few ulp off, two products and a sum are rounded:
5e-7 of |a| + |b|, and the output's own rounding."""
import pytest
import torch

import latent64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def near(got, want, dtype, sizes, what):
    latent64.check(got, (want, latent64.half_step(dtype) * want.abs() + 5e-7 * sizes), what)


def sizes(x, pairs):
    n = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :n], x[..., n:])
    s = a.abs() + b.abs()
    return torch.stack([s, s], -1).flatten(-2) if pairs else torch.cat([s, s], -1)


def frequencies(dim):
    return (10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) * 2 / dim)).float()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("B,T,H,dim", [(1, 1, 1, 2), (2, 7, 3, 6), (1, 300, 5, 64), (3, 33, 1, 32),
                                       (2, 5, 4, 256), (1, 2000, 2, 64), (2, 9, 2, 24)])
def test_rotate(B, T, H, dim, pairs, dtype):
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(T + dim)
    x = torch.randn(B, T, H, dim, generator=gen).to(dtype)
    freq = frequencies(dim)
    for at in (None, torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, T), generator=gen).int(),
               torch.randint(0, 1 << 20, (B, T), generator=gen).int()):
        where = torch.arange(T).expand(B, T) if at is None else at
        for inverse in (False, True):
            y = kda.rotate(x.cuda(), freq.cuda(), positions=None if at is None else at.cuda(),
                           pairs=pairs, inverse=inverse)
            want = latent64.rotate(x.double(), where[..., None], freq, pairs, inverse)
            near(y, want, dtype, sizes(x.double(), pairs), f"{pairs} {inverse}")


def test_rotate_in_place_strided_and_three_dimensional():
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(2)
    wide = torch.randn(2, 40, 3, 200, generator=gen)
    freq = frequencies(64)
    for dtype, lo in ((BF, 128), (BF, 129), (F32, 100), (F32, 101)):
        w = wide.to(dtype).cuda()
        before = w.clone()
        x = w[..., lo:lo + 64]
        want = latent64.rotate(x.double().cpu(), torch.arange(40)[:, None].expand(2, 40, 1), freq)
        got = kda.rotate(x, freq.cuda(), out=x)
        assert got.data_ptr() == x.data_ptr()
        near(x, want, dtype, sizes(before[..., lo:lo + 64].double().cpu(), True), "in place")
        assert torch.equal(w[..., :lo], before[..., :lo])
        assert torch.equal(w[..., lo + 64:], before[..., lo + 64:])
        flat = before[:, :, 0, lo:lo + 64]
        assert torch.equal(kda.rotate(flat, freq.cuda()), x[:, :, 0])


def test_rotate_back_is_the_gradient():
    """<rotate(x), g> = <x, rotate back(g)>, and back undoes it."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(5)
    x, g = (torch.randn(2, 30, 4, 64, generator=gen).cuda() for _ in range(2))
    freq = frequencies(64).cuda()
    for pairs in (True, False):
        y = kda.rotate(x, freq, pairs=pairs)
        dx = kda.rotate(g, freq, pairs=pairs, inverse=True)
        a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
        assert abs(float(a - b)) <= 1e-6 * float((y.double() * g.double()).abs().sum())
        again = kda.rotate(y, freq, pairs=pairs, inverse=True)
        assert float((again - x).abs().max()) <= 2e-6 * float(x.abs().max()) * 2


def plain_append(cache, latent, k_rope, table, lengths, new, freq, pairs):
    """The cache after it, in the cache's type, and where keys were rotated."""
    n_pages, page, _ = cache.shape
    want, turned = cache.double().clone(), torch.zeros(cache.shape, dtype=torch.bool)
    B, T, C = latent.shape
    for b in range(B):
        n = T if new is None else min(max(int(new[b]), 0), T)
        for t in range(n):
            at = int(lengths[b]) - n + t
            if at < 0 or at // page >= table.shape[1]:
                continue
            pg = int(table[b, at // page])
            if not 0 <= pg < n_pages:
                continue
            want[pg, at % page, :C] = latent[b, t].double()
            if k_rope is not None:
                r = k_rope[b, t].double()
                if freq is not None:
                    r = latent64.rotate(r, torch.tensor(at), freq, pairs)
                want[pg, at % page, C:] = r
                turned[pg, at % page, C:] = True
    return want, turned


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,C,R,page,odd", [
    (1, 1, 4, 512, 64, 64, False), (3, 5, 2, 128, 32, 16, False), (2, 70, 3, 256, 64, 32, False),
    (2, 9, 1, 100, 6, 7, True), (2, 4, 2, 128, 0, 16, False), (40, 1, 3, 512, 64, 64, False),
    (2, 33, 2, 128, 64, 128, True)])
def test_append(B, T, H, C, R, page, odd, dtype):
    """Ragged rows, idle ones, pages outside the cache, a length that the table
    does not hold, a position before 0; nothing else is touched."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(B * 31 + T)
    wide, n_pages = 2 + -(-2 * T // page), B * (2 + -(-2 * T // page)) + 2
    table = torch.randperm(n_pages, generator=gen)[:B * wide].view(B, wide).int()
    new = torch.randint(0, T + 1, (B,), generator=gen).int()
    lengths = new + torch.randint(0, T + 1, (B,), generator=gen).int()
    new[0], lengths[0] = T, wide * page + 1        # its last token has no place
    if B > 1:
        table[1, -1], table[1, 0] = n_pages, -1
        lengths[1], new[1] = T, T
    if B > 2:
        lengths[2], new[2] = 2, T                  # begins before position 0
    pad = 1 if odd else 0
    down = torch.randn(B, T, C + R + 3, generator=gen).to(dtype).cuda()[..., pad:C + R + pad] \
        if odd else torch.randn(B, T, C + R, generator=gen).to(dtype).cuda()
    latent, k_rope = down[..., :C], (down[..., C:] if R else None)
    q = torch.randn(B, T, H, R, generator=gen).to(dtype).cuda() if R else None
    for pairs in (True, False):
        for n in (new, None):
            cache = torch.randn(n_pages, page, C + R, generator=gen).to(dtype).cuda()
            want, turned = plain_append(cache.cpu(), latent.cpu(), None if k_rope is None else
                                        k_rope.cpu(), table, lengths, n,
                                        frequencies(R) if R else None, pairs)
            got = kda.latent_append(latent, k_rope, cache, table.cuda(), lengths.cuda(),
                                    inv_freq=frequencies(R).cuda() if R else None,
                                    new=None if n is None else n.cuda(), q_rope=q, pairs=pairs)
            out = cache.double().cpu()
            assert torch.equal(out[~turned], want[~turned])
            if not R:
                assert got is None
                continue
            near(out, want, dtype, 8.0 * turned, "cache")
            have = torch.full((B,), T) if n is None else n.clamp(0, T)
            for b in range(B):
                at = int(lengths[b]) - int(have[b]) + torch.arange(T)
                live = (torch.arange(T) < have[b]) & (at >= 0)
                ref = torch.where(live[:, None, None], latent64.rotate(
                    q[b].double().cpu(), at[:, None].expand(T, H), frequencies(R), pairs),
                    q[b].double().cpu())
                near(got[b], ref, dtype, sizes(q[b].double().cpu(), pairs) * live[:, None, None],
                     "queries")


def test_append_copies_keys_without_frequencies():
    import gated_delta_rule_21_gb300 as kda
    cache = torch.zeros(3, 8, 40, device="cuda")
    latent, k = torch.randn(1, 5, 32, device="cuda"), torch.randn(1, 5, 8, device="cuda")
    k[0, 2, 3] = float("inf")
    kda.latent_append(latent, k, cache, torch.tensor([[2, 0]], dtype=torch.int32, device="cuda"),
                      torch.tensor([10], dtype=torch.int32, device="cuda"))
    assert torch.equal(torch.cat([cache[2, 5:], cache[0, :2]]), torch.cat([latent, k], -1)[0])
    assert not cache[1].any() and not cache[2, :5].any() and not cache[0, 2:].any()


def test_append_at_offsets_past_32_bits():
    import gated_delta_rule_21_gb300 as kda
    page, width = 128, 576
    n_pages = 2 ** 31 // (page * width) + 3
    cache = torch.zeros(n_pages, page, width, dtype=BF, device="cuda")
    latent = torch.randn(1, 2, 512, device="cuda").to(BF)
    k = torch.randn(1, 2, 64, device="cuda").to(BF)
    kda.latent_append(latent, k, cache, torch.tensor([[n_pages - 1]], dtype=torch.int32,
                                                     device="cuda"),
                      torch.tensor([128], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache[-1, -2:], torch.cat([latent, k], -1)[0])
    assert not cache[:-1].any() and not cache[-1, :-2].any()

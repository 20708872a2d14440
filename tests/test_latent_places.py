"""GPU test of new tokens that have no place in the paged cache: behind the table's
room, or on a page outside the cache.  By the documentation they are not stored and
nobody sees them, themselves included; their queries are rotated and see the
sequence's other tokens up to their own position.  The expected values are
made token by token from that, with no code of the other tests' plain form."""
import pytest
import torch

import latent64
from test_latent_rotate import frequencies

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WAYS = [("simt", F32), ("simt", BF), ("tc", BF)]

# page table, length, new tokens (of T = 5), pages of 8 tokens, 6 of them
ROWS = [([0, 1], 19, 5),        # positions 14 to 18, room for 16
        ([2, 6], 11, 5),        # the second page is outside: 6, 7 have a place, 8 to 10 not
        ([-1, 3], 12, 4),       # the first one is
        ([4, 5], 30, 2),        # both new tokens far behind the room
        ([9, 9], 10, 3),        # no pages at all
        ([-3, 7], 3, 5)]        # nor here; two of them before position 0


@pytest.mark.parametrize("impl,dtype", WAYS)
def test_tokens_without_a_place(impl, dtype):
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(1)
    B, T, H, C, R, page, n_pages = len(ROWS), 5, 3, 128, 32, 8, 6
    table = torch.tensor([r[0] for r in ROWS], dtype=torch.int32)
    lengths, new = (torch.tensor([r[i] for r in ROWS], dtype=torch.int32) for i in (1, 2))
    cache = torch.randn(n_pages, page, C + R, generator=gen).to(dtype)
    latent = torch.randn(B, T, C, generator=gen).to(dtype)
    k = torch.randn(B, T, R, generator=gen).to(dtype)
    q = torch.randn(B, T, H, C, generator=gen).to(dtype)
    r = torch.randn(B, T, H, R, generator=gen).to(dtype)
    freq = frequencies(R)
    dev = cache.cuda()
    turned = kda.latent_append(latent.cuda(), k.cuda(), dev, table.cuda(), lengths.cuda(),
                               inv_freq=freq.cuda(), new=new.cuda(), q_rope=r.cuda())
    o, lse = kda.latent_step(q.cuda(), turned, dev, table.cuda(), lengths.cuda(), scale=0.1,
                             new=new.cuda(), return_lse=True, impl=impl)
    after, turned = dev.cpu(), turned.cpu()
    want, written = cache.clone(), set()
    for b, (pages, length, n) in enumerate(ROWS):
        for t in range(T):
            at = length - n + t
            if t >= n or at < 0:            # not there
                assert torch.equal(turned[b, t], r[b, t])
                assert not o[b, t].any() and bool((lse[b, :, t] == -torch.inf).all())
                continue
            ref = latent64.rotate(r[b, t].double(), torch.full((H,), at), freq)
            assert float((turned[b, t].double() - ref).abs().max()) <= \
                float(ref.abs().max()) * (2.0 ** -8 * 1.01 if dtype == BF else 2e-6)
            if at < len(pages) * page and 0 <= pages[at // page] < n_pages:
                written.add((pages[at // page], at % page))
                want[pages[at // page], at % page, :C] = latent[b, t]
            # who is seen: the positions up to its own that have a place
            seen = [(pages[j // page], j % page) for j in range(at + 1)
                    if j < len(pages) * page and 0 <= pages[j // page] < n_pages]
            if not seen:
                assert not o[b, t].any() and bool((lse[b, :, t] == -torch.inf).all())
                continue
            tokens = torch.stack([after[i] for i in seen]).double()
            (v, tol), (l, l_tol) = latent64.step(
                q[b, t:t + 1].double(), turned[b, t:t + 1].double(), tokens,
                torch.ones(len(seen), dtype=torch.bool), torch.tensor([len(seen)]), 0.1, impl, dtype)
            latent64.check(o[b, t], (v[0], tol[0]), f"o of {b}, {t}")
            latent64.check(lse[b, :, t], (l[0], l_tol[0]), f"lse of {b}, {t}")
    assert torch.equal(after[..., :C], want[..., :C])
    for i in range(n_pages):
        for j in range(page):
            assert (i, j) in written or torch.equal(after[i, j], cache[i, j])
    assert written == {(1, 6), (1, 7), (2, 6), (2, 7), (3, 0), (3, 1), (3, 2), (3, 3)}

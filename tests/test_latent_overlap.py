"""Outputs of the latent attention's row kernels whose rows lie over each other (a
stride smaller than a row) are refused, on the host and before anything is enqueued: two
of their rows would be written in no order.  No GPU is needed."""
import pytest

import gated_delta_rule_21_gb300 as kda
from gated_delta_rule_21_gb300 import build as kbuild

FAKE = 0x10000      # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


@pytest.mark.parametrize("strides", [(0, 128, 64), (512, 0, 64), (512, 128, 0), (512, 128, 63),
                                     (512, -128, 32), (-63, 128, 64)])
def test_rotate_refuses_rows_over_each_other(L, strides):
    d = kda.kda_rotate_desc(2, 4, 2, 64, 1, 1, 0, 0, 0, 0, *strides)   # (x may be broadcast)
    assert L.kda_rotate(d, FAKE, None, FAKE, FAKE, None) == 1


@pytest.mark.parametrize("page_stride,token_stride", [(0, 576), (64 * 576, 0), (64 * 576, 575),
                                                      (100, 576), (64 * 576, -512)])
def test_append_refuses_places_over_each_other(L, page_stride, token_stride):
    s = kda.kda_latent_cache(2, 1, 4, 8, 20, 64, 512, 64, 1, page_stride, token_stride, 2048, 2048,
                             512, 256, 256, 64, 512, 512, 64, 64)
    assert L.kda_latent_append(s, FAKE, FAKE, None, FAKE, 1, FAKE, FAKE, None, FAKE, None, None) == 1


@pytest.mark.gpu
def test_rows_that_are_not_over_each_other_are_served():
    """Strides of dimensions of 1 are not looked at; pages and tokens may lie in either
    order, and a row's heads may lie apart."""
    import torch
    x = torch.randn(1, 3, 1, 32, device="cuda")
    freq = torch.rand(16, device="cuda")
    y = torch.empty(1, 3, 1, 32, device="cuda").as_strided((1, 3, 1, 32), (0, 32, 0, 1))
    want = kda.rotate(x, freq)
    assert torch.equal(kda.rotate(x, freq, out=y), want)
    wide = torch.zeros(3, 5, 1, 40, device="cuda")
    out = wide[:, 2:3, :, 4:36].transpose(0, 1)
    kda.rotate(x, freq, out=out)
    assert torch.equal(out, want) and not wide[:, :2].any() and not wide[..., :4].any()
    # the heads' rows of a transposed tensor, backwards in memory
    heads = torch.empty(2, 4, 1, 32, device="cuda").transpose(0, 2)      # [1, 4, 2, 32]
    x = torch.randn(1, 4, 2, 32, device="cuda")
    assert torch.equal(kda.rotate(x, freq, out=heads), kda.rotate(x, freq))
    latent, k = torch.randn(1, 9, 128, device="cuda"), torch.randn(1, 9, 32, device="cuda")
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    n = torch.tensor([9], dtype=torch.int32, device="cuda")
    pages_first = torch.zeros(3, 8, 160, device="cuda")
    tokens_first = torch.zeros(8, 3, 160, device="cuda").transpose(0, 1)
    for cache in (pages_first, tokens_first):
        kda.latent_append(latent, k, cache, table, n, inv_freq=freq)
    assert torch.equal(pages_first, tokens_first) and pages_first[2].any()

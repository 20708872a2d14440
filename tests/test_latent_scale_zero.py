"""GPU test of the latent attention with a scale of 0 on the tensor cores: all
tokens weigh alike, and the call takes no longer than with another scale.  (Made row by
row, as rows that are not finite are, this size takes hundreds of times as long; the bound
is 8 times, of the fastest of five calls.)"""
import pytest
import torch

import latent64
from test_latent_prompt import compare, inputs, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def fastest(x, scale, ws, seg):
    times = []
    for _ in range(6):
        a, z = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        run(x, seg, "tc", scale=scale, workspace=ws)
        z.record()
        z.synchronize()
        times.append(a.elapsed_time(z))
    return min(times[1:])


@pytest.mark.parametrize("packed", [False, True])
def test_scale_of_zero_takes_no_longer(packed):
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(1)
    B, T, H, K, R, V = 1, 2048, 4, 128, 64, 128
    x, x64 = inputs(B, T, H, K, R, V, BF, gen)
    seg = None
    if packed:
        seg = torch.ones(1, T, dtype=torch.int32)
        seg[0, 700:1500], seg[0, 1490:1500] = 2, 0
    d_o = torch.randn(B, T, H, V, generator=gen).to(BF).cuda()
    ws = kda.alloc_latent_workspace(B, T, H, R, backward=True)
    dev = None if seg is None else seg.cuda()
    for scale in (0.0, -0.0):
        compare(run(x, dev, "tc", d_o, scale=scale, workspace=ws),
                latent64.prompt(x64, scale, seg, "tc", BF, d_o.double()))
    assert kda.read_device_status(ws) == 0
    assert fastest(x, 0.0, ws, dev) <= 8 * fastest(x, 0.1, ws, dev)


def test_scale_of_zero_and_values_that_are_not_finite():
    """0 times an infinite or undefined product is not a number, as in the definition;
    it reaches the tokens that see it."""
    gen = torch.Generator().manual_seed(2)
    x, _ = inputs(1, 300, 2, 64, 32, 64, BF, gen, strided=False)
    clean = run(x, None, "tc", scale=0.0)["o"]
    x["k"][0, 170, 0, 3] = float("inf")
    got = run(x, None, "tc", scale=0.0)["o"]
    assert got[0, 170:, 0].isnan().all()
    assert torch.equal(got[0, :170], clean[0, :170]) and torch.equal(got[:, :, 1], clean[:, :, 1])

"""GPU test of latent attention calls at once on three streams, each with its own
workspace that all its calls share."""
import pytest
import torch

from test_latent_prompt import inputs, run
from test_latent_rotate import frequencies
from test_latent_step import places

BF = torch.bfloat16


@pytest.mark.gpu
def test_prompts_and_steps_on_two_streams_while_a_third_appends():
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(10)
    B, H, C, R, T = 5, 32, 512, 64, 700
    made = []
    for s in range(2):
        lengths = torch.full((B,), 1000 + 300 * s, dtype=torch.int32)
        table, n_pages = places(lengths, 64, 24, gen)
        a = [torch.randn(B, 1, H, C, generator=gen).to(BF).cuda(),
             torch.randn(B, 1, H, R, generator=gen).to(BF).cuda(),
             torch.randn(n_pages, 64, C + R, generator=gen).to(BF).cuda(), table.cuda(),
             lengths.cuda()]
        x, _ = inputs(1, T, 4, 128, 64, 128, BF, gen, strided=False)
        d_o = torch.randn(1, T, 4, 128, generator=gen).to(BF).cuda()
        ws = (kda.alloc_latent_step_workspace(B, 1, H, C),
              kda.alloc_latent_workspace(1, T, 4, 64, backward=True))
        made.append((a, x, d_o, ws, kda.latent_step(*a, scale=0.07), run(x, None, "auto", d_o)))
    # the third one fills a cache of its own, 8 prompts of 48 tokens one after another
    table = torch.randperm(24, generator=gen).view(3, 8).int().cuda()
    latent = torch.randn(3, 384, C, generator=gen).to(BF).cuda()
    k = torch.randn(3, 384, R, generator=gen).to(BF).cuda()
    r = torch.randn(3, 384, H, R, generator=gen).to(BF).cuda()
    freq = frequencies(R).cuda()
    ends = [torch.full((3,), 48 * (i + 1), dtype=torch.int32, device="cuda") for i in range(8)]

    def append(cache, i, **kw):
        part = slice(48 * i, 48 * (i + 1))
        return kda.latent_append(latent[:, part], k[:, part], cache, table, ends[i],
                                 inv_freq=freq, q_rope=r[:, part], **kw)

    alone, busy = (torch.zeros(24, 48, C + R, dtype=BF, device="cuda") for _ in range(2))
    turned = [append(alone, i) for i in range(8)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    steps, prompts, appended = ([], []), ([], []), []
    for i in range(8):
        for s, (a, x, d_o, ws, _, _) in enumerate(made):
            steps[s].append(kda.latent_step(*a, scale=0.07, workspace=ws[0], stream=streams[s]))
            prompts[s].append(run(x, None, "auto", d_o, workspace=ws[1], stream=streams[s]))
        appended.append(append(busy, i, stream=streams[2]))
    torch.cuda.synchronize()
    for s, (_, _, _, ws, o, want) in enumerate(made):
        for y in steps[s]:
            assert torch.equal(y, o)
        for y in prompts[s]:
            for n in want:
                assert torch.equal(y[n], want[n]), n
        assert all(kda.read_device_status(w) == 0 for w in ws)
    assert torch.equal(busy, alone)
    assert all(torch.equal(a, b) for a, b in zip(appended, turned))

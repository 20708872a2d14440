"""GPU tests of the state space operator at the sizes where the kernels take
their other forms: 64 columns per state CTA, several heads per output CTA,
several blocks per prep CTA, fp32 that AUTO puts on the tensor cores.

Each shape is chosen by the rule that selects the form (restated beside it).
The plain 64-bit form runs on the GPU, all rows at once, token by token.
Tolerances as in test_ssm.py."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

F32, F64 = torch.float32, torch.float64


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def plain(x, dt, z, w, bias, A, db, D, ids, state, window, dims):
    """The recurrence on [B, T, ..] tensors of 64 bits."""
    B, T, H, P, N, G = dims
    y = torch.zeros(B, T, H, P, dtype=F64, device=x.device)
    begun = torch.zeros(B, dtype=torch.bool, device=x.device)
    prev = torch.zeros(B, dtype=torch.int32, device=x.device)
    for t in range(T):
        now = ids[:, t]
        live = now != 0
        start = live & (now != prev)
        reset = start & begun
        begun, prev = begun | live, now
        state = torch.where(reset[:, None, None, None], 0.0, state)
        window = torch.where(reset[:, None, None], 0.0, window)
        full = torch.cat([window, x[:, t:t + 1]], 1)
        u = plain64.silu((full * w.t()).sum(1) + bias)
        xs = u[:, :H * P].view(B, H, P)
        bs, cs = (v.reshape(B, G, N).repeat_interleave(H // G, 1)
                  for v in u[:, H * P:].split(G * N, 1))
        d = plain64.softplus(dt[:, t] + db)
        new = torch.exp(d * A)[..., None, None] * state \
            + (d[..., None] * bs)[..., None] * xs[:, :, None]
        state = torch.where(live[:, None, None, None], new, state)
        window = torch.where(live[:, None, None], full[:, 1:], window)
        out = (cs[:, :, None] @ state)[:, :, 0] + D[:, None] * xs
        y[:, t] = out * plain64.silu(z[:, t]).view(B, H, P) * live[:, None, None]
    return y, state, window


def check(dims, dtype, packed, impl="auto", seed=0):
    import gated_delta_rule_21_gb300 as kda
    B, T, H, P, N, G = dims
    gen = torch.Generator(device="cuda").manual_seed(seed + T + H)

    def rand(*s, std=1.0, mean=0.0, to=F32):
        return plain64.cast(mean + std * torch.randn(*s, generator=gen, device="cuda"), to)

    hp, ch = H * P, H * P + 2 * G * N
    proj = rand(B, T, -(-(hp + ch + H) // 8) * 8, to=dtype)
    z, x, dt = ([p[..., a:b] for p in proj] for a, b in
                ((0, hp), (hp, hp + ch), (hp + ch, hp + ch + H)))
    w, bias, db, D = rand(ch, 4, std=0.5), rand(ch, std=0.1), rand(H, mean=-3.0), rand(H, mean=1.0)
    A = plain64.cast(-(1 + 15 * torch.rand(H, generator=gen, device="cuda")), F32)
    s0, c0 = rand(B, H, N, P, std=0.3), rand(B, 3, ch, to=dtype)
    ids = torch.ones(B, T, dtype=torch.int32)
    if packed:          # runs of every row at other places, some padding, an empty row
        cpu = torch.Generator().manual_seed(seed)
        for b in range(B):
            cuts = sorted(torch.randint(1, T, (6,), generator=cpu).tolist())
            for i, c in enumerate(cuts):
                ids[b, c:] = i + 2
            ids[b, cuts[2]:cuts[2] + 9] = 0
        ids[B // 2] = 0
    ids = ids.cuda()
    ws = kda.alloc_ssm_workspace(*dims, dtype=dtype, impl=impl)
    y, s, c = kda.ssm_fwd(x[0], dt[0], w[0], A[0], head_dim=P, state_dim=N, conv_bias=bias[0],
                          dt_bias=db[0], D=D[0], z=z[0], initial_state=s0[0], conv_state=c0[0],
                          segment_ids=ids if packed else None, output_final_state=True,
                          workspace=ws, impl=impl)
    assert kda.read_device_status(ws) == 0
    yr, sr, cr = plain(x[1], dt[1], z[1], w[1], bias[1], A[1], db[1], D[1], ids, s0[1], c0[1], dims)
    d = (y.double() - yr).abs()
    if dtype == F32:
        assert d.max() <= 2e-5 * yr.abs().max(), d.max() / yr.abs().max()
    else:
        assert d.max() <= 2 ** -5 * yr.abs().max(), d.max() / yr.abs().max()
        assert d.norm() <= 5e-3 * yr.norm(), d.norm() / yr.norm()
    d = (s.double() - sr).abs()
    assert d.max() <= 2e-5 * sr.abs().max(), d.max() / sr.abs().max()
    assert torch.equal(c.double(), cr)
    assert not y[ids == 0].any()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dims", [(2, 300, 40, 64, 64, 1), (2, 257, 20, 128, 128, 4)])
def test_states_of_64_columns(dims, packed):
    B, _, H, P, _, _ = dims
    assert 2 * B * H * (P // 64) > sms()
    check(dims, torch.bfloat16, packed)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype,dims", [
    (torch.bfloat16, (8, 500, 78, 64, 32, 1)), (torch.bfloat16, (5, 600, 66, 128, 32, 2)),
    (torch.bfloat16, (6, 513, 56, 32, 64, 1)), (torch.float32, (6, 513, 54, 32, 64, 2))])
def test_several_heads_per_output_cta(dims, dtype, packed):
    """4 heads in the first shape, 2 in the others: with that many there are
    still 4 CTAs per SM.  Every shape but the third leaves a last CTA with fewer."""
    B, T, H, _, _, G = dims
    assert B * -(-T // 128) * G * -(-(H // G) // 2) >= 4 * sms()
    check(dims, dtype, packed, impl="tc")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype,dims", [
    (torch.bfloat16, (16, 1000, 16, 32, 64, 16)), (torch.bfloat16, (24, 900, 8, 64, 128, 8)),
    (torch.bfloat16, (40, 700, 16, 32, 32, 8)), (torch.float32, (12, 800, 8, 32, 128, 8))])
def test_several_blocks_per_prep_cta(dims, dtype, packed):
    """Two blocks and more per CTA where the tiles make 12 waves of the SMs."""
    B, T, _, _, N, G = dims
    tile = 32 if dtype == torch.float32 or N == 32 else 64
    assert B * -(-T // 128) * G * 2 * N // tile >= 12 * sms()
    check(dims, dtype, packed, impl="tc")


@pytest.mark.parametrize("packed", [False, True])
def test_auto_in_fp32_at_both_sides_of_its_rule(packed):
    """2^26 products of states and tokens."""
    import gated_delta_rule_21_gb300 as kda
    for dims in ((1, 1000, 16, 64, 64, 2), (1, 1100, 16, 64, 64, 2)):
        B, T, H, P, N, G = dims
        on_tc = B * T * H * P * N > 2 ** 26
        assert (kda.ssm_workspace_size(*dims, dtype=F32) ==
                kda.ssm_workspace_size(*dims, dtype=F32, impl="tc" if on_tc else "simt"))
        check(dims, F32, packed)

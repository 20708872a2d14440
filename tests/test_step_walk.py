"""GPU tests of the single-token steps where a CTA walks many units: more
units than three on every SM three times over, and idle sequences in every
place between active ones.

The plain 64-bit form runs on the GPU, all sequences at once.  Tolerances as
in test_step.py: one rounding of the output, 1e-5 of the largest value for the
fp32 arithmetic before it, copies equal."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu


def near(got, ref, dtype, what, f32=1e-5):
    tol = torch.finfo(dtype).eps / 2 * 1.01 * ref.abs() + f32 * ref.abs().amax() + 1e-30
    bad = (got.double() - ref).abs() - tol
    assert bad.max() <= 0, f"{what}: {int((bad > 0).sum())} of {bad.numel()} off, by up to {bad.max():.3e}"


def idle_rows(pattern, B, H, tiles, gen):
    """Sequences that are idle.  A CTA's units are `stride` (sequence, head)
    pairs apart, so its n-th unit belongs to a sequence b with b H / stride = n."""
    stride = 3 * torch.cuda.get_device_properties(0).multi_processor_count // tiles
    turn = torch.arange(B) * H // stride
    assert int(turn[-1]) >= 3, "every CTA walks four units or more"
    if pattern == "every second":
        return turn % 2 == 1
    if pattern == "two of three":
        return turn % 3 != 0
    return torch.rand(B, generator=gen) < 0.5


def slots_of(idle, n_slots, gen):
    s = torch.randperm(n_slots, generator=gen)[:idle.numel()].to(torch.int32)
    s[idle] = torch.tensor([-1, n_slots, -9, 2 ** 31 - 1], dtype=torch.int32).repeat(
        idle.numel())[:int(idle.sum())]
    return s.cuda()


PATTERNS = ["every second", "two of three", "half of them"]
KDA = [(1300, 2, 32, 32, True), (128, 33, 64, 128, True), (64, 32, 128, 128, True),
       (330, 7, 128, 64, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,K,V,conv", KDA)
@pytest.mark.parametrize("pattern", PATTERNS)
def test_kda_step_walks(B, H, K, V, conv, dtype, pattern):
    import gated_delta_rule_21_gb300 as kda
    cpu = torch.Generator().manual_seed(B + H)
    gen = torch.Generator(device="cuda").manual_seed(B + H)
    f32 = torch.float32

    def rand(*s, std=1.0, to=dtype):
        return plain64.cast(std * torch.randn(*s, generator=gen, device="cuda"), to)

    n_slots, ch = B + 5, H * (2 * K + V)
    idle = idle_rows(pattern, B, H, 2 if V == 128 else 1, cpu)
    slots = slots_of(idle, n_slots, cpu)
    on = (~idle).cuda()
    at = slots[on].long()
    state, state64 = rand(n_slots, H, K, V, std=0.3, to=f32)
    cache, cache64 = rand(n_slots, 3, ch)
    w, w64 = rand(ch, 4, std=0.5, to=f32)
    ws = kda.alloc_step_workspace(B, H)
    for _ in range(3):
        x, x64 = rand(B, ch, std=1.0 if conv else K ** -0.5)
        g, g64 = plain64.cast(-5 * torch.rand(B, H, K, generator=gen, device="cuda"), f32)
        beta, beta64 = plain64.cast(torch.rand(B, H, generator=gen, device="cuda"), f32)
        q, k, v = (t.unflatten(1, (H, -1)) for t in x.split([H * K, H * K, H * V], 1))
        o = kda.step(q, k, v, g, beta, state, slots=slots, conv_w=w if conv else None,
                     conv_state=cache if conv else None, l2norm_qk=conv, workspace=ws)
        u = x64[on]
        if conv:
            full = torch.cat([cache64[at], u[:, None]], 1)
            cache64[at] = full[:, 1:]
            u = plain64.silu((full * w64.t()).sum(1))
        q, k, v = (t.unflatten(1, (H, -1)) for t in u.split([H * K, H * K, H * V], 1))
        if conv:
            q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        s = state64[at] * torch.exp(g64[on])[..., None]
        rest = v - (k[..., None] * s).sum(2)
        s += (beta64[on][..., None] * k)[..., None] * rest[:, :, None]
        state64[at] = s
        want = torch.zeros(B, H, V, dtype=torch.float64, device="cuda")
        want[on] = K ** -0.5 * (q[..., None] * s).sum(2)
        near(o, want, dtype, "o")
        near(state, state64, f32, "state")
        assert torch.equal(cache.double(), cache64)
    assert int(ws.sum()) == 0


SSM = [(1400, 2, 32, 32, 1), (128, 33, 64, 64, 3), (96, 24, 128, 128, 2), (330, 8, 64, 128, 8)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,P,N,G", SSM)
@pytest.mark.parametrize("pattern", PATTERNS)
def test_ssm_step_walks(B, H, P, N, G, dtype, pattern):
    import gated_delta_rule_21_gb300 as kda
    cpu = torch.Generator().manual_seed(B * 3 + H)
    gen = torch.Generator(device="cuda").manual_seed(B * 3 + H)
    f32 = torch.float32

    def rand(*s, std=1.0, mean=0.0, to=f32):
        return plain64.cast(mean + std * torch.randn(*s, generator=gen, device="cuda"), to)

    n_slots, hp, ch = B + 5, H * P, H * P + 2 * G * N
    idle = idle_rows(pattern, B, H, 2 if P == 128 else 1, cpu)
    slots = slots_of(idle, n_slots, cpu)
    on = (~idle).cuda()
    at = slots[on].long()
    state, state64 = rand(n_slots, H, N, P, std=0.3)
    conv, conv64 = rand(n_slots, 3, ch, to=dtype)
    (w, w64), (bias, bias64) = rand(ch, 4, std=0.5), rand(ch, std=0.1)
    (db, db64), (D, D64) = rand(H, mean=-3.0), rand(H, mean=1.0)
    A, A64 = plain64.cast(-(1 + 15 * torch.rand(H, generator=gen, device="cuda")), f32)
    ws = kda.alloc_step_workspace(B, H)
    for _ in range(3):
        proj, proj64 = rand(B, hp + ch + H + 3, to=dtype)
        z, x, dt = proj[:, :hp], proj[:, hp:hp + ch], proj[:, hp + ch:hp + ch + H]
        y = kda.ssm_step(x, dt, w, A, state, conv, head_dim=P, state_dim=N, conv_bias=bias,
                         dt_bias=db, D=D, z=z, slots=slots, workspace=ws)
        z, x, dt = (t[on] for t in proj64.split([hp, ch, H, 3], 1)[:3])
        full = torch.cat([conv64[at], x[:, None]], 1)
        conv64[at] = full[:, 1:]
        u = plain64.silu((full * w64.t()).sum(1) + bias64)
        xs = u[:, :hp].unflatten(1, (H, P))
        bs, cs = (t.unflatten(1, (G, N)).repeat_interleave(H // G, 1)
                  for t in u[:, hp:].split([G * N, G * N], 1))
        d = plain64.softplus(dt + db64)
        s = torch.exp(d * A64)[..., None, None] * state64[at] \
            + (d[..., None] * bs)[..., None] * xs[:, :, None]
        state64[at] = s
        want = torch.zeros(B, H, P, dtype=torch.float64, device="cuda")
        want[on] = ((cs[..., None] * s).sum(2) + D64[:, None] * xs) \
            * plain64.silu(z).unflatten(1, (H, P))
        near(y, want, dtype, "y")
        near(state, state64, f32, "state")
        assert torch.equal(conv.double(), conv64)
    assert int(ws.sum()) == 0

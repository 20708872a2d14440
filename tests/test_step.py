"""GPU tests of the single-token steps (kda_step, kda_ssm_step) against the
plain 64-bit recurrences.

Tolerances.  The outputs are rounded once to their type (eps / 2 relative to
the value).  Everything before is fp32: the state is one product and one
multiply-add from its old value, off by a few 2^-24 of the terms; the factors
exp, SiLU, softplus and rsqrt are off by a few ulp, and a sum over at most 128
keys in 16 or fewer sequential terms adds 2^-24 * 24 of its terms' sizes.  1e-5
of the largest value of the tensor covers these; the cached inputs of the
convolution are copies and are equal."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu


def near(got, ref, dtype, what, f32=1e-5):
    got = got.double().cpu()
    tol = torch.finfo(dtype).eps / 2 * 1.01 * ref.abs() + f32 * ref.abs().amax() + 1e-30
    bad = (got - ref).abs() - tol
    assert bad.max() <= 0, f"{what}: {(bad > 0).sum()} of {bad.numel()} off, by up to {bad.max():.3e}"


def rand(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, dtype=torch.float64) * std


def places(B, n_slots, idle, gen):
    s = torch.randperm(n_slots, generator=gen)[:B].to(torch.int32)
    for i in range(idle):
        s[(2 * i + 1) % B] = (-1, n_slots, -7, 2 ** 31 - 1)[i % 4]
    return s


SSM = [(1, 1, 32, 32, 1), (3, 4, 64, 128, 2), (2, 6, 128, 64, 3), (40, 8, 64, 128, 8),
       (5, 3, 128, 128, 1), (160, 2, 32, 64, 1), (1, 32, 128, 128, 1), (7, 5, 64, 32, 5)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,P,N,G", SSM)
@pytest.mark.parametrize("slim", [False, True])
def test_ssm_step(B, H, P, N, G, dtype, slim):
    """Three tokens in a row; ``slim`` leaves out bias, D, gate and slots."""
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(B * 7 + H)
    ch, hp = H * P + 2 * G * N, H * P
    n_slots = B if slim else B + 3
    slots = None if slim else places(B, n_slots, B // 3, gen)
    w, w64 = plain64.cast(rand(gen, ch, 4, std=0.5), torch.float32)
    A, A64 = plain64.cast(-(1 + 15 * torch.rand(H, generator=gen, dtype=torch.float64)),
                          torch.float32)
    bias, bias64 = plain64.cast(rand(gen, ch, std=0.1), torch.float32)
    db, db64 = plain64.cast(rand(gen, H) - 3, torch.float32)
    D, D64 = plain64.cast(1 + rand(gen, H), torch.float32)
    state, state64 = plain64.cast(rand(gen, n_slots, H, N, P, std=0.3), torch.float32)
    conv, conv64 = plain64.cast(rand(gen, n_slots, 3, ch), dtype)
    state, conv, w, A = state.cuda(), conv.cuda(), w.cuda(), A.cuda()
    opt = {} if slim else dict(conv_bias=bias.cuda(), dt_bias=db.cuda(), D=D.cuda(),
                               slots=slots.cuda())
    op = plain64.Ssm(w64, A64, H, P, N, G) if slim else \
        plain64.Ssm(w64, A64, H, P, N, G, bias64, db64, D64)
    ws = kda.alloc_step_workspace(B, H)
    for _ in range(3):
        proj, proj64 = plain64.cast(rand(gen, B, hp + ch + H + 3), dtype)
        z, x, dt = (proj.cuda()[:, a:b] for a, b in ((0, hp), (hp, hp + ch), (hp + ch, hp + ch + H)))
        y = kda.ssm_step(x, dt, w, A, state, conv, head_dim=P, state_dim=N,
                         z=None if slim else z, workspace=ws, **opt)
        want = torch.zeros(B, H, P, dtype=torch.float64)
        for b in range(B):
            k = b if slim else int(slots[b])
            if 0 <= k < n_slots:
                want[b], state64[k], conv64[k] = op.token(
                    proj64[b, hp:hp + ch], proj64[b, hp + ch:hp + ch + H],
                    None if slim else proj64[b, :hp], state64[k], conv64[k])
        near(y, want, dtype, "y")
        near(state, state64, torch.float32, "state")
        assert torch.equal(conv.cpu().double(), conv64)
    assert int(ws.sum()) == 0      # the counters are left as they were found


KDA = [(1, 1, 32, 32), (3, 4, 64, 128), (2, 6, 128, 64), (40, 7, 128, 128), (160, 2, 32, 64),
       (1, 32, 128, 128), (5, 3, 64, 32)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,K,V", KDA)
@pytest.mark.parametrize("conv", [False, True])
def test_kda_step(B, H, K, V, dtype, conv):
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(B * 5 + H)
    ch = H * (2 * K + V)
    n_slots = B + 2
    slots = places(B, n_slots, B // 3, gen)
    w, w64 = plain64.cast(rand(gen, ch, 4, std=0.5), torch.float32)
    state, state64 = plain64.cast(rand(gen, n_slots, H, K, V, std=0.3), torch.float32)
    cache, cache64 = plain64.cast(rand(gen, n_slots, 3, ch), dtype)
    state, cache, w = state.cuda(), cache.cuda(), w.cuda()
    ws = kda.alloc_step_workspace(B, H)
    for _ in range(3):
        qkv = rand(gen, B, ch + 8)
        if not conv:
            qkv[:, :2 * H * K] /= K ** 0.5
        qkv, qkv64 = plain64.cast(qkv, dtype)
        g, g64 = plain64.cast(-5 * torch.rand(B, H, K, generator=gen, dtype=torch.float64),
                              torch.float32)
        beta, beta64 = plain64.cast(torch.rand(B, H, generator=gen, dtype=torch.float64),
                                    torch.float32)
        dev = qkv.cuda()
        q, k, v = (dev[:, a:b].unflatten(1, (H, -1)) for a, b in
                   ((0, H * K), (H * K, 2 * H * K), (2 * H * K, ch)))
        o = kda.step(q, k, v, g.cuda(), beta.cuda(), state, slots=slots.cuda(),
                     conv_w=w if conv else None, conv_state=cache if conv else None,
                     l2norm_qk=conv, workspace=ws)
        want = torch.zeros(B, H, V, dtype=torch.float64)
        for b in range(B):
            s = int(slots[b])
            if not 0 <= s < n_slots:
                continue
            x = qkv64[b, :ch]
            if conv:
                full = torch.cat([cache64[s], x[None]])
                cache64[s] = full[1:]
                x = plain64.silu((full * w64.t()).sum(0))
            qi, ki, vi = x[:H * K].view(H, K), x[H * K:2 * H * K].view(H, K), x[2 * H * K:].view(H, V)
            if conv:
                qi, ki = (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (qi, ki))
            want[b], state64[s] = plain64.delta_token(qi, ki, vi, g64[b], beta64[b], state64[s],
                                                      K ** -0.5)
        near(o, want, dtype, "o")
        near(state, state64, torch.float32, "state")
        if conv:
            assert torch.equal(cache.cpu().double(), cache64)
    assert int(ws.sum()) == 0


def test_a_cache_whose_offsets_pass_32_bits():
    """The last places of a cache of more than 2^31 state values."""
    import gated_delta_rule_21_gb300 as kda
    H, D = 32, 128
    n_slots = 2 ** 31 // (H * D * D) + 5
    state = torch.zeros(n_slots, H, D, D, device="cuda")
    gen = torch.Generator().manual_seed(3)
    s0, s64 = plain64.cast(rand(gen, H, D, D, std=0.3), torch.float32)
    slot = n_slots - 1
    state[slot] = s0.cuda()
    q, k, v = (plain64.cast(rand(gen, 1, H, D, std=0.1), torch.float32) for _ in range(3))
    g, g64 = plain64.cast(-torch.rand(1, H, D, generator=gen, dtype=torch.float64), torch.float32)
    beta, b64 = plain64.cast(torch.rand(1, H, generator=gen, dtype=torch.float64), torch.float32)
    o = kda.step(q[0].cuda(), k[0].cuda(), v[0].cuda(), g.cuda(), beta.cuda(), state,
                 slots=torch.tensor([slot], dtype=torch.int32, device="cuda"))
    want, s64 = plain64.delta_token(q[1][0], k[1][0], v[1][0], g64[0], b64[0], s64, D ** -0.5)
    near(o[0], want, torch.float32, "o")
    near(state[slot], s64, torch.float32, "state")
    assert not state[:slot].any()


def test_step_follows_chunk_fwd():
    """A prompt through chunk_fwd and its next tokens one by one against the
    fp64 oracle over the whole sequence."""
    import gated_delta_rule_21_gb300 as kda
    import kda_inputs as ki
    import oracle
    T, n = 70, 6
    w = ki.custom_workload(2, T, 3, 64, 64, dtype="f32", init_state_std=0.1)
    x = ki.make_inputs(w, seed=4)
    names = ("q", "k", "v", "g", "beta")
    head = [x[k][:, :T - n].contiguous().cuda() for k in names]
    _, state = kda.chunk_fwd(*head, scale=x["scale"], initial_state=x["initial_state"].cuda(),
                             output_final_state=True)
    o_ref, s_ref = oracle.kda_forward(*[x[k] for k in names], x["scale"],
                                      initial_state=x["initial_state"])
    for t in range(T - n, T):
        o = kda.step(*[x[k][:, t].contiguous().cuda() for k in names], state, scale=x["scale"])
        assert abs(o.double().cpu().numpy() - o_ref[:, t]).max() <= 1e-4
    assert abs(state.double().cpu().numpy() - s_ref).max() <= 1e-4


def test_step_in_a_graph_and_on_another_stream():
    import gated_delta_rule_21_gb300 as kda
    gen = torch.Generator().manual_seed(11)
    B, H, P, N, G = 4, 4, 64, 128, 2
    ch = H * P + 2 * G * N
    t = {k: v.cuda().float() for k, v in dict(
        x=rand(gen, B, ch), dt=rand(gen, B, H), w=rand(gen, ch, 4), A=-rand(gen, H).abs(),
        state=rand(gen, B, H, N, P), conv=rand(gen, B, 3, ch)).items()}
    ws = kda.alloc_step_workspace(B, H)

    def go(state, conv, **kw):
        return kda.ssm_step(t["x"], t["dt"], t["w"], t["A"], state, conv, head_dim=P,
                            state_dim=N, **kw)

    s1, c1 = t["state"].clone(), t["conv"].clone()
    want = [go(s1, c1) for _ in range(2)]
    s2, c2 = t["state"].clone(), t["conv"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = go(s2, c2, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = go(s2, c2, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want[1]) and torch.equal(s1, s2) and torch.equal(c1, c2)

"""Calls with an explicit stream: what they allocate and zero is in that
stream's order, as if the call were made under torch.cuda.stream(stream)."""
import contextlib
import types

import pytest
import torch

import gated_delta_rule_21_gb300 as kda

ENTRIES = {
    "chunk_fwd": 5, "chunk_fwd_scan": 5, "chunk_bwd": 6, "chunk_fwd_save": 5,
    "chunk_bwd_from_saved": 7, "short_conv_silu": 4, "chunk_fwd_host": 5, "step": 6, "ssm_fwd": 4,
    "ssm_step": 6, "block_norm": 2, "block_norm_bwd": 4}
KEYWORDS = {"ssm_fwd": dict(head_dim=32, state_dim=32), "ssm_step": dict(head_dim=32, state_dim=32)}


def test_every_entry_runs_under_its_stream(monkeypatch):
    """On the CPU: arguments that every entry refuses, and a stream that
    records whether it was entered by then."""
    entered = []

    @contextlib.contextmanager
    def under(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    side = types.SimpleNamespace(cuda_stream=7, device=None)
    four, bad = torch.zeros(1, 2, 1, 32), torch.zeros(1, 3, 1, 32)
    for name, n in ENTRIES.items():
        args = [four] + [bad] * (n - 1)
        with pytest.raises((ValueError, TypeError)):
            getattr(kda, name)(*args, stream=side, **KEYWORDS.get(name, {}))
        assert entered == [side], name
        entered.clear()
        with pytest.raises((ValueError, TypeError)):
            getattr(kda, name)(*args, **KEYWORDS.get(name, {}))
        assert not entered, name


def busy():
    """The current stream works for some milliseconds, and what it allocates
    next is memory that holds no zeros."""
    room = torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del room
    torch.cuda._sleep(20_000_000)


@pytest.mark.gpu
def test_a_step_without_a_workspace_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(1)
    B, H, K, V = 8, 4, 128, 128
    ch = H * (2 * K + V)

    def rand(*s, std=1.0):
        return std * torch.randn(*s, generator=gen, device="cuda")

    x = rand(B, ch).bfloat16()
    q, k, v = (t.unflatten(1, (H, -1)) for t in x.split([H * K, H * K, H * V], 1))
    g, beta, w = -rand(B, H, K).abs(), torch.sigmoid(rand(B, H)), rand(ch, 4, std=0.5)
    state, cache = rand(B, H, K, V, std=0.3), rand(B, 3, ch).bfloat16()

    def go(state, cache, **kw):
        return kda.step(q, k, v, g, beta, state, conv_w=w, conv_state=cache, l2norm_qk=True, **kw)

    s1, c1 = state.clone(), cache.clone()
    want = [go(s1, c1, workspace=kda.alloc_step_workspace(B, H)) for _ in range(4)]
    s2, c2 = state.clone(), cache.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    got = [go(s2, c2, stream=side) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(s1, s2) and torch.equal(c1, c2)
    assert torch.equal(c2, x[:, None].expand(-1, 3, -1))


@pytest.mark.gpu
def test_prompts_and_norms_without_a_workspace_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rand(*s, std=1.0):
        return std * torch.randn(*s, generator=gen, device="cuda")

    H, P, N = 4, 64, 64
    ch = H * P + 2 * N
    x, dt, w, A = rand(2, 300, ch).bfloat16(), rand(2, 300, H).bfloat16(), rand(ch, 4), -rand(H).abs()
    ids = torch.ones(2, 300, dtype=torch.int32, device="cuda")
    ids[:, 120:] = 2
    y, wp, gate = rand(500, 264).bfloat16(), rand(264), rand(5, 264).bfloat16()
    d = rand(500, 264).bfloat16()

    def go(**kw):
        a = kda.ssm_fwd(x, dt, w, A, head_dim=P, state_dim=N, segment_ids=ids,
                        output_final_state=True, **kw)
        out, _, stats = kda.block_norm(y, wp, gate=gate, save_stats=True, **kw)
        b = kda.block_norm_bwd(y, wp, stats, d, gate=gate, **kw)
        return [*a, out, stats, *(t for t in b if t is not None)]

    want = go()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    got = go(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))

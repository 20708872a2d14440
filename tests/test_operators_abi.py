"""Refusals of the state space, single-token and block-norm entry points, on
the host and before anything is enqueued: no GPU is needed."""
import ctypes

import pytest
import torch

import gated_delta_rule_21_gb300 as kda
from gated_delta_rule_21_gb300 import build as kbuild

FAKE = 0x10000      # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def ssm_shape(B=1, T=64, H=4, P=64, N=128, G=1, dtype=1, xs=(4096, 512), zs=(4096, 256),
              ds=(64, 4)):
    return kda.kda_ssm_shape(B, T, H, P, N, G, dtype, *xs, *zs, *ds)


def ssm_fwd(L, impl=0, nbytes=1 << 30, ws=FAKE, xbc=FAKE, dt=FAKE, z=FAKE, w=FAKE, A=FAKE,
            s0=None, c0=None, y=FAKE, fs=None, co=None, **shape):
    return L.kda_ssm_fwd(ssm_shape(**shape), xbc, dt, z, w, None, A, None, None, s0, c0, None, y,
                         fs, co, ws, nbytes, impl, None)


@pytest.mark.parametrize("kw,want", [
    (dict(xbc=None), 1), (dict(dt=None), 1), (dict(w=None), 1), (dict(A=None), 1),
    (dict(y=None), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(G=0), 1),
    (dict(H=4, G=3), 1), (dict(dtype=5), 1), (dict(impl=9), 1),
    (dict(P=48), 2), (dict(N=256), 2), (dict(N=16), 2), (dict(B=1 << 15, T=1 << 15), 2),
    (dict(H=1 << 18, P=128), 2),
    (dict(xbc=FAKE + 8), 3), (dict(z=FAKE + 2), 3), (dict(s0=FAKE + 4), 3), (dict(y=FAKE + 8), 3),
    (dict(xs=(4096, 516)), 3), (dict(zs=(4092, 256)), 3), (dict(ws=FAKE + 16), 3),
    (dict(ws=None), 4), (dict(nbytes=64), 4)])
def test_ssm_fwd_refuses(L, kw, want):
    assert ssm_fwd(L, **kw) == want


def test_ssm_fwd_strides_of_a_gate_that_is_absent_are_not_read(L):
    assert ssm_fwd(L, z=None, zs=(3, 5), nbytes=64) == 4


def test_ssm_fwd_on_the_cuda_cores_needs_no_alignment(L):
    odd = dict(xbc=FAKE + 2, z=FAKE + 6, s0=FAKE + 4, c0=FAKE + 2, y=FAKE + 2, fs=FAKE + 4,
               co=FAKE + 2, xs=(40001, 517), zs=(40001, 517))
    assert ssm_fwd(L, impl=kda.IMPLS["simt"], nbytes=64, **odd) == 4
    assert ssm_fwd(L, impl=kda.IMPLS["simt"], nbytes=64, w=FAKE + 4) == 3
    assert ssm_fwd(L, impl=kda.IMPLS["tc"], nbytes=64, **odd) == 3


def ssm_step(L, xbc=FAKE, dt=FAKE, w=FAKE, A=FAKE, slots=None, n_slots=4, conv=FAKE, state=FAKE,
             y=FAKE, ws=FAKE, nbytes=1 << 20, **shape):
    return L.kda_ssm_step(ssm_shape(**dict(dict(T=1), **shape)), xbc, dt, None, w, None, A, None,
                          None, slots, n_slots, conv, state, y, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(xbc=None), 1), (dict(conv=None), 1), (dict(state=None), 1), (dict(y=None), 1),
    (dict(T=2), 1), (dict(n_slots=0), 1), (dict(B=5), 1), (dict(H=4, G=3), 1), (dict(P=16), 2),
    (dict(w=FAKE + 4), 3), (dict(state=FAKE + 4), 3), (dict(ws=FAKE + 16), 3),
    (dict(ws=None), 4), (dict(nbytes=128), 4)])
def test_ssm_step_refuses(L, kw, want):
    assert ssm_step(L, **kw) == want


def step(L, q=FAKE, g=FAKE, conv_w=None, conv=None, slots=None, n_slots=4, state=FAKE, o=FAKE,
         scale=0.1, ws=FAKE, nbytes=1 << 20, shape=(1, 1, 4, 128, 128, 1)):
    return L.kda_step(kda.kda_shape(*shape), q, FAKE, FAKE, 512, 512, 512, g, FAKE, scale, conv_w,
                      conv, 0, slots, n_slots, state, o, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(g=None), 1), (dict(state=None), 1), (dict(o=None), 1),
    (dict(conv_w=FAKE), 1), (dict(conv=FAKE), 1), (dict(scale=float("nan")), 1),
    (dict(shape=(1, 2, 4, 128, 128, 1)), 1), (dict(shape=(9, 1, 4, 128, 128, 1)), 1),
    (dict(n_slots=0), 1), (dict(shape=(1, 1, 4, 96, 128, 1)), 2), (dict(state=FAKE + 8), 3),
    (dict(conv_w=FAKE + 4, conv=FAKE), 3), (dict(ws=FAKE + 128), 3), (dict(ws=None), 4),
    (dict(nbytes=256), 4)])
def test_step_refuses(L, kw, want):
    assert step(L, **kw) == want


def desc(rows=8, dim=64, dtype=1, act=1, gate_rows=8, scale=1.0, eps=1e-6):
    return kda.kda_norm_desc(rows, dim, dtype, act, gate_rows, scale, eps)


def norm(L, y=FAKE, w=FAKE, gate=None, w_pre=None, out=FAKE, x=None, **d):
    return L.kda_block_norm_fwd(desc(**d), y, w, None, gate, w_pre, out, x, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(y=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(w_pre=FAKE), 1),
    (dict(x=FAKE), 1), (dict(rows=0), 1), (dict(dim=0), 1), (dict(dtype=3), 1), (dict(act=4), 1),
    (dict(act=-1), 1), (dict(gate=FAKE, gate_rows=3), 1), (dict(gate=FAKE, gate_rows=0), 1),
    (dict(scale=float("nan")), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(dim=16385), 2), (dict(rows=1 << 31), 2)])
def test_block_norm_refuses(L, kw, want):
    assert norm(L, **kw) == want


def test_block_norm_in_place_keeps_nothing_for_the_backward(L):
    """The backward reads the residual, so out cannot replace it then."""
    args = [desc(), FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, None]
    assert L.kda_block_norm_fwd(*args) == 1


def norm_bwd(L, stats=FAKE, res=None, gate=None, w_pre=None, d_out=FAKE, d_x=None, dy=FAKE,
             d_res=None, d_gate=None, dw=FAKE, dw_pre=None, ws=FAKE, nbytes=1 << 30, **d):
    return L.kda_block_norm_bwd(desc(**d), FAKE, FAKE, res, gate, w_pre, stats, d_out, d_x, dy,
                                d_res, d_gate, dw, dw_pre, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(stats=None), 1), (dict(dy=None), 1), (dict(dw=None), 1), (dict(d_out=None), 1),
    (dict(d_x=FAKE), 1), (dict(w_pre=FAKE), 1), (dict(dw_pre=FAKE), 1), (dict(d_res=FAKE), 1),
    (dict(d_gate=FAKE), 1), (dict(gate=FAKE, gate_rows=5), 1), (dict(dim=16385), 2),
    (dict(ws=FAKE + 4), 3), (dict(ws=None), 4), (dict(nbytes=100), 4)])
def test_block_norm_bwd_refuses(L, kw, want):
    assert norm_bwd(L, **kw) == want


def test_workspace_sizes(L):
    assert kda.step_workspace_size(3, 70) == 256 + 1024     # header, 4 bytes per sequence and head
    assert kda.step_workspace_size(0, 4) == 0 and kda.step_workspace_size(1 << 20, 1 << 20) == 0
    assert kda.ssm_workspace_size(1, 64, 4, 64, 128, 1, impl="simt") > 0
    assert kda.ssm_workspace_size(1, 64, 4, 40, 128, 1) == 0
    assert kda.block_norm_workspace_size(8, 20000) == 0
    assert kda.block_norm_workspace_size(8, 64, gate_rows=3) == 0
    # a unit's sums of dw_post and dw_pre, and of the gate where rows share one
    one = kda.block_norm_workspace_size(1, 64)
    assert one == 2 * 64 * 4
    assert kda.block_norm_workspace_size(8192, 4096, gate_rows=4) >= \
        kda.block_norm_workspace_size(8192, 4096, gate_rows=8192)


def test_python_checks_come_before_the_library():
    cpu = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        kda.block_norm(cpu, torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        kda.ssm_fwd(cpu[None], cpu[None], cpu, cpu, head_dim=32, state_dim=32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.step(cpu[None], cpu[None], cpu[None], cpu[None], cpu, cpu)
    assert ctypes.sizeof(kda.kda_ssm_shape) == 80 and ctypes.sizeof(kda.kda_norm_desc) == 40


def test_a_gate_that_is_broadcast_over_leading_rows_is_refused():
    """Each gate row serves consecutive rows: [B,1,D] and [1,1,D] beside
    [B,T,D] are what broadcasting means, [1,T,D] is not; [B,T/2,D] can only
    mean consecutive rows."""
    y = torch.zeros(2, 6, 8)
    for shape in ((2, 6, 8), (2, 1, 8), (1, 1, 8), (2, 3, 8), (2, 8), (4, 8), (1, 8), (8,)):
        kda._norm_desc(y, torch.zeros(shape), "silu", 1.0, 1e-6)
    for shape in ((1, 6, 8), (1, 2, 8)):
        with pytest.raises(ValueError, match="consecutive"):
            kda._norm_desc(y, torch.zeros(shape), "silu", 1.0, 1e-6)
    kda._norm_desc(torch.zeros(12, 8), torch.zeros(4, 8), "silu", 1.0, 1e-6)
    with pytest.raises(ValueError, match="consecutive"):
        kda._norm_desc(torch.zeros(2, 3, 4, 8), torch.zeros(2, 1, 4, 8), "silu", 1.0, 1e-6)
    kda._norm_desc(torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 1, 8), "silu", 1.0, 1e-6)

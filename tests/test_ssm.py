"""GPU tests of the state space operator on prompts (kda_ssm_fwd) against the
plain 64-bit recurrence, and of prompts followed by single tokens.

Tolerances.  fp32: the scan is fp32 (2^-24 per operation; decays multiply an
old state's error by less than one, so a state is off by about the length of
its memory times 2^-24 of its terms) and y adds up to 128 products: 2e-5 of
the largest value.  bf16: y is rounded once, 2^-9 on average and eps / 2 =
2^-8 at most of the value; the tensor-core path also rounds the operands of
its products for y to bf16 (see the kernel), each product by up to 2^-7, whose
sum over many terms stays near 2^-8 of the terms' root sum of squares: rel-L2
5e-3 and 2^-5 of the largest value elementwise.  The final state is fp32-grade
on both paths: 2e-5."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu


def rand(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, dtype=torch.float64) * std


class Case:
    def __init__(self, B, T, H, P, N, G, dtype, ids=None, init=False, slim=False, seed=0,
                 A=(1, 16), dt=(-3.0, 1.0)):
        gen = torch.Generator().manual_seed(seed + T * 3 + H)
        self.dims, self.dtype, self.ids = (B, T, H, P, N, G), dtype, ids
        ch, hp = H * P + 2 * G * N, H * P
        f32 = torch.float32
        width = -(-(hp + ch + H) // 8) * 8
        self.proj = plain64.cast(rand(gen, B, T, width), dtype)
        self.w = plain64.cast(rand(gen, ch, 4, std=0.5), f32)
        u = torch.rand(H, generator=gen, dtype=torch.float64)
        self.A = plain64.cast(-(A[0] + (A[1] - A[0]) * u), f32)
        self.bias = plain64.cast(rand(gen, ch, std=0.1), f32)
        self.db = plain64.cast(dt[0] + dt[1] * rand(gen, H), f32)
        self.D = plain64.cast(1 + rand(gen, H, std=0.2), f32)
        self.s0 = plain64.cast(rand(gen, B, H, N, P, std=0.3), f32) if init else None
        self.c0 = plain64.cast(rand(gen, B, 3, ch), dtype) if init else None
        self.slim = slim

    def parts(self, proj):
        B, T, H, P, N, G = self.dims
        a, b = H * P, 2 * H * P + 2 * G * N
        return proj[..., a:b], proj[..., b:b + H], proj[..., :a]

    def gpu(self, impl="auto", upto=None, **kw):
        import gated_delta_rule_21_gb300 as kda
        B, T, H, P, N, G = self.dims
        x, dt, z = self.parts(self.proj[0].cuda()[:, :upto])
        opt = {} if self.slim else dict(conv_bias=self.bias[0].cuda(), dt_bias=self.db[0].cuda(),
                                        D=self.D[0].cuda(), z=z)
        if self.s0 is not None:
            opt.update(initial_state=self.s0[0].cuda(), conv_state=self.c0[0].cuda())
        if self.ids is not None:
            opt["segment_ids"] = self.ids[:, :upto].contiguous().cuda()
        out = kda.ssm_fwd(x, dt, self.w[0].cuda(), self.A[0].cuda(), head_dim=P, state_dim=N,
                          output_final_state=True, impl=impl, **opt, **kw)
        torch.cuda.synchronize()
        return out

    def plain(self):
        B, T, H, P, N, G = self.dims
        op = plain64.Ssm(self.w[1], self.A[1], H, P, N, G) if self.slim else plain64.Ssm(
            self.w[1], self.A[1], H, P, N, G, self.bias[1], self.db[1], self.D[1])
        ch = H * P + 2 * G * N
        ys, ss, cs = [], [], []
        for b in range(B):
            x, dt, z = self.parts(self.proj[1][b])
            s0 = self.s0[1][b] if self.s0 is not None else torch.zeros(H, N, P, dtype=torch.float64)
            c0 = self.c0[1][b] if self.c0 is not None else torch.zeros(3, ch, dtype=torch.float64)
            y, s, c = op.row(x, dt, None if self.slim else z,
                             None if self.ids is None else self.ids[b], s0, c0)
            ys.append(y)
            ss.append(s)
            cs.append(c)
        return torch.stack(ys), torch.stack(ss), torch.stack(cs)

    def check(self, impl="auto"):
        (y, s, c), (yr, sr, cr) = self.gpu(impl), self.plain()
        d = (y.double().cpu() - yr).abs()
        if self.dtype == torch.float32:
            assert d.max() <= 2e-5 * yr.abs().max() + 1e-30, d.max()
        else:
            assert d.max() <= 2 ** -5 * yr.abs().max() + 1e-30, d.max()
            assert d.norm() <= 5e-3 * yr.norm() + 1e-30, d.norm() / yr.norm()
        d = (s.double().cpu() - sr).abs()
        assert d.max() <= 2e-5 * sr.abs().max() + 1e-30, d.max() / sr.abs().max()
        assert torch.equal(c.double().cpu(), cr)
        if self.ids is not None:
            assert not y.cpu()[self.ids == 0].any()


IMPLS = [(torch.float32, "simt"), (torch.float32, "tc"), (torch.bfloat16, "simt"),
         (torch.bfloat16, "auto")]
DIMS = [(1, 1, 1, 32, 32, 1), (2, 3, 2, 64, 64, 1), (1, 65, 3, 128, 32, 3), (2, 128, 4, 32, 128, 2),
        (1, 129, 8, 64, 128, 1), (1, 300, 2, 128, 128, 1), (3, 257, 5, 64, 64, 5),
        (1, 640, 4, 32, 64, 2)]


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("init", [False, True])
def test_prompt(dims, dtype, impl, init):
    Case(*dims, dtype, init=init).check(impl)


@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_parts_left_out(dtype, impl):
    Case(2, 200, 4, 64, 128, 2, dtype, slim=True, dt=(0.0, 1.0)).check(impl)


ROWS = {
    "short runs": [1] * 3 + [2] + [3] * 2 + [0] * 2 + [4] * 60 + [5] + [6] * 63 + [7] * 2,
    "padding first": [0] * 5 + [1] * 100 + [0] * 3 + [1] * 40,
    "padding last": [1] * 90 + [2] * 40 + [0] * 70,
    "empty": [0] * 140,
    "one token": [0] * 66 + [3] + [0] * 10,
    "same id after padding": [2] * 2 + [0] + [2] * 2 + [0] * 130 + [2] * 70,
    "every token": list(range(1, 200)),
    "at the edges": [1] * 64 + [2] * 64 + [3] * 128 + [4] * 2,
    "long run": [7] * 400,
}


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("init", [False, True])
def test_packed_rows(dtype, impl, init):
    T = max(map(len, ROWS.values()))
    ids = torch.zeros(len(ROWS), T, dtype=torch.int32)
    for i, r in enumerate(ROWS.values()):
        ids[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    Case(len(ROWS), T, 2, 32, 64, 1, dtype, ids=ids, init=init).check(impl)


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("A,dt", [((0.0, 0.0), (-3.0, 1.0)), ((1e-4, 1e-3), (-5.0, 0.5)),
                                  ((50.0, 400.0), (2.0, 1.0)), ((1.0, 16.0), (-60.0, 1.0))])
def test_decays_from_none_to_total(dtype, impl, A, dt):
    Case(1, 400, 4, 64, 64, 1, dtype, init=True, A=A, dt=dt).check(impl)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_follow_a_prompt(dtype):
    """Prompt to T - 5, then five tokens: y and states of the whole."""
    import gated_delta_rule_21_gb300 as kda
    c = Case(2, 150, 4, 64, 128, 2, dtype, init=True)
    B, T, H, P, N, G = c.dims
    yr, sr, cr = c.plain()
    _, state, conv = c.gpu(upto=T - 5)
    for t in range(T - 5, T):
        x, dt, z = c.parts(c.proj[0][:, t].cuda())
        y = kda.ssm_step(x, dt, c.w[0].cuda(), c.A[0].cuda(), state, conv, head_dim=P,
                         state_dim=N, conv_bias=c.bias[0].cuda(), dt_bias=c.db[0].cuda(),
                         D=c.D[0].cuda(), z=z)
        tol = (2e-5 if dtype == torch.float32 else 2 ** -7) * yr[:, t].abs().max()
        assert (y.double().cpu() - yr[:, t]).abs().max() <= tol
    assert (state.double().cpu() - sr).abs().max() <= 2e-5 * sr.abs().max()
    assert torch.equal(conv.double().cpu(), cr)


def test_calls_repeat_bit_for_bit_and_run_in_a_graph():
    import gated_delta_rule_21_gb300 as kda
    c = Case(2, 300, 4, 64, 128, 2, torch.bfloat16, init=True)
    ws = kda.alloc_ssm_workspace(*c.dims)
    first = c.gpu(workspace=ws)
    again = c.gpu(workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    x, dt, z = c.parts(c.proj[0].cuda())
    w, A = c.w[0].cuda(), c.A[0].cuda()
    want = kda.ssm_fwd(x, dt, w, A, head_dim=64, state_dim=128, z=z, workspace=ws)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = kda.ssm_fwd(x, dt, w, A, head_dim=64, state_dim=128, z=z, workspace=ws)[0]
    held.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, held)


@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_padding_may_hold_anything(dtype, impl):
    """NaN and infinities at padding change nothing, bit for bit."""
    ids = torch.ones(3, 300, dtype=torch.int32)
    ids[0, 250:] = 0
    ids[1, :70] = 0
    ids[1, 200:230] = 0
    ids[2] = 0
    clean = Case(3, 300, 2, 64, 64, 1, dtype, ids=ids, init=True)
    want = clean.gpu(impl)
    for bad in (float("nan"), float("inf"), -float("inf")):
        c = Case(3, 300, 2, 64, 64, 1, dtype, ids=ids, init=True)
        c.proj[0][ids == 0] = bad
        got = c.gpu(impl)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_a_reset_ends_what_came_before(dtype, impl):
    """A run of NaN leaves the blocks after it untouched."""
    ids = torch.ones(1, 600, dtype=torch.int32)
    ids[0, 128:] = 2
    c = Case(1, 600, 2, 32, 64, 1, dtype, ids=ids)
    want = c.gpu(impl)
    c.proj[0][0, :128] = float("nan")
    got = c.gpu(impl)
    assert torch.equal(want[0][0, 128:], got[0][0, 128:]) and torch.equal(want[1], got[1])


def test_segments_of_the_fp32_kernel_agree_with_one_chain():
    """Few heads and a long row (many segments) against many rows (one)."""
    import gated_delta_rule_21_gb300 as kda
    c = Case(1, 1500, 1, 32, 32, 1, torch.float32, init=True)
    c.check("simt")
    assert kda.ssm_workspace_size(1, 1500, 1, 32, 32, 1, torch.float32, "simt") > \
        kda.ssm_workspace_size(1, 60, 1, 32, 32, 1, torch.float32, "simt")


def test_device_status_is_clean():
    import gated_delta_rule_21_gb300 as kda
    c = Case(2, 300, 4, 64, 128, 2, torch.bfloat16)
    ws = kda.alloc_ssm_workspace(*c.dims)
    c.gpu(workspace=ws)
    assert kda.read_device_status(ws) == 0

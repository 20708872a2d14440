"""GPU tests of the state space operator on values at the edges: step widths,
inputs and cached states that are not finite, decays of any size.

What is not finite may reach only what the recurrence lets it reach: tokens of
its own run from its own place on, and the state if that run is the last.
Everything else stays within the tolerances of test_ssm.py."""
import pytest
import torch

from test_ssm import IMPLS, Case

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def near(got, ref, dtype, what):
    """Finite exactly where the plain form is, and near it there."""
    got = got.double().cpu()
    ok = ref.isfinite()
    assert torch.equal(got.isfinite(), ok), \
        f"{what}: {int((got.isfinite() != ok).sum())} of {ok.numel()} finite in one form only"
    got, ref = got[ok], ref[ok]
    if ref.numel() == 0:
        return
    d = (got - ref).abs()
    if dtype == torch.float32:
        assert d.max() <= 2e-5 * ref.abs().max() + 1e-30, (what, d.max())
    else:
        assert d.max() <= 2 ** -5 * ref.abs().max() + 1e-30, (what, d.max())
        assert d.norm() <= 5e-3 * ref.norm() + 1e-30, (what, d.norm() / ref.norm())


def check(c, impl):
    (y, s, conv), (yr, sr, cr) = c.gpu(impl), c.plain()
    near(y, yr, c.dtype, "y")
    near(s, sr, torch.float32, "state")
    assert torch.equal(conv.double().cpu().nan_to_num(9.0), cr.nan_to_num(9.0))


def put(c, part, b, t, index, value):
    """Sets one input of token t of row b: part 0 xbc, 1 dt, 2 z."""
    for proj in c.proj:
        c.parts(proj[b])[part][t, index] = value


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_step_widths_that_are_not_finite(dtype, impl, value):
    """In one head, at the first and a later token, in a row of one run and in
    a row of several that share blocks.  (-inf is a step of width 0.)"""
    T = 300
    ids = torch.ones(4, T, dtype=torch.int32)
    ids[2, 40:60], ids[2, 60:] = 2, 3
    ids[3, 30:200], ids[3, 200:] = 0, 2
    c = Case(4, T, 3, 32, 64, 1, dtype, ids=ids, init=True)
    put(c, 1, 0, 0, 1, value)
    put(c, 1, 1, 77, 0, value)
    put(c, 1, 2, 45, 2, value)
    put(c, 1, 2, 61, 0, value)
    put(c, 1, 3, 7, 1, value)
    put(c, 1, 3, 90, 1, value)          # padding: nothing
    check(c, impl)


def between(dtype, every, size):
    """Widths of about 1e-3 and 8 by turns: short runs of tokens that remember
    each other behind sums of decays that have run far, and outputs of which one
    term is nearly all."""
    c = Case(2, 400, 3, 32, 64, 1, dtype, init=True, A=(size, 2 * size), dt=(0.0, 0.0))
    for proj in c.proj:
        dt = c.parts(proj)[1]
        dt[...] = -7.0 if size < 1e3 else -14.0      # |A| d near 0.3 and 1
        dt[:, ::every] = 8.0
    return c


def test_outputs_of_one_term_in_fp32():
    check(between(torch.float32, 2, 300.0), "tc")


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("size", [40.0, 400.0, 4000.0, 3e37])
def test_decays_of_any_size(dtype, impl, size):
    """|A| d of 80 to 1e38 at every token: only a token's own term is left, and
    its factor d must not carry the rounding of the sums around it."""
    c = Case(2, 260, 3, 64, 64, 1, dtype, init=True, A=(size, 1.5 * size), dt=(2.0, 1.0))
    check(c, impl)


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("every", [2, 5])
@pytest.mark.parametrize("size", [300.0, 1e6])
def test_small_decays_between_total_ones(dtype, impl, every, size):
    check(between(dtype, every, size), impl)


def runs(T):
    """A whole row, runs that share blocks, runs and padding."""
    ids = torch.ones(3, T, dtype=torch.int32)
    ids[1, 40:60], ids[1, 60:150], ids[1, 150:] = 2, 3, 4
    ids[2, :9], ids[2, 100:140], ids[2, 140:260], ids[2, 260:] = 0, 0, 2, 0
    return ids


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("what", ["x", "B", "C", "z"])
@pytest.mark.parametrize("G", [1, 2])
def test_inputs_that_are_not_finite(dtype, impl, value, what, G):
    """Neither earlier tokens nor other runs of the same block see them."""
    T, H, P, N = 300, 4, 64, 32
    c = Case(3, T, H, P, N, G, dtype, ids=runs(T), init=True)
    part, at = {"x": (0, P + 5), "B": (0, H * P + 3), "C": (0, H * P + G * N + 17),
                "z": (2, 2 * P + 40)}[what]
    for b, t in ((0, 130), (0, 290), (1, 30), (1, 45), (1, 170), (2, 90), (2, 115), (2, 150)):
        put(c, part, b, t, at, value)
    check(c, impl)


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("value", [NAN, INF])
def test_caches_that_are_not_finite(dtype, impl, value):
    """A state and a convolution cache reach the row's first run only."""
    T, H, P, N = 300, 4, 32, 64
    c = Case(3, T, H, P, N, 1, dtype, ids=runs(T), init=True)
    for i in range(2):
        c.s0[i][:, 1, 7, 20] = value
        c.c0[i][1, 1, H * P + 9] = value
        c.c0[i][2, 2, 2 * P + 3] = value
    check(c, impl)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [200, 1])
def test_slices_of_a_projection_of_any_width(dtype, T):
    """3 heads: the slices begin and lie at odd places.  The CUDA cores serve
    them; the strides of one token or one row mean nothing on either path."""
    H, P, N = 3, 32, 64
    c = Case(2, T, H, P, N, 1, dtype, init=True)
    width = 2 * H * P + 2 * N + H
    for i, to in enumerate((dtype, torch.float64)):
        room = torch.zeros(2, T, width + 1, dtype=to)
        room[..., 1:] = c.proj[i][..., :width]
        c.proj = (*c.proj[:i], room[..., 1:], *c.proj[i + 1:])
    c.check("simt")


def test_strides_of_a_dimension_of_one_are_not_read():
    import gated_delta_rule_21_gb300 as kda
    c = Case(1, 1, 2, 32, 32, 1, torch.bfloat16)
    x, dt, z = c.parts(c.proj[0].cuda())
    w, A = c.w[0].cuda(), c.A[0].cuda()
    want = kda.ssm_fwd(x, dt, w, A, head_dim=32, state_dim=32, z=z)[0]
    x, z = (t.as_strided(t.shape, (7, 13, 1)) for t in (x, z))
    got = kda.ssm_fwd(x, dt, w, A, head_dim=32, state_dim=32, z=z)[0]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("scale", [1.0, 3e4, 2e-5])
@pytest.mark.parametrize("dims", [(2, 300, 4, 64, 128, 2), (3, 257, 5, 128, 32, 1)])
def test_states_are_formed_to_fp32_grade(dtype, impl, scale, dims):
    """In the 2-norm, for inputs of any size: operands of 22 bits are off by 2^-23
    each, products and sums by 2^-24 a step; 1e-6 covers ten of them."""
    c = Case(*dims, dtype, init=True)
    for i in range(2):
        for part in c.parts(c.proj[i])[::2]:
            part *= scale
    c.proj = (c.proj[0], c.proj[0].double())
    (_, s, _), (_, sr, _) = c.gpu(impl), c.plain()
    d = s.double().cpu() - sr
    assert d.norm() <= 1e-6 * sr.norm(), d.norm() / sr.norm()


@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("size", [1e30, 1e4])
def test_what_is_masked_scales_nothing(dtype, impl, size):
    """Large finite values at padding, and (up to 1e4 times the others) in another
    run of the same block, cost the rest no digits."""
    T = 300
    ids = torch.ones(2, T, dtype=torch.int32)
    ids[:, 60:100], ids[:, 100:] = 2, 3
    ids[:, 20:30] = 0
    ids[:, 290:] = 0
    c = Case(2, T, 3, 64, 64, 1, dtype, ids=ids)
    big = ids == (0 if size > 1e5 else 2)
    for proj in c.proj:
        proj[..., 3 * 64:2 * 3 * 64 + 2 * 64][big] = size        # xbc
    c.proj = (c.proj[0], c.proj[0].double())
    (y, s, _), (yr, sr, _) = c.gpu(impl), c.plain()
    d = s.double().cpu() - sr
    assert d.norm() <= 1e-6 * sr.norm(), d.norm() / sr.norm()
    for run in (1, 3):
        near(y.cpu()[ids == run], yr[ids == run], dtype, "y")


@pytest.mark.parametrize("T", [70, 400])
@pytest.mark.parametrize("scale", [1.0, 1e3, 1e-3])
@pytest.mark.parametrize("init,tol", [(False, 2.5e-3), (True, 3.2e-3)])
def test_outputs_are_off_by_little_more_than_their_own_rounding(T, scale, init, tol):
    """bf16 outputs in the 2-norm.  Rounding to bf16 is off by at most 2^-9 of the
    binade, 1.7e-3 in the mean.  From zero states: that of y, and a quarter of
    that of each of C and B (sums of 128 terms) and of x and the factors (2^-12):
    2.0e-3.  Where a state enters that is all of y, that of C, S and y: 3.0e-3."""
    c = Case(2, T, 4, 64, 128, 2, torch.bfloat16, init=init)
    for part in c.parts(c.proj[0])[::2]:
        part *= scale
    c.proj = (c.proj[0], c.proj[0].double())
    y, yr = c.gpu("tc")[0], c.plain()[0]
    d = y.double().cpu() - yr
    assert d.norm() <= tol * yr.norm(), d.norm() / yr.norm()


@pytest.mark.parametrize("impl", ["simt", "tc"])
@pytest.mark.parametrize("dims", [(2, 300, 4, 64, 128, 2), (1, 400, 3, 128, 64, 1)])
def test_fp32_outputs_are_formed_to_fp32_grade(dims, impl):
    """From zero states, in the 2-norm: x and the factors are two parts of 22 bits,
    C and B three of 24, a factor's exponential is off by 2^-22: below 1e-6."""
    c = Case(*dims, torch.float32)
    y, yr = c.gpu(impl)[0], c.plain()[0]
    d = y.double().cpu() - yr
    assert d.norm() <= 1e-6 * yr.norm(), d.norm() / yr.norm()

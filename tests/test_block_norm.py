"""GPU tests of the block norms (kda_block_norm_fwd / _bwd) against the plain
64-bit form and its derivatives.

Tolerances.  An output of type t is rounded once: half a step, eps(t) / 2
relative to the value.  Before that the kernel works in fp32: a sum of D
squares and a handful of products, each off by 2^-24; with sums of at most
16 sequential terms per thread and a tree, the relative error of a norm stays
below 32 * 2^-24 = 2e-6, and an output that adds terms is off by that much of
the largest of them.  4e-6 of the largest value in the row (or tensor) covers
both norms.  Column sums over rows add up to `rows` terms in fp32: 2^-24 *
(rows per thread + 64) of the sum of the terms' sizes."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

F32 = 4e-6


def near(got, ref, dtype, size, what):
    """Within one rounding of the value and F32 of `size`."""
    got = got.double().cpu()
    tol = torch.finfo(dtype).eps / 2 * 1.01 * ref.abs() + F32 * size
    bad = (got - ref).abs() - tol
    assert bad.max() <= 0, f"{what}: {(bad > 0).sum()} of {bad.numel()} off, by up to {bad.max():.3e}"


def make(rows, D, dtype, gate_rows, res, pre, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + rows * 31 + D)

    def rand(*s, std=1.0):
        return torch.randn(*s, generator=g, dtype=torch.float64) * std

    x = {"y": plain64.cast(rand(rows, D), dtype),
         "gate": plain64.cast(rand(gate_rows, D, std=2.0), dtype) if gate_rows else None,
         "residual": plain64.cast(rand(rows, D, std=2.0), dtype) if res else None,
         "w_post": plain64.cast(1 + rand(D, std=0.2), torch.float32),
         "w_pre": plain64.cast(1 + rand(D, std=0.2), torch.float32) if pre else None,
         "d_out": plain64.cast(rand(rows, D), dtype),
         "d_x": plain64.cast(rand(rows, D), dtype) if pre else None}
    dev = {k: None if v is None else v[0].cuda() for k, v in x.items()}
    ref = {k: None if v is None else v[1] for k, v in x.items()}
    return dev, ref


def term_sizes(ref, out, act, scale, eps, d_out):
    """The largest terms that the gradients of residual, gate and y add up:
    at D = 1, say, those of y cancel down to eps and their rounding stays."""
    def inv(v):
        return torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)

    r = ref["d_out"].abs().amax() if d_out else torch.zeros(())
    if ref["w_pre"] is not None:
        r = r + (inv(out) * ref["d_x"] * ref["w_pre"]).abs().amax()
    u = (ref["y"] * inv(ref["y"]) * ref["w_post"]).abs().amax()
    a = d = torch.ones((), dtype=torch.float64)
    if ref["gate"] is not None:
        g = ref["gate"].clone().requires_grad_()
        a = plain64.GATES[act](g)
        d, = torch.autograd.grad(a.sum(), g)
        a, d = a.detach().abs().amax(), d.abs().amax()
    return {"residual": r, "gate": abs(scale) * u * d * r,
            "y": abs(scale) * inv(ref["y"]).amax() * a * ref["w_post"].abs().amax() * r}


def check(dev, ref, dtype, act, scale=0.7, eps=1e-6, d_out=True, backward=True):
    import gated_delta_rule_21_gb300 as kda
    kw = dict(residual=dev["residual"], gate=dev["gate"], gate_act=act, scale=scale,
              w_pre=dev["w_pre"], eps=eps)
    out, x, stats = kda.block_norm(dev["y"], dev["w_post"], save_stats=True, **kw)
    leaf = {k: ref[k].clone().requires_grad_() for k in
            ("y", "gate", "residual", "w_post", "w_pre") if ref[k] is not None}
    o, xr = plain64.block_norm(leaf["y"], leaf["w_post"], leaf.get("residual"), leaf.get("gate"),
                               act, scale, leaf.get("w_pre"), eps)
    near(out, o.detach(), dtype, o.detach().abs().amax(-1, keepdim=True), "out")
    if xr is not None:
        near(x, xr.detach(), dtype, xr.detach().abs().amax(-1, keepdim=True), "x")
    else:
        assert x is None
    if not backward:
        return
    got = kda.block_norm_bwd(dev["y"], dev["w_post"], stats, dev["d_out"] if d_out else None,
                             d_x=dev["d_x"], **kw)
    loss = 0.0
    if d_out:
        loss = (o * ref["d_out"]).sum()
    if xr is not None:
        loss = loss + (xr * ref["d_x"]).sum()
    loss.backward()
    rows = ref["y"].shape[0]
    size = term_sizes(ref, o.detach(), act, scale, eps, d_out)
    dy, dres, dgate, dw_post, dw_pre = got
    for t, name in ((dy, "y"), (dres, "residual"), (dgate, "gate")):
        if name not in leaf:
            assert t is None
            continue
        want = leaf[name].grad
        # a gate row sums the gradients of the rows it serves
        per = rows // want.shape[0]
        near(t, want, dtype, 4 * size[name] * per ** 0.5, f"d{name}")
    for t, name in ((dw_post, "w_post"), (dw_pre, "w_pre")):
        if name not in leaf:
            assert t is None
            continue
        want = leaf[name].grad
        # every term of a column sum is a product of O(1) values here
        near(t, want, torch.float32, 4 * (want.abs().amax() + rows ** 0.5), f"d{name}")


CASES = [(1, 1), (3, 7), (5, 24), (37, 64), (2, 128), (300, 128), (4, 1000), (3, 1001), (9, 4096),
         (700, 512), (2, 8192), (3, 5181), (2, 16384), (1, 16383), (2, 12288 + 8), (64, 33)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", CASES)
def test_norms_gate_each_and_their_gradients(rows, D, dtype):
    dev, ref = make(rows, D, dtype, rows, True, True)
    check(dev, ref, dtype, "sigmoid")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", CASES)
def test_gated_norm_alone(rows, D, dtype):
    dev, ref = make(rows, D, dtype, rows, False, False, seed=1)
    check(dev, ref, dtype, "silu")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,gates,D", [(6, 2, 40), (1200, 3, 128), (1200, 600, 128),
                                          (40, 1, 4096), (900, 450, 1000), (1216, 4, 96),
                                          (15, 5, 16384), (1, 1, 64), (800, 2, 77),
                                          (2000, 1000, 17)])
def test_gate_rows_shared_by_rows(rows, gates, D, dtype):
    dev, ref = make(rows, D, dtype, gates, True, True, seed=2)
    check(dev, ref, dtype, "tanh")


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu", "tanh"])
@pytest.mark.parametrize("res,pre", [(False, True), (True, False)])
@pytest.mark.parametrize("gates", [0, 33, 3])
def test_parts_left_out(act, res, pre, gates):
    dev, ref = make(33, 200, torch.float32, gates, res, pre, seed=3)
    check(dev, ref, torch.float32, act, scale=-1.3, eps=0.0)


def test_only_the_second_norms_gradient():
    dev, ref = make(21, 264, torch.bfloat16, 21, True, True, seed=4)
    check(dev, ref, torch.bfloat16, "sigmoid", d_out=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pointers_that_are_not_aligned(dtype):
    dev, ref = make(19, 256, dtype, 19, True, True, seed=5)
    for k in ("y", "gate", "residual", "d_out", "d_x"):
        room = torch.empty(19 * 256 + 1, dtype=dtype, device="cuda")
        room[1:].copy_(dev[k].flatten())
        dev[k] = room[1:].view(19, 256)
    check(dev, ref, dtype, "sigmoid")


def test_gradient_against_differences():
    """The loss along a random direction, differenced in 64 bits: the step
    1e-5 leaves about 1e-9 of the loss, the gradients 2e-6 of its terms."""
    import gated_delta_rule_21_gb300 as kda
    dev, ref = make(12, 80, torch.float32, 4, True, True, seed=6)
    kw = dict(residual=dev["residual"], gate=dev["gate"], gate_act="silu", scale=0.5,
              w_pre=dev["w_pre"], eps=1e-3)
    _, _, stats = kda.block_norm(dev["y"], dev["w_post"], save_stats=True, **kw)
    grads = dict(zip(("y", "residual", "gate", "w_post", "w_pre"), kda.block_norm_bwd(
        dev["y"], dev["w_post"], stats, dev["d_out"], d_x=dev["d_x"], **kw)))
    gen = torch.Generator().manual_seed(1)
    for name, grad in grads.items():
        way = torch.randn(ref[name].shape, generator=gen, dtype=torch.float64)

        def loss(h):
            at = dict(ref, **{name: ref[name] + h * way})
            o, x = plain64.block_norm(at["y"], at["w_post"], at["residual"], at["gate"], "silu",
                                      0.5, at["w_pre"], 1e-3)
            return (o * ref["d_out"]).sum() + (x * ref["d_x"]).sum()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = grad.double().cpu() * way
        assert (terms.sum() - want).abs() <= 1e-5 * terms.abs().sum() + 1e-6, name


def test_rows_of_zeros_and_values_that_are_not_finite():
    import gated_delta_rule_21_gb300 as kda
    dev, ref = make(6, 136, torch.bfloat16, 6, True, True, seed=7)
    y = dev["y"].clone()
    y[1] = 0
    y[3, 5] = float("nan")
    y[4, 9] = float("inf")
    kw = dict(residual=dev["residual"], gate=dev["gate"], w_pre=dev["w_pre"])
    out, x = kda.block_norm(y, dev["w_post"], **kw)
    ok = [0, 1, 2, 5]
    o, xr = plain64.block_norm(y[ok].double().cpu(), ref["w_post"], ref["residual"][ok],
                               ref["gate"][ok], w_pre=ref["w_pre"])
    near(out[ok], o, torch.bfloat16, o.abs().amax(), "out")
    near(x[ok], xr, torch.bfloat16, xr.abs().amax(), "x")
    assert x[3].isnan().all() and x[4, 9].isnan() and out[4, 9].isnan()


def test_out_may_be_the_residual_and_calls_repeat_bit_for_bit():
    import gated_delta_rule_21_gb300 as kda
    dev, _ = make(400, 264, torch.bfloat16, 8, True, True, seed=8)
    kw = dict(gate=dev["gate"], w_pre=dev["w_pre"])
    out, x, stats = kda.block_norm(dev["y"], dev["w_post"], residual=dev["residual"],
                                   save_stats=True, **kw)
    room = dev["residual"].clone()
    out2, x2 = kda.block_norm(dev["y"], dev["w_post"], residual=room, out=room, **kw)
    assert torch.equal(out, out2) and torch.equal(x, x2)
    bwd = [kda.block_norm_bwd(dev["y"], dev["w_post"], stats, dev["d_out"], d_x=dev["d_x"],
                              residual=dev["residual"], **kw) for _ in range(2)]
    for a, b in zip(*bwd):
        assert torch.equal(a, b)


def test_another_stream_and_a_graph():
    import gated_delta_rule_21_gb300 as kda
    dev, _ = make(64, 264, torch.bfloat16, 64, True, True, seed=9)
    kw = dict(residual=dev["residual"], gate=dev["gate"], w_pre=dev["w_pre"])
    want = kda.block_norm(dev["y"], dev["w_post"], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kda.block_norm(dev["y"], dev["w_post"], stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = kda.block_norm(dev["y"], dev["w_post"], **kw)
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-14, 1e14])
def test_outputs_of_any_size_before_the_second_norm(dtype, scale):
    """The second norm takes the scale out again: gradients of size 1 from
    statistics whose cube fp32 does not hold."""
    dev, ref = make(21, 264, dtype, 21, False, True, seed=10)
    check(dev, ref, dtype, "sigmoid", scale=scale, eps=0.0, d_out=False)

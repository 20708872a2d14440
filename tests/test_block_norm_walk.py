"""GPU tests of the block norms where a CTA walks many rows, so that its staged
rows wrap around, in every layout of a row.

The plain 64-bit form and its derivatives run on the GPU.  Tolerances as in
test_block_norm.py; a thread adds up fewer than 100 rows of a column here."""
import pytest
import torch

import plain64
from test_block_norm import F32, term_sizes

pytestmark = pytest.mark.gpu


def near(got, ref, dtype, size, what):
    tol = torch.finfo(dtype).eps / 2 * 1.01 * ref.abs() + F32 * size
    bad = (got.double() - ref).abs() - tol
    assert bad.max() <= 0, f"{what}: {int((bad > 0).sum())} of {bad.numel()} off, by up to {bad.max():.3e}"


def check(rows, D, dtype, gates, act, res, pre, shift=0, scale=0.7, eps=1e-6):
    import gated_delta_rule_21_gb300 as kda
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    f32 = torch.float32

    def weight():
        return plain64.cast(1 + 0.2 * torch.randn(D, generator=g, device="cuda"), f32)

    def tensor(n, std=1.0):     # `shift` elements off a 16-byte boundary
        t = torch.empty(n * D + shift, dtype=dtype, device="cuda")[shift:].view(n, D)
        t.copy_(std * torch.randn(n, D, generator=g, device="cuda"))
        return t, t.double()

    x = {"y": tensor(rows), "gate": tensor(gates, 2.0) if gates else None,
         "residual": tensor(rows, 2.0) if res else None, "w_post": weight(),
         "w_pre": weight() if pre else None, "d_out": tensor(rows),
         "d_x": tensor(rows) if pre else None}
    dev = {k: None if v is None else v[0] for k, v in x.items()}
    ref = {k: None if v is None else v[1] for k, v in x.items()}
    kw = dict(residual=dev["residual"], gate=dev["gate"], gate_act=act, scale=scale,
              w_pre=dev["w_pre"], eps=eps)
    out, xo, stats = kda.block_norm(dev["y"], dev["w_post"], save_stats=True, **kw)
    got = kda.block_norm_bwd(dev["y"], dev["w_post"], stats, dev["d_out"], d_x=dev["d_x"], **kw)
    leaf = {k: ref[k].clone().requires_grad_() for k in
            ("y", "gate", "residual", "w_post", "w_pre") if ref[k] is not None}
    o, xr = plain64.block_norm(leaf["y"], leaf["w_post"], leaf.get("residual"), leaf.get("gate"),
                               act, scale, leaf.get("w_pre"), eps)
    near(out, o.detach(), dtype, o.detach().abs().amax(-1, keepdim=True), "out")
    loss = (o * ref["d_out"]).sum()
    if pre:
        near(xo, xr.detach(), dtype, xr.detach().abs().amax(-1, keepdim=True), "x")
        loss = loss + (xr * ref["d_x"]).sum()
    loss.backward()
    size = term_sizes(ref, o.detach(), act, scale, eps, True)
    for t, name in zip(got, ("y", "residual", "gate", "w_post", "w_pre")):
        if name not in leaf:
            assert t is None
            continue
        want = leaf[name].grad
        if name in size:
            near(t, want, dtype, 4 * size[name] * (rows // want.shape[0]) ** 0.5, f"d{name}")
        else:
            near(t, want, f32, 4 * (want.abs().amax() + rows ** 0.5), f"d{name}")


# The forward has at most 8 CTAs of 256 threads on an SM, a row group of
# (threads of a row) for each 256: these rows are five turns and more of the forward,
# and of the backward's one or two CTAs per SM with them.
BF16 = [(300001, 40), (100003, 128), (7001, 4096), (3501, 8192), (3001, 16384), (7001, 2292),
        (2001, 12002), (60001, 77), (7001, 2291), (2001, 9001)]
FP32 = [(300001, 20), (14001, 2048), (7001, 4096), (3001, 8192), (2001, 16384), (60001, 77),
        (7001, 2047), (5001, 4095), (2001, 9001)]


@pytest.mark.parametrize("rows,D", BF16)
def test_bf16_gate_each(rows, D):
    check(rows, D, torch.bfloat16, rows, "sigmoid", True, True)


@pytest.mark.parametrize("rows,D", FP32)
def test_fp32_gate_each(rows, D):
    check(rows, D, torch.float32, rows, "silu", True, True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,gates,D", [(100000, 4, 128), (100000, 25000, 128), (6000, 3, 4096),
                                          (6000, 1500, 2291), (6000, 2, 2292), (2000, 400, 16384),
                                          (60000, 5, 77)])
def test_gate_rows_shared_by_many_rows(rows, gates, D, dtype):
    check(rows, D, dtype, gates, "tanh", True, True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(7001, 4096), (3001, 8192), (60001, 128)])
def test_rows_that_are_not_aligned_and_parts_left_out(rows, D, dtype):
    check(rows, D, dtype, rows, "sigmoid", False, True, shift=1)
    check(rows, D, dtype, 0, "none", True, False, shift=1)

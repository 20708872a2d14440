"""The example layer: single tokens after a prompt equal one prompt over all, and
its weights' gradients are those of the plain form in 64 bits.

fp32 on either side.  The matrix products of the layer are torch's, whose fp32 sums
of up to 1024 terms are off by 1e-6 or so of their terms' sizes; scores that are 2e-5
off (latent64.py) change a weight by 4e-5 of itself, which bounds what the whole
differs by."""
import importlib.util
import os

import pytest
import torch

import latent64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    path = os.path.join(ROOT, "examples", "latent_layer.py")
    spec = importlib.util.spec_from_file_location("latent_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("batch,length,tokens", [(2, 150, 6), (1, 1, 3), (3, 64, 2)])
def test_tokens_after_a_prompt(batch, length, tokens):
    assert load().compare(batch, length, tokens) < 1e-4


def test_tokens_after_a_prompt_bf16():
    """Activations are rounded to bf16 at half a dozen places either way, at other
    ones in the absorbed form: 2^-9 each in the 2-norm."""
    assert load().compare(2, 200, 4, torch.bfloat16) < 2e-2


def test_gradients():
    mod = load()
    layer = mod.Layer(torch.float32, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    h = torch.randn(2, 70, mod.WIDTH, generator=gen, device="cuda")
    up = torch.randn(2, 70, mod.WIDTH, generator=gen, device="cuda")
    for w in layer.weights():
        w.requires_grad_()
    layer.train(h).backward(up)
    got = [w.grad.double() for w in layer.weights()]
    q_w, down, k_up, v_up, out = [w.detach().double().requires_grad_() for w in layer.weights()]
    x = h.double()
    q, q_rope = (x @ q_w).unflatten(-1, (mod.HEADS, -1)).split([mod.KEY, mod.ROPE], -1)
    latent, k_rope = (x @ down).split([mod.LATENT, mod.ROPE], -1)
    at = torch.arange(70, device="cuda").expand(2, 70)
    q_rope = latent64.rotate(q_rope, at[..., None], layer.freq)
    k_rope = latent64.rotate(k_rope, at, layer.freq)
    k = torch.einsum("btc,hcd->bthd", latent, k_up)
    v = torch.einsum("btc,hcd->bthd", latent, v_up)
    s = torch.einsum("bihd,bjhd->bhij", q, k) + torch.einsum("bihd,bjd->bhij", q_rope, k_rope)
    p = torch.softmax((s * mod.SCALE).masked_fill(
        torch.ones(70, 70, dtype=torch.bool, device="cuda").triu(1), -torch.inf), -1)
    o = torch.einsum("bhij,bjhd->bihd", p, v)
    (o.flatten(-2) @ out).backward(up.double())
    for a, b in zip(got, (w.grad for w in (q_w, down, k_up, v_up, out))):
        assert float((a - b).norm() / b.norm()) < 1e-4

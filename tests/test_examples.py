"""The example stack: single tokens after a prompt equal one prompt over all.

Both ways round activations to bf16 at the same places but for q, k, v (the
prompt rounds them between its kernels, the token step does not) and the
tensor-core products; each such rounding is 2^-9 of a value, and a dozen of
them in two layers stay below 2e-2 of the outputs' 2-norm."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_recurrent_stack():
    path = os.path.join(ROOT, "examples", "recurrent_stack.py")
    spec = importlib.util.spec_from_file_location("recurrent_stack", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.compare() < 2e-2
    assert mod.compare(batch=1, length=3, tokens=3, seed=5) < 2e-2


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("length", [1, 2])
def test_prompts_shorter_than_the_convolution(length):
    assert load("recurrent_stack").compare(batch=2, length=length, tokens=4, seed=6) < 2e-2


def test_tokens_share_a_workspace_per_stream(monkeypatch):
    import torch
    mod = load("recurrent_stack")
    made = []
    alloc = mod.kda.alloc_step_workspace
    monkeypatch.setattr(mod.kda, "alloc_step_workspace", lambda *a: made.append(a) or alloc(*a))
    stack = mod.Stack()
    h = torch.randn(3, 8, mod.WIDTH, device="cuda").bfloat16()
    _, _, states = stack.prompt(h)
    for _ in range(3):
        stack.token(h[:, 0].contiguous(), states)
    assert len(made) == 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.token(h[:, 0].contiguous(), states)
    side.synchronize()
    assert len(made) == 2

"""A latent attention layer, as it stands between a stack's recurrent ones: in
training, on a prompt and on single tokens.

In training and on prompts keys and values are expanded from the latents
(rotate, latent_fwd, latent_bwd).  On single tokens the expansions are moved to
the queries and the output, and the heads attend to the cached latents themselves
(latent_append, latent_step).  main() checks that the tokens' outputs are those of
a prompt that holds them all, and says how long a token takes.

    python examples/latent_layer.py
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_21_gb300 as kda  # noqa: E402

WIDTH, HEADS, KEY, ROPE, VALUE, LATENT = 512, 8, 128, 64, 128, 512
SCALE = (KEY + ROPE) ** -0.5
PAGE = 64


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, q_rope, k_rope):
        o, lse = kda.latent_fwd(q, k, v, q_rope=q_rope, k_rope=k_rope, scale=SCALE, save_lse=True)
        ctx.save_for_backward(q, k, v, q_rope, k_rope, o, lse)
        return o

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, q_rope, k_rope, o, lse = ctx.saved_tensors
        return kda.latent_bwd(q, k, v, o, lse, d_o.contiguous(), q_rope=q_rope, k_rope=k_rope,
                              scale=SCALE)


class Rotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, freq):
        ctx.save_for_backward(freq)
        return kda.rotate(x, freq)

    @staticmethod
    def backward(ctx, g):
        return kda.rotate(g, ctx.saved_tensors[0], inverse=True), None


class Layer:
    def __init__(self, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def mat(*n):
            return (torch.randn(*n, generator=gen, device=device) * n[-2] ** -0.5).to(dtype)

        self.q, self.down = mat(WIDTH, HEADS * (KEY + ROPE)), mat(WIDTH, LATENT + ROPE)
        self.k_up, self.v_up = mat(HEADS, LATENT, KEY), mat(HEADS, LATENT, VALUE)
        self.out = mat(HEADS * VALUE, WIDTH)
        self.freq = 10000.0 ** (-torch.arange(0, ROPE, 2, device=device) / ROPE)
        self.workspace = {}

    def weights(self):
        return [self.q, self.down, self.k_up, self.v_up, self.out]

    def _inputs(self, h):
        q, q_rope = (h @ self.q).unflatten(-1, (HEADS, KEY + ROPE)).split([KEY, ROPE], -1)
        latent, k_rope = (h @ self.down).split([LATENT, ROPE], -1)
        return q, q_rope, latent, k_rope

    # -- training, and a prompt without a cache: [B, T, WIDTH] ------------------------
    def train(self, h):
        q, q_rope, latent, k_rope = self._inputs(h)
        k = torch.einsum("btc,hcd->bthd", latent, self.k_up)
        v = torch.einsum("btc,hcd->bthd", latent, self.v_up)
        o = Attend.apply(q, k, v, Rotate.apply(q_rope, self.freq), Rotate.apply(k_rope, self.freq))
        return o.flatten(-2) @ self.out

    # -- serving: T new tokens of each sequence, `lengths` with these ---------------------
    def serve(self, h, cache, table, lengths, new=None):
        q, q_rope, latent, k_rope = self._inputs(h)
        q_rope = kda.latent_append(latent, k_rope, cache, table, lengths, inv_freq=self.freq,
                                   new=new, q_rope=q_rope)
        rows = h.shape[0], h.shape[1], torch.cuda.current_stream().cuda_stream
        if rows not in self.workspace:      # one for each stream that makes such calls
            self.workspace[rows] = kda.alloc_latent_step_workspace(*rows[:2], HEADS, LATENT)
        o = kda.latent_step(torch.einsum("bthd,hcd->bthc", q, self.k_up), q_rope, cache, table,
                            lengths, scale=SCALE, new=new, workspace=self.workspace[rows])
        return torch.einsum("bthc,hcd->bthd", o, self.v_up).flatten(-2) @ self.out


def pages(batch, length, dtype, device="cuda", seed=0):
    """An empty cache for `batch` sequences of up to `length` tokens, its pages
    scattered, and their table."""
    wide = -(-length // PAGE)
    order = torch.randperm(batch * wide, generator=torch.Generator().manual_seed(seed))
    cache = torch.empty(batch * wide, PAGE, LATENT + ROPE, dtype=dtype, device=device)
    return cache, order.view(batch, wide).int().to(device)


def compare(batch=2, length=150, tokens=6, dtype=torch.float32, seed=0):
    """Relative 2-norm of the difference between a prompt of everything and a
    prompt into the cache with single tokens after it."""
    layer = Layer(dtype, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    h = torch.randn(batch, length + tokens, WIDTH, generator=gen, device="cuda").to(dtype)
    cache, table = pages(batch, length + tokens, dtype)
    made = []
    for lo, hi in [(0, length)] + [(length + i, length + i + 1) for i in range(tokens)]:
        lengths = torch.full((batch,), hi, dtype=torch.int32, device="cuda")
        made.append(layer.serve(h[:, lo:hi], cache, table, lengths))
    want = layer.train(h).double()
    return float((torch.cat(made, 1).double() - want).norm() / want.norm())


def main():
    print(f"tokens after a prompt against one prompt: {compare():.2e} apart (2-norm, fp32)")
    layer = Layer()
    for w in layer.weights():
        w.requires_grad_()
    h = torch.randn(2, 1024, WIDTH, device="cuda").bfloat16()
    layer.train(h).float().square().mean().backward()
    print("gradient norms:", [f"{float(w.grad.float().norm()):.2e}" for w in layer.weights()])
    with torch.no_grad():
        h = torch.randn(32, 1, WIDTH, device="cuda").bfloat16()
        cache, table = pages(32, 4096, torch.bfloat16)
        cache.normal_()
        lengths = torch.full((32,), 4000, dtype=torch.int32, device="cuda")
        for n in (20, 200):
            torch.cuda.synchronize()
            t = time.perf_counter()
            for _ in range(n):
                layer.serve(h, cache, table, lengths)
            torch.cuda.synchronize()
        print(f"one token for 32 sequences: {(time.perf_counter() - t) / n * 1e6:.0f} us")


if __name__ == "__main__":
    main()

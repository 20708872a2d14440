"""A prompt and then single tokens through a small stack of recurrent layers.

Two layers, a Kimi Delta Attention layer and a selective state space layer,
each between the norms around its block:

    h, x = block_norm(block(x), residual=h, gate=..., scale=..., w_pre=...)

The prompt runs in chunks (short_conv_silu + chunk_fwd, ssm_fwd) and leaves
the states behind; the tokens that follow go one by one through step and
ssm_step on those states.  main() checks that the tokens' outputs are those
of a prompt that holds them all, and says how long a token takes.

    python examples/recurrent_stack.py
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_21_gb300 as kda  # noqa: E402

WIDTH, HEADS, KEY = 512, 4, 128             # of the delta rule layer (values: 128 too)
SSM_HEADS, SSM_DIM, STATES, GROUPS = 8, 64, 128, 2
SCALE = 0.5                                 # of each block's output


class Stack:
    def __init__(self, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def mat(n, m):
            return (torch.randn(n, m, generator=gen, device=device) * n ** -0.5).bfloat16()

        def vec(*n, std=1.0, mean=0.0):
            return mean + std * torch.randn(*n, generator=gen, device=device)

        hk, inner = HEADS * KEY, SSM_HEADS * SSM_DIM
        self.channels = inner + 2 * GROUPS * STATES
        self.qkv, self.gates = mat(WIDTH, 3 * hk), mat(WIDTH, 2 * hk + HEADS)
        self.conv_w, self.o_norm, self.out = vec(3 * hk, 4, std=0.4), vec(KEY, std=0.1, mean=1.0), \
            mat(hk, WIDTH)
        self.proj = mat(WIDTH, inner + self.channels + SSM_HEADS)
        self.ssm_conv, self.ssm_out = vec(self.channels, 4, std=0.4), mat(inner, WIDTH)
        self.A = -torch.exp(vec(SSM_HEADS, std=0.5))
        self.dt_bias, self.D = vec(SSM_HEADS, std=0.5, mean=-3.0), vec(SSM_HEADS, std=0.1, mean=1.0)
        self.norms = vec(5, WIDTH, std=0.1, mean=1.0)        # before, and two around each block
        self.block_gates = vec(2, 1, WIDTH).bfloat16()       # one for every row
        self.workspace = {}

    # -- what both ways share ------------------------------------------------
    def _delta_inputs(self, x):
        q, k, v = (x @ self.qkv).unflatten(-1, (3, HEADS, KEY)).unbind(-3)
        gates = (x @ self.gates).float()
        g, z, beta = gates.split([HEADS * KEY, HEADS * KEY, HEADS], -1)
        g = torch.nn.functional.logsigmoid(g).clamp(min=-5).unflatten(-1, (HEADS, KEY))
        return q, k, v, g.contiguous(), torch.sigmoid(beta).contiguous(), \
            z.bfloat16().unflatten(-1, (HEADS, KEY)).contiguous()

    def _delta_output(self, o, z):
        o, _ = kda.block_norm(o, self.o_norm, gate=z)        # a norm and a gate per head
        return o.flatten(-2) @ self.out

    def _around(self, block, y, h):
        return kda.block_norm(y.contiguous(), self.norms[1 + 2 * block], residual=h,
                              gate=self.block_gates[block], gate_act="tanh", scale=SCALE,
                              w_pre=self.norms[2 + 2 * block])

    def _enter(self, h):
        return kda.block_norm(h, self.norms[0])[0]

    # -- a prompt: [B, T, WIDTH] ------------------------------------------------
    def prompt(self, h):
        x = self._enter(h)
        q, k, v, g, beta, z = self._delta_inputs(x)
        raw = torch.cat([t.flatten(-2) for t in (q, k, v)], -1)
        # the convolution goes on from the last three inputs, zeros before the prompt
        # (a row of several sequences or with padding has them elsewhere)
        conv = torch.nn.functional.pad(raw, (0, 0, 3, 0))[:, -3:].contiguous()
        q, k, v = kda.short_conv_silu(q.contiguous(), k.contiguous(), v.contiguous(),
                                      self.conv_w, l2norm_qk=True)
        o, state = kda.chunk_fwd(q, k, v, g, beta, output_final_state=True)
        h, x = self._around(0, self._delta_output(o, z), h)
        zz, xbc, dt = self._ssm_inputs(x)
        y, ssm_state, ssm_conv = kda.ssm_fwd(
            xbc, dt, self.ssm_conv, self.A, head_dim=SSM_DIM, state_dim=STATES,
            dt_bias=self.dt_bias, D=self.D, z=zz, output_final_state=True)
        h, x = self._around(1, y.flatten(-2) @ self.ssm_out, h)
        return x, h, {"delta": state, "delta_conv": conv, "ssm": ssm_state, "ssm_conv": ssm_conv}

    def _ssm_inputs(self, x):
        return (x @ self.proj).split([SSM_HEADS * SSM_DIM, self.channels, SSM_HEADS], -1)

    def _workspace(self, rows):
        """One for each stream that makes tokens of so many sequences."""
        key = rows, torch.cuda.current_stream().cuda_stream
        if key not in self.workspace:
            self.workspace[key] = kda.alloc_step_workspace(rows, max(HEADS, SSM_HEADS))
        return self.workspace[key]

    # -- one token per sequence: [B, WIDTH]; the states move on in place ------
    def token(self, h, states, slots=None):
        ws = self._workspace(h.shape[0])
        x = self._enter(h)
        q, k, v, g, beta, z = self._delta_inputs(x)
        o = kda.step(q, k, v, g, beta, states["delta"], slots=slots, conv_w=self.conv_w,
                     conv_state=states["delta_conv"], l2norm_qk=True, workspace=ws)
        h, x = self._around(0, self._delta_output(o, z), h)
        zz, xbc, dt = self._ssm_inputs(x)
        y = kda.ssm_step(xbc, dt, self.ssm_conv, self.A, states["ssm"], states["ssm_conv"],
                         head_dim=SSM_DIM, state_dim=STATES, dt_bias=self.dt_bias, D=self.D, z=zz,
                         slots=slots, workspace=ws)
        h, x = self._around(1, y.flatten(-2) @ self.ssm_out, h)
        return x, h


def compare(batch=2, length=200, tokens=8, seed=0):
    """Relative 2-norm of the difference between the tokens' outputs and
    those of one prompt over everything."""
    stack = Stack(seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    h = torch.randn(batch, length + tokens, WIDTH, generator=gen, device="cuda").bfloat16()
    whole, _, _ = stack.prompt(h)
    _, _, states = stack.prompt(h[:, :length].contiguous())
    made = [stack.token(h[:, length + i].contiguous(), states)[0] for i in range(tokens)]
    made, want = torch.stack(made, 1).double(), whole[:, length:].double()
    return float((made - want).norm() / want.norm())


def main():
    print(f"tokens after a prompt against one prompt: {compare():.2e} apart (2-norm)")
    stack = Stack()
    h = torch.randn(32, 1024, WIDTH, device="cuda").bfloat16()
    _, _, states = stack.prompt(h)
    h = h[:, 0].contiguous()
    for n in (20, 200):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            stack.token(h, states)
        torch.cuda.synchronize()
    print(f"one token for 32 sequences: {(time.perf_counter() - t) / n * 1e6:.0f} us")


if __name__ == "__main__":
    main()

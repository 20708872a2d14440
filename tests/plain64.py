"""The state space operator, the single-token steps and the block norms
written down plainly in 64 bits on the CPU, for the tests to compare with."""
import torch

TAPS = 4


def silu(x):
    return x / (1 + torch.exp(-x))


def softplus(x):
    return torch.log1p(torch.exp(-x.abs())) + x.clamp(min=0)


def cast(x, dtype):
    """Values of ``dtype`` and the same values in 64 bits."""
    y = x.to(dtype)
    return y, y.double()


class Ssm:
    """The operator on one row, token by token.  Inputs are 64-bit."""

    def __init__(self, w, A, H, P, N, G, bias=None, dt_bias=None, D=None):
        self.w, self.A, self.H, self.P, self.N, self.G = w, A, H, P, N, G
        self.bias = torch.zeros(w.shape[0], dtype=torch.float64) if bias is None else bias
        self.dt_bias = torch.zeros(H, dtype=torch.float64) if dt_bias is None else dt_bias
        self.D = torch.zeros(H, dtype=torch.float64) if D is None else D

    def token(self, x, dt, z, state, window):
        """(y, state, window) after one token; window [3, channels]."""
        H, P, N, G = self.H, self.P, self.N, self.G
        full = torch.cat([window, x[None]])
        u = silu((full * self.w.t()).sum(0) + self.bias)
        xs = u[:H * P].view(H, P)
        bs = u[H * P:H * P + G * N].view(G, N).repeat_interleave(H // G, 0)
        cs = u[H * P + G * N:].view(G, N).repeat_interleave(H // G, 0)
        d = softplus(dt + self.dt_bias)
        state = torch.exp(d * self.A)[:, None, None] * state \
            + (d[:, None] * bs)[:, :, None] * xs[:, None, :]
        y = (cs[:, :, None] * state).sum(1) + self.D[:, None] * xs
        if z is not None:
            y = y * silu(z).view(H, P)
        return y, state, full[1:]

    def row(self, x, dt, z, ids, state, window):
        y = torch.zeros(x.shape[0], self.H, self.P, dtype=torch.float64)
        begun, prev = False, 0
        for t in range(x.shape[0]):
            now = 1 if ids is None else int(ids[t])
            if now and now != prev:
                if begun:
                    state, window = torch.zeros_like(state), torch.zeros_like(window)
                begun = True
            prev = now
            if now:
                y[t], state, window = self.token(x[t], dt[t], None if z is None else z[t],
                                                 state, window)
        return y, state, window


def delta_token(q, k, v, g, beta, state, scale):
    """One token of the delta rule for all heads: (o, state)."""
    state = torch.exp(g)[:, :, None] * state
    rest = v - (k[:, :, None] * state).sum(1)
    state = state + (beta[:, None] * k)[:, :, None] * rest[:, None, :]
    return scale * (q[:, :, None] * state).sum(1), state


GATES = {"none": lambda a: a, "sigmoid": torch.sigmoid, "tanh": torch.tanh, "silu": silu}


def block_norm(y, w_post, residual=None, gate=None, act="sigmoid", scale=1.0, w_pre=None,
               eps=1e-6):
    """(out, x or None) for [rows, D] tensors; gate has rows that divide theirs."""
    u = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w_post
    if gate is not None:
        u = u * GATES[act](gate).repeat_interleave(y.shape[0] // gate.shape[0], 0)
    out = scale * u if residual is None else residual + scale * u
    if w_pre is None:
        return out, None
    return out, out / torch.sqrt((out * out).mean(-1, keepdim=True) + eps) * w_pre

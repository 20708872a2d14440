"""The latent attention written down plainly in 64 bits, for the tests to
compare with, and how far off a kernel may be, term by term.

Errors.  A score is off by at most ``es``: a sum of up to 576 products in fp32,
whose partial sums stay below about 30 for these inputs; a few dozen roundings
of 2^-24 of them in fp32 (2e-5), and as many of 2^-23 in the tensor cores'
accumulator (1e-4).  A weight p = exp(s - lse) is then off by 2 es of itself, and
where it is rounded to bf16 for the tensor cores by 2^-8 more; the same holds for
ds = p (dp - D).  A sum over weights is off by that much of the sum of its terms'
sizes.  Outputs are rounded once, by eps / 2 of their type."""
import torch

ES = {"simt": 2e-5, "tc": 1e-4}
ROUND = {"simt": 0.0, "tc": 2.0 ** -8}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 * 1.001


def mask(T, seg=None):
    """[T, T] of one row: who sees whom."""
    i = torch.arange(T)
    on = i[:, None] >= i
    if seg is None:
        return on
    seg = seg.cpu().long()
    run = torch.cat([torch.zeros(1, dtype=torch.long), (seg[1:] != seg[:-1]).long()]).cumsum(0)
    return on & (run[:, None] == run) & (seg != 0)[:, None]


def softmax(s, on):
    s = torch.where(on, s, -torch.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e300)
    e = torch.exp(s - top)
    n = e.sum(-1, keepdim=True)
    lse = (top + torch.log(n)).squeeze(-1)
    return e / torch.where(n > 0, n, 1.0), lse


def prompt(x, scale, seg=None, impl="simt", dtype=torch.float32, d_o=None):
    """x: dict of 64-bit q, k, v, q_rope, k_rope ([B,T,H,.], [B,T,R]; on any
    device).  Returns {name: (value, tolerance)}."""
    q, k, v = (x[n].transpose(1, 2) for n in "qkv")
    K = q.shape[-1]
    if x.get("q_rope") is not None:
        q = torch.cat([q, x["q_rope"].transpose(1, 2)], -1)
        k = torch.cat([k, x["k_rope"][:, None].expand(-1, k.shape[1], -1, -1)], -1)
    B, H, T, _ = q.shape
    on = torch.stack([mask(T, None if seg is None else seg[b]) for b in range(B)])[:, None]
    on = on.to(q.device)
    p, lse = softmax(q @ k.transpose(-1, -2) * scale, on)
    es, half = ES[impl], half_step(dtype)
    w = 2 * es + ROUND[impl]
    o = p @ v
    size = p @ v.abs()
    got = {"o": (o, half * o.abs() + w * size)}
    got["lse"] = (lse, es + 1e-6 * lse.abs().nan_to_num(posinf=0.0))
    if d_o is not None:
        up = d_o.transpose(1, 2)
        pt = p.transpose(-1, -2)
        dv = pt @ up
        got["dv"] = (dv, half * dv.abs() + w * (pt @ up.abs()))
        dp = up @ v.transpose(-1, -2)
        D = (up * o).sum(-1, keepdim=True)
        ds = p * (dp - D)
        # D is made from the rounded o; sums of 128 products
        off = (up.abs() * got["o"][1]).sum(-1, keepdim=True)
        e = w * ds.abs() + p * (off + 1e-6 * (up.abs() @ v.abs().transpose(-1, -2)))
        et = e.transpose(-1, -2)
        dq, dk = scale * ds @ k, scale * ds.transpose(-1, -2) @ q
        eq, ek = abs(scale) * e @ k.abs(), abs(scale) * et @ q.abs()
        for n, a, b in (("dq", dq, eq), ("dk", dk, ek)):
            got[n] = (a[..., :K], half * a[..., :K].abs() + b[..., :K])
        if q.shape[-1] > K:
            got["dq_rope"] = (dq[..., K:], half * dq[..., K:].abs() + eq[..., K:])
            s = dk[..., K:].sum(1)
            got["dk_rope"] = (s, half * s.abs() + ek[..., K:].sum(1) +
                              1e-6 * dk[..., K:].abs().sum(1))
    return {n: tuple(t.transpose(1, 2) if n not in ("lse", "dk_rope") else t for t in pair)
            for n, pair in got.items()}


def step(q, q_rope, tokens, there, seen, scale, impl="simt", dtype=torch.float32):
    """One sequence: q [T,H,C], q_rope [T,H,R] or None, tokens [n, C + R] with
    ``there`` [n], seen [T].  Returns (o, tolerance), (lse, tolerance)."""
    C = q.shape[-1]
    s = q @ tokens[:, :C].t()
    if q_rope is not None:
        s = s + q_rope @ tokens[:, C:].t()
    on = (torch.arange(tokens.shape[0]) < seen[:, None])[:, None] & there
    p, lse = softmax(s * scale, on)
    o = p @ tokens[:, :C]
    w = 2 * ES[impl] + ROUND[impl]
    return (o, half_step(dtype) * o.abs() + w * (p @ tokens[:, :C].abs())), \
        (lse, ES[impl] + 1e-6 * lse.abs().nan_to_num(posinf=0.0))


def rotate(x, at, freq, pairs=True, inverse=False):
    """x [..., dim] at positions [...] (64-bit)."""
    angle = at.double()[..., None] * freq.double()
    c, s = torch.cos(angle), torch.sin(angle)
    if inverse:
        s = -s
    n = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :n], x[..., n:])
    u, v = a * c - b * s, b * c + a * s
    return torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)


def check(got, want, what):
    """Elementwise; -inf and NaN in the same places."""
    ref, tol = (t.cpu() for t in want)
    got = got.double().cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(ref.shape)}"
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad = ~(same | ((got - ref).abs() <= tol + 1e-30))
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{float(got[i])}, not {float(ref[i])} +- {float(tol[i]):.3e}")

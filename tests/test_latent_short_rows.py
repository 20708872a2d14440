"""GPU tests of D = d_o . o in the latent attention's gradients on the tensor
cores: every query that sees at most 1024 keys has it from the products, whatever
its tile holds and whatever its run is packed behind, and not from the rounded o.

The values are about 8 with a spread of 0.1, so that o's rounding (2^-9 of 8) moves D
by a fifth of what ds = p (dp - D) is made of, where D from the products does not.

Tolerance of D from the products, sum p dp / sum p: a weight is off by 2 es of itself
(latent64.py), dp by 1e-6 of its terms' sizes, and a sum of up to 1024 terms, of which a
thread adds one after another no more than 300, by 300 roundings of 2^-24 of its terms'
sizes, in both sums.  Of D from the stored o, for queries with more keys: o's rounding, as in
latent64.py."""
import pytest
import torch

import latent64
from test_latent_prompt import inputs, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def want(x, scale, seg, d_o):
    """{name: (value, tolerance)} of the gradients; x in 64 bits."""
    q, k, v = (x[n].transpose(1, 2) for n in "qkv")
    K = q.shape[-1]
    if x["q_rope"] is not None:
        q = torch.cat([q, x["q_rope"].transpose(1, 2)], -1)
        k = torch.cat([k, x["k_rope"][:, None].expand(-1, k.shape[1], -1, -1)], -1)
    T, up = q.shape[2], d_o.transpose(1, 2)
    on = latent64.mask(T, None if seg is None else seg[0]).to(q.device)
    p, _ = latent64.softmax(q @ k.transpose(-1, -2) * scale, on)
    es, half = latent64.ES["tc"], latent64.half_step(BF)
    w = 2 * es + latent64.ROUND["tc"]
    o = p @ v
    dp = up @ v.transpose(-1, -2)
    D = (up * o).sum(-1, keepdim=True)
    ds = p * (dp - D)
    e_dp = 1e-6 * (up.abs() @ v.abs().transpose(-1, -2))
    made = (p * (2 * es * (dp - D).abs() + e_dp + 600 * 2.0 ** -24 * dp.abs())).sum(-1, keepdim=True)
    stored = (up.abs() * (half * o.abs() + w * (p @ v.abs()))).sum(-1, keepdim=True)
    few = (on.sum(-1) <= 1024)[:, None]
    e = w * ds.abs() + p * (torch.where(few, 1.01 * made, stored) + e_dp)
    dq, eq = scale * ds @ k, scale * e @ k.abs()
    dk, ek = scale * ds.transpose(-1, -2) @ q, scale * e.transpose(-1, -2) @ q.abs()
    got = {n: (a[..., :K].transpose(1, 2), (half * a[..., :K].abs() + b[..., :K]).transpose(1, 2))
           for n, a, b in (("dq", dq, eq), ("dk", dk, ek))}
    if q.shape[-1] > K:
        a, b = dq[..., K:], eq[..., K:]
        got["dq_rope"] = (a.transpose(1, 2), (half * a.abs() + b).transpose(1, 2))
        a, s = dk[..., K:], dk[..., K:].sum(1)
        got["dk_rope"] = (s, half * s.abs() + ek[..., K:].sum(1) + 1e-6 * a.abs().sum(1))
    return got


@pytest.mark.parametrize("T,edges", [
    (2210, [0, 1100, 1160, 2180, 2200]),   # short runs behind long ones, in one tile; padding
    (1300, [0, 30, 1040, 1300]),           # 1010 keys that lie on 17 tiles of 64
    (2048, [0, 1024, 1025, 2048]),
    (1500, None), (700, None), (700, [0, 333, 334, 690])])
@pytest.mark.parametrize("K,R,V", [(64, 0, 128), (128, 64, 128)])
def test_rows_with_few_keys(T, edges, K, R, V):
    gen = torch.Generator().manual_seed(T + K)
    x, x64 = inputs(1, T, 2, K, R, V, BF, gen, strided=False)
    x["v"] = (8 + 0.1 * torch.randn(1, T, 2, V, generator=gen)).to(BF).cuda()
    x64["v"] = x["v"].double()
    d_o = torch.randn(1, T, 2, V, generator=gen).to(BF).cuda()
    seg = None
    if edges:
        seg = torch.zeros(1, T, dtype=torch.int32)
        for i, (a, z) in enumerate(zip(edges, edges[1:])):
            seg[0, a:z] = i + 1
    got = run(x, None if seg is None else seg.cuda(), "tc", d_o)
    for n, pair in want(x64, (K + R) ** -0.5, seg, d_o.double()).items():
        latent64.check(got[n], pair, n)

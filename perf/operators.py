"""What is measured of the operators that carry a layer's state from a prompt
into single tokens and that stand around its blocks.

Five kinds of call, each with its plain form, its value in 64 bits and the
call a user makes:

* ``ssm``       a prompt through the selective state space operator (short
                causal convolution, SiLU, scan over the tokens, skip, gate);
* ``ssm_step``  one new token per sequence on the cached states;
* ``kda_step``  one new token per sequence through the delta rule;
* ``norm``      the norm after a block, its gate and residual scale, and the
                norm before the next block, forward;
* ``norm_train``  the same forward and backward.
"""
import math

import torch

own = False

W = 4          # taps of the short convolution
CHUNK = 64     # tokens per chunk of the plain scan
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a short prompt of a small model: launches and latency count
        {"name": "ssm short prompt", "op": "ssm", "B": 1, "T": 197, "H": 8, "P": 64, "N": 128,
         "G": 1, "dtype": "bf16", "rows": "full", "init": False},
        # a packed row of 25 documents, 32 heads of 128 channels
        {"name": "ssm packed", "op": "ssm", "B": 1, "T": 8192, "H": 32, "P": 128, "N": 128,
         "G": 1, "dtype": "bf16", "rows": "packed", "init": False},
        # two long prompts that go on from cached states, 64 heads in 8 groups
        {"name": "ssm long prompts", "op": "ssm", "B": 2, "T": 8192, "H": 64, "P": 64, "N": 128,
         "G": 8, "dtype": "bf16", "rows": "full", "init": True},
        # prompts of unequal lengths in 32 bits (evaluation of a small model)
        {"name": "ssm ragged f32", "op": "ssm", "B": 3, "T": 997, "H": 6, "P": 32, "N": 64,
         "G": 2, "dtype": "f32", "rows": "ragged", "init": True},
        # one user's next token: latency
        {"name": "ssm token, 1 user", "op": "ssm_step", "B": 1, "slots": 1, "H": 32, "P": 128,
         "N": 128, "G": 1, "dtype": "bf16", "idle": 0},
        # a serving batch with a few idle places, states scattered over a cache
        {"name": "ssm token, 128 users", "op": "ssm_step", "B": 128, "slots": 160, "H": 64,
         "P": 64, "N": 128, "G": 8, "dtype": "bf16", "idle": 3},
        # one user's next token through the delta rule, with its convolution
        {"name": "kda token, 1 user", "op": "kda_step", "B": 1, "slots": 1, "H": 32, "K": 128,
         "V": 128, "dtype": "bf16", "conv": True, "idle": 0},
        # a serving batch through the delta rule
        {"name": "kda token, 120 users", "op": "kda_step", "B": 120, "slots": 160, "H": 32,
         "K": 128, "V": 128, "dtype": "bf16", "conv": True, "idle": 5},
        # between two blocks while single tokens are made
        {"name": "norm 5 rows", "op": "norm", "R": 5, "D": 4096, "dtype": "bf16", "gate": "each",
         "act": "sigmoid", "res": True, "pre": True},
        # between two blocks of a long prompt
        {"name": "norm 8192 rows", "op": "norm", "R": 8192, "D": 4096, "dtype": "bf16",
         "gate": "each", "act": "silu", "res": True, "pre": True},
        # a training step between two blocks, one gate for each of 4 sequences
        {"name": "norm training", "op": "norm_train", "R": 8192, "D": 4096, "dtype": "bf16",
         "gate": "group", "groups": 4, "act": "tanh", "res": True, "pre": True},
        # a training step of the gated norm of each head of the delta rule's output
        {"name": "head norm training", "op": "norm_train", "R": 131072, "D": 128,
         "dtype": "bf16", "gate": "each", "act": "sigmoid", "res": False, "pre": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["ssm", "ssm", "ssm_step", "kda_step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "ssm":
        while True:
            c = {"op": op, "B": _log(rng, 1, 6), "T": _log(rng, 1, 8192), "H": _log(rng, 1, 64),
                 "P": rng.choice([32, 64, 128]), "N": rng.choice([32, 64, 128]), "G": 1,
                 "dtype": dtype, "rows": rng.choice(["full", "full", "packed", "ragged"]),
                 "init": rng.random() < 0.5}
            c["G"] = rng.choice([g for g in (1, 2, 4, 8) if c["H"] % g == 0])
            cost = c["B"] * c["T"] * c["H"]
            if cost <= 1 << 20 and cost * c["P"] <= 1 << 26:
                return c
    if op == "ssm_step":
        b = _log(rng, 1, 128)
        h = _log(rng, 1, 64)
        return {"op": op, "B": b, "slots": b + rng.randrange(0, 33), "H": h,
                "P": rng.choice([32, 64, 128]), "N": rng.choice([32, 64, 128]),
                "G": rng.choice([g for g in (1, 2, 4, 8) if h % g == 0]), "dtype": dtype,
                "idle": rng.choice([0, b // 4])}
    if op == "kda_step":
        b = _log(rng, 1, 120)
        return {"op": op, "B": b, "slots": b + rng.randrange(0, 33), "H": _log(rng, 1, 32),
                "K": rng.choice([32, 64, 128]), "V": rng.choice([32, 64, 128]), "dtype": dtype,
                "conv": rng.random() < 0.6, "idle": rng.choice([0, b // 4])}
    while True:
        gate = rng.choice(["none", "each", "group"])
        groups = rng.randrange(1, 9) if gate == "group" else 1
        c = {"op": op, "R": groups * _log(rng, 1, 65536 // groups), "D": _log(rng, 24, 16384),
             "dtype": dtype, "gate": gate, "groups": groups,
             "act": rng.choice(["none", "sigmoid", "silu", "tanh"]),
             "res": rng.random() < 0.7, "pre": rng.random() < 0.7}
        if rng.random() < 0.6:
            c["D"] = -(-c["D"] // 8) * 8
        if c["R"] * c["D"] * SIZE[dtype] <= 8192 * 4096 * 2:
            return c


# --------------------------------------------------------------------------
# inputs


def _rand(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _round_up(n, m):
    return -(-n // m) * m


def _ssm_weights(c, gen):
    h, ch = c["H"], c["H"] * c["P"] + 2 * c["G"] * c["N"]
    u = torch.rand(2, h, generator=gen, device="cuda")
    step = torch.exp(math.log(1e-3) + u[0] * (math.log(1e-1) - math.log(1e-3)))
    return {"conv_w": _rand(gen, ch, W, std=0.5), "conv_bias": _rand(gen, ch, std=0.1),
            "A": -(1 + 15 * u[1]), "D": 1 + _rand(gen, h, std=0.1),
            # the step width softplus(dt_bias) is spread over its logarithm
            "dt_bias": step + torch.log(-torch.expm1(-step))}


def _segment_ids(c, gen):
    """Row layouts: whole rows, documents packed with a little padding, or
    one prompt per row of its own length (one row of several is empty)."""
    b, t = c["B"], c["T"]
    if c["rows"] == "full":
        return None
    cpu = torch.Generator().manual_seed(gen.initial_seed())
    ids = torch.zeros(b, t, dtype=torch.int32)
    if c["rows"] == "ragged":
        for r in range(b):
            n = int(torch.randint(1, t + 1, (1,), generator=cpu)) if r else t
            ids[r, :0 if (r == 1 and b > 2) else n] = 1
        return ids.cuda()
    n = max(1, min(25, t // 40))
    for r in range(b):
        cuts = torch.randperm(max(t - 1, 1), generator=cpu)[:n - 1].add(1).sort().values.tolist()
        edges = [0] + [x for x in cuts if x < t] + [t]
        for i in range(len(edges) - 1):
            ids[r, edges[i]:edges[i + 1]] = i + 1
        ids[r, max(1, t - t // 64):] = 0
    return ids.cuda()


def _slots(c, gen):
    """Each sequence's place in the cache; idle sequences have place -1."""
    s = torch.randperm(c["slots"], generator=gen, device="cuda")[:c["B"]].to(torch.int32)
    if c["idle"]:
        s[torch.randperm(c["B"], generator=gen, device="cuda")[:c["idle"]]] = -1
    return s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op = c["op"]
    s = {"c": c, "op": op}
    if op in ("ssm", "ssm_step"):
        dt = DT[c["dtype"]]
        hp, ch = c["H"] * c["P"], c["H"] * c["P"] + 2 * c["G"] * c["N"]
        s.update(_ssm_weights(c, gen))
        rows = (c["B"], c["T"]) if op == "ssm" else (c["B"],)
        # one projection gives z, the channels of the convolution and dt
        proj = _rand(gen, *rows, _round_up(hp + ch + c["H"], 8))
        s["z"], s["xbc"], s["dt"] = (t for t in proj.to(dt).split(
            [hp, ch, c["H"], proj.shape[-1] - hp - ch - c["H"]], -1)[:3])
        if op == "ssm":
            s["seg"] = _segment_ids(c, gen)
            s["state"] = _rand(gen, c["B"], c["H"], c["N"], c["P"], std=0.1) if c["init"] else None
            s["conv"] = _rand(gen, c["B"], W - 1, ch).to(dt) if c["init"] else None
        else:
            s["state"] = _rand(gen, c["slots"], c["H"], c["N"], c["P"], std=0.1)
            s["conv"] = _rand(gen, c["slots"], W - 1, ch).to(dt)
            s["slots"] = _slots(c, gen)
    elif op == "kda_step":
        dt, b, h, k, v = DT[c["dtype"]], c["B"], c["H"], c["K"], c["V"]
        q, kk = _rand(gen, b, h, k), _rand(gen, b, h, k)
        if not c["conv"]:
            q, kk = q / q.norm(dim=-1, keepdim=True), kk / kk.norm(dim=-1, keepdim=True)
        s["q"], s["k"], s["v"] = q.to(dt), kk.to(dt), _rand(gen, b, h, v).to(dt)
        s["g"] = torch.log(torch.sigmoid(_rand(gen, b, h, k))).clamp(min=-5)
        s["beta"] = torch.sigmoid(_rand(gen, b, h))
        s["state"] = _rand(gen, c["slots"], h, k, v, std=0.1)
        s["slots"] = _slots(c, gen)
        s["conv_w"] = _rand(gen, h * (2 * k + v), W, std=0.5) if c["conv"] else None
        s["conv"] = _rand(gen, c["slots"], W - 1, h * (2 * k + v)).to(dt) if c["conv"] else None
    else:
        dt, r, d = DT[c["dtype"]], c["R"], c["D"]
        s["y"] = _rand(gen, r, d).to(dt)
        s["w_post"] = 1 + _rand(gen, d, std=0.2)
        s["w_pre"] = 1 + _rand(gen, d, std=0.2) if c["pre"] else None
        s["res"] = _rand(gen, r, d, std=2.0).to(dt) if c["res"] else None
        n = {"none": 0, "each": r, "group": c.get("groups", 1)}[c["gate"]]
        s["gate"] = _rand(gen, n, d).to(dt) if n else None
        s["d_res"] = _rand(gen, r, d).to(dt)
        s["d_pre"] = _rand(gen, r, d).to(dt) if c["pre"] else None
    if own:
        s["ws"] = _workspace(s, c)
    return s


def _workspace(s, c):
    """The scratch memory that a program keeps beside its weights."""
    import gated_delta_rule_21_gb300 as kda
    if c["op"] == "ssm":
        return kda.alloc_ssm_workspace(c["B"], c["T"], c["H"], c["P"], c["N"], c["G"],
                                       dtype=DT[c["dtype"]])
    if c["op"] in ("ssm_step", "kda_step"):
        return kda.alloc_step_workspace(c["B"], c["H"])
    if c["op"] == "norm_train":
        return kda.alloc_block_norm_workspace(
            c["R"], c["D"], gate_rows=0 if s["gate"] is None else s["gate"].shape[0])
    return None


NORM_EPS, NORM_SCALE = 1e-6, 0.7


# --------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _own(s)
    return {"ssm": _ssm_plain, "ssm_step": _ssm_step_plain, "kda_step": _kda_step_plain,
            "norm": _norm_plain, "norm_train": _norm_train_plain}[s["op"]](s)


def _own(s):
    import gated_delta_rule_21_gb300 as kda
    c, op = s["c"], s["op"]
    if op == "ssm":
        y, state, conv = kda.ssm_fwd(
            s["xbc"], s["dt"], s["conv_w"], s["A"], head_dim=c["P"], state_dim=c["N"],
            conv_bias=s["conv_bias"], dt_bias=s["dt_bias"], D=s["D"], z=s["z"],
            initial_state=s["state"], conv_state=s["conv"], segment_ids=s["seg"],
            output_final_state=True, workspace=s["ws"])
        return {"y": y, "state": state, "conv": conv}
    if op == "ssm_step":
        y = kda.ssm_step(s["xbc"], s["dt"], s["conv_w"], s["A"], s["state"], s["conv"],
                         head_dim=c["P"], state_dim=c["N"], conv_bias=s["conv_bias"],
                         dt_bias=s["dt_bias"], D=s["D"], z=s["z"], slots=s["slots"],
                         workspace=s["ws"])
        return {"y": y, "state": s["state"], "conv": s["conv"]}
    if op == "kda_step":
        o = kda.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"],
                     conv_w=s["conv_w"], conv_state=s["conv"], l2norm_qk=c["conv"],
                     workspace=s["ws"])
        return {"o": o, "state": s["state"], "conv": s["conv"]}
    act = {"gate": s["gate"], "gate_act": c["act"], "residual": s["res"], "w_pre": s["w_pre"],
           "scale": NORM_SCALE, "eps": NORM_EPS}
    if op == "norm":
        out, x = kda.block_norm(s["y"], s["w_post"], **act)
        return {"out": out, "x": x}
    out, x, stats = kda.block_norm(s["y"], s["w_post"], save_stats=True, **act)
    dy, dres, dgate, dw_post, dw_pre = kda.block_norm_bwd(
        s["y"], s["w_post"], stats, s["d_res"], d_x=s["d_pre"], workspace=s["ws"], **act)
    return {"out": out, "x": x, "dy": dy, "dres": dres, "dgate": dgate, "dw_post": dw_post,
            "dw_pre": dw_pre}


def _silu(x):
    return x * torch.sigmoid(x)


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _runs(seg, b, t, device):
    """Of every token: whether it counts, its place in its run, whether its
    run is the row's first, and how many resets lie at or before it."""
    at = torch.arange(t, device=device).expand(b, t)
    if seg is None:
        one = torch.ones(b, t, dtype=torch.bool, device=device)
        return one, at, one, torch.zeros_like(at)
    before = torch.cat([torch.zeros_like(seg[:, :1]), seg[:, :-1]], 1)
    live = seg != 0
    start = live & (seg != before)
    number = start.cumsum(1)
    begun = torch.where(start, at, torch.zeros_like(at)).cummax(1).values
    return live, at - begun, number == 1, (start & (number > 1)).cumsum(1)


def _ssm_plain(s):
    c, dtype = s["c"], s["xbc"].dtype
    b, t, h, p, n, g = (c[k] for k in "BTHPNG")
    x = s["xbc"].float()
    dev, ch = x.device, x.shape[-1]
    live, place, first, resets = _runs(s["seg"], b, t, dev)
    past = s["conv"].float() if s["conv"] is not None else torch.zeros(b, W - 1, ch, device=dev)

    def tap(i):     # the input i tokens before, from the cache before the row's first run
        moved = torch.cat([torch.zeros(b, min(i, t), ch, device=dev), x[:, :max(t - i, 0)]], 1)
        if i == 0:
            return moved
        old = past.gather(1, (W - 1 + place - i).clamp(0, W - 2)[..., None].expand(-1, -1, ch))
        keep = (place >= i)[..., None]
        return torch.where(keep, moved, torch.where(first[..., None] & live[..., None], old, 0.0))

    u = _silu(sum(s["conv_w"][:, W - 1 - i] * tap(i) for i in range(W)) + s["conv_bias"])
    xs, bs, cs = u.split([h * p, g * n, g * n], -1)
    step = _softplus(s["dt"].float() + s["dt_bias"]) * live[..., None]
    nc = -(-t // CHUNK)
    room = nc * CHUNK - t

    def cut(v, *dims):      # [B, T, ...] as chunks, the last one filled up
        v = torch.cat([v, torch.zeros(b, room, *v.shape[2:], dtype=v.dtype, device=dev)], 1)
        return v.reshape(b, nc, CHUNK, *dims)

    xs, bs, cs = cut(xs, h, p), cut(bs, g, n), cut(cs, g, n)
    step = cut(step, h)
    count = torch.cat([resets, resets[:, -1:].expand(b, room)], 1).reshape(b, nc, CHUNK)
    far = (step.double() * s["A"].double()).cumsum(2)           # [B, nc, CHUNK, H]
    same = (count[:, :, :, None] == count[:, :, None, :]).tril()
    decay = torch.exp((far[:, :, :, None] - far[:, :, None]).clamp(max=0)).float()
    decay = decay * same[..., None]                             # [B, nc, r, j, H]
    dot = torch.einsum("bcrgn,bcjgn->bcrjg", cs, bs).repeat_interleave(h // g, -1)
    xd = xs * step[..., None]
    y = torch.einsum("bcrjh,bcjhp->bcrhp", dot * decay, xd)
    # what each chunk adds to the state, and the states that enter the chunks
    tail = torch.exp((far[:, :, -1:] - far)).float() * (count == count[:, :, -1:])[..., None]
    bh = bs.repeat_interleave(h // g, 3)
    add = torch.einsum("bcjhn,bcjhp->bchnp", bh * tail[..., None], xd)
    s0 = s["state"] if s["state"] is not None else torch.zeros(b, h, n, p, device=dev)
    add = torch.cat([s0[:, None], add], 1)
    end = torch.cat([torch.zeros_like(count[:, 0, :1]), count[:, :, -1]], 1)   # [B, nc + 1]
    sums = torch.cat([torch.zeros(b, 1, h, dtype=torch.float64, device=dev), far[:, :, -1]], 1)
    sums = sums.cumsum(1)
    over = torch.exp((sums[:, :, None] - sums[:, None]).clamp(max=0)).float()
    over = over * (end[:, :, None] == end[:, None]).tril()[..., None]
    states = torch.einsum("bcdh,bdhnp->bchnp", over, add)       # entering each chunk, and the last
    enter = torch.exp(far).float() * (count == end[:, :-1, None])[..., None]
    ch_ = cs.repeat_interleave(h // g, 3)
    y = y + torch.einsum("bcrhn,bchnp->bcrhp", ch_ * enter[..., None], states[:, :-1])
    y = (y + xs * s["D"][:, None]).reshape(b, nc * CHUNK, h, p)[:, :t]
    y = y * _silu(s["z"].float().reshape(b, t, h, p)) * live[..., None, None]
    # the last inputs of the sequence that the row ends with
    at = torch.arange(t, device=dev).expand(b, t)
    last = torch.where(live, at, torch.full_like(at, -1)).max(1).values
    age = torch.arange(W - 2, -1, -1, device=dev).expand(b, W - 1)
    lc = last.clamp(min=0)[:, None]
    here = place.gather(1, lc)
    new = x.gather(1, (lc - age).clamp(min=0)[..., None].expand(-1, -1, ch))
    old = past.gather(1, (W - 1 + here - age).clamp(0, W - 2)[..., None].expand(-1, -1, ch))
    old = torch.where(first.gather(1, lc)[..., None], old, torch.zeros_like(old))
    conv = torch.where((here >= age)[..., None], new, old)
    conv = torch.where((last >= 0)[:, None, None], conv, past)
    return {"y": y.to(dtype), "state": states[:, -1].contiguous(), "conv": conv.to(dtype)}


def _window(s, x, active, place):
    """The last W inputs of every sequence; shifts the cached ones."""
    win = torch.cat([s["conv"][place].float(), x[:, None]], 1)
    s["conv"][place[active]] = win[active, 1:].to(s["conv"].dtype)
    return win


def _ssm_step_plain(s):
    c, dtype = s["c"], s["xbc"].dtype
    b, h, p, n, g = (c[k] for k in "BHPNG")
    active = s["slots"] >= 0
    place = s["slots"].clamp(min=0).long()
    win = _window(s, s["xbc"].float(), active, place)
    u = _silu((win * s["conv_w"].t()).sum(1) + s["conv_bias"])
    xs, bs, cs = u.split([h * p, g * n, g * n], -1)
    xs = xs.reshape(b, h, p)
    bs, cs = (v.reshape(b, g, n).repeat_interleave(h // g, 1) for v in (bs, cs))
    step = _softplus(s["dt"].float() + s["dt_bias"])
    keep = torch.exp(step * s["A"])
    state = s["state"][place] * keep[..., None, None]
    state = state + (bs * step[..., None])[..., None] * xs[:, :, None]
    s["state"][place[active]] = state[active]
    y = (cs[..., None] * state).sum(2) + xs * s["D"][:, None]
    y = y * _silu(s["z"].float().reshape(b, h, p)) * active[:, None, None]
    return {"y": y.to(dtype), "state": s["state"], "conv": s["conv"]}


def _kda_step_plain(s):
    c, dtype = s["c"], s["q"].dtype
    b, h, k, v = (c[n] for n in "BHKV")
    active = s["slots"] >= 0
    place = s["slots"].clamp(min=0).long()
    q, kk, vv = (s[n].float() for n in "qkv")
    if c["conv"]:
        x = torch.cat([t.reshape(b, -1) for t in (q, kk, vv)], 1)
        u = _silu((_window(s, x, active, place) * s["conv_w"].t()).sum(1))
        q, kk, vv = u.split([h * k, h * k, h * v], -1)
        q, kk, vv = q.reshape(b, h, k), kk.reshape(b, h, k), vv.reshape(b, h, v)
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        kk = kk * torch.rsqrt((kk * kk).sum(-1, keepdim=True) + 1e-6)
    state = s["state"][place] * torch.exp(s["g"])[..., None]
    left = vv - (kk[..., None] * state).sum(2)
    state = state + (s["beta"][..., None] * kk)[..., None] * left[:, :, None]
    s["state"][place[active]] = state[active]
    o = k ** -0.5 * (q[..., None] * state).sum(2) * active[:, None, None]
    return {"o": o.to(dtype), "state": s["state"], "conv": s["conv"]}


def _gate(a, act):
    """The gate's value and its derivative."""
    if act == "none":
        return a, torch.ones_like(a)
    if act == "tanh":
        v = torch.tanh(a)
        return v, 1 - v * v
    v = torch.sigmoid(a)
    return (v, v * (1 - v)) if act == "sigmoid" else (a * v, v * (1 + a * (1 - v)))


def _norm_parts(s):
    y = s["y"].float()
    r, d = y.shape
    inv = torch.rsqrt((y * y).sum(-1, keepdim=True) / d + NORM_EPS)
    n = y * inv
    u = n * s["w_post"]
    a, da = (None, None)
    if s["gate"] is not None:
        a, da = (v.repeat_interleave(r // s["gate"].shape[0], 0)
                 for v in _gate(s["gate"].float(), s["c"]["act"]))
    out = NORM_SCALE * (u if a is None else u * a)
    if s["res"] is not None:
        out = out + s["res"].float()
    inv2 = torch.rsqrt((out * out).sum(-1, keepdim=True) / d + NORM_EPS)
    return inv, n, u, a, da, out, inv2


def _norm_plain(s):
    out, inv2 = _norm_parts(s)[-2:]
    x = (out * inv2 * s["w_pre"]).to(s["y"].dtype) if s["c"]["pre"] else None
    return {"out": out.to(s["y"].dtype), "x": x}


def _norm_train_plain(s):
    dtype, (r, d) = s["y"].dtype, s["y"].shape
    inv, n, u, a, da, out, inv2 = _norm_parts(s)
    d_out = s["d_res"].float()
    x = dw_pre = None
    if s["c"]["pre"]:
        n2 = out * inv2
        x = (n2 * s["w_pre"]).to(dtype)
        up = s["d_pre"].float()
        dw_pre = (up * n2).double().sum(0).float()
        up = up * s["w_pre"]
        d_out = d_out + inv2 * (up - n2 * ((up * n2).sum(-1, keepdim=True) / d))
    du = NORM_SCALE * (d_out if a is None else d_out * a)
    dgate = None
    if a is not None:
        each = NORM_SCALE * d_out * u * da
        dgate = each.double().reshape(s["gate"].shape[0], -1, d).sum(1).to(dtype)
    dw_post = (du * n).double().sum(0).float()
    dn = du * s["w_post"]
    dy = inv * (dn - n * ((dn * n).sum(-1, keepdim=True) / d))
    return {"out": out.to(dtype), "x": x, "dy": dy.to(dtype),
            "dres": d_out.to(dtype) if s["res"] is not None else None, "dgate": dgate,
            "dw_post": dw_post, "dw_pre": dw_pre}


# --------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["op"] in ("ssm", "ssm_step"):
        hp, bc, hn = c["H"] * c["P"], 2 * c["G"] * c["N"], c["H"] * c["N"] * c["P"]
        tok = c["B"] * c["T"] if c["op"] == "ssm" else c["B"] - c["idle"]
        wts = 4 * ((hp + bc) * (W + 1) + 3 * c["H"])
        n = tok * e * (3 * hp + bc + c["H"]) + wts      # z, channels, dt in; y out
        if c["op"] == "ssm":
            held = c["B"] * (4 * hn + e * (W - 1) * (hp + bc))
            n += held * (2 if c["init"] else 1) + (4 * tok if c["rows"] != "full" else 0)
        else:
            n += 2 * tok * (4 * hn + e * (W - 1) * (hp + bc)) + 4 * c["B"]
        return {"bytes": n, "flops": 4 * tok * hn + tok * (hp + bc) * 2 * W}
    if c["op"] == "kda_step":
        tok, kv, ch = c["B"] - c["idle"], c["K"] * c["V"], c["H"] * (2 * c["K"] + c["V"])
        n = tok * (e * (ch + c["H"] * c["V"]) + 4 * c["H"] * (c["K"] + 1) + 8 * c["H"] * kv)
        n += (2 * tok * e * (W - 1) * ch + 4 * W * ch) if c["conv"] else 0
        return {"bytes": n + 4 * c["B"], "flops": 7 * tok * c["H"] * kv}
    rd = c["R"] * c["D"]
    gate = {"none": 0, "each": rd, "group": c.get("groups", 1) * c["D"]}[c["gate"]]
    n = e * (rd * (2 + c["res"] + c["pre"]) + gate) + 4 * c["D"] * (1 + c["pre"])
    f = 12 * rd
    if c["op"] == "norm_train":     # y, gate, residual and the two gradients in, theirs out
        n += e * (rd * (3 + 2 * c["res"] + c["pre"]) + 2 * gate) + 8 * c["D"] * (1 + c["pre"])
        f += 24 * rd
    return {"bytes": n, "flops": f}


# --------------------------------------------------------------------------
# the definitions in 64 bits, token by token and row by row


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    return {"ssm": _ssm_exact, "ssm_step": _token_exact, "kda_step": _delta_exact,
            "norm": _norm_exact, "norm_train": _norm_exact}[c["op"]](s, c)


def _ssm_token(c, s, u, dt, state):
    """One token of the recurrence: (y without the gate, state)."""
    h, p, g, n = c["H"], c["P"], c["G"], c["N"]
    x = u[:, :h * p].view(-1, h, p)
    heads = torch.arange(h, device=u.device) // (h // g)
    bb = u[:, h * p:h * p + g * n].view(-1, g, n)[:, heads]
    cc = u[:, h * p + g * n:].view(-1, g, n)[:, heads]
    width = torch.nn.functional.softplus(dt + s["dt_bias"].double(), threshold=700.0)
    state = torch.exp(width * s["A"].double())[:, :, None, None] * state \
        + (width[:, :, None] * bb)[:, :, :, None] * x[:, :, None, :]
    return torch.matmul(cc[:, :, None, :], state)[:, :, 0] + s["D"].double()[:, None] * x, state


def _ssm_exact(s, c):
    b, t, h, p, n = c["B"], c["T"], c["H"], c["P"], c["N"]
    x, z, dt = s["xbc"].double(), s["z"].double(), s["dt"].double()
    ch = x.shape[-1]
    state = x.new_zeros(b, h, n, p) if s["state"] is None else s["state"].double()
    win = x.new_zeros(b, W - 1, ch) if s["conv"] is None else s["conv"].double()
    taps, bias = s["conv_w"].double().t().contiguous(), s["conv_bias"].double()
    y = x.new_zeros(b, t, h, p)
    ids = s["seg"].tolist() if s["seg"] is not None else [[1] * t] * b
    for r in (range(b) if s["seg"] is not None else [slice(0, b)]):
        rows = slice(r, r + 1) if isinstance(r, int) else r
        st, wi, begun, prev = state[rows], win[rows], False, 0
        for i in range(t):
            now = ids[r][i] if isinstance(r, int) else 1
            if now and now != prev:
                if begun:
                    st, wi = torch.zeros_like(st), torch.zeros_like(wi)
                begun = True
            prev = now
            if not now:
                continue
            full = torch.cat([wi, x[rows, i:i + 1]], 1)
            pre = (full * taps).sum(1) + bias
            yi, st = _ssm_token(c, s, pre / (1 + torch.exp(-pre)), dt[rows, i], st)
            y[rows, i], wi = yi, full[:, 1:]
        state[rows], win[rows] = st, wi
    gate = z / (1 + torch.exp(-z))
    return {"y": y * gate.reshape(b, t, h, p), "state": state, "conv": win}


def _advance(s, new, conv_w, bias):
    """The cached inputs of the active sequences moved on by one token, and
    what the convolution makes of them."""
    conv = s["conv"].double()
    out = new.new_zeros(new.shape)
    for i, k in enumerate(s["slots"].tolist()):
        if k >= 0:
            full = torch.cat([conv[k], new[i:i + 1]], 0)
            pre = (full * conv_w.double().t()).sum(0) + bias
            out[i], conv[k] = pre / (1 + torch.exp(-pre)), full[1:]
    return out, conv


def _token_exact(s, c):
    new, z = s["xbc"].double(), s["z"].double()
    u, conv = _advance(s, new, s["conv_w"], s["conv_bias"].double())
    state = s["state"].double()
    y = new.new_zeros(c["B"], c["H"], c["P"])
    for i, k in enumerate(s["slots"].tolist()):
        if k >= 0:
            yi, st = _ssm_token(c, s, u[i:i + 1], s["dt"][i:i + 1].double(), state[k:k + 1])
            y[i], state[k] = yi[0], st[0]
    return {"y": y * (z / (1 + torch.exp(-z))).reshape(y.shape), "state": state, "conv": conv}


def _delta_exact(s, c):
    b, h, k, v = c["B"], c["H"], c["K"], c["V"]
    q, kk, vv = (s[n].double().reshape(b, -1) for n in "qkv")
    conv = None
    if c["conv"]:
        u, conv = _advance(s, torch.cat([q, kk, vv], 1), s["conv_w"], 0.0)
        q, kk, vv = u[:, :h * k], u[:, h * k:2 * h * k], u[:, 2 * h * k:]
    state, o = s["state"].double(), q.new_zeros(b, h, v)
    for i, place in enumerate(s["slots"].tolist()):
        if place < 0:
            continue
        qi, ki, vi = q[i].view(h, k), kk[i].view(h, k), vv[i].view(h, v)
        if c["conv"]:
            qi = qi / torch.sqrt((qi ** 2).sum(1, keepdim=True) + 1e-6)
            ki = ki / torch.sqrt((ki ** 2).sum(1, keepdim=True) + 1e-6)
        st = state[place] * torch.exp(s["g"][i].double())[:, :, None]
        rest = vi - torch.matmul(ki[:, None], st)[:, 0]
        st = st + s["beta"][i].double()[:, None, None] * ki[:, :, None] * rest[:, None]
        state[place], o[i] = st, torch.matmul(qi[:, None], st)[:, 0] / math.sqrt(k)
    return {"o": o, "state": state, "conv": conv}


def _norm_exact(s, c):
    """The forward written down, the gradients by differentiating it."""
    train = c["op"] == "norm_train"
    leaf = {k: s[k].double().requires_grad_(train) for k in
            ("y", "w_post", "w_pre", "res", "gate") if s[k] is not None}
    rows, d = leaf["y"].shape

    def rms(v, w):
        return v / torch.sqrt(torch.mean(v ** 2, -1, keepdim=True) + NORM_EPS) * w

    u = rms(leaf["y"], leaf["w_post"])
    if "gate" in leaf:
        f = {"none": lambda a: a, "tanh": torch.tanh, "sigmoid": torch.sigmoid,
             "silu": torch.nn.functional.silu}[c["act"]]
        a = f(leaf["gate"])
        u = (u.view(a.shape[0], -1, d) * a[:, None]).view(rows, d)
    out = NORM_SCALE * u + leaf.get("res", 0.0)
    x = rms(out, leaf["w_pre"]) if c["pre"] else None
    if not train:
        return {"out": out, "x": x}
    loss = (out * s["d_res"].double()).sum()
    if x is not None:
        loss = loss + (x * s["d_pre"].double()).sum()
    loss.backward()
    got = {k: v.grad for k, v in leaf.items()}
    return {"out": out.detach(), "x": None if x is None else x.detach(), "dy": got["y"],
            "dres": got.get("res"), "dgate": got.get("gate"), "dw_post": got["w_post"],
            "dw_pre": got.get("w_pre")}

"""What is measured of the attention over one shared latent vector a token,
the layers that stand between a stack's recurrent ones, and of the cache and
the position rotation that serve it.

Five kinds of call, each with its plain form, its value in 64 bits and the
call a user makes:

* ``rotate``  the position rotation of queries or keys, or of their gradients
              back;
* ``append``  new tokens' latents and rotated keys into a paged cache, the
              queries rotated on the way;
* ``step``    the absorbed form: a few new queries per sequence over the paged
              latents;
* ``fwd``     the expanded form: a prompt, causal within its runs;
* ``train``   the expanded form forward and backward.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BASE = 10000.0     # of the rotation's frequencies


def listed():
    return [
        # the queries of a long prompt
        {"name": "rotate prompt", "op": "rotate", "B": 1, "T": 8192, "H": 32, "R": 64,
         "dtype": "bf16", "pairs": True, "inverse": False, "far": 0},
        # gradients rotated back, in 32 bits, far into a long text
        {"name": "rotate back f32", "op": "rotate", "B": 3, "T": 997, "H": 6, "R": 32,
         "dtype": "f32", "pairs": False, "inverse": True, "far": 1000000},
        # one user's next token: latency
        {"name": "append 1 token", "op": "append", "B": 1, "T": 1, "H": 32, "C": 512, "R": 64,
         "page": 64, "most": 1000, "dtype": "bf16", "pairs": True, "ragged": False, "idle": 0},
        # prompts of unequal lengths, four at once
        {"name": "append prompts", "op": "append", "B": 4, "T": 2048, "H": 32, "C": 512, "R": 64,
         "page": 64, "most": 8192, "dtype": "bf16", "pairs": True, "ragged": True, "idle": 0},
        # one user's next token over a short text: latency
        {"name": "step 1 user", "op": "step", "B": 1, "T": 1, "H": 32, "C": 512, "R": 64,
         "page": 64, "most": 1000, "dtype": "bf16", "ragged": False, "idle": 0},
        # a serving batch of unequal lengths with a few idle places
        {"name": "step 120 users", "op": "step", "B": 120, "T": 1, "H": 32, "C": 512, "R": 64,
         "page": 64, "most": 8192, "dtype": "bf16", "ragged": True, "idle": 5},
        # two long texts, 64 heads
        {"name": "step long texts", "op": "step", "B": 2, "T": 1, "H": 64, "C": 512, "R": 64,
         "page": 128, "most": 131072, "dtype": "bf16", "ragged": False, "idle": 0},
        # a few drafted tokens per sequence, in 32 bits (evaluation of a small model)
        {"name": "step drafts f32", "op": "step", "B": 3, "T": 4, "H": 6, "C": 128, "R": 32,
         "page": 16, "most": 997, "dtype": "f32", "ragged": True, "idle": 1},
        # a short prompt of a small model: launches and latency count
        {"name": "fwd short prompt", "op": "fwd", "B": 1, "T": 197, "H": 8, "K": 128, "R": 64,
         "V": 128, "dtype": "bf16", "rows": "full"},
        # a packed row of 25 documents, 32 heads
        {"name": "fwd packed", "op": "fwd", "B": 1, "T": 8192, "H": 32, "K": 128, "R": 64,
         "V": 128, "dtype": "bf16", "rows": "packed"},
        # a training step of a long row, 32 heads
        {"name": "train long", "op": "train", "B": 1, "T": 8192, "H": 32, "K": 128, "R": 64,
         "V": 128, "dtype": "bf16", "rows": "full"},
        # rows of unequal lengths in 32 bits
        {"name": "train ragged f32", "op": "train", "B": 3, "T": 997, "H": 6, "K": 64, "R": 32,
         "V": 64, "dtype": "f32", "rows": "ragged"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "step", "step", "fwd", "fwd", "train", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = {"op": op, "dtype": dtype}
    if op == "rotate":
        c.update(R=rng.choice([32, 64]), pairs=rng.random() < 0.5, inverse=rng.random() < 0.5,
                 far=rng.choice([0, _log(rng, 1, 1 << 24)]))
        while True:
            c.update(B=_log(rng, 1, 8), T=_log(rng, 1, 8192), H=_log(rng, 1, 32))
            if c["B"] * c["T"] * c["H"] * SIZE[dtype] <= 8192 * 32 * 2:
                return c
    if op == "append":
        c.update(C=rng.choice([128, 256, 512]), R=rng.choice([32, 64]), pairs=rng.random() < 0.5,
                 page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.6)
        while True:
            c.update(B=_log(rng, 1, 64), T=_log(rng, 1, 2048), H=_log(rng, 1, 32))
            if c["B"] * c["T"] * c["H"] * SIZE[dtype] <= 4 * 2048 * 32 * 2:
                break
        c["most"] = c["T"] + _log(rng, 1, 4096)
        c["idle"] = rng.choice([0, c["B"] // 4])
        return c
    if op == "step":
        c.update(C=rng.choice([128, 256, 512]), R=rng.choice([0, 32, 64]),
                 page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
        while True:
            c.update(B=_log(rng, 1, 120), T=_log(rng, 1, 6), H=_log(rng, 1, 64),
                     most=_log(rng, 1, 65536))
            rows = c["T"] * c["H"]
            if c["B"] * c["most"] <= 2 * 131072 and \
                    c["B"] * rows * c["most"] <= (1 << 24 if dtype == "bf16" else 1 << 21):
                break
        c["most"] = max(c["most"], c["T"])
        c["idle"] = rng.choice([0, c["B"] // 4])
        return c
    c.update(K=rng.choice([32, 64, 128]), R=rng.choice([0, 32, 64]), V=rng.choice([32, 64, 128]),
             rows=rng.choice(["full", "full", "packed", "ragged"]))
    if rng.random() < 0.5:
        c.update(K=128, R=64, V=128)
    while True:
        # (a training row of one token has no gradient of queries and keys)
        c.update(B=_log(rng, 1, 6), T=_log(rng, 2 if op == "train" else 1, 8192),
                 H=_log(rng, 1, 32))
        if c["B"] * c["H"] * c["T"] ** 2 <= (1 << 31 if dtype == "bf16" else 1 << 25):
            return c


# --------------------------------------------------------------------------
# inputs


def _rand(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda")


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


def _paged(c, gen, s):
    """The cache of a serving program: pages of tokens scattered over it, a
    table of each sequence's pages (-1 behind the last), each sequence's
    length with its new tokens, and how many of these there are."""
    b, t, page, most = c["B"], c["T"], c["page"], c["most"]
    new = torch.full((b,), t, device="cuda")
    length = torch.full((b,), most, device="cuda")
    if c["ragged"]:
        new = _ints(gen, 1, t, b)
        new[0] = t
        length = torch.maximum(_ints(gen, 1, most, b), new)
    if c["idle"]:
        out = torch.randperm(b, generator=gen, device="cuda")[:c["idle"]]
        new[out], length[out] = 0, 0
    wide = -(-most // page)
    used = -(-length // page)
    at = torch.arange(wide, device="cuda")
    held = at < used[:, None]
    n_pages = b * wide + 3
    pages = torch.randperm(n_pages, generator=gen, device="cuda")[:n_pages - 3]
    table = torch.where(held, pages.view(b, wide), -1)
    s["cache"] = _rand(gen, n_pages, page, c["C"] + c["R"]).to(DT[c["dtype"]])
    s["table"], s["lengths"], s["new"] = table.int(), length.int(), new.int()
    if not c["ragged"] and not c["idle"]:
        s["new"] = None


def _frequencies(r):
    return (BASE ** (-2.0 * torch.arange(r // 2, device="cuda", dtype=torch.float64) / r)).float()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    op, dt = c["op"], DT[c["dtype"]]
    s = {"c": c, "op": op}
    b, t, h, r = c["B"], c["T"], c["H"], c["R"]
    if op == "rotate":
        s["freq"] = _frequencies(r)
        s["x"] = _rand(gen, b, t, h, r).to(dt)
        start = _ints(gen, 0, c["far"], b) if c["far"] else torch.zeros(b, device="cuda")
        s["positions"] = (start[:, None] + torch.arange(t, device="cuda")).int() if c["far"] else None
    elif op == "append":
        _paged(c, gen, s)
        s["freq"] = _frequencies(r)
        # one projection gives the latent and the key that is rotated, another the queries
        down = _rand(gen, b, t, c["C"] + r).to(dt)
        s["latent"], s["k_rope"] = down.split([c["C"], r], -1)
        s["q_rope"] = _rand(gen, b, t, h, 128 + r).to(dt)[..., 128:]
    elif op == "step":
        _paged(c, gen, s)
        std = 2.0 * ((128 + r) / (c["C"] + r)) ** 0.5      # scores of a deviation of about 2
        s["q"] = _rand(gen, b, t, h, c["C"], std=std).to(dt)
        s["q_rope"] = _rand(gen, b, t, h, r, std=std).to(dt) if r else None
        s["scale"] = (128 + r) ** -0.5
    else:
        k, v = c["K"], c["V"]
        q = _rand(gen, b, t, h, k + r, std=1.5).to(dt)
        s["q"], s["q_rope"] = q[..., :k], q[..., k:] if r else None
        # the expanded keys and values lie side by side, as one projection of the latents
        kv = _rand(gen, b, t, h, k + v).to(dt)
        s["k"], s["v"] = kv.split([k, v], -1)
        s["k_rope"] = _rand(gen, b, t, r).to(dt) if r else None
        s["seg"] = _segment_ids(c, gen)
        s["scale"] = (k + r) ** -0.5
        if op == "train":
            s["d_o"] = _rand(gen, b, t, h, v).to(dt)
    if own:
        s["ws"] = _workspace(c)
    return s


def _workspace(c):
    """The scratch memory that a program keeps beside its weights."""
    import gated_delta_rule_21_gb300 as kda
    if c["op"] == "step":
        return kda.alloc_latent_step_workspace(c["B"], c["T"], c["H"], c["C"])
    if c["op"] in ("fwd", "train"):
        return kda.alloc_latent_workspace(c["B"], c["T"], c["H"], c["R"],
                                          backward=c["op"] == "train")
    return None


# --------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _own(s)
    return {"rotate": _rotate_plain, "append": _append_plain, "step": _step_plain,
            "fwd": _fwd_plain, "train": _train_plain}[s["op"]](s)


def _own(s):
    import gated_delta_rule_21_gb300 as kda
    c, op = s["c"], s["op"]
    if op == "rotate":
        return {"y": kda.rotate(s["x"], s["freq"], positions=s["positions"], pairs=c["pairs"],
                                inverse=c["inverse"])}
    if op == "append":
        q = kda.latent_append(s["latent"], s["k_rope"], s["cache"], s["table"], s["lengths"],
                              inv_freq=s["freq"], new=s["new"], q_rope=s["q_rope"],
                              pairs=c["pairs"])
        return {"q_rope": q, "cache": s["cache"]}
    if op == "step":
        return {"o": kda.latent_step(s["q"], s["q_rope"], s["cache"], s["table"], s["lengths"],
                                     scale=s["scale"], new=s["new"], workspace=s["ws"])}
    with_rope = {"q_rope": s["q_rope"], "k_rope": s["k_rope"], "scale": s["scale"],
                 "segment_ids": s["seg"], "workspace": s["ws"]}
    if op == "fwd":
        return {"o": kda.latent_fwd(s["q"], s["k"], s["v"], **with_rope)}
    o, lse = kda.latent_fwd(s["q"], s["k"], s["v"], save_lse=True, **with_rope)
    dq, dk, dv, dq_rope, dk_rope = kda.latent_bwd(s["q"], s["k"], s["v"], o, lse, s["d_o"],
                                                  **with_rope)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dq_rope": dq_rope, "dk_rope": dk_rope}


def _turned(x, positions, freq, pairs, inverse):
    """x [B, T, H, R] rotated at positions [B, T]."""
    r = x.shape[-1]
    angle = positions.double()[..., None, None] * freq.double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if inverse:
        sin = -sin
    x = x.float()
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :r // 2], x[..., r // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _rotate_plain(s):
    c, x = s["c"], s["x"]
    at = s["positions"]
    if at is None:
        at = torch.arange(c["T"], device=x.device).expand(c["B"], -1)
    return {"y": _turned(x, at, s["freq"], c["pairs"], c["inverse"]).to(x.dtype)}


def _places(s):
    """Of every new token: its position, and whether it counts."""
    t = torch.arange(s["c"]["T"], device="cuda")
    new = s["lengths"] * 0 + s["c"]["T"] if s["new"] is None else s["new"]
    return (s["lengths"] - new)[:, None] + t, t < new[:, None]


def _append_plain(s):
    c, dt = s["c"], s["latent"].dtype
    at, live = _places(s)
    k = _turned(s["k_rope"][:, :, None], at, s["freq"], c["pairs"], False)[:, :, 0].to(dt)
    q = _turned(s["q_rope"], at, s["freq"], c["pairs"], False).to(dt)
    q = torch.where(live[..., None, None], q, s["q_rope"])
    safe = torch.where(live, at, 0)
    pages = s["table"].long().gather(1, safe // c["page"])[live]
    s["cache"][pages, safe[live] % c["page"]] = torch.cat([s["latent"], k], -1)[live]
    return {"q_rope": q, "cache": s["cache"]}


def _step_plain(s):
    c, dt = s["c"], s["q"].dtype
    at, live = _places(s)
    q = s["q"] if s["q_rope"] is None else torch.cat([s["q"], s["q_rope"]], -1)
    kv = s["cache"][s["table"].long().clamp(min=0)].flatten(1, 2).float()      # [B, tokens, C + R]
    score = torch.einsum("bthd,bsd->bths", q.float(), kv) * s["scale"]
    seen = torch.arange(kv.shape[1], device=kv.device) <= at[..., None]
    seen = (seen & live[..., None])[:, :, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bths,bsc->bthc", p, kv[..., :c["C"]]) / torch.where(total > 0, total, 1.0)
    return {"o": o.to(dt)}


def _mask(seg, t, device):
    """[B or 1, 1, T, T]: which token sees which."""
    i = torch.arange(t, device=device)
    causal = i[:, None] >= i
    if seg is None:
        return causal[None, None]
    change = torch.cat([torch.ones_like(seg[:, :1]), (seg[:, 1:] != seg[:, :-1]).int()], 1)
    run = change.cumsum(1)
    same = (run[:, :, None] == run[:, None]) & (seg != 0)[:, :, None]
    return (same & causal)[:, None]


def _scores(s):
    """Heads in front: queries, keys, values, and the softmax's weights."""
    q, k, v = (s[n].float().transpose(1, 2) for n in "qkv")
    if s["q_rope"] is not None:
        q = torch.cat([q, s["q_rope"].float().transpose(1, 2)], -1)
        shared = s["k_rope"].float()[:, None].expand(-1, k.shape[1], -1, -1)
        k = torch.cat([k, shared], -1)
    seen = _mask(s["seg"], q.shape[2], q.device)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return q, k, v, p.div_(torch.where(total > 0, total, 1.0))


def _fwd_plain(s):
    _, _, v, p = _scores(s)
    return {"o": torch.matmul(p, v).transpose(1, 2).to(s["q"].dtype).contiguous()}


def _train_plain(s):
    c, dt = s["c"], s["q"].dtype
    q, k, v, p = _scores(s)

    def back(x):
        return x.transpose(1, 2).to(dt).contiguous()

    o = torch.matmul(p, v)
    up = s["d_o"].float().transpose(1, 2)
    dv = torch.matmul(p.transpose(-1, -2), up)
    ds = torch.matmul(up, v.transpose(-1, -2))
    ds = ds.sub_((up * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    n = c["K"]
    with_rope = c["R"] > 0
    return {"o": back(o), "dq": back(dq[..., :n]), "dk": back(dk[..., :n]), "dv": back(dv),
            "dq_rope": back(dq[..., n:]) if with_rope else None,
            "dk_rope": dk[..., n:].sum(1).to(dt) if with_rope else None}


# --------------------------------------------------------------------------
# what a pass cannot do without


def _pairs_seen(c):
    """How many (query, key) pairs the rows of a prompt hold, on average where
    their runs are drawn."""
    b, t = c["B"], c["T"]
    if c["rows"] == "full":
        return b * t * (t + 1) // 2
    if c["rows"] == "ragged":     # lengths uniform in 1 .. t, the first row whole, one empty
        rest = max(0, b - 1 - (1 if b > 2 else 0))
        return int(t * (t + 1) / 2 + rest * (t * t / 6 + t / 2))
    n = max(1, min(25, t // 40))  # n runs cut at random: the mean square of a run is 2 t^2 / n (n + 1)
    return int(b * (t * t / (n + 1) + t / 2))


def work(case):
    c = case
    e, b, t, h, r = SIZE[c["dtype"]], c["B"], c["T"], c["H"], c["R"]
    if c["op"] == "rotate":
        n = b * t * h * r
        return {"bytes": 2 * e * n + 2 * r + (4 * b * t if c["far"] else 0), "flops": 3 * n}
    if c["op"] in ("append", "step"):
        live = b - c["idle"]
        # half of the new tokens and of the lengths where rows are ragged
        new = live * (t + 1) // 2 if c["ragged"] else live * t
        held = live * (c["most"] + 1) // 2 if c["ragged"] else live * c["most"]
        table = 4 * (-(-held // c["page"]) + 2 * b)
        if c["op"] == "append":
            n = e * new * 2 * (c["C"] + r) + 2 * e * b * t * h * r
            return {"bytes": n + 4 * (2 * b + new) + 2 * r, "flops": 3 * new * (h + 1) * r}
        n = e * held * (c["C"] + r) + e * new * h * (2 * c["C"] + r)
        ratio = new / max(live, 1)
        return {"bytes": n + table, "flops": int(2 * held * ratio * h * (2 * c["C"] + r))}
    k, v = c["K"], c["V"]
    tok = b * t
    n = e * tok * (h * (2 * k + r + 2 * v) + r) + (4 * tok if c["rows"] != "full" else 0)
    f = 2 * _pairs_seen(c) * h * (k + r + v)
    if c["op"] == "train":      # the inputs and d_o again for the gradients, and these
        n += e * tok * (h * (2 * k + r + 2 * v) + r)
        f += 2 * _pairs_seen(c) * h * (3 * (k + r) + 2 * v)
    return {"bytes": n, "flops": f}


# --------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    return {"rotate": _rotate_exact, "append": _append_exact, "step": _step_exact,
            "fwd": _prompt_exact, "train": _prompt_exact}[c["op"]](s, c)


def _spin(x, at, freq, pairs, sign):
    """Rows of x as complex numbers, turned by at * freq."""
    x = x.double()
    shape = x.shape
    half = shape[-1] // 2
    pair = x.unflatten(-1, (half, 2)) if pairs else x.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.exp(1j * sign * at.double()[..., None] * freq.double())
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    return (z if pairs else z.transpose(-1, -2)).reshape(shape)


def _rotate_exact(s, c):
    at = torch.arange(c["T"], device="cuda")[None].expand(c["B"], -1) \
        if s["positions"] is None else s["positions"]
    at = at[:, :, None].expand(-1, -1, c["H"])
    return {"y": _spin(s["x"], at, s["freq"], c["pairs"], -1.0 if c["inverse"] else 1.0)}


def _append_exact(s, c):
    cache, q = s["cache"].double(), s["q_rope"].double()
    for b in range(c["B"]):
        n = c["T"] if s["new"] is None else int(s["new"][b])
        if n == 0:
            continue
        at = int(s["lengths"][b]) - n + torch.arange(n, device="cuda")
        k = _spin(s["k_rope"][b, :n], at, s["freq"], c["pairs"], 1.0)
        page = s["table"][b].long()[torch.div(at, c["page"], rounding_mode="floor")]
        slot = page * c["page"] + torch.remainder(at, c["page"])
        flat = cache.view(-1, cache.shape[-1])
        flat[slot, :c["C"]] = s["latent"][b, :n].double()
        flat[slot, c["C"]:] = k
        q[b, :n] = _spin(s["q_rope"][b, :n], at[:, None].expand(-1, c["H"]), s["freq"],
                         c["pairs"], 1.0)
    return {"q_rope": q, "cache": cache}


def _step_exact(s, c):
    o = torch.zeros(c["B"], c["T"], c["H"], c["C"], dtype=torch.float64, device="cuda")
    flat = s["cache"].view(-1, c["C"] + c["R"])
    slot = torch.arange(c["page"], device="cuda")
    for b in range(c["B"]):
        n, length = (c["T"] if s["new"] is None else int(s["new"][b])), int(s["lengths"][b])
        if length == 0:
            continue
        rows = (s["table"][b].long()[:, None] * c["page"] + slot).view(-1)[:length]
        kv = flat[rows].double()
        for i in range(n):
            last = length - n + i + 1
            score = torch.matmul(s["q"][b, i].double(), kv[:last, :c["C"]].t())
            if c["R"]:
                score = score + torch.matmul(s["q_rope"][b, i].double(), kv[:last, c["C"]:].t())
            o[b, i] = torch.matmul(torch.softmax(score * s["scale"], -1), kv[:last, :c["C"]])
    return {"o": o}


def _prompt_exact(s, c):
    """Run by run and head by head; the gradients by differentiating."""
    train = c["op"] == "train"
    names = [n for n in ("q", "k", "v", "q_rope", "k_rope") if s[n] is not None]
    o = torch.zeros(c["B"], c["T"], c["H"], c["V"], dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names}
    ids = None if s["seg"] is None else s["seg"].tolist()
    for b in range(c["B"]):
        cuts = [0] + ([] if ids is None else
                      [t for t in range(1, c["T"]) if ids[b][t] != ids[b][t - 1]]) + [c["T"]]
        for lo, hi in zip(cuts, cuts[1:]):
            if ids is not None and ids[b][lo] == 0:
                continue
            above = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").triu(1)
            for h in range(c["H"]):
                x = {n: (s[n][b, lo:hi] if n == "k_rope" else s[n][b, lo:hi, h]).double()
                     .requires_grad_(train) for n in names}
                score = x["q"] @ x["k"].t()
                if c["R"]:
                    score = score + x["q_rope"] @ x["k_rope"].t()
                score = (score * s["scale"]).masked_fill(above, -math.inf)
                out = torch.softmax(score, -1) @ x["v"]
                o[b, lo:hi, h] = out.detach()
                if not train:
                    continue
                out.backward(s["d_o"][b, lo:hi, h].double())
                for n in names:
                    if n == "k_rope":
                        grads[n][b, lo:hi] += x[n].grad
                    else:
                        grads[n][b, lo:hi, h] = x[n].grad
    if not train:
        return {"o": o}
    return {"o": o, "dq": grads["q"], "dk": grads["k"], "dv": grads["v"],
            "dq_rope": grads.get("q_rope"), "dk_rope": grads.get("k_rope")}

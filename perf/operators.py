"""The attention layer's operators on the event history, as cases to measure: rotary positions,
the append to a paged key/value cache, attention of a chunk of new tokens over that cache, and the
block norm (norms before and after a block with its gate and residual scale), forward and backward.

A case's lengths follow from the case alone (``lens_seed``); the values of its inputs from the seed
given to ``prepare``.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BIG = 2**31 - 1


def listed():
    return [
        # training: q and k (16 + 16 heads) of a batch of event histories, before the window attention
        dict(name="rotary_train", op="rotary", dtype="bf16", lens_seed=1, B=256, n_lo=32, n_hi=1024,
             ctx_lo=0, ctx_hi=0, h=32, dh=64, rot=64, interleaved=False, factor=1.0, inverse=False),
        # the gradient of partly rotated fp32 heads, interleaved pairs, far positions of a scaled context
        dict(name="rotary_inverse_f32", op="rotary", dtype="f32", lens_seed=2, B=7, n_lo=1, n_hi=4001,
             ctx_lo=100000, ctx_hi=1000000, h=6, dh=128, rot=96, interleaved=True, factor=8.0,
             inverse=True),
        # serving, one new event for each of 64 users
        dict(name="append_decode", op="append", dtype="bf16", lens_seed=3, B=64, n_lo=1, n_hi=1,
             ctx_lo=200, ctx_hi=4000, hq=16, hk=16, dh=64, page=32, rot=64, interleaved=False,
             factor=1.0),
        # serving, the first chunks of new histories: shared heads, long ragged chunks
        dict(name="append_chunk", op="append", dtype="bf16", lens_seed=4, B=48, n_lo=0, n_hi=2047,
             ctx_lo=0, ctx_hi=500, hq=32, hk=8, dh=128, page=64, rot=64, interleaved=True,
             factor=4.0),
        # serving, one event of three users: the latency of a step
        dict(name="decode_small", op="chunk", dtype="bf16", lens_seed=5, B=3, n_lo=1, n_hi=1,
             ctx_lo=100, ctx_hi=1500, hq=16, hk=16, dh=64, page=16, window=0),
        # serving, one event for each of 64 users with long ragged histories, 4 heads on each kv head
        dict(name="decode_long", op="chunk", dtype="bf16", lens_seed=6, B=64, n_lo=1, n_hi=1,
             ctx_lo=1000, ctx_hi=16000, hq=32, hk=8, dh=128, page=64, window=0),
        # serving, sessions of a few hundred new events (some users with none) in a 256-event window
        dict(name="chunk_window", op="chunk", dtype="bf16", lens_seed=7, B=48, n_lo=0, n_hi=700,
             ctx_lo=0, ctx_hi=3000, hq=16, hk=16, dh=64, page=16, window=256),
        # serving, a long chunk late in a long context: the matrix products count
        dict(name="chunk_long", op="chunk", dtype="bf16", lens_seed=8, B=2, n_lo=4000, n_hi=4100,
             ctx_lo=12000, ctx_hi=12200, hq=16, hk=4, dh=128, page=128, window=0),
        # serving step: one row per user between two blocks
        dict(name="norm_decode", op="norm", dtype="bf16", lens_seed=9, B=64, n_lo=1, n_hi=1, d=1024,
             gate="sample", sigmoid=True, post=True, backward=False),
        # training forward between two blocks, a gate for every element
        dict(name="norm_forward", op="norm", dtype="bf16", lens_seed=10, B=256, n_lo=32, n_hi=1024,
             d=2048, gate="token", sigmoid=True, post=True, backward=False),
        # training backward, one gate per user shared by the user's events
        dict(name="norm_backward", op="norm", dtype="bf16", lens_seed=11, B=256, n_lo=32, n_hi=1024,
             d=1024, gate="sample", sigmoid=False, post=True, backward=True),
        # an odd width in fp32, no norm after the block
        dict(name="norm_backward_f32", op="norm", dtype="f32", lens_seed=12, B=9, n_lo=1, n_hi=2001,
             d=1001, gate="token", sigmoid=True, post=False, backward=True),
    ]


def _logu(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "chunk", "chunk", "chunk", "norm", "norm"])
    c = dict(op=op, dtype="bf16", lens_seed=rng.randrange(1 << 30))
    if op == "norm":
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["B"] = _logu(rng, 1, 300)
        d = _logu(rng, 64, 8192)
        c["d"] = d if rng.random() < 0.3 else max(8, d // 8 * 8)
        most = max(1, (1 << 27) // (c["d"] * c["B"]))       # elements of the largest listed case
        c["n_hi"] = _logu(rng, 1, min(4000, most))
        c["n_lo"] = rng.randint(min(1, c["n_hi"]), c["n_hi"])
        c["gate"] = rng.choice(["none", "token", "sample"])
        c["sigmoid"] = rng.random() < 0.5
        c["post"] = rng.random() < 0.7
        c["backward"] = rng.random() < 0.5
        return c
    c["dh"] = rng.choice([32, 64, 64, 128, 128])
    c["ctx_lo"] = 0
    if op in ("rotary", "append"):
        c["rot"] = rng.choice([c["dh"], c["dh"], c["dh"] // 2, 2 * rng.randint(1, c["dh"] // 2)])
        c["interleaved"] = rng.random() < 0.5
        c["factor"] = rng.choice([1.0, 2.0, 8.0])
        c["B"] = _logu(rng, 1, 200)
        c["n_hi"] = _logu(rng, 1, max(1, min(4000, (1 << 16) // c["B"])))
        c["n_lo"] = rng.randint(0, c["n_hi"]) if c["n_hi"] > 1 else 1
    if op == "rotary":
        c["dtype"] = rng.choice(["bf16", "f32"])
        c["h"] = rng.randint(1, 32)
        c["ctx_hi"] = _logu(rng, 1, 1000000)
        c["inverse"] = rng.random() < 0.5
        return c
    c["page"] = rng.choice([16, 32, 64, 128])
    c["hk"] = rng.choice([1, 2, 4, 8, 16])
    c["hq"] = c["hk"] * rng.choice([g for g in (1, 2, 3, 4, 8) if g * c["hk"] <= 32])
    if op == "append":
        c["ctx_hi"] = _logu(rng, 1, 4000)
        return c
    kind = rng.choice(["one", "few", "chunk"])
    c["window"] = rng.choice([0, 0, _logu(rng, 1, 4000)])
    if kind == "chunk":
        c["n_hi"] = _logu(rng, 20, 4000)
        c["ctx_hi"] = _logu(rng, 1, 12000)
        most = (1 << 31) // (c["hq"] * c["n_hi"] * (c["n_hi"] + c["ctx_hi"]))
        if most < 1:
            c["hk"], c["hq"], most = 1, 4, (1 << 31) // (4 * c["n_hi"] * (c["n_hi"] + c["ctx_hi"]))
        c["B"] = _logu(rng, 1, max(1, min(64, most)))
        c["n_lo"] = rng.randint(0, c["n_hi"] - 1)
        return c
    c["n_hi"] = 1 if kind == "one" else rng.randint(2, 16)
    c["n_lo"] = 1
    c["ctx_hi"] = _logu(rng, 50, 60000)
    most = 64 * 16000 * 8 * 128 // (c["hk"] * c["dh"] * c["ctx_hi"])
    c["B"] = _logu(rng, 1, max(1, min(256, most)))
    return c


def _lengths(c):
    """(new tokens of each sample, tokens of each sample before them), from the case alone."""
    r = random.Random(c["lens_seed"])
    n = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    if sum(n) == 0:
        n[0] = 1
    ctx = [r.randint(c.get("ctx_lo", 0), c.get("ctx_hi", 0)) for _ in range(c["B"])]
    return n, ctx


def work(c):
    n, ctx = _lengths(c)
    T, es = sum(n), 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rotary":
        return {"bytes": 2 * T * c["h"] * c["dh"] * es, "flops": 3 * T * c["h"] * c["rot"]}
    if c["op"] == "append":
        return {"bytes": 2 * T * (c["hq"] + 2 * c["hk"]) * c["dh"] * es,
                "flops": 3 * T * (c["hq"] + c["hk"]) * c["rot"]}
    if c["op"] == "norm":
        rows, extra = (7, 24) if c["backward"] else (4, 10)
        rows += {"token": 2 if c["backward"] else 1}.get(c["gate"], 0)
        return {"bytes": rows * T * c["d"] * es, "flops": extra * T * c["d"]}
    w = c["window"] or BIG
    seen = pairs = 0
    for a, b in zip(n, ctx):
        if not a:
            continue
        seen += min(a + b, a + w - 1)
        full = max(0, min(a, w - b))      # rows whose window still reaches the first token
        pairs += full * b + full * (full + 1) // 2 + (a - full) * w
    return {"bytes": seen * c["hk"] * c["dh"] * 2 * es + 2 * T * c["hq"] * c["dh"] * es
            + 4 * T * c["hq"], "flops": 4 * c["dh"] * c["hq"] * pairs}


def _spec(c):
    """The rotary settings of a case: a context scaled by ``factor`` was trained at 2048 tokens."""
    scaled = c["factor"] != 1.0
    return dict(rot=c["rot"], interleaved=c["interleaved"], base=10000.0, factor=c["factor"],
                trained_len=2048 if scaled else 0, low=1.0, high=32.0,
                mscale=1.0 + 0.1 * math.log(c["factor"]) if scaled else 1.0)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    n, ctx = _lengths(c)
    T, B = sum(n), c["B"]

    def rand(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(c=c, T=T, max_n=max(n))
    s["offsets"] = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=dev)
    kv_len = [a + b for a, b in zip(n, ctx)]
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
    if c["op"] == "norm":
        d = c["d"]
        s["f"], s["a"] = rand(T, d), rand(T, d)      # a: the residual stream before (after) the block
        s["a"] += 0.5 * rand(T, 1)
        s["gate"] = {"none": lambda: None, "token": lambda: rand(T, d),
                     "sample": lambda: rand(B, d)}[c["gate"]]()
        s["w_pre"] = 1.0 + 0.2 * rand(d, dtype=torch.float32)
        s["w_post"] = 1.0 + 0.2 * rand(d, dtype=torch.float32) if c["post"] else None
        s["alpha"], s["eps"] = 0.7, 1e-6
        if c["backward"]:
            s["dy"], s["dn"] = rand(T, d), rand(T, d)
        return s
    dh = c["dh"]
    if c["op"] == "rotary":
        s["x"] = rand(T, c["h"], dh)
        return s
    hk, hq, page = c["hk"], c["hq"], c["page"]
    pages = [-(-x // page) for x in kv_len]
    P, width = sum(pages) + 3, max(1, max(pages))
    order = torch.randperm(P, generator=g, device=dev, dtype=torch.int64)
    table = torch.full((B, width), -1, dtype=torch.int64, device=dev)
    col = torch.arange(width, device=dev)
    first = torch.tensor([0] + list(np.cumsum(pages)), device=dev)
    held = col < torch.tensor(pages, device=dev)[:, None]
    table = torch.where(held, order[(first[:-1, None] + col).clamp(max=P - 1)], table)
    if c["op"] == "append":
        qkv = rand(T, hq + 2 * hk, dh)               # one projection's output, used in place
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["cache_k"], s["cache_v"] = rand(P, hk, page, dh), rand(P, hk, page, dh)
        s["table"] = table.to(torch.int32)
        return s
    s["q"] = 1.5 * rand(T, hq, dh)
    s["scale"] = dh ** -0.5
    s["window"] = c["window"] or None
    s["cache_k"], s["cache_v"] = rand(P, hk, page, dh), rand(P, hk, page, dh)
    # rows that hold no token are memory that was never written
    pos = torch.arange(width * page, device=dev)
    live = torch.zeros(P * page, dtype=torch.bool, device=dev)
    at = (table.clamp(min=0)[:, :, None] * page + torch.arange(page, device=dev)).reshape(B, -1)
    live[at[(pos < s["kv_len"][:, None]) & held.repeat_interleave(page, 1)]] = True
    dead = ~live.view(P, 1, page, 1)
    s["cache_k"].masked_fill_(dead, math.nan)
    s["cache_v"].masked_fill_(dead, math.nan)
    if c["window"]:      # pages behind every window have been given back
        low = s["kv_len"] - torch.tensor(n, device=dev) - c["window"] + 1
        table = torch.where((col + 1) * page <= low[:, None], torch.full_like(table, -1), table)
    s["table"] = table.to(torch.int32)
    return s


# --------------------------------------------------------------- the framework's calls
def _own(s):
    from recsys_context_personalised_b200 import gdpa as G
    c, off = s["c"], s["offsets"]
    if c["op"] == "rotary":
        return G.rotary(G.rotary_spec(**_spec(c)), s["x"], offsets=off, kv_len=s["kv_len"],
                        inverse=c["inverse"])
    if c["op"] == "append":
        q = G.cache_append(s["k"], s["v"], off, s["kv_len"], s["table"], s["cache_k"],
                           s["cache_v"], spec=G.rotary_spec(**_spec(c)), q=s["q"])
        return q, s["cache_k"], s["cache_v"]
    if c["op"] == "chunk":
        return G.chunk_fwd(s["q"], off, s["kv_len"], s["table"], s["cache_k"], s["cache_v"],
                           s["scale"], max_n=s["max_n"], window=s["window"])
    kw = dict(gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], alpha=s["alpha"],
              eps=s["eps"], sigmoid=c["sigmoid"], offsets=off if c["gate"] == "sample" else None)
    if c["backward"]:
        return G.block_norm_bwd(s["a"], s["f"], dy=s["dy"], dn=s["dn"], **kw)
    return G.block_norm_fwd(s["a"], s["f"], **kw)


# --------------------------------------------------------------- the plain forms
def _rows(s):
    """(sample of each token, its place among the sample's new tokens, its position)"""
    off = s["offsets"].long()
    t = torch.arange(s["T"], device=off.device)
    b = torch.searchsorted(off[1:], t, right=True)
    i = t - off[b]
    return b, i, s["kv_len"].long()[b] - (off[1:] - off[:-1])[b] + i


def _turn(x, pos, c, inverse):
    sp = _spec(c)
    half = sp["rot"] // 2
    w = sp["base"] ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    part = 1.0
    if sp["factor"] != 1.0:
        part = ((sp["trained_len"] * w / (2 * math.pi) - sp["low"]) / (sp["high"] - sp["low"])).clamp(0, 1)
    w = w * (part + (1 - part) / sp["factor"])
    ang = pos.double()[:, None] * w * (-1.0 if inverse else 1.0)
    cos, sin = ((f(ang) * sp["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))
    x = x.float()
    y = x.clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if sp["interleaved"] else (
        slice(0, half), slice(half, 2 * half))
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., first] * sin + x[..., second] * cos
    return y


def _plain_chunk(s):
    c = s["c"]
    off, kv_len, table = s["offsets"].long(), s["kv_len"].long(), s["table"].long()
    B, hk, page, dh = c["B"], c["hk"], c["page"], c["dh"]
    g, N, L = c["hq"] // hk, s["max_n"], table.shape[1] * page
    key = torch.arange(L, device=off.device)
    n = off[1:] - off[:-1]
    row = torch.arange(N, device=off.device)
    pos = (kv_len - n)[:, None] + row                                        # [B, N]
    see = (key <= pos[:, :, None]) & (row < n[:, None])[:, :, None]          # [B, N, L]
    if s["window"]:
        see &= key > pos[:, :, None] - s["window"]
    some = see.any(1)[:, None, :, None]                                      # keys that any row sees
    k, v = (x[table.clamp(min=0)].transpose(1, 2).reshape(B, hk, L, dh).float()
            for x in (s["cache_k"], s["cache_v"]))
    zero = torch.zeros((), device=off.device)
    k, v = torch.where(some, k, zero), torch.where(some, v, zero)
    q = s["q"][(off[:-1, None] + row).clamp(max=s["T"] - 1)].float()         # [B, N, hq, dh]
    q = q.view(B, N, hk, g, dh).permute(0, 2, 3, 1, 4).reshape(B, hk, g * N, dh)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, hk, g, N, L)
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, zero, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, hk, g * N, L) @ v).view(B, hk, g, N, dh) / torch.where(l == 0, zero + 1, l)
    lse = (l.log() + m).squeeze(-1)                                          # [B, hk, g, N]
    b, i, _ = _rows(s)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, c["hq"], dh)[b, i]
    lse = lse.permute(1, 2, 0, 3).reshape(c["hq"], B, N)[:, b, i]
    return o.to(s["q"].dtype), lse


def _plain_norm(s):
    c, eps, alpha = s["c"], s["eps"], s["alpha"]
    dt = s["a"].dtype
    f, a = s["f"].float(), s["a"].float()
    b = _rows(s)[0] if c["gate"] == "sample" else None
    z = None if s["gate"] is None else s["gate"].float()
    act = torch.ones((), device=f.device) if z is None else (1 / (1 + torch.exp(-z)) if c["sigmoid"] else z)
    full = act if b is None else act[b]

    def inv(x):
        return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)

    fh = f * inv(f) if c["post"] else f
    u = fh * s["w_post"] if c["post"] else f
    if not c["backward"]:
        y = a + alpha * full * u
        return y.to(dt), (y * inv(y) * s["w_pre"]).to(dt)
    dn, ry = s["dn"].float(), inv(a)
    yh, t = a * ry, dn * s["w_pre"]
    G = s["dy"].float() + ry * (t - yh * (t * yh).mean(-1, keepdim=True))
    du = alpha * full * G
    dgate = dw_post = None
    if z is not None:
        dgate = alpha * G * u
        if b is not None:
            dgate = torch.zeros_like(z).index_add_(0, b, dgate)
        if c["sigmoid"]:
            dgate = dgate * act * (1 - act)
        dgate = dgate if b is not None else dgate.to(dt)
    df = du
    if c["post"]:
        t = du * s["w_post"]
        df = inv(f) * (t - fh * (t * fh).mean(-1, keepdim=True))
        dw_post = (du * fh).sum(0)
    return G.to(dt), df.to(dt), dgate, dw_post, (dn * yh).sum(0)


def run(s):
    if own:
        return _own(s)
    c = s["c"]
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "chunk":
        return _plain_chunk(s)
    b, i, pos = _rows(s)
    if c["op"] == "rotary":
        return _turn(s["x"], pos, c, c["inverse"]).to(s["x"].dtype)
    page = s["table"].long()[b, pos // c["page"]]
    s["cache_k"][page, :, pos % c["page"]] = _turn(s["k"], pos, c, False).to(s["k"].dtype)
    s["cache_v"][page, :, pos % c["page"]] = s["v"]
    return _turn(s["q"], pos, c, False).to(s["q"].dtype), s["cache_k"], s["cache_v"]


# --------------------------------------------------------------- the definitions, in 64 bits
def _exact_turn(x, pos, c, inverse):
    """Each pair as a complex number, multiplied by mscale * exp(i pos w)."""
    sp = _spec(c)
    R = sp["rot"]
    freq = []
    for i in range(R // 2):
        w = sp["base"] ** (-2.0 * i / R)
        keep = 1.0
        if sp["factor"] != 1.0:
            r = sp["trained_len"] * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (r - sp["low"]) / (sp["high"] - sp["low"])))
        freq.append(w * keep + (1.0 - keep) * w / sp["factor"])
    w = torch.tensor(freq, dtype=torch.float64, device=x.device)
    z = torch.polar(torch.full((len(pos), R // 2), sp["mscale"], dtype=torch.float64, device=x.device),
                    torch.tensor(pos, dtype=torch.float64, device=x.device)[:, None] * w)
    z = (z.conj() if inverse else z)[:, None]
    y = x.double()
    head, rest = y[..., :R], y[..., R:]
    pairs = head.unflatten(-1, (-1, 2)) if sp["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    out = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * z)
    out = out if sp["interleaved"] else out.transpose(-1, -2)
    return torch.cat([out.flatten(-2), rest], -1)


def exact(c, seed):
    s = prepare(c, seed)
    n, ctx = _lengths(c)
    pos = [p for a, b in zip(n, ctx) for p in range(b, b + a)]
    if c["op"] == "rotary":
        return _exact_turn(s["x"], pos, c, c["inverse"])
    if c["op"] == "append":
        ck, cv = s["cache_k"].double(), s["cache_v"].double()
        k, table, t = _exact_turn(s["k"], pos, c, False), s["table"].tolist(), 0
        rows = [table[b][p // c["page"]] * c["page"] + p % c["page"]
                for b in range(c["B"]) for p in range(ctx[b], ctx[b] + n[b])]
        rows = torch.tensor(rows, device=k.device)
        for cache, new in ((ck, k), (cv, s["v"].double())):
            flat = cache.transpose(1, 2).reshape(-1, c["hk"], c["dh"])
            flat[rows] = new
            cache.copy_(flat.view(-1, c["page"], c["hk"], c["dh"]).transpose(1, 2))
        return _exact_turn(s["q"], pos, c, False), ck, cv
    if c["op"] == "norm":
        return _exact_norm(s, n)
    o = torch.zeros_like(s["q"], dtype=torch.float64)
    lse = torch.full((c["hq"], s["T"]), -math.inf, dtype=torch.float64, device=o.device)
    g, t0 = c["hq"] // c["hk"], 0
    for b in range(c["B"]):
        if not n[b]:
            continue
        low = max(0, ctx[b] - c["window"] + 1) if c["window"] else 0
        p = torch.arange(low, ctx[b] + n[b], device=o.device)
        page, at = s["table"][b].long()[p // c["page"]], p % c["page"]
        me = torch.arange(ctx[b], ctx[b] + n[b], device=o.device)[:, None]
        hidden = p > me
        if c["window"]:
            hidden |= p <= me - c["window"]
        for j in range(c["hq"]):
            k, v = (x[page, j // g, at].double() for x in (s["cache_k"], s["cache_v"]))
            x = (s["q"][t0:t0 + n[b], j].double() @ k.T) * s["scale"]
            x.masked_fill_(hidden, -math.inf)
            lse[j, t0:t0 + n[b]] = torch.logsumexp(x, -1)
            o[t0:t0 + n[b], j] = torch.softmax(x, -1) @ v
        t0 += n[b]
    return o, lse


def _exact_norm(s, n):
    """The forward's formula in 64 bits; the backward by differentiating that formula."""
    c = s["c"]
    if s["f"].numel() > 1 << 29:
        return None
    a, f = s["a"].double(), s["f"].double()
    z = None if s["gate"] is None else s["gate"].double()
    w_pre = s["w_pre"].double()
    w_post = None if s["w_post"] is None else s["w_post"].double()

    def norm(x, w):
        return x * w * torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"])

    def branch(f, z, w_post):
        v = f if w_post is None else norm(f, w_post)
        if z is not None:
            v = v * (torch.sigmoid(z) if c["sigmoid"] else z).repeat_interleave(
                torch.tensor(n, device=v.device), 0) if c["gate"] == "sample" else v * (
                torch.sigmoid(z) if c["sigmoid"] else z)
        return s["alpha"] * v

    if not c["backward"]:
        y = a + branch(f, z, w_post)
        return y, norm(y, w_pre)
    a.requires_grad_(), w_pre.requires_grad_()
    da, dw_pre = torch.autograd.grad(norm(a, w_pre), (a, w_pre), s["dn"].double())
    da = da + s["dy"].double()
    leaves = [x.requires_grad_() for x in (f, z, w_post) if x is not None]
    grads = iter(torch.autograd.grad(branch(f, z, w_post), leaves, da))
    df, dz, dw_post = (next(grads) if x is not None else None for x in (f, z, w_post))
    return da, df, dz, dw_post, dw_pre

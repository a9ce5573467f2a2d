"""Cases of the operators that run between the adapter layers of a decoder's
attention block: what each is called with, its plain form, its definition in
64 bits, and what one pass has to move and compute.

  assign  pages and slots of a step's tokens, from the requests' lengths
  rotary  rotation of q and k by positions with several axes, k and v stored
          in the paged cache
  attend  attention of new tokens over the paged cache
  norm    the norms after and before a block with its gate and residual scale

``own`` false: elementary torch operations; true: the framework's operators.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _es(dtype):
    return 2 if dtype == "bf16" else 4


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of 128 requests: one token each, some just ended
        {"name": "assign_decode_128", "op": "assign", "requests": 128, "max_len": 4096, "max_new": 1,
         "page_size": 16, "ended": 0.05, "short": False},
        # a large mixed step: thousands of requests, prompts among them, the pool runs dry
        {"name": "assign_prompts_2000", "op": "assign", "requests": 2000, "max_len": 8000, "max_new": 150,
         "page_size": 32, "ended": 0.1, "short": True},
        # one token of one request: 32 query and 8 key heads of 128, as a 4096 -> (4096, 1024, 1024) layer has
        {"name": "rotary_1_token", "op": "rotary", "tokens": 1, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "axes": 1, "interleaved": False, "page_size": 16, "src": "f32", "dtype": "bf16",
         "far": 131072},
        # the decode batch of 128 tokens, positions of image and video tokens (time, height, width)
        {"name": "rotary_128_3axes", "op": "rotary", "tokens": 128, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "axes": 3, "interleaved": False, "page_size": 16, "src": "f32", "dtype": "bf16",
         "far": 32768},
        # prompts: an odd number of tokens, part of each head rotated, adjacent pairs
        {"name": "rotary_8191_partial", "op": "rotary", "tokens": 8191, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 64, "axes": 2, "interleaved": True, "page_size": 64, "src": "f32", "dtype": "bf16",
         "far": 1000000},
        # one request, a short context: latency
        {"name": "attend_1x700", "op": "attend", "requests": 1, "new": 1, "max_len": 700, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page_size": 16, "dtype": "bf16", "window": 0, "full": True,
         "by_head": False},
        # the decode batch of 128 requests with ragged contexts, empty ones among them
        {"name": "attend_128_ragged", "op": "attend", "requests": 128, "new": 1, "max_len": 4096, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page_size": 16, "dtype": "bf16", "window": 0, "full": False,
         "by_head": False},
        # two requests with long contexts, odd lengths, a cache laid out by head
        {"name": "attend_2x100003", "op": "attend", "requests": 2, "new": 1, "max_len": 100003, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page_size": 64, "dtype": "bf16", "window": 0, "full": True,
         "by_head": True},
        # the largest: 64 requests of up to 16384 positions
        {"name": "attend_64x16384", "op": "attend", "requests": 64, "new": 1, "max_len": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page_size": 32, "dtype": "bf16", "window": 0, "full": False,
         "by_head": False},
        # float32 layers: several drafted tokens a request, a window, pages of an odd size
        {"name": "attend_f32_drafts", "op": "attend", "requests": 16, "new": 4, "max_len": 2500, "heads": 12,
         "kv_heads": 4, "head_dim": 80, "page_size": 5, "dtype": "f32", "window": 1000, "full": False,
         "by_head": False},
        # the decode batch between two layers 4096 wide: both norms and a gate
        {"name": "norm_128x4096", "op": "norm", "rows": 128, "d": 4096, "kind": "rms", "post": True, "pre": True,
         "gate": "none", "y": "f32", "h": "bf16", "x": "bf16"},
        # a batch of prompts: layer norms with biases, a gate for each token
        {"name": "norm_8191x4096_gated", "op": "norm", "rows": 8191, "d": 4096, "kind": "layer", "post": True,
         "pre": True, "gate": "token", "y": "f32", "h": "f32", "x": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "rotary", "attend", "attend", "norm"])
    if op == "assign":
        return {"op": op, "requests": _log(rng, 1, 4000), "max_len": _log(rng, 16, 10000),
                "max_new": rng.choice([1, 1, _log(rng, 2, 150)]), "page_size": rng.choice([1, 5, 16, 32, 64, 100, 128]),
                "ended": rng.choice([0.0, 0.1]), "short": rng.random() < 0.3}
    if op == "rotary":
        hd = 8 * rng.randint(2, 32)
        kv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 8000), "heads": kv * rng.randint(1, 6), "kv_heads": kv,
                "head_dim": hd, "rot_dim": rng.choice([hd, 2 * rng.randint(1, hd // 2)]), "axes": rng.randint(1, 4),
                "interleaved": rng.random() < 0.5, "page_size": rng.choice([1, 5, 16, 32, 64, 100, 128]),
                "src": rng.choice(["f32", "f32", "bf16"]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "far": _log(rng, 100, 1000000)}
    if op == "attend":
        kv = rng.choice([1, 2, 4, 8])
        new = rng.choice([1, 1, 1, rng.randint(2, 5)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        hd = 8 * rng.randint(2, 32)
        requests = _log(rng, 1, 192)
        # in all no more bytes of cache than the largest case reads
        room = 500000 * 4096 // (2 * kv * hd * _es(dtype) * new)
        return {"op": op, "requests": requests, "new": new, "max_len": _log(rng, new, max(new, min(100000, room // requests))),
                "heads": kv * rng.randint(1, 20), "kv_heads": kv, "head_dim": hd,
                "page_size": rng.choice([1, 5, 16, 16, 32, 64, 100, 128]), "dtype": dtype,
                "window": rng.choice([0, 0, 0, _log(rng, 1, 4000)]), "full": rng.random() < 0.3,
                "by_head": rng.random() < 0.3}
    d = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)])
    return {"op": op, "rows": _log(rng, 1, max(1, min(8000, 20000000 // d))), "d": d,
            "kind": rng.choice(["rms", "layer"]), "post": rng.random() < 0.7, "pre": rng.random() < 0.8,
            "gate": rng.choice(["none", "channel", "token"]), "y": rng.choice(["f32", "f32", "bf16"]),
            "h": rng.choice(["f32", "bf16"]), "x": rng.choice(["f32", "bf16", "bf16"])}


# ---- what the caller has in hand ----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _assign_sizes(c):
    R, ps = c["requests"], c["page_size"]
    width = -(-(c["max_len"] + c["max_new"]) // ps)
    return R, ps, width, R * c["max_new"]


def _prepare_assign(c, g):
    R, ps, P, T = _assign_sizes(c)
    old = _lengths(g, R, 0, c["max_len"])
    if c["max_new"] == 1:
        new = torch.ones_like(old)
    else:  # half of them decode, the others bring a prompt or a part of one
        new = torch.where(torch.rand(R, generator=g, device="cuda") < 0.5, torch.ones_like(old),
                          _lengths(g, R, 0, c["max_new"]))
    ended = torch.rand(R, generator=g, device="cuda") < c["ended"]
    new = torch.where(ended, torch.full_like(new, -1), new)
    held = (old + ps - 1) // ps
    n_pages = R * P
    pages = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64)
    col = torch.arange(P, device="cuda")
    first = torch.cumsum(held, 0) - held
    table = torch.where(col[None] < held[:, None], pages[(first[:, None] + col[None]).clamp(max=n_pages - 1)],
                        torch.full((), -1, device="cuda", dtype=torch.int64))
    n_held = held.sum()
    # the free pages lie in a ring, from a place somewhere in it
    free = n_pages - n_held
    free = free // 64 if c["short"] else free
    head = _lengths(g, 1, 0, n_pages)[0] + 5 * n_pages
    at = torch.arange(n_pages, device="cuda")
    k = (at - head) % n_pages
    ring = torch.where(k < free, pages[(n_held + k).clamp(max=n_pages - 1)],
                       torch.full((), -1, device="cuda", dtype=torch.int64))
    st = {"old": old.int(), "new": new.int(), "table": table.int(), "ring": ring.int(),
          "cursor": torch.stack([head, head + free])}
    st["max_tokens"] = T
    if own:
        from lora_normal_form_amd import block
        st["rows"] = block.Rows(R, T, device=old.device)
    return st


def _rotary_sections(c):
    """Axis of each rotary pair: contiguous sections, one an axis."""
    n = c["rot_dim"] // 2
    return [min(c["axes"] - 1, i * c["axes"] // max(1, n)) for i in range(n)]


def _prepare_rotary(c, g):
    T, D, Hq, Hk, ps = c["tokens"], c["head_dim"], c["heads"], c["kv_heads"], c["page_size"]
    y = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device="cuda").to(DT[c["src"]])
    n = c["rot_dim"] // 2
    freq = 500000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / max(1, n))
    axis = torch.tensor(_rotary_sections(c), device="cuda", dtype=torch.int32)
    pos = torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
    n_pages = -(-(T + 2) // ps) + 3
    slot = torch.randperm(n_pages * ps, generator=g, device="cuda")[:T]
    slot = torch.where(torch.rand(T, generator=g, device="cuda") < 0.01, torch.full_like(slot, -1), slot)
    dt = DT[c["dtype"]]
    kc = torch.randn((n_pages, ps, Hk, D), generator=g, device="cuda").to(dt)
    vc = torch.randn((n_pages, ps, Hk, D), generator=g, device="cuda").to(dt)
    st = {"y": y, "freq": freq, "axis": axis, "pos": pos, "slot": slot, "k": kc, "v": vc}
    if own:
        from lora_normal_form_amd import block
        st["cache"] = block.KVCache(kc, vc)
        st["rotary"] = block.Rotary(freq, D, axis=axis, n_axes=c["axes"], interleaved=c["interleaved"])
        st["q_out"] = torch.empty((T, Hq, D), device="cuda", dtype=dt)
    return st


def _prepare_attend(c, g):
    R, new, L, ps = c["requests"], c["new"], c["max_len"], c["page_size"]
    Hq, Hk, D = c["heads"], c["kv_heads"], c["head_dim"]
    dt = DT[c["dtype"]]
    total = torch.full((R,), L, device="cuda", dtype=torch.int64) if c["full"] else _lengths(g, R, 0, L)
    P = -(-L // ps)
    n_pages = R * P + 1
    table = torch.randperm(n_pages, generator=g, device="cuda")[:R * P].view(R, P).int()
    shape = (n_pages, Hk, ps, D) if c["by_head"] else (n_pages, ps, Hk, D)
    kc = torch.empty(shape, device="cuda", dtype=dt).normal_(generator=g)
    vc = torch.empty(shape, device="cuda", dtype=dt).normal_(generator=g)
    if c["by_head"]:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    q = torch.randn((R * new, Hq, D), generator=g, device="cuda").to(dt)
    # the new tokens of a request are its newest positions: each sees up to its own
    back = torch.arange(new - 1, -1, -1, device="cuda")
    row_len = (total[:, None] - back[None]).clamp(min=0).reshape(-1).int()
    row_req = torch.arange(R, device="cuda").repeat_interleave(new).int()
    st = {"k": kc, "v": vc, "q": q, "table": table, "row_len": row_len, "row_req": row_req}
    if own:
        from lora_normal_form_amd import block
        st["attention"] = block.PagedAttention(block.KVCache(kc, vc), Hq, R * new, window=c["window"])
        st["out"] = torch.empty_like(q)
    return st


ALPHA, BETA, EPS = 0.7, 1.0, 1e-5


def _prepare_norm(c, g):
    T, d = c["rows"], c["d"]

    def vec(mean, on):
        return mean + 0.2 * torch.randn(d, generator=g, device="cuda") if on else None

    layer = c["kind"] == "layer"
    st = {"y": (3.0 * torch.randn((T, d), generator=g, device="cuda") + 0.5).to(DT[c["y"]]),
          "h": (2.0 * torch.randn((T, d), generator=g, device="cuda")).to(DT[c["h"]]),
          "post_w": vec(1.0, c["post"]), "post_b": vec(0.0, c["post"] and layer),
          "pre_w": vec(1.0, c["pre"]), "pre_b": vec(0.0, c["pre"] and layer), "gate": None}
    if c["gate"] == "channel":
        st["gate"] = torch.randn(d, generator=g, device="cuda")
    elif c["gate"] == "token":
        st["gate"] = torch.randn((T, d), generator=g, device="cuda")
    if own:
        from lora_normal_form_amd import block
        st["norm"] = block.ResidualNorm(d, kind=c["kind"], post=c["post"], post_weight=st["post_w"],
                                        post_bias=st["post_b"], pre=c["pre"], pre_weight=st["pre_w"],
                                        pre_bias=st["pre_b"], h_scale=BETA, y_scale=ALPHA, eps=EPS)
        st["h_out"] = torch.empty_like(st["h"])
        st["x"] = torch.empty((T, d), device="cuda", dtype=DT[c["x"]]) if c["pre"] else None
    return st


def prepare(case, seed):
    g = _gen(seed)
    st = {"assign": _prepare_assign, "rotary": _prepare_rotary, "attend": _prepare_attend,
          "norm": _prepare_norm}[case["op"]](case, g)
    st["case"] = case
    return st


# ---- one pass ------------------------------------------------------------------------------------

def _run_assign(st):
    c, table, ring, cursor = st["case"], st["table"], st["ring"], st["cursor"]
    if own:
        from lora_normal_form_amd import block
        r = block.assign_pages(st["old"], st["new"], table, ring, cursor, c["page_size"], st["rows"])
        return {"table": table, "ring": ring, "cursor": r.cursor, "seq_len": r.seq_len, "cu_len": r.cu_len,
                "slot": r.slot, "req": r.req, "pos": r.pos, "len": r.len, "counts": r.counts}
    ps, P, cap, T = c["page_size"], table.shape[1], ring.shape[0], st["max_tokens"]
    o, n = st["old"].long(), st["new"].long()
    grows = n >= 0
    add = n.clamp(min=0)
    held = (o + ps - 1) // ps
    upto = (o + add + ps - 1) // ps
    fits = grows & (upto <= P)
    want = torch.where(fits, upto - held, 0)
    need = torch.cumsum(want, 0)
    base = need - want
    head, tail = cursor[0], cursor[1]
    placed = fits & ((want == 0) | (need <= tail - head))  # in the requests' order, all of its pages or none
    col = torch.arange(P, device=o.device)
    j = col[None] - held[:, None]
    takes = (j >= 0) & (j < want[:, None]) & placed[:, None]
    table.copy_(torch.where(takes, ring[(head + base[:, None] + j) % cap], table))
    gone = torch.where(grows, 0, held)
    gbase = torch.cumsum(gone, 0) - gone
    to = torch.where(col[None] < gone[:, None], (tail + gbase[:, None] + col[None]) % cap, cap)
    ring.copy_(torch.cat([ring, ring[:1]]).index_put((to.reshape(-1),), table.reshape(-1))[:cap])
    cu = torch.cat([torch.zeros(1, device=o.device, dtype=torch.int64), torch.cumsum(add, 0)])
    t = torch.arange(T, device=o.device)
    req = torch.searchsorted(cu, t, right=True) - 1
    rq = req.clamp(max=o.shape[0] - 1)
    live = (req < o.shape[0]) & placed[rq]
    pos = o[rq] + t - cu[rq]
    page = table[rq, (pos // ps).clamp(max=P - 1)].long()
    taken = torch.where(placed & (want > 0), need, 0).amax()
    counts = torch.stack([torch.where(placed, add, 0).sum(), taken, (grows & ~placed).sum(), gone.sum()])
    return {"table": table, "ring": ring, "cursor": torch.stack([head + taken, tail + gone.sum()]),
            "seq_len": torch.where(placed, o + add, torch.where(grows, o, 0)).int(), "cu_len": cu.int(),
            "slot": torch.where(live, page * ps + pos % ps, -1), "req": torch.where(live, req, -1).int(),
            "pos": torch.where(live, pos, 0).int(), "len": torch.where(live, pos + 1, 0).int(), "counts": counts.int()}


def _split(y, c):
    T, D, Hq, Hk = y.shape[0], c["head_dim"], c["heads"], c["kv_heads"]
    return (y[:, :Hq * D].view(T, Hq, D), y[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D),
            y[:, (Hq + Hk) * D:].view(T, Hk, D))


def _pairs(c):
    n = c["rot_dim"] // 2
    i = torch.arange(n, device="cuda")
    return (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + n)


def _turned(z, cos, sin, c):
    """z [T][H][D] with its pairs rotated."""
    ia, ib = _pairs(c)
    a, b = z[..., ia], z[..., ib]
    out = z.clone()
    out[..., ia] = a * cos[:, None] - b * sin[:, None]
    out[..., ib] = a * sin[:, None] + b * cos[:, None]
    return out


def _run_rotary(st):
    c = st["case"]
    q, k, v = _split(st["y"], c)
    if own:
        st["rotary"].store(q, k, v, st["pos"], st["slot"], st["cache"], st["q_out"])
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    angle = st["pos"].double()[st["axis"].long()].T * st["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dt = st["k"].dtype
    kc, vc = st["k"].flatten(0, 1), st["v"].flatten(0, 1)
    # tokens without a slot rewrite the row that the first one with a slot gets
    some = (st["slot"] >= 0)
    src = torch.where(some, torch.arange(len(some), device="cuda"), torch.argmax(some.int()))
    to = st["slot"][src]
    live = (to >= 0)[:, None, None]
    at = to.clamp(min=0)
    kc[at] = torch.where(live, _turned(k.float(), cos, sin, c).to(dt)[src], kc[at])
    vc[at] = torch.where(live, v.to(dt)[src], vc[at])
    return {"q": _turned(q.float(), cos, sin, c).to(dt), "k": st["k"], "v": st["v"]}


def _run_attend(st):
    c = st["case"]
    if own:
        one = c["new"] == 1
        return st["attention"].forward(st["q"], st["table"], st["row_len"], st["out"],
                                       row_req=None if one else st["row_req"])
    q, table, n = st["q"], st["table"], st["row_len"].long()
    N, Hq, D = q.shape
    Hk, ps, L = c["kv_heads"], c["page_size"], c["max_len"]
    t = torch.arange(L, device=q.device)
    page = table.long()[:, t // ps]
    K = st["k"][page, t % ps].permute(0, 2, 3, 1).float()  # [R][Hk][D][L]
    s = torch.matmul(q.float().view(-1, c["new"], Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).flatten(2, 3), K)
    del K
    s = s.view(s.shape[0], Hk, c["new"], Hq // Hk, L) * (1.0 / math.sqrt(D))
    first = (n - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(n)
    seen = ((t >= first[:, None]) & (t < n[:, None])).view(-1, 1, c["new"], 1, L)
    s = torch.where(seen, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-37)
    V = st["v"][page, t % ps].permute(0, 2, 1, 3).float()
    o = torch.matmul(p.flatten(2, 3), V).view(-1, Hk, c["new"], Hq // Hk, D)
    return o.permute(0, 2, 1, 3, 4).reshape(N, Hq, D).to(q.dtype)


def _normed(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w
    return v if b is None else v + b


def _run_norm(st):
    c = st["case"]
    if own:
        st["norm"].forward(st["y"], st["h"], st["h_out"], st["x"], gate=st["gate"])
        return {"h": st["h_out"], "x": st["x"]}
    z = st["y"].float()
    if c["post"]:
        z = _normed(z, c["kind"], st["post_w"], st["post_b"])
    if st["gate"] is not None:
        z = z * st["gate"]
    h = BETA * st["h"].float() + ALPHA * z
    x = _normed(h, c["kind"], st["pre_w"], st["pre_b"]).to(DT[c["x"]]) if c["pre"] else None
    return {"h": h.to(st["h"].dtype), "x": x}


RUN = {"assign": _run_assign, "rotary": _run_rotary, "attend": _run_attend, "norm": _run_norm}


def run(state):
    return RUN[state["case"]["op"]](state)


# ---- what a pass has to move and compute --------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "assign":
        R, ps, P, T = _assign_sizes(c)
        tokens = R if c["max_new"] == 1 else R * c["max_new"] // 4
        moved = tokens / ps + c["ended"] * R * c["max_len"] / 2 / ps
        return {"bytes": 16 * R + 4 + 20 * T + 8 * moved + 48, "flops": 0}
    if c["op"] == "rotary":
        n = c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["head_dim"]
        turned = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot_dim"]
        return {"bytes": n * (_es(c["src"]) + _es(c["dtype"])) + c["tokens"] * (4 * c["axes"] + 8) + 6 * c["rot_dim"],
                "flops": 3 * turned}
    if c["op"] == "attend":
        rows, mean = c["requests"] * c["new"], c["max_len"] if c["full"] else c["max_len"] / 2
        seen = min(mean, c["window"]) if c["window"] else mean
        read = min(mean, seen + c["new"] - 1) * c["requests"]
        return {"bytes": read * 2 * c["kv_heads"] * c["head_dim"] * _es(c["dtype"]) + 4 * read / c["page_size"]
                + 2 * rows * c["heads"] * c["head_dim"] * _es(c["dtype"]) + 4 * rows,
                "flops": 4 * rows * seen * c["heads"] * c["head_dim"]}
    n = c["rows"] * c["d"]
    vectors = 4 * c["d"] * (1 + (c["kind"] == "layer")) * (c["post"] + c["pre"])
    gate = {"none": 0, "channel": 4 * c["d"], "token": 4 * n}[c["gate"]]
    return {"bytes": n * (_es(c["y"]) + 2 * _es(c["h"]) + (_es(c["x"]) if c["pre"] else 0)) + vectors + gate,
            "flops": n * (3 + 4 * c["post"] + 4 * c["pre"])}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_rotary(c, st):
    y = st["y"].double()
    q, k, v = (t.clone() for t in _split(y, c))
    n = c["rot_dim"] // 2
    for i, ax in enumerate(_rotary_sections(c)):
        ang = st["pos"][ax].double() * 500000.0 ** (-i / max(1, n))
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, n + i)
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]
        for z in (q, k):
            w = torch.complex(z[:, :, a], z[:, :, b]) * turn
            z[:, :, a], z[:, :, b] = w.real, w.imag
    ps = c["page_size"]
    kc, vc = st["k"].double(), st["v"].double()
    live = torch.nonzero(st["slot"] >= 0)[:, 0]
    to = st["slot"][live]
    kc[to // ps, to % ps] = k[live]
    vc[to // ps, to % ps] = v[live]
    return {"q": q, "k": kc, "v": vc}


def _exact_attend(c, st):
    ps, Hk, G = c["page_size"], c["kv_heads"], c["heads"] // c["kv_heads"]
    out = torch.zeros_like(st["q"], dtype=torch.float64)
    lens, table = st["row_len"].tolist(), st["table"].long()
    for i, n in enumerate(lens):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n <= lo:
            continue
        pages = table[i // c["new"], : -(-n // ps)]
        K = st["k"][pages].flatten(0, 1)[lo:n].double().transpose(0, 1).contiguous()
        V = st["v"][pages].flatten(0, 1)[lo:n].double().transpose(0, 1).contiguous()
        q = st["q"][i].double().view(Hk, G, -1)
        p = torch.softmax(torch.bmm(q, K.transpose(1, 2).contiguous()) / math.sqrt(q.shape[-1]), -1)
        out[i] = torch.bmm(p, V).view(c["heads"], -1)
    return out


def _exact_norm(c, st):
    def norm(z, w, b):
        mu = z.mean(1, keepdim=True) if c["kind"] == "layer" else 0.0
        z = (z - mu) / ((z - mu).square().mean(1, keepdim=True) + EPS).sqrt() * w.double()
        return z if b is None else z + b.double()

    z = st["y"].double()
    z = norm(z, st["post_w"], st["post_b"]) if c["post"] else z
    z = z if st["gate"] is None else z * st["gate"].double()
    h = BETA * st["h"].double() + ALPHA * z
    return {"h": h, "x": norm(h, st["pre_w"], st["pre_b"]) if c["pre"] else None}


def exact(case, seed):
    if case["op"] == "assign":
        return None  # whole numbers
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "attend": _exact_attend, "norm": _exact_norm}[case["op"]](case, st)

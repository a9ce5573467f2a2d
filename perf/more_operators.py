"""Cases of the operators around a paged cache whose requests share pages, keep
only a window, or norm their heads: what each is called with, its plain form,
its definition in 64 bits, and what one pass has to move and compute.

  fork     requests that continue others (samples of one prompt, beams), are
           cut back, end or lose the pages between sinks and window: pages
           shared, copied and given back
  compact  positions of a request that stay moved together (accepted tokens of
           a tree of drafts, an evicted context) and the pages behind given back
  heads    norms of each head of q and k, rotary positions and the cache store
           in one pass
  sinks    attention with a sliding window and first tokens that stay visible
  shared   attention of rows whose contexts begin with the same positions

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
        # parallel samples: 8 prompts of 4 beams each, every beam goes on from one of its prompt's
        {"name": "fork_beams_32", "op": "fork", "requests": 32, "beams": 4, "max_len": 2048, "page_size": 16,
         "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "moved": 0.6, "ended": 0.0, "cut": 0.0, "window": 0,
         "sinks": 0, "short": False},
        # a large server between two steps: some requests end, some forget the middle of their context, some
        # drafts are taken back, the pool runs dry
        {"name": "fork_1000_mixed", "op": "fork", "requests": 1000, "beams": 2, "max_len": 8000, "page_size": 32,
         "kv_heads": 2, "head_dim": 64, "dtype": "bf16", "moved": 0.2, "ended": 0.1, "cut": 0.3, "window": 4096,
         "sinks": 64, "short": True},
        # a tree of 24 drafted tokens a request: the accepted path moves together
        {"name": "compact_drafts_64", "op": "compact", "requests": 64, "max_len": 1000, "tail": 24, "share": 0.2,
         "page_size": 16, "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "by_head": False},
        # half of each long context evicted
        {"name": "compact_evict_16x16000", "op": "compact", "requests": 16, "max_len": 16000, "tail": 16000,
         "share": 0.5, "page_size": 64, "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "by_head": True},
        # one token of one request: 32 query and 8 key heads of 128, as a 4096 -> (4096, 1024, 1024) layer has
        {"name": "heads_1_token", "op": "heads", "tokens": 1, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "axes": 1, "interleaved": False, "kind": "rms", "own_weights": False, "page_size": 16,
         "src": "f32", "dtype": "bf16", "far": 131072},
        # prompts: an odd number of tokens, part of each head rotated, layer norms with weights of each head
        {"name": "heads_8191_layer", "op": "heads", "tokens": 8191, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 64, "axes": 2, "interleaved": False, "kind": "layer", "own_weights": True, "page_size": 64,
         "src": "f32", "dtype": "bf16", "far": 1000000},
        # one request far behind its window: latency
        {"name": "sinks_1x9000", "op": "sinks", "requests": 1, "new": 1, "max_len": 9000, "window": 1024, "sinks": 4,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "dtype": "bf16", "full": True, "freed": False},
        # the decode batch of 128 ragged contexts, the pages between sinks and window given back
        {"name": "sinks_128x32000", "op": "sinks", "requests": 128, "new": 1, "max_len": 32000, "window": 4096,
         "sinks": 16, "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "dtype": "bf16", "full": False,
         "freed": True},
        # float32 layers: drafted tokens, sinks over several tiles, pages of an odd size
        {"name": "sinks_f32_drafts", "op": "sinks", "requests": 16, "new": 4, "max_len": 2500, "window": 500,
         "sinks": 37, "heads": 12, "kv_heads": 4, "head_dim": 80, "page_size": 5, "dtype": "f32", "full": False,
         "freed": False},
        # four samples of one prompt: latency
        {"name": "shared_4x1000", "op": "shared", "groups": 1, "rows": 4, "new": 1, "prefix": 1000, "suffix": 60,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "dtype": "bf16", "full": True, "empty": 0.0},
        # the decode batch behind one long system prompt
        {"name": "shared_128x8192", "op": "shared", "groups": 1, "rows": 128, "new": 1, "prefix": 8192, "suffix": 512,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "dtype": "bf16", "full": False, "empty": 0.05},
        # the largest: eight documents with 64 questions each, drafted tokens among the rows
        {"name": "shared_8x64x32000", "op": "shared", "groups": 8, "rows": 64, "new": 2, "prefix": 32000,
         "suffix": 1500, "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 64, "dtype": "bf16", "full": False,
         "empty": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fork", "compact", "heads", "sinks", "shared", "shared"])
    ps, kv = rng.choice([1, 5, 16, 16, 32, 64, 100, 128]), rng.choice([1, 2, 4, 8])
    hd, dtype = 8 * rng.randint(2, 32), rng.choice(["bf16", "bf16", "f32"])
    row = 2 * kv * hd * _es(dtype)  # bytes of a position
    if op == "fork":
        beams = rng.choice([1, 2, 4, 5])
        requests = beams * _log(rng, 1, 1500 // beams)
        window = rng.choice([0, 0, _log(rng, 16, 3000)])
        return {"op": op, "requests": requests, "beams": beams,
                "max_len": _log(rng, 16, max(16, min(10000, (1 << 31) // (row * requests)))), "page_size": ps,
                "kv_heads": kv, "head_dim": hd, "dtype": dtype, "moved": rng.choice([0.1, 0.7]),
                "ended": rng.choice([0.0, 0.1]), "cut": rng.choice([0.0, 0.3]), "window": window,
                "sinks": rng.choice([0, rng.randint(1, 70)]) if window else 0, "short": rng.random() < 0.3}
    if op == "compact":
        requests = _log(rng, 1, 100)
        most = _log(rng, 16, max(16, min(20000, (1 << 30) // (row * requests))))
        return {"op": op, "requests": requests, "max_len": most,
                "tail": rng.choice([min(most, rng.randint(1, 64)), most]), "share": rng.choice([0.1, 0.5, 0.9]),
                "page_size": ps, "kv_heads": kv, "head_dim": hd, "dtype": dtype, "by_head": rng.random() < 0.3}
    if op == "heads":
        return {"op": op, "tokens": _log(rng, 1, 8000), "heads": kv * rng.randint(1, 6), "kv_heads": kv,
                "head_dim": hd, "rot_dim": rng.choice([hd, 2 * rng.randint(1, hd // 2)]), "axes": rng.randint(1, 4),
                "interleaved": rng.random() < 0.5, "kind": rng.choice(["rms", "rms", "layer"]),
                "own_weights": rng.random() < 0.3, "page_size": ps, "src": rng.choice(["f32", "f32", "bf16"]),
                "dtype": dtype, "far": _log(rng, 100, 1000000)}
    if op == "sinks":
        window, sinks, new = _log(rng, 8, 4096), _log(rng, 1, 200), rng.choice([1, 1, rng.randint(2, 5)])
        requests = _log(rng, 1, max(1, min(192, (1 << 31) // (row * (window + sinks) * new))))
        return {"op": op, "requests": requests, "new": new,
                "max_len": _log(rng, new, max(new, min(40000, (1 << 34) // (row * requests)))), "window": window,
                "sinks": sinks, "heads": kv * rng.randint(1, 20), "kv_heads": kv, "head_dim": hd, "page_size": ps,
                "dtype": dtype, "full": rng.random() < 0.3, "freed": rng.random() < 0.5}
    groups = _log(rng, 1, 12)
    rows, new = _log(rng, 1, 1000 // groups), rng.choice([1, 1, rng.randint(2, 4)])
    heads = kv * rng.randint(1, 12)
    # in all no more products, and no more scores, than the largest case has
    room = min(4 * 10 ** 11 // (4 * hd * (1 if dtype == "bf16" else 16)), 10 ** 9) // (groups * rows * new * heads)
    return {"op": op, "groups": groups, "rows": rows, "new": new,
            "prefix": _log(rng, 1, max(1, min(32000, room, (1 << 31) // (row * groups)))),
            "suffix": _log(rng, new, max(new, min(2000, (1 << 31) // (row * groups * rows)))), "heads": heads,
            "kv_heads": kv, "head_dim": hd, "page_size": ps, "dtype": dtype, "full": rng.random() < 0.3,
            "empty": rng.choice([0.0, 0.1])}


# ---- what the caller has in hand ----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _chance(g, n, p):
    return torch.rand(n, generator=g, device="cuda") < p


def _cache(c, g, n_pages, by_head=False):
    Hk, ps, D = c["kv_heads"], c["page_size"], c["head_dim"]
    shape = (n_pages, Hk, ps, D) if by_head else (n_pages, ps, Hk, D)
    k, v = (torch.empty(shape, device="cuda", dtype=DT[c["dtype"]]).normal_(generator=g) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if by_head else (k, v)


def _fork_sizes(c):
    width = -(-c["max_len"] // c["page_size"]) + 1
    return width, c["requests"] * width + 64


def _prepare_fork(c, g):
    R, ps, B = c["requests"], c["page_size"], c["beams"]
    P, n_pages = _fork_sizes(c)
    r = torch.arange(R, device="cuda")
    # beams of one prompt share the whole pages of a common part
    length = _lengths(g, R, 0, c["max_len"])
    first = r // B * B
    common = torch.minimum((length[first] * torch.rand(R, generator=g, device="cuda")[first]).long(),
                           length.view(-1, B).amin(1)[r // B]) // ps
    held = (length + ps - 1) // ps
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    col = torch.arange(P, device="cuda")
    lead = torch.where((col[None] < common[:, None]), first[:, None], r[:, None])
    table = torch.where(col[None] < held[:, None], pages[lead * P + col[None]], -1)
    used = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    used[table[table >= 0]] = True
    free = pages[~used[pages]]
    n_free = min(free.shape[0], 5) if c["short"] else free.shape[0]
    head = int(_lengths(g, 1, 0, n_pages)[0]) + 5 * n_pages
    ring = torch.full((n_pages,), -1, dtype=torch.int64, device="cuda")
    ring[(head + torch.arange(n_free, device="cuda")) % n_pages] = free[:n_free]
    parent = torch.where(_chance(g, R, c["moved"]), first + _lengths(g, R, 0, B - 1), r)
    parent = torch.where(_chance(g, R, c["ended"]), -1, parent)
    keep = torch.where(_chance(g, R, c["cut"]), length[parent.clamp(min=0)] - _lengths(g, R, 0, 8), c["max_len"])
    k, v = _cache(c, g, n_pages)
    st = {"len": length.int(), "parent": parent.int(), "keep": keep.clamp(min=0).int(), "table": table.int(),
          "ring": ring.int(), "cursor": torch.tensor([head, head + n_free], device="cuda"), "k": k, "v": v}
    if own:
        from lora_normal_form_amd import block
        st["cache"] = block.KVCache(k, v)
        st["fork"] = block.Fork(R, P, n_pages, device=k.device)
    return st


def _prepare_compact(c, g):
    R, ps, L = c["requests"], c["page_size"], c["max_len"]
    P = -(-L // ps)
    n_pages = R * P + 3
    length = _lengths(g, R, L // 2, L)
    start = (length - c["tail"]).clamp(min=0)
    # the places that stay: any of the tail's, in order
    W = c["tail"]
    stay = _chance(g, (R, W), c["share"]) & (start[:, None] + torch.arange(W, device="cuda") < length[:, None])
    n_kept = stay.sum(1)
    order = torch.argsort((~stay).int(), dim=1, stable=True)
    kept = torch.where(torch.arange(W, device="cuda") < n_kept[:, None], start[:, None] + order, -1)
    table = torch.randperm(n_pages, generator=g, device="cuda")[:R * P].view(R, P)
    k, v = _cache(c, g, n_pages, c["by_head"])
    # the free pages' ring is empty at first; its cursor has come some way
    st = {"len": length.int(), "start": start.int(), "kept": kept.int().contiguous(), "n_kept": n_kept.int(),
          "table": table.int().contiguous(), "ring": torch.full((n_pages,), -1, dtype=torch.int32, device="cuda"),
          "cursor": torch.full((2,), 7 * n_pages + 5, dtype=torch.int64, device="cuda"), "k": k, "v": v,
          "parent": torch.arange(R, device="cuda", dtype=torch.int32)}
    if own:
        from lora_normal_form_amd import block
        st["cache"] = block.KVCache(k, v)
        st["fork"] = block.Fork(R, P, n_pages, device=k.device)
        st["new_len"] = torch.empty(R, dtype=torch.int32, device="cuda")
    return st


def _sections(c):
    """Axis of each rotary pair: contiguous sections, one an axis."""
    n = c["rot_dim"] // 2
    return [min(c["axes"] - 1, i * c["axes"] // max(1, n)) for i in range(n)]


EPS = 1e-6


def _prepare_heads(c, g):
    T, D, Hq, Hk, ps = c["tokens"], c["head_dim"], c["heads"], c["kv_heads"], c["page_size"]
    y = (2.0 * torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device="cuda") + 0.3).to(DT[c["src"]])
    n = c["rot_dim"] // 2
    freq = 500000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / max(1, n))
    axis = torch.tensor(_sections(c), device="cuda", dtype=torch.int32)
    pos = torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
    n_pages = -(-(T + 2) // ps) + 3
    slot = torch.randperm(n_pages * ps, generator=g, device="cuda")[:T]
    slot = torch.where(_chance(g, T, 0.01), -1, slot)
    k, v = _cache(c, g, n_pages)

    def vec(heads, mean):
        shape = (heads, D) if c["own_weights"] else (D,)
        return mean + 0.2 * torch.randn(shape, generator=g, device="cuda")

    st = {"y": y, "freq": freq, "axis": axis, "pos": pos, "slot": slot, "k": k, "v": v, "q_w": vec(Hq, 1.0),
          "k_w": vec(Hk, 1.0), "q_b": vec(Hq, 0.0) if c["kind"] == "layer" else None,
          "k_b": vec(Hk, 0.0) if c["kind"] == "layer" else None}
    if own:
        from lora_normal_form_amd import block
        st["cache"] = block.KVCache(k, v)
        st["rotary"] = block.Rotary(freq, D, axis=axis, n_axes=c["axes"], interleaved=c["interleaved"])
        st["norm"] = block.HeadNorm(D, c["kind"], st["q_w"], st["k_w"], st["q_b"], st["k_b"], eps=EPS)
        st["q_out"] = torch.empty((T, Hq, D), device="cuda", dtype=DT[c["dtype"]])
    return st


def _prepare_sinks(c, g):
    R, new, L, ps = c["requests"], c["new"], c["max_len"], c["page_size"]
    total = torch.full((R,), L, device="cuda", dtype=torch.int64) if c["full"] else _lengths(g, R, 0, L)
    P = -(-L // ps)
    col = torch.arange(P, device="cuda")
    if c["freed"]:  # no page lies wholly between the sinks and the first row's window
        low = (total - (new - 1)).clamp(min=0)[:, None] - c["window"]
        held = (col * ps < total[:, None]) & ((col * ps < c["sinks"]) | ((col + 1) * ps > low))
        n_pages = R * min(P, -(-(c["window"] + new) // ps) + -(-c["sinks"] // ps) + 3) + 1
    else:
        held = (col * ps < total[:, None])
        n_pages = R * P + 1
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    at = torch.cumsum(held.view(-1).long(), 0).view(R, P) - 1
    table = torch.where(held, pages[at.clamp(min=0, max=n_pages - 1)], -1).int()
    k, v = _cache(c, g, n_pages)
    q = torch.randn((R * new, c["heads"], c["head_dim"]), generator=g, device="cuda").to(DT[c["dtype"]])
    back = torch.arange(new - 1, -1, -1, device="cuda")
    row_len = (total[:, None] - back[None]).clamp(min=0).reshape(-1).int()
    row_req = torch.arange(R, device="cuda").repeat_interleave(new).int()
    st = {"k": k, "v": v, "q": q, "table": table, "row_len": row_len, "row_req": row_req}
    if own:
        from lora_normal_form_amd import block
        st["attention"] = block.PagedAttention(block.KVCache(k, v), c["heads"], R * new, window=c["window"],
                                               sinks=c["sinks"])
        st["out"] = torch.empty_like(q)
    return st


def _prepare_shared(c, g):
    G, B, new, ps = c["groups"], c["rows"], c["new"], c["page_size"]
    R = G * B
    prefix = torch.full((G,), c["prefix"], device="cuda", dtype=torch.int64) if c["full"] else \
        _lengths(g, G, c["prefix"] // 2, c["prefix"])
    prefix = prefix // ps * ps  # requests fork at whole pages
    own_len = torch.full((R,), c["suffix"], device="cuda", dtype=torch.int64) if c["full"] else \
        _lengths(g, R, min(new, c["suffix"]), c["suffix"])
    total = prefix.repeat_interleave(B) + own_len
    total = torch.where(_chance(g, R, c["empty"]), 0, total)
    Pp, Ps = -(-c["prefix"] // ps), -(-c["suffix"] // ps) + 1
    P = Pp + Ps
    n_pages = G * Pp + R * Ps + 1
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    col = torch.arange(P, device="cuda")
    r = torch.arange(R, device="cuda")
    pp = (prefix // ps).repeat_interleave(B)[:, None]
    mine = pages[(G * Pp + r[:, None] * Ps + (col - pp).clamp(min=0, max=Ps - 1))]
    table = torch.where(col < pp, pages[(r // B)[:, None] * Pp + col.clamp(max=Pp - 1)], mine)
    table = torch.where(col - pp < Ps, table, -1).int()
    k, v = _cache(c, g, n_pages)
    q = torch.randn((R * new, c["heads"], c["head_dim"]), generator=g, device="cuda").to(DT[c["dtype"]])
    back = torch.arange(new - 1, -1, -1, device="cuda")
    row_len = (total[:, None] - back[None]).clamp(min=0).reshape(-1).int()
    st = {"k": k, "v": v, "q": q, "table": table, "row_len": row_len,
          "row_req": r.repeat_interleave(new).int(), "shared_len": prefix.int(),
          "group": (torch.arange(G + 1, device="cuda") * B * new).int()}
    if own:
        from lora_normal_form_amd import block
        st["attention"] = block.SharedAttention(block.KVCache(k, v), c["heads"], R * new, G)
        st["out"] = torch.empty_like(q)
    return st


PREPARE = {"fork": _prepare_fork, "compact": _prepare_compact, "heads": _prepare_heads, "sinks": _prepare_sinks,
           "shared": _prepare_shared}


def prepare(case, seed):
    st = PREPARE[case["op"]](case, _gen(seed))
    st["case"] = case
    return st


# ---- one pass ------------------------------------------------------------------------------------

def _forked(length, parent, keep, table, ring, cursor, ps, n_pages, window=0, sinks=0):
    """The new table, lengths, ring, cursor, counts and pages to copy."""
    R, P = table.shape
    cap = ring.shape[0]
    p = parent.long()
    lives = (p >= 0) & (p < R)
    src = p.clamp(min=0, max=R - 1)
    held_len = length.long().clamp(min=0, max=P * ps)
    n = torch.where(lives, torch.minimum(held_len[src], keep.long().clamp(min=0)), 0)
    col = torch.arange(P, device=table.device)
    whole, part = n // ps, n % ps
    t = table.long()
    inside = (t >= 0) & (t < n_pages)
    entry = torch.where((col < ((n + ps - 1) // ps)[:, None]) & inside[src], t[src], -1)
    if window:
        entry = torch.where((col * ps >= sinks) & ((col + 1) * ps <= n[:, None] - window), -1, entry)
    full = torch.zeros(n_pages + 1, dtype=torch.bool, device=t.device)
    before = torch.zeros_like(full)
    is_full = (col < whole[:, None]) & (entry >= 0)
    full[torch.where(is_full, entry, n_pages).view(-1)] = True
    had = inside & (col < ((held_len + ps - 1) // ps)[:, None])
    before[torch.where(had, t, n_pages).view(-1)] = True
    last = entry.gather(1, whole.clamp(max=P - 1)[:, None])[:, 0]
    last = torch.where(part > 0, last, -1)
    at = torch.where(last >= 0, last, n_pages)
    r = torch.arange(R, device=t.device)
    keeper = torch.full((n_pages + 1,), R, device=t.device).scatter_reduce(0, at, r, "amin")
    wants = (last >= 0) & (full[at] | (keeper[at] != r))
    need = torch.cumsum(wants.long(), 0)
    head, tail = cursor[0], cursor[1]
    avail = (tail - head).clamp(min=0, max=cap)
    gets = wants & (need <= avail)
    refused = wants & ~gets
    fresh = ring.long()[(head + need - 1) % cap]
    new_last = torch.where(gets, fresh, torch.where(refused, -1, last))
    entry = torch.where((col == whole[:, None]) & (part > 0)[:, None], new_last[:, None], entry)
    keeper[n_pages] = R
    gone = before[:n_pages] & ~full[:n_pages] & (keeper[:n_pages] == R)
    rank = torch.cumsum(gone.long(), 0) - 1
    n_gone, taken = gone.long().sum(), gets.long().sum()
    to = torch.where(gone & (rank < cap), (tail + rank) % cap, cap)
    ring_out = torch.cat([ring, ring[:1]]).index_put((to,), torch.arange(n_pages, device=t.device).int())[:cap]
    seq = torch.where(refused, whole * ps, n)
    counts = torch.stack([(seq > 0).long().sum(), taken, refused.long().sum(), n_gone])
    return {"table": entry.int(), "ring": ring_out, "cursor": torch.stack([head + taken, tail + n_gone]),
            "seq_len": seq.int(), "counts": counts.int(), "src": torch.where(gets, last, -1).int(),
            "dst": torch.where(gets, fresh, -1).int(), "n": torch.where(gets, part, 0).int()}


def _run_fork(st):
    c, table, ring, cursor = st["case"], st["table"], st["ring"], st["cursor"]
    if own:
        from lora_normal_form_amd import block
        f = block.fork_pages(st["len"], st["parent"], table, ring, cursor, c["page_size"], st["fork"],
                             keep=st["keep"], window=c["window"], sinks=c["sinks"])
        block.copy_pages(st["cache"], f.src, f.dst, f.n)
        return {"table": f.table, "ring": ring, "cursor": f.cursor, "seq_len": f.seq_len, "counts": f.counts,
                "src": f.src, "dst": f.dst, "n": f.n, "k": st["k"], "v": st["v"]}
    k, v = st["k"], st["v"]
    f = _forked(st["len"], st["parent"], st["keep"], table, ring, cursor, c["page_size"], k.shape[0], c["window"],
                c["sinks"])
    ring.copy_(f["ring"])
    # requests without a copy rewrite what the first one with a copy does
    some = f["dst"] >= 0
    first = torch.argmax(some.int())
    pick = torch.where(some, torch.arange(len(some), device="cuda"), first)
    src, dst = f["src"].long()[pick].clamp(min=0), f["dst"].long()[pick].clamp(min=0)
    upto = (torch.arange(c["page_size"], device="cuda") < f["n"].long()[pick][:, None])[:, :, None, None]
    for z in (k, v):
        z[dst] = torch.where(upto, z[src], z[dst])
    return dict(f, ring=ring, k=k, v=v)


def _run_compact(st):
    c, ps, table = st["case"], st["case"]["page_size"], st["table"]
    if own:
        from lora_normal_form_amd import block
        block.compact(st["cache"], table, st["start"], st["kept"], st["n_kept"], new_len=st["new_len"])
        f = block.fork_pages(st["len"], st["parent"], table, st["ring"], st["cursor"], ps, st["fork"],
                             keep=st["new_len"])
        return {"table": f.table, "ring": st["ring"], "cursor": f.cursor, "seq_len": f.seq_len, "counts": f.counts,
                "k": st["k"], "v": st["v"]}
    start, kept, t = st["start"].long(), st["kept"].long(), table.long()
    W = kept.shape[1]
    j = torch.arange(W, device="cuda")
    to = start[:, None] + j
    live = (j < st["n_kept"][:, None]) & (kept >= to)
    last = table.shape[1] * ps - 1
    kept, to = kept.clamp(min=0, max=last), to.clamp(max=last)
    s_at = (t.gather(1, kept // ps) * ps + kept % ps)[live]
    d_at = (t.gather(1, to // ps) * ps + to % ps)[live]
    for z in (st["k"], st["v"]):
        rows = z[s_at // ps, s_at % ps]
        z[d_at // ps, d_at % ps] = rows
    new_len = (start + st["n_kept"]).int()
    f = _forked(st["len"], st["parent"], new_len, table, st["ring"], st["cursor"], ps, st["k"].shape[0])
    st["ring"].copy_(f["ring"])
    return {"table": f["table"], "ring": st["ring"], "cursor": f["cursor"], "seq_len": f["seq_len"],
            "counts": f["counts"], "k": st["k"], "v": st["v"]}


def _split(y, c):
    T, D, Hq, Hk = y.shape[0], c["head_dim"], c["heads"], c["kv_heads"]
    return (y[:, :Hq * D].view(T, Hq, D), y[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D),
            y[:, (Hq + Hk) * D:].view(T, Hk, D))


def _normed(z, kind, w, b):
    z = z.float()
    if kind == "layer":
        z = z - z.mean(-1, keepdim=True)
    z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * w
    return z if b is None else z + b


def _turned(z, cos, sin, c):
    """z [T][H][D] with its pairs rotated."""
    n = c["rot_dim"] // 2
    i = torch.arange(n, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + n)
    a, b = z[..., ia], z[..., ib]
    out = z.clone()
    out[..., ia] = a * cos[:, None] - b * sin[:, None]
    out[..., ib] = a * sin[:, None] + b * cos[:, None]
    return out


def _run_heads(st):
    c = st["case"]
    q, k, v = _split(st["y"], c)
    if own:
        st["rotary"].store(q, k, v, st["pos"], st["slot"], st["cache"], st["q_out"], norm=st["norm"])
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    angle = st["pos"].double()[st["axis"].long()].T * st["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dt = st["k"].dtype
    kc, vc = st["k"].flatten(0, 1), st["v"].flatten(0, 1)
    # tokens without a slot rewrite the row that the first one with a slot gets
    some = st["slot"] >= 0
    src = torch.where(some, torch.arange(len(some), device="cuda"), torch.argmax(some.int()))
    to = st["slot"][src]
    live = (to >= 0)[:, None, None]
    at = to.clamp(min=0)
    k1 = _turned(_normed(k, c["kind"], st["k_w"], st["k_b"]), cos, sin, c).to(dt)
    kc[at] = torch.where(live, k1[src], kc[at])
    vc[at] = torch.where(live, v.to(dt)[src], vc[at])
    return {"q": _turned(_normed(q, c["kind"], st["q_w"], st["q_b"]), cos, sin, c).to(dt), "k": st["k"], "v": st["v"]}


def _softmax_parts(s):
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-37)


def _run_sinks(st):
    c = st["case"]
    if own:
        return st["attention"].forward(st["q"], st["table"], st["row_len"], st["out"],
                                       row_req=None if c["new"] == 1 else st["row_req"])
    q, table, new, ps = st["q"], st["table"].long(), c["new"], c["page_size"]
    N, Hq, D = q.shape
    Hk = c["kv_heads"]
    n = st["row_len"].long().view(-1, new)
    # the first tokens, and the positions that some row's window holds
    S, W, L = min(c["sinks"], c["max_len"]), min(c["window"] + new - 1, c["max_len"]), c["max_len"]
    low = (n[:, -1:] - W).clamp(min=0)
    t = torch.cat([torch.arange(S, device=q.device).expand(n.shape[0], S),
                   low + torch.arange(W, device=q.device)], 1)
    first = torch.cat([torch.ones_like(t[:, :S], dtype=torch.bool), t[:, S:] >= S], 1)  # (each position once)
    tc = t.clamp(max=L - 1)
    page = table.gather(1, tc // ps)
    there = first & (page >= 0)
    page = page.clamp(min=0)
    nr = n[:, :, None]
    seen = there[:, None] & (t[:, None] < nr) & ((t[:, None] >= nr - c["window"]) | (t[:, None] < S))
    K = st["k"][page, tc % ps].permute(0, 2, 3, 1).float()
    s = torch.matmul(q.float().view(-1, new, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).flatten(2, 3), K)
    del K
    s = s.view(s.shape[0], Hk, new, Hq // Hk, S + W) * (1.0 / math.sqrt(D))
    p = _softmax_parts(torch.where(seen[:, None, :, None], s, float("-inf")))
    V = st["v"][page, tc % ps].permute(0, 2, 1, 3).float()
    o = torch.matmul(p.flatten(2, 3), V).view(-1, Hk, new, Hq // Hk, D)
    return o.permute(0, 2, 1, 3, 4).reshape(N, Hq, D).to(q.dtype)


def _run_shared(st):
    c = st["case"]
    if own:
        return st["attention"].forward(st["q"], st["table"], st["row_len"], st["group"], st["shared_len"], st["out"],
                                       row_req=None if c["new"] == 1 else st["row_req"])
    q, table, new, ps = st["q"], st["table"].long(), c["new"], c["page_size"]
    N, Hq, D = q.shape
    Hk, G, B = c["kv_heads"], c["groups"], c["rows"]
    n, prefix = st["row_len"].long(), st["shared_len"].long()
    X, Y = c["prefix"], c["suffix"]
    # the prefix, once for all rows of a group
    t = torch.arange(X, device=q.device)
    page = table[::B][:, t // ps].clamp(min=0)
    K = st["k"][page, t % ps].permute(0, 2, 3, 1).float()  # [G][Hk][D][X]
    qg = q.float().view(G, B * new, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(qg, K).view(G, Hk, B * new, Hq // Hk, X)
    del K
    s = s.permute(0, 2, 1, 3, 4).reshape(N, Hk, Hq // Hk, X)
    seen_x = (t < prefix.repeat_interleave(B * new)[:, None]) & (t < n[:, None])
    # what each request has of its own
    own_t = prefix.repeat_interleave(B)[:, None] + torch.arange(Y, device=q.device)
    page_y = table.gather(1, (own_t // ps).clamp(max=table.shape[1] - 1)).clamp(min=0)
    K = st["k"][page_y, own_t % ps].permute(0, 2, 3, 1).float()  # [R][Hk][D][Y]
    sy = torch.matmul(q.float().view(-1, new, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).flatten(2, 3), K)
    del K
    sy = sy.view(-1, Hk, new, Hq // Hk, Y).permute(0, 2, 1, 3, 4).reshape(N, Hk, Hq // Hk, Y)
    seen_y = own_t.repeat_interleave(new, 0) < n[:, None]
    s = torch.where(seen_x[:, None, None], s, float("-inf"))
    sy = torch.where(seen_y[:, None, None], sy, float("-inf"))
    p = _softmax_parts(torch.cat([s, sy], -1) * (1.0 / math.sqrt(D)))
    del s, sy
    V = st["v"][page, t % ps].permute(0, 2, 1, 3).float()
    px = p[..., :X].view(G, B * new, Hk, Hq // Hk, X).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o = torch.matmul(px, V).view(G, Hk, B * new, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(N, Hq, D)
    del px, V
    V = st["v"][page_y, own_t % ps].permute(0, 2, 1, 3).float()
    py = p[..., X:].reshape(-1, new, Hk, Hq // Hk, Y).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o = o + torch.matmul(py, V).view(-1, Hk, new, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(N, Hq, D)
    return o.to(q.dtype)


RUN = {"fork": _run_fork, "compact": _run_compact, "heads": _run_heads, "sinks": _run_sinks, "shared": _run_shared}


def run(state):
    return RUN[state["case"]["op"]](state)


# ---- what a pass has to move and compute --------------------------------------------------------

def work(case):
    c = case
    row = 2 * c["kv_heads"] * c["head_dim"] * _es(c["dtype"])  # bytes of a position
    if c["op"] == "fork":
        R, ps = c["requests"], c["page_size"]
        P, n_pages = _fork_sizes(c)
        copies = min(5, c["moved"] * R / 2) if c["short"] else c["moved"] * R * (1 - 1 / c["beams"]) / 2
        moved = copies * (ps - 1) / 2 * row * 2
        return {"bytes": 4 * R * c["max_len"] / 2 / ps + 4 * R * P + 28 * R + moved, "flops": 0}
    if c["op"] == "compact":
        held = 0.75 * c["max_len"]
        kept = c["requests"] * min(c["tail"], held) * c["share"]
        return {"bytes": kept * (2 * row + 4) + 8 * c["requests"] * held / c["page_size"] + 24 * c["requests"], "flops": 0}
    if c["op"] == "heads":
        n = c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["head_dim"]
        turned = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["head_dim"]
        return {"bytes": n * (_es(c["src"]) + _es(c["dtype"])) + c["tokens"] * (4 * c["axes"] + 8) + 6 * c["rot_dim"]
                + 8 * c["head_dim"] * (c["heads"] + c["kv_heads"] if c["own_weights"] else 2), "flops": 8 * turned}
    rows, es = 0, _es(c["dtype"])
    if c["op"] == "sinks":
        rows, L = c["requests"] * c["new"], c["max_len"]
        span = min(L, c["window"] + c["sinks"])
        # lengths are even over 0 .. L (or all L): what a request sees of them
        seen = span if c["full"] else span - span * span / (2 * L)
        read = (seen + c["new"] - 1) * c["requests"]
    else:
        rows = c["groups"] * c["rows"] * c["new"]
        share = 1.0 if c["full"] else 0.75
        x, y = c["prefix"] * share, c["suffix"] * (1.0 if c["full"] else 0.5)
        live = 1 - c["empty"]
        read, seen = c["groups"] * x + c["groups"] * c["rows"] * y * live, (x + y) * live
    return {"bytes": read * row + 4 * read / c["page_size"] + 2 * rows * c["heads"] * c["head_dim"] * es + 4 * rows,
            "flops": 4 * rows * seen * c["heads"] * c["head_dim"]}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _copied(z, st, c, moves):
    """z in 64 bits with the rows moved: moves are (from page, place, to page, place)."""
    out = z.double()
    if moves:
        m = torch.tensor(moves, device=z.device).T
        out[m[2], m[3]] = z[m[0], m[1]].double()
    return out


def _exact_fork(c, st):
    """The pages to copy, request by request (whole numbers need no exact value)."""
    ps, R = c["page_size"], c["requests"]
    length, parent, keep = st["len"].tolist(), st["parent"].tolist(), st["keep"].tolist()
    table, ring = st["table"].tolist(), st["ring"].tolist()
    head, tail = st["cursor"].tolist()
    full, partial = set(), {}
    for r in range(R):
        n = min(length[parent[r]], keep[r]) if parent[r] >= 0 else 0
        t = table[parent[r]]
        for i in range(n // ps):
            if c["window"] and i * ps >= c["sinks"] and (i + 1) * ps <= n - c["window"]:
                continue
            full.add(t[i])
        if n % ps:
            partial.setdefault(t[n // ps], []).append((r, n % ps))
    wants = sorted((r, page, n) for page, who in partial.items()
                   for i, (r, n) in enumerate(sorted(who)) if i > 0 or page in full)
    moves = []
    for (r, page, n), place in zip(wants, range(head, tail)):
        moves += [(page, i, ring[place % len(ring)], i) for i in range(n)]
    return {"table": None, "ring": None, "cursor": None, "seq_len": None, "counts": None, "src": None, "dst": None,
            "n": None, "k": _copied(st["k"], st, c, moves), "v": _copied(st["v"], st, c, moves)}


def _exact_compact(c, st):
    ps = c["page_size"]
    k, v = st["k"].double(), st["v"].double()
    for r, (a, n) in enumerate(zip(st["start"].tolist(), st["n_kept"].tolist())):
        t = st["table"][r].long()
        src, dst = st["kept"][r, :n].long(), a + torch.arange(n, device="cuda")
        for z, was in ((k, st["k"]), (v, st["v"])):
            z[t[dst // ps], dst % ps] = was[t[src // ps], src % ps].double()
    return {"table": None, "ring": None, "cursor": None, "seq_len": None, "counts": None, "k": k, "v": v}


def _exact_heads(c, st):
    y = st["y"].double()
    q, k, v = (t.clone() for t in _split(y, c))
    for z, w, b in ((q, st["q_w"], st["q_b"]), (k, st["k_w"], st["k_b"])):
        if c["kind"] == "layer":
            z -= z.sum(-1, keepdim=True) / c["head_dim"]
        z /= (z.square().sum(-1, keepdim=True) / c["head_dim"] + EPS).sqrt()
        z *= w.double()
        if b is not None:
            z += b.double()
    n = c["rot_dim"] // 2
    for i, ax in enumerate(_sections(c)):
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


def _exact_rows(c, st, seen):
    """Attention row by row over the positions that seen(length) lists."""
    ps, Hk, G = c["page_size"], c["kv_heads"], c["heads"] // c["kv_heads"]
    out = torch.zeros_like(st["q"], dtype=torch.float64)
    table = st["table"].long()
    for i, n in enumerate(st["row_len"].tolist()):
        if n <= 0:
            continue
        t = seen(n)
        pages = table[i // c["new"], t // ps]
        K = st["k"][pages, t % ps].double().transpose(0, 1).contiguous()
        V = st["v"][pages, t % ps].double().transpose(0, 1).contiguous()
        q = st["q"][i].double().view(Hk, G, -1)
        p = torch.softmax(torch.bmm(q, K.transpose(1, 2).contiguous()) / math.sqrt(q.shape[-1]), -1)
        out[i] = torch.bmm(p, V).view(c["heads"], -1)
    return out


def _exact_sinks(c, st):
    def seen(n):
        t = torch.arange(n, device="cuda")
        return t[(t >= n - c["window"]) | (t < c["sinks"])]

    return _exact_rows(c, st, seen)


def _exact_shared(c, st):
    return _exact_rows(c, st, lambda n: torch.arange(n, device="cuda"))


EXACT = {"fork": _exact_fork, "compact": _exact_compact, "heads": _exact_heads, "sinks": _exact_sinks,
         "shared": _exact_shared}


def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))

"""Multi-projection layers built on the single-layer library: the attention
input projections q, k, v, and the FFN's gated up projection.

"How does Scute plug into vLLM?" (paper-daily.com explainer of "Scute:
Exact Batched Serving for PEFT Adapters Beyond LoRA"): the base GEMM is split
into q, k and v when OFT is present, because each projection has its own
rotation of the input; otherwise q, k and v are one GEMM over the stacked
weights. "What problem is it solving?" and "The big picture": (IA)^3
multiplies the keys, the values and the FFN intermediate silu(x W_g) (.)
x W_u by learned vectors; the first two are s slots of the k and v
projections, the last (products reorder) the s slot of the up projection.

QKV, fused   one layer over W_qkv = [W_q; W_k; W_v] ([d_q + d_k + d_v][d_in]).
             Each tenant's per-projection slots, as the library folds them
             (read back with scute_read_slot), become one normal-form
             adapter: s and b concatenated (ones / zeros on projections the
             tenant leaves alone), one own term with the A' stacked and the
             B' block diagonal (its rank the sum of theirs), and, when the
             tenant rotates, one rotation per projection (the identity where
             it does not): the layer's projections are set to the q / k / v
             column ranges and the adapter loads with
             scute_load_adapter_proj, so OFT tenants keep the single GEMM.
             VeRA: each projection has its own shared pair, so the fused
             layer's pair is theirs side by side, A_sh stacked and B_sh
             block diagonal (its rank the sum of theirs), and a tenant's d
             and e are its projections' concatenated (d zero on projections
             without its VeRA term). Exact.
QKV, split   three layers and three forwards; any method.
FFN          a gate layer (base weight only) and the up layer with the
             tenants' adapters ((IA)^3's l on its s slot), then
             scute_silu_gate: h = silu(g) (.) u.
Attention    one step of a block's attention half around the fused QKV layer:
             norm, q / k / v, rotary positions and the paged cache, attention,
             the output projection (any method), residual and next norm.

    python -m lora_normal_form_amd.multiproj [--out PATH]   (timing on one GPU)
"""

from __future__ import annotations

import argparse
import dataclasses
import json
import statistics
import sys

import numpy as np

from . import convert, scute


# ---- workloads -----------------------------------------------------------------------------

def projection_workloads(tenants, n_tok, d_in, d_outs, seed, vera_rank=0, dtype="bf16",
                         none_frac=0.0):
    """One synthetic workload per projection sharing x and the tokens'
    tenants. tenants: list of per-projection AdapterSpec tuples (None: the
    tenant leaves that projection alone). Returns (workloads, tenant of each
    token (-1: none))."""
    from synth import WorkloadSpec, make_workload
    rng = np.random.default_rng(seed)
    tt = rng.integers(0, len(tenants), size=n_tok)
    tt[rng.random(n_tok) < none_frac] = -1
    wls, x = [], None
    for p, d_out in enumerate(d_outs):
        specs, ids = [], {}
        for t, per in enumerate(tenants):
            if per[p] is not None:
                ids[t] = len(specs)
                specs.append(per[p])
        ta = np.array([ids.get(int(t), -1) if t >= 0 else -1 for t in tt], dtype=np.int64)
        wl = make_workload(WorkloadSpec(f"proj{p}", dtype, d_in, d_out, n_tok, specs,
                                        vera_rank=vera_rank, assign="explicit", token_adapter=ta,
                                        seed=seed + 1 + p))
        if x is None:
            x = wl.x
        else:
            wl = dataclasses.replace(wl, x=x)
        wls.append((wl, ids))
    return wls, tt


# ---- QKV ---------------------------------------------------------------------------------------

class QKVSplit:
    """q, k and v as three layers (any method); forward returns the three outputs."""

    def __init__(self, wls, device=0, flags=0):
        from . import workload as glue
        self.parts = [glue.load(wl, device=device, flags=flags) for wl, _ in wls]

    def forward(self):
        for ld in self.parts:
            ld.layer.forward(ld.batch, ld.x, ld.W, ld.y)
        return [ld.y for ld in self.parts]

    def close(self):
        for ld in self.parts:
            ld.batch.close()
            ld.layer.close()


def fused_vera_pair(wls):
    """The fused layer's shared VeRA pair from the projections' pairs: A_sh
    [sum r][d_in] stacked, B_sh [sum d_out][sum r] block diagonal; with the
    projections' ranks. None when no projection has a pair."""
    ranks = [wl.vera_rank for wl, _ in wls]
    if not any(ranks):
        return None
    d_in, d_outs = wls[0][0].d_in, [wl.d_out for wl, _ in wls]
    A = np.zeros((sum(ranks), d_in))
    B = np.zeros((sum(d_outs), sum(ranks)))
    r0 = c0 = 0
    for (wl, _), r, d in zip(wls, ranks, d_outs):
        if r:
            A[r0:r0 + r] = wl.A_sh
            B[c0:c0 + d, r0:r0 + r] = wl.B_sh
        r0, c0 = r0 + r, c0 + d
    return A, B, ranks


def fused_slots(per_proj, d_outs, vera_ranks=None):
    """One normal-form adapter's arrays from a tenant's per-projection folded
    slots (None for a projection it leaves alone). "R_proj" is None when no
    projection rotates, else one rotation per projection (None: identity).
    vera_ranks: each projection's shared-pair rank (needed with a VeRA term)."""
    d_in = None
    for sl in per_proj:
        if sl is None:
            continue
        if sl["A"] is not None:
            d_in = sl["A"].shape[1]
    rot = [sl is not None and sl["R_minus_I"] is not None for sl in per_proj]
    blks = {sl["R_minus_I"].shape[1] for sl, r in zip(per_proj, rot) if r}
    if len(blks) > 1:
        raise ValueError("rotations of different block sizes need the split q / k / v layers")
    s = np.concatenate([sl["s"] if sl is not None and sl["s"] is not None else np.ones(d)
                        for sl, d in zip(per_proj, d_outs)])
    b = np.concatenate([sl["b"] if sl is not None and sl["b"] is not None else np.zeros(d)
                        for sl, d in zip(per_proj, d_outs)])
    has_s = any(sl is not None and sl["s"] is not None for sl in per_proj)
    has_b = any(sl is not None and sl["b"] is not None for sl in per_proj)
    terms = [(p, sl["A"], sl["B"]) for p, sl in enumerate(per_proj) if sl is not None and sl["A"] is not None]
    out = {"s": s if has_s else None, "b": b if has_b else None, "rank": 0, "A": None, "B": None,
           "R_proj": None, "blk": 0, "vd": None, "ve": None}
    has_v = [sl is not None and sl["vd"] is not None for sl in per_proj]
    if any(has_v):
        if vera_ranks is None:
            raise ValueError("a VeRA term needs the projections' shared-pair ranks")
        out["vd"] = np.concatenate([sl["vd"] if v else np.zeros(r)
                                    for sl, v, r in zip(per_proj, has_v, vera_ranks)])
        out["ve"] = np.concatenate([sl["ve"] if v else np.ones(d)
                                    for sl, v, d in zip(per_proj, has_v, d_outs)])
    if blks:
        blk = blks.pop()
        out["blk"] = blk
        out["R_proj"] = [np.eye(blk)[None] + sl["R_minus_I"] if r else None for sl, r in zip(per_proj, rot)]
    if terms:
        r = sum(A.shape[0] for _, A, _ in terms)
        A = np.zeros((r, d_in))
        B = np.zeros((sum(d_outs), r))
        k = 0
        offs = np.concatenate([[0], np.cumsum(d_outs)])
        for p, Ap, Bp in terms:
            A[k:k + Ap.shape[0]] = Ap
            B[offs[p]:offs[p + 1], k:k + Ap.shape[0]] = Bp
            k += Ap.shape[0]
        out.update(rank=r, A=A, B=B)
    return out


def fused_layer(wls, n_tenants, device=0):
    """The q / k / v layer over the stacked weights with every tenant's fused
    normal-form adapter loaded (device -1: a host-only layer)."""
    from . import workload as glue
    d_outs = [wl.d_out for wl, _ in wls]
    wl0 = wls[0][0]
    hosts = [glue.load(wl, device=-1, plan=False) for wl, _ in wls]
    layer = scute.Layer(wl0.d_in, sum(d_outs), wl0.dtype, max_adapters=max(1, n_tenants), device=device)
    pair = fused_vera_pair(wls)
    ranks = pair[2] if pair else None
    fused = []
    for t in range(n_tenants):
        per = [convert.slots(h.layer, ids[t], wl.d_in, wl.d_out, wl.vera_rank) if t in ids else None
               for (wl, ids), h in zip(wls, hosts)]
        fused.append(None if all(p is None for p in per) else fused_slots(per, d_outs, ranks))
    if pair is not None and any(f is not None and f["vd"] is not None for f in fused):
        if device >= 0:
            import torch
            dev = torch.device("cuda", device)
            A_f, B_f = glue.to_device(pair[0], wl0.dtype, dev), glue.to_device(pair[1], wl0.dtype, dev)
        else:  # (a host-only layer keeps the pointers without reading them)
            A_f, B_f = pair[0], pair[1]
        layer.set_vera_shared(A_f, B_f, sum(ranks))
    if any(f is not None and f["R_proj"] is not None for f in fused):
        if any(d % 64 for d in d_outs[:-1]):
            raise ValueError("rotations per projection need q and k widths that are multiples of 64")
        layer.set_projections(np.cumsum(d_outs))
    for t, f in enumerate(fused):
        if f is None:
            continue
        if f["R_proj"] is not None:
            layer.load_proj(t, f["R_proj"], f["blk"], rank=f["rank"], c=1.0, A=f["A"], B=f["B"], s=f["s"],
                            b=f["b"], vd=f["vd"], ve=f["ve"])
        else:
            layer.load(t, "nf", rank=f["rank"], c=1.0, A=f["A"], B=f["B"], s=f["s"], b=f["b"], vd=f["vd"],
                       ve=f["ve"])
    for h in hosts:
        h.layer.close()
    return layer


class QKVFused:
    """q, k and v as one layer over the stacked weights (any method: rotations
    per projection, the projections' VeRA pairs side by side); forward
    returns the three column slices."""

    def __init__(self, wls, tenant_of_token, n_tenants, device=0, flags=0):
        import torch
        from . import workload as glue
        self.d_outs = [wl.d_out for wl, _ in wls]
        wl0 = wls[0][0]
        self.layer = fused_layer(wls, n_tenants, device)
        dev = torch.device("cuda", device)
        W = np.concatenate([wl.W for wl, _ in wls], 0)
        self.x = glue.to_device(wl0.x, wl0.dtype, dev)
        self.W = glue.to_device(W, wl0.dtype, dev)
        self.y = torch.empty((wl0.n, sum(self.d_outs)), dtype=torch.float32, device=dev)
        self.batch = self.layer.plan(np.asarray(tenant_of_token), flags=flags)

    def forward(self):
        self.layer.forward(self.batch, self.x, self.W, self.y)
        offs = np.concatenate([[0], np.cumsum(self.d_outs)])
        return [self.y[:, offs[p]:offs[p + 1]] for p in range(len(self.d_outs))]

    def close(self):
        self.batch.close()
        self.layer.close()


# ---- FFN ---------------------------------------------------------------------------------------

class GatedUp:
    """h = silu(x W_g) (.) up(x): the gate projection (base weight only) and
    the up projection with the tenants' adapters ((IA)^3's l on s)."""

    def __init__(self, wl_up, W_gate, device=0):
        import torch
        from . import workload as glue
        self.up = glue.load(wl_up, device=device)
        gate_wl = dataclasses.replace(wl_up, name=wl_up.name + "_gate", W=W_gate, adapters=[],
                                      token_adapter=np.full(wl_up.n, -1), A_sh=None, B_sh=None)
        self.gate = glue.load(gate_wl, device=device)
        self.h = torch.empty_like(self.up.y)

    def forward(self):
        g, u = self.gate, self.up
        g.layer.forward(g.batch, g.x, g.W, g.y)
        u.layer.forward(u.batch, u.x, u.W, u.y)
        scute.scute_silu_gate(g.y, u.y, self.h)
        return self.h

    def close(self):
        for ld in (self.gate, self.up):
            ld.batch.close()
            ld.layer.close()


# ---- attention ---------------------------------------------------------------------------------

class AttentionStep:
    """One step of a decoder block's attention half for a batch of n rows:

        x = N_in(h);  q, k, v = the fused layer;  q and k rotated, k and v into
        the paged cache;  a = attention;  o = out(a)
        h' = h_scale h + y_scale (gate (.) N_post(o));  x' = N_out(h')

    qkv: a QKVFused over projections of n_heads, n_kv_heads and n_kv_heads
    heads of head_dim columns. wl_out: the output projection's workload (d_in
    n_heads head_dim, its own tenants), whose rows' inputs the attention
    writes. The rows are the requests' new tokens in the requests' order; rows past the last token, and those of
    a request that found no pages, go through the layers and are skipped by the
    cache and the attention. So is a request with tokens past the last row:
    it keeps its length and may bring them again.

    Whose adapters a row runs under: without `tenants` those that the two plans
    give row i in every step, which fits steps whose rows stay their requests'
    (one_each, or the same new lengths every time). tenants: int32 [2][n_requests]
    on the GPU, each request's adapter in the q / k / v layer and in the output
    projection (-1: none); every row then runs under its request's, whichever
    row it is, in layers that take the rows' adapters from the GPU
    (scute_layer_forward_noalloc: its sizes, its speed). `tenants` stays the
    step's, to be written where a request changes hands. A caller who knows the
    new lengths may plan a step's rows instead and hand the plans to forward.

    The step keeps the requests' lengths, pages and free pages on the GPU:
    table [n_requests][pages_per_request], ring (n_pages free pages at first),
    state (cursor and lengths, as in block.Rows). A forward moves them on by its
    last launch, so a captured forward is a new step whenever it is replayed.
    like: another step of the same sizes, whose cache, table, ring and state this
    one works on too: one with rows for prompts and a one_each step take turns.
    one_each: row i is request i's, with one token or, where the request brings
    none, ends or finds no page, empty (n is n_requests; more tokens are
    refused); the attention then streams the cache. freq (float64 [pairs]), axis, n_axes
    and interleaved as in block.Rotary; norm_in, norm_post, norm_out: float32
    weights [d] (norm_post None: no norm on o). head_norm: a block.HeadNorm of q's
    and k's heads before they are rotated. window, sinks: as in block.PagedAttention.

    groups > 0: rows whose contexts begin with the same pages read those
    positions once (block.SharedAttention, without a window): `group`
    [groups + 1] and `shared_len` [groups] say which, by row, zero at first and
    to be written by the caller. forks: requests may go on from others, be cut
    back or keep some of their positions (fork, keep_only); they then end by
    fork, and a negative new_len is a request without tokens. Steps with forks that
    share a cache (like) have one window and the same sinks."""

    head_norm = group = shared_len = None
    forks = False

    def __init__(self, qkv, wl_out, n_heads, n_kv_heads, head_dim, n_requests, pages_per_request, page_size,
                 n_pages, freq, axis=None, n_axes=1, interleaved=False, norm_in=None, norm_post=None, norm_out=None,
                 kind="rms", eps=1e-5, h_scale=1.0, y_scale=1.0, window=0, one_each=False, device=0,
                 tenants=None, like=None, head_norm=None, sinks=0, groups=0, forks=False):
        import torch
        from . import block
        from . import workload as glue
        if list(qkv.d_outs) != [n_heads * head_dim, n_kv_heads * head_dim, n_kv_heads * head_dim]:
            raise ValueError("the q / k / v projections must be n_heads, n_kv_heads and n_kv_heads heads wide")
        n, d = qkv.x.shape
        if wl_out.n != n or wl_out.d_in != n_heads * head_dim or wl_out.d_out != d:
            raise ValueError("the output projection must take the heads of every row back to the layer's width")
        if one_each and n != n_requests:
            raise ValueError("one_each needs a row for each request")
        dev, dt = qkv.x.device, qkv.x.dtype
        shape = (n_pages, page_size, n_kv_heads, head_dim)
        if like is not None and (like.cache.k.shape, like.table.shape, like.cache.dtype, like.cache.device) != (
                shape, (n_requests, pages_per_request), dt, dev):
            raise ValueError("like: a step whose requests, pages, heads, type or device are others")
        if like is not None and like.forks != bool(forks):
            raise ValueError("like: requests end by fork in both steps or in none")
        if like is not None and forks and (like.window, like.window and like.sinks) != (window, window and sinks):
            raise ValueError("like: forks give back pages behind the window, which has to be the same in both steps")
        if groups and (window or sinks):
            raise ValueError("groups: rows that share positions see all of theirs, without a window")
        if tenants is not None and (tenants.dtype != torch.int32 or tenants.shape != (2, n_requests)):
            raise ValueError("tenants must be int32 [2][n_requests]")
        self.qkv, self.out = qkv, glue.load(wl_out, device=device)
        self.one_each = one_each
        q, k, v = (qkv.y[:, a:b] for a, b in zip((0, *np.cumsum(qkv.d_outs)), np.cumsum(qkv.d_outs)))
        self.q, self.k, self.v = (t.unflatten(1, (-1, head_dim)) for t in (q, k, v))
        self.rows = block.Rows(n_requests, n, dev)
        if like is None:
            self.cache = block.KVCache(torch.zeros(shape, dtype=dt, device=dev), torch.zeros(shape, dtype=dt, device=dev))
            self.table = torch.zeros((n_requests, pages_per_request), dtype=torch.int32, device=dev)
            self.ring = torch.arange(n_pages, dtype=torch.int32, device=dev)
            self.rows.cursor.copy_(torch.tensor([0, n_pages]))
            self.state = self.rows.state.clone()
        else:
            self.cache, self.table, self.ring, self.state = like.cache, like.table, like.ring, like.state
            self.rows.state.copy_(self.state)
        self.rotary = block.Rotary(freq, head_dim, axis=axis, n_axes=n_axes, interleaved=interleaved)
        self.head_norm, self.window, self.sinks = head_norm, window, sinks
        if groups:
            self.attention = block.SharedAttention(self.cache, n_heads, n, groups)
            self.group = torch.zeros(groups + 1, dtype=torch.int32, device=dev)
            self.shared_len = torch.zeros(groups, dtype=torch.int32, device=dev)
        else:
            self.attention = block.PagedAttention(self.cache, n_heads, window=window, sinks=sinks)
        self.forks = bool(forks)
        if forks:
            self._fork = block.Fork(n_requests, pages_per_request, n_pages, dev)
            self._new_len, self._keep = (torch.zeros(n_requests, dtype=torch.int32, device=dev) for _ in range(2))
            self._same = torch.arange(n_requests, dtype=torch.int32, device=dev)
        self.norm_in = block.ResidualNorm(d, kind, pre_weight=norm_in, eps=eps, device=dev)
        self.norm_out = block.ResidualNorm(d, kind, post=norm_post is not None, post_weight=norm_post,
                                           pre_weight=norm_out, h_scale=h_scale, y_scale=y_scale, eps=eps, device=dev)
        # (column 0: rows of no request)
        self._ids = torch.full((2, n_requests + 1), -1, dtype=torch.int32, device=dev)
        self.tenants = None if tenants is None else self._ids[:, 1:].copy_(tenants)
        self._column, self._row_ids = (torch.empty(s, dtype=torch.int32, device=dev) for s in ((n,), (2, n)))
        self.q_rot = torch.empty((n, n_heads, head_dim), dtype=dt, device=dev)
        self.a = self.out.x.view(n, n_heads, head_dim)
        block.settle(dev)

    def forward(self, h, new_len, h_out, x_out, pos=None, gate=None, plans=None):
        """h [n][d] the residual stream; new_len int32 [n_requests] on the GPU
        (negative: the request ends); pos int32 [n_axes][n] (None: every axis
        at the token's position); plans: this step's (q / k / v plan, output
        projection plan) in place of the step's own, each of n rows (of
        self.qkv.layer and self.out.layer; the caller keeps them until the
        stream has run the step, a graph's as long as the graph). Writes and
        returns (h_out, x_out); self.rows holds the step's rows (block.Rows).
        Runs on torch's current stream of the tensors' device, the layers too."""
        import torch
        from . import block
        rows, s = self.rows, block.current_stream(self.cache.index)
        if plans is not None and [p.info()["n"] for p in plans] != 2 * [rows.max_tokens]:
            raise ValueError(f"plans must be two plans of {rows.max_tokens} rows")
        cursor, seq_len = block.split_state(self.state, rows.n_requests)
        if self.forks:
            block._vector(new_len, rows.n_requests, torch.int32, "new_len")
            new_len = torch.clamp(new_len, min=0, out=self._new_len)
        block.assign_pages(seq_len, new_len, self.table, self.ring, cursor, self.cache.page_size, rows, stream=s,
                           fit_rows=True, one_each=self.one_each)
        qkv, out = self.qkv, self.out
        self.norm_in.forward(None, h, None, qkv.x, stream=s)
        ids = self._row_ids if self.tenants is not None and plans is None else (None, None)
        plans = plans or (qkv.batch, out.batch)
        if ids[0] is not None:
            torch.add(rows.req, 1, out=self._column)
            torch.index_select(self._ids, 1, self._column, out=self._row_ids)
        self._layer(qkv, plans[0], ids[0], s)
        if pos is None:
            pos = rows.pos if self.rotary.n_axes == 1 else rows.pos.expand(self.rotary.n_axes, -1)
        self.rotary.store(self.q, self.k, self.v, pos, rows.slot, self.cache, self.q_rot, stream=s,
                          norm=self.head_norm)
        req = None if self.one_each else rows.req
        if self.group is None:
            self.attention.forward(self.q_rot, self.table, rows.len, self.a, row_req=req, stream=s)
        else:
            self.attention.forward(self.q_rot, self.table, rows.len, self.group, self.shared_len, self.a, row_req=req,
                                   stream=s)
        self._layer(out, plans[1], ids[1], s)
        self.norm_out.forward(out.y, h, h_out, x_out, gate=gate, stream=s)
        # (last, so that a call that was refused on its way may be made again)
        torch.add(rows.state, 0, out=self.state)
        return h_out, x_out

    def fork(self, parent, keep=None, drop=False):
        """Between two steps: request r goes on from the first keep[r] positions
        (None: all) of request parent[r], as in block.fork_pages (outside the
        requests: it ends). drop: pages that rows from here on do not see
        through the window go back, so the request cannot be cut back past them
        later, and one that is refused (its length says so) is ended or read again
        from its start where the window is not whole pages. Returns the block.Fork
        that says what came of it."""
        import torch
        from . import block
        if not self.forks:
            raise ValueError("a step made without forks")
        f, s = self._fork, block.current_stream(self.cache.index)
        cursor, seq_len = block.split_state(self.state, self.rows.n_requests)
        block.fork_pages(seq_len, parent, self.table, self.ring, cursor, self.cache.page_size, f, keep=keep,
                         window=self.window if drop else 0, sinks=self.sinks if drop else 0, stream=s)
        block.copy_pages(self.cache, f.src, f.dst, f.n, stream=s)
        torch.add(f.table, 0, out=self.table)
        torch.add(f.state, 0, out=self.state)
        return f

    def keep_only(self, start, kept, n_kept, drop=False):
        """Between two steps: of its positions from start[r] on request r keeps
        n_kept[r], those in kept[r] (ascending), moved together (block.compact: the
        drafts that were accepted, a cache with positions evicted), and gives back
        the pages behind. The pages from start[r] on must be the request's alone.
        Returns the block.Fork of that."""
        from . import block
        if not self.forks:
            raise ValueError("a step made without forks")
        s = block.current_stream(self.cache.index)
        block.compact(self.cache, self.table, start, kept, n_kept, new_len=self._keep, stream=s)
        return self.fork(self._same, self._keep, drop=drop)

    @staticmethod
    def _layer(ld, plan, ids, stream):
        if ids is None:
            ld.layer.forward(plan, ld.x, ld.W, ld.y, stream=stream)
        else:
            ld.layer.forward_noalloc(ids, ld.x, ld.W, ld.y, stream=stream)

    def close(self):
        self.out.batch.close()
        self.out.layer.close()


# ---- timing ------------------------------------------------------------------------------------

def _time(torch, fn, iters=200, reps=7):
    for _ in range(20):
        fn()
    torch.cuda.synchronize()
    ts = []
    for _ in range(reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(iters):
            fn()
        e1.record()
        torch.cuda.synchronize()
        ts.append(e0.elapsed_time(e1) * 1e3 / iters)
    return statistics.median(ts)


def qkv_tenants(with_oft: bool, with_vera: bool = False):
    from synth import AdapterSpec
    L, Dr, I3 = AdapterSpec("lora", rank=16), AdapterSpec("dora", rank=16), AdapterSpec("ia3")
    ten = [(L, L, L)] * 8 + [(Dr, Dr, Dr)] * 6 + [(None, I3, I3)] * 6
    if with_oft:
        O = AdapterSpec("oft", blk=32)
        ten = ten[:16] + [(O, O, O)] * 4
    if with_vera:
        V = AdapterSpec("vera")
        ten = ten[:4] + [(V, V, V)] * 4 + ten[8:]
    return ten


def run():
    import torch
    rows = []
    d_in, d_outs, n = 4096, (4096, 1024, 1024), 128
    for with_oft, with_vera in ((False, False), (True, False), (True, True)):
        ten = qkv_tenants(with_oft, with_vera)
        wls, tt = projection_workloads(ten, n, d_in, d_outs, seed=11, vera_rank=256 if with_vera else 0)
        sp = QKVSplit(wls)
        t_split = _time(torch, sp.forward)
        sp.close()
        name = "lora+dora+ia3(k,v)" + ("+oft" if with_oft else "") + ("+vera" if with_vera else "")
        rows.append({"layer": "qkv", "tenants": name, "route": "split", "us": t_split})
        fu = QKVFused(wls, tt, len(ten))
        t_fused = _time(torch, fu.forward)
        fu.close()
        rows.append({"layer": "qkv", "tenants": name, "route": "fused", "us": t_fused})
        print(f"multiproj: {rows[-1]}", file=sys.stderr, flush=True)
    # prefill: 2048 tokens with the OFT tenants (the fused layer takes the
    # prefill path, its projections ending on 256-column tiles)
    wls, tt = projection_workloads(qkv_tenants(True), 2048, d_in, d_outs, seed=12)
    sp = QKVSplit(wls)
    t_split = _time(torch, sp.forward, iters=50)
    sp.close()
    fu = QKVFused(wls, tt, len(qkv_tenants(True)))
    t_fused = _time(torch, fu.forward, iters=50)
    fu.close()
    name = "lora+dora+ia3(k,v)+oft, 2048 tok"
    rows += [{"layer": "qkv", "tenants": name, "route": "split", "us": t_split},
             {"layer": "qkv", "tenants": name, "route": "fused", "us": t_fused}]
    print(f"multiproj: {rows[-1]}", file=sys.stderr, flush=True)
    from synth import make_config
    up = make_config(3)  # FFN up 4096 -> 14336, 256 tokens, (IA)^3 + VeRA tenants
    Wg = np.random.default_rng(5).normal(0.0, 1.0 / np.sqrt(up.d_in), size=up.W.shape)
    gu = GatedUp(up, Wg)
    t_gated = _time(torch, gu.forward)
    t_up = _time(torch, lambda: gu.up.layer.forward(gu.up.batch, gu.up.x, gu.up.W, gu.up.y))
    gu.close()
    rows.append({"layer": "ffn_up_gated", "tenants": up.name, "route": "gate + up + silu_gate", "us": t_gated})
    rows.append({"layer": "ffn_up_gated", "tenants": up.name, "route": "up only", "us": t_up})
    for context in (512, 4096):
        rows += attention_rows(torch, context)
        print(f"multiproj: {rows[-1]}", file=sys.stderr, flush=True)
    return rows


def attention_rows(torch, context, n=128, heads=32, kv_heads=8, head_dim=128, page_size=16):
    """The attention step of n requests with `context` positions each (one
    token a step), and its operators one by one."""
    from synth import AdapterSpec, WorkloadSpec, make_workload
    d = heads * head_dim
    ten = qkv_tenants(False)
    wls, tt = projection_workloads(ten, n, d, (d, kv_heads * head_dim, kv_heads * head_dim), seed=13)
    wl_out = make_workload(WorkloadSpec("out", "bf16", d, d, n, [AdapterSpec("lora", rank=16)] * 4, assign="explicit",
                                        token_adapter=np.asarray(tt) % 4, seed=14))
    fu = QKVFused(wls, tt, len(ten))
    dev = fu.x.device
    freq = 500000.0 ** (-torch.arange(head_dim // 2, dtype=torch.float64, device=dev) / (head_dim // 2))
    pages = -(-(context + 1) // page_size)
    ones = torch.ones(d, device=dev)
    st = AttentionStep(fu, wl_out, heads, kv_heads, head_dim, n, pages, page_size, n * pages, freq, norm_in=ones,
                       norm_out=ones, one_each=True)
    h, new = torch.randn((n, d), device=dev), torch.ones(n, dtype=torch.int32, device=dev)
    h_out, x_out = torch.empty_like(h), torch.empty((n, d), dtype=fu.x.dtype, device=dev)
    # every request holds `context` positions; the timed steps bring the same next token again
    from . import block
    grown, rows = block.Rows(n, n * context, dev), st.rows
    block.assign_pages(st.rows.seq_len, new * context, st.table, st.ring, st.rows.cursor, page_size, grown)

    def step():
        st.state.copy_(grown.state)
        return st.forward(h, new, h_out, x_out)

    parts = [("attention step", step),
             ("norm + pages + rotary", lambda: (
                 st.norm_in.forward(None, h, None, fu.x),
                 block.assign_pages(grown.seq_len, new, st.table, st.ring, grown.cursor, page_size, rows),
                 st.rotary.store(st.q, st.k, st.v, rows.pos, rows.slot, st.cache, st.q_rot))),
             ("attention over the cache", lambda: st.attention.forward(st.q_rot, st.table, rows.len, st.a)),
             ("residual + norm", lambda: st.norm_out.forward(st.out.y, h, h_out, x_out))]
    got = [{"layer": "attention", "tenants": f"{n} requests, {context} positions", "route": name,
            "us": _time(torch, fn, iters=50)} for name, fn in parts]
    st.close()
    fu.close()
    return got


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--out", default=None)
    a = ap.parse_args()
    rows = run()
    if a.out:
        with open(a.out, "w") as f:
            json.dump(rows, f, indent=1)
    print("| layer | tenants | route | µs / forward |\n|---|---|---|---|")
    for r in rows:
        print(f"| {r['layer']} | {r['tenants']} | {r['route']} | {r['us']:.2f} |")


if __name__ == "__main__":
    main()

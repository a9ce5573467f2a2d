"""Operators on pages that requests share (fork_pages, copy_pages, compact)
against plain loops. Whole numbers and moved values are equal, bit for bit."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _int(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def fork_ref(length, parent, keep, table, ring, head, tail, ps, n_pages, window=0, sinks=0):
    """The step in plain loops."""
    R, P = table.shape
    cap, ring = len(ring), ring.copy()
    held_len = [min(max(0, int(n)), P * ps) for n in length]
    new, pos = [], []
    for r in range(R):
        p = int(parent[r])
        n = held_len[p] if 0 <= p < R else 0
        if keep is not None:
            n = min(n, max(0, int(keep[r])))
        row = [-1] * P
        for c in range(-(-n // ps)):
            e = int(table[p, c])
            unseen = window > 0 and c * ps >= sinks and (c + 1) * ps <= n - window
            row[c] = e if 0 <= e < n_pages and not unseen else -1
        new.append(row)
        pos.append(n)
    before = {int(e) for r in range(R) for e in table[r, :-(-held_len[r] // ps)] if 0 <= e < n_pages}
    whole = {new[r][c] for r in range(R) for c in range(pos[r] // ps)} - {-1}
    partly = {}
    for r in range(R):
        if pos[r] % ps and new[r][pos[r] // ps] >= 0:
            partly.setdefault(new[r][pos[r] // ps], []).append(r)
    free = max(0, min(cap, tail - head))
    src, dst, cnt = [-1] * R, [-1] * R, [0] * R
    taken = refused = 0
    for r in range(R):
        c, n = divmod(pos[r], ps)
        e = new[r][c] if n else -1
        if e < 0 or (e not in whole and partly[e][0] == r):
            continue
        if taken < free:
            src[r], dst[r], cnt[r] = e, int(ring[(head + taken) % cap]), n
            new[r][c] = dst[r]
            taken += 1
        else:
            new[r][c], pos[r] = -1, pos[r] - n
            refused += 1
    gone = sorted(before - whole - set(partly))
    for j, e in enumerate(gone):
        ring[(tail + j) % cap] = e
    return {"table": np.array(new).reshape(R, P), "seq_len": np.array(pos), "src": np.array(src), "dst": np.array(dst),
            "n": np.array(cnt), "cursor": np.array([head + taken, tail + len(gone)]),
            "counts": np.array([sum(n > 0 for n in pos), taken, refused, len(gone)])}, ring


def _case(seed, R, P, ps, beams=2, spare=7, share_free=1.0, bad=False):
    """Requests that share the first pages of their group's first."""
    rng = np.random.default_rng(seed)
    n_pages = R * P + spare
    length = rng.integers(0, P * ps + 1, size=R)
    length[rng.random(R) < 0.1] = 0
    pages = rng.permutation(n_pages)
    table = np.full((R, P), -1, np.int64)
    k = 0
    for r in range(R):
        lead = r // beams * beams
        both = min(int(length[r]), int(length[lead])) // ps
        share = int(rng.integers(0, both + 1)) if r != lead else 0
        held = -(-int(length[r]) // ps)
        table[r, :share] = table[lead, :share]
        table[r, share:held] = pages[k:k + held - share]
        k += held - share
    free = int((n_pages - k) * share_free)
    head = int(rng.integers(0, 3 * n_pages))
    ring = np.full(n_pages, -9, np.int64)
    for j in range(free):
        ring[(head + j) % n_pages] = pages[k + j]
    parent = np.arange(R)
    for r in range(R):
        lead, x = r // beams * beams, rng.random()
        if x < 0.5:
            parent[r] = min(R - 1, lead + int(rng.integers(0, beams)))
        elif x < 0.6:
            parent[r] = rng.choice([-1, -5, R, R + 9])
    keep = np.where(rng.random(R) < 0.4, length[np.clip(parent, 0, max(0, R - 1))] - rng.integers(0, 2 * ps, size=R) if R else 0, P * ps)
    if bad and R:  # entries that hold no page, lengths past the table, negative ones
        table[rng.random((R, P)) < 0.1] = n_pages + 3
        length[0], length[-1] = P * ps + 99, -4
    return length, parent, keep, table, ring, head, head + free, n_pages


FORKS = [
    (0, 1, 16, {}, 0, 0), (1, 1, 1, {}, 0, 0), (1, 5, 4, dict(beams=1), 0, 0), (1, 5, 4, dict(beams=1), 3, 0),
    (5, 6, 4, dict(beams=5), 0, 0), (64, 9, 16, dict(beams=4), 0, 0), (64, 9, 16, dict(beams=4, share_free=0.02), 0, 0),
    (64, 300, 5, dict(beams=3), 200, 7), (64, 300, 5, dict(beams=3, bad=True), 31, 0),
    (63, 40, 16, dict(beams=9, bad=True, share_free=0.0), 0, 0), (300, 12, 1, dict(beams=2), 4, 3),
    (1023, 9, 16, dict(beams=4, share_free=0.1), 40, 16), (1025, 9, 16, dict(beams=4), 16, 100000),
    (2500, 5, 128, dict(beams=6, share_free=0.05), 0, 0), (3, 2500, 2, dict(beams=3), 1, 0),
    (17, 300, 5, dict(beams=3, bad=True), 31, 0), (256, 30, 4, dict(beams=4, share_free=0.1), 40, 3), (257, 30, 4, dict(beams=4), 40, 3),
    (2, 4093, 1, dict(beams=2), 0, 0), (2, 4092, 1, dict(beams=2), 1000, 70)]


@pytest.mark.parametrize("R, P, ps, kw, window, sinks", FORKS)
@pytest.mark.parametrize("cut", [False, True])
def test_fork_matches_loops(R, P, ps, kw, window, sinks, cut):
    length, parent, keep, table, ring, head, tail, n_pages = _case(R + P, R, P, ps, **kw)
    want, ring_want = fork_ref(length, parent, keep if cut else None, table, ring, head, tail, ps, n_pages, window, sinks)
    wide = torch.full((R, P + 3), -5, dtype=torch.int32, device=DEV)
    wide[:, :P] = _int(table.reshape(R, P))
    ring_d, cur = _int(ring), torch.tensor([head, tail], device=DEV)
    f = block.Fork(R, P, n_pages, DEV)
    len_d, par_d, keep_d = _int(length), _int(parent), _int(keep) if cut else None
    for again in range(2):  # the inputs stand, so a second call does the same (and its marks were cleared)
        for name in ("table", "seq_len", "src", "dst", "n", "cursor", "counts"):
            getattr(f, name).fill_(-77)
        block.fork_pages(len_d, par_d, wide[:, :P], ring_d, cur, ps, f, keep=keep_d, window=window, sinks=sinks)
        torch.cuda.synchronize()
        for name, v in want.items():
            assert np.array_equal(getattr(f, name).cpu().numpy(), v), (again, name)
        assert np.array_equal(ring_d.cpu().numpy(), ring_want), again
    assert bool((wide[:, P:] == -5).all()) and np.array_equal(wide[:, :P].cpu().numpy(), table.reshape(R, P))


def test_fork_steps_in_a_graph():
    """Captured steps of assign, fork and copies: requests grow, fork from each
    other, are cut back and end. Pages are never lost, a request's last page is
    its own, and what every request reads at its positions is what it wrote or
    took over."""
    R, P, ps, n_pages, H, D = 24, 8, 4, 150, 2, 8
    rng = np.random.default_rng(8)
    k = torch.zeros((n_pages, ps, H, D), device=DEV)
    cache = block.KVCache(k, torch.zeros_like(k))
    ring = torch.arange(n_pages, dtype=torch.int32, device=DEV)
    rows, f = block.Rows(R, 64, DEV), block.Fork(R, P, n_pages, DEV)
    f.state[:2] = torch.tensor([0, n_pages])
    table = torch.full((R, P), -1, dtype=torch.int32, device=DEV)
    new_d, par_d, keep_d = _int(np.zeros(R)), _int(np.arange(R)), _int(np.zeros(R))
    token = torch.zeros(64, device=DEV)
    rot = block.Rotary(torch.zeros(0, dtype=torch.float64, device=DEV), D)
    q, q_out = torch.zeros((64, H, D), device=DEV), torch.empty((64, H, D), device=DEV)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        block.assign_pages(f.seq_len, new_d, table, ring, f.cursor, ps, rows, fit_rows=True)
        kv = token[:, None, None].expand(64, H, D).contiguous()
        rot.store(q, kv, kv, rows.pos, rows.slot, cache, q_out)
        block.fork_pages(rows.seq_len, par_d, table, ring, rows.cursor, ps, f, keep=keep_d)
        block.copy_pages(cache, f.src, f.dst, f.n)
        table.copy_(f.table)
    f.state.zero_()
    f.state[:2] = torch.tensor([0, n_pages])
    said = [[] for _ in range(R)]
    stamp = 0
    for step in range(50):
        new = rng.integers(0, 4, size=R)
        parent = np.where(rng.random(R) < 0.3, rng.integers(-1, R, size=R), np.arange(R))
        cut = rng.random(R) < 0.2
        new_d.copy_(_int(new)), par_d.copy_(_int(parent)), keep_d.copy_(_int(np.where(cut, rng.integers(0, P * ps, size=R), P * ps)))
        stamp_row = stamp + np.arange(64)
        token.copy_(torch.tensor(stamp_row, dtype=F32))
        stamp += 64
        graph.replay()
        torch.cuda.synchronize()
        req, pos = rows.req.tolist(), rows.pos.tolist()
        for t in range(64):
            if req[t] >= 0:
                assert pos[t] == len(said[req[t]])
                said[req[t]].append(float(stamp_row[t]))
        seq, keep = f.seq_len.tolist(), keep_d.tolist()
        said = [said[p][:seq[r]] if 0 <= p < R else [] for r, p in enumerate(parent)]
        assert [len(x) for x in said] == seq
        tab, kk, vv = table.tolist(), cache.k.cpu(), cache.v.cpu()
        holders = {}
        for r in range(R):
            for c in range(-(-seq[r] // ps)):
                holders.setdefault(tab[r][c], []).append((r, c))
            for t, x in enumerate(said[r]):
                for z in (kk, vv):
                    assert bool((z[tab[r][t // ps], t % ps] == x).all()), (step, r, t)
        for r in range(R):
            if seq[r] % ps:
                assert len(holders[tab[r][seq[r] // ps]]) == 1, (step, r)
        h, t = f.cursor.tolist()
        assert sorted(list(holders) + [int(ring[c % n_pages]) for c in range(h, t)]) == list(range(n_pages)), step


def test_fork_on_another_stream():
    length, parent, keep, table, ring, head, tail, n_pages = _case(3, 64, 9, 16, beams=4)
    want, _ = fork_ref(length, parent, keep, table, ring, head, tail, 16, n_pages)
    s = torch.cuda.Stream()
    args = [_int(length), _int(parent), _int(table), _int(ring), torch.tensor([head, tail], device=DEV)]
    keep_d, f = _int(keep), block.Fork(64, 9, n_pages, DEV)
    s.wait_stream(torch.cuda.current_stream())
    block.fork_pages(*args, 16, f, keep=keep_d, stream=s)
    s.synchronize()
    for name, v in want.items():
        assert np.array_equal(getattr(f, name).cpu().numpy(), v), name


# ---- copies -----------------------------------------------------------------------------------------

def _cache(n_pages, ps, heads, dim, dt, by_head, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (n_pages, heads, ps, dim) if by_head else (n_pages, ps, heads, dim)
    k, v = (torch.randn(shape, generator=g).to(dt) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if by_head else (k, v)


def _on_gpu(z, by_head):
    return z.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if by_head else z.to(DEV)


LAYOUTS = [(1, 1, 8, F32, False), (16, 8, 128, BF16, False), (5, 3, 80, F32, True), (64, 1, 256, F32, False),
           (100, 2, 8, BF16, True), (7, 11, 24, BF16, False)]


@pytest.mark.parametrize("ps, heads, dim, dt, by_head", LAYOUTS)
def test_copies(ps, heads, dim, dt, by_head):
    n_pages, m = 40, 23
    k, v = _cache(n_pages, ps, heads, dim, dt, by_head)
    rng = np.random.default_rng(ps)
    dst = rng.permutation(n_pages)[:m]
    rest = np.setdiff1d(np.arange(n_pages), dst)
    src = rng.choice(rest, size=m)
    n = rng.integers(0, ps + 1, size=m)
    n[0], n[1], n[2], n[3], dst[4], src[5], dst[6] = ps + 5, 0, -3, ps, -1, n_pages, src[6]
    kd, vd = _on_gpu(k, by_head), _on_gpu(v, by_head)
    block.copy_pages(block.KVCache(kd, vd), _int(src), _int(dst), _int(n))
    for z, got in ((k.clone(), kd), (v.clone(), vd)):
        want = z.clone()
        for s, d, c in zip(src, dst, n):
            if 0 <= s < n_pages and 0 <= d < n_pages and c > 0:
                want[d, :c] = z[s, :c]
        assert torch.equal(got.cpu(), want)


def test_many_copies():
    k, v = _cache(9001, 2, 1, 8, F32, False)
    kd, vd = k.to(DEV), v.to(DEV)
    block.copy_pages(block.KVCache(kd, vd), _int(np.arange(4500)), _int(4500 + np.arange(4500)), _int(np.full(4500, 2)))
    assert torch.equal(kd[4500:9000].cpu(), k[:4500]) and torch.equal(vd[4500:9000].cpu(), v[:4500])
    assert torch.equal(kd[9000].cpu(), k[9000])


# ---- positions moved together -----------------------------------------------------------------------------

def _compact_ref(z, table, start, kept, n_kept, ps):
    z, was = z.clone(), z.clone()
    R, P = table.shape
    for r in range(R):
        a = max(0, int(start[r]))
        for j in range(min(max(0, int(n_kept[r])), kept.shape[1])):
            s, d = int(kept[r, j]), a + j
            if d < s < P * ps:
                ps_, pd = int(table[r, s // ps]), int(table[r, d // ps])
                if 0 <= ps_ < z.shape[0] and 0 <= pd < z.shape[0]:
                    z[pd, d % ps] = was[ps_, s % ps]
    return z


@pytest.mark.parametrize("ps, heads, dim, dt, by_head", LAYOUTS)
@pytest.mark.parametrize("R, P, share", [(1, 40, 0.5), (7, 9, 0.2), (5, 30, 0.95)])
def test_compact_matches_loops(ps, heads, dim, dt, by_head, R, P, share):
    rng = np.random.default_rng(R + ps)
    n_pages = R * P + 2
    table = rng.permutation(n_pages)[:R * P].reshape(R, P)
    L = P * ps
    start = rng.integers(0, L // 2 + 1, size=R)
    stay = [np.nonzero(rng.random(L - a) < share)[0] + a for a in start]
    W = max(len(s) for s in stay) + 2
    kept, n_kept = np.full((R, W), -1), np.array([len(s) for s in stay])
    for r, s in enumerate(stay):
        kept[r, :len(s)] = s
    if R > 1:  # places that keep what they held, pages that are not there, rows without anything
        if n_kept[0] > 2:
            kept[0, 1], kept[0, 2] = -8, L + 5
        table[1, rng.integers(0, P)] = -1
        n_kept[2], start[2] = 0, -3
        n_kept[3] = W + 9
    k, v = _cache(n_pages, ps, heads, dim, dt, by_head, seed=P)
    kd, vd = _on_gpu(k, by_head), _on_gpu(v, by_head)
    new_len = _int(np.full(R, -1))
    wide = torch.full((R, W + 5), 1, dtype=torch.int32, device=DEV)
    wide[:, :W] = _int(kept)
    block.compact(block.KVCache(kd, vd), _int(table), _int(start), wide[:, :W], _int(n_kept), new_len=new_len)
    for z, got in ((k, kd), (v, vd)):
        assert torch.equal(got.cpu(), _compact_ref(z, table, start, kept, n_kept, ps))
    assert new_len.tolist() == [max(0, int(a)) + min(int(n), W) for a, n in zip(start, n_kept)]


@pytest.mark.parametrize("R, heads, dim, dt", [(2, 1, 8, F32), (9, 2, 128, BF16), (40, 4, 128, F32), (70, 8, 128, BF16)])
def test_compact_columns_of_each_width(R, heads, dim, dt):
    """32, 64, 128 and 256 bytes, lists of several trips of each."""
    rng, P, ps, W = np.random.default_rng(R), 80, 16, 1100
    table = rng.permutation(R * P).reshape(R, P)
    k, v = _cache(R * P, ps, heads, dim, dt, False, seed=R)
    kd, vd = k.to(DEV), v.to(DEV)
    start = rng.integers(0, 9, size=R)
    kept = np.stack([np.sort(rng.choice(np.arange(10, P * ps), W, replace=False)) for _ in range(R)])
    n_kept = rng.integers(W - 60, W + 1, size=R)
    block.compact(block.KVCache(kd, vd), _int(table), _int(start), _int(kept), _int(n_kept))
    for z, got in ((k, kd), (v, vd)):
        want = z.clone()
        for r in range(R):
            n, src = n_kept[r], torch.as_tensor(kept[r][:n_kept[r]])
            to, t = start[r] + torch.arange(n), torch.as_tensor(table[r])
            at = src > to
            src, to = src[at], to[at]
            want[t[to // ps], to % ps] = z[t[src // ps], src % ps]
        same = torch.equal(got.cpu(), want)
        assert same


def test_compact_nothing_kept():
    k, v = _cache(4, 2, 1, 8, F32, False)
    kd, vd, new_len = k.to(DEV), v.to(DEV), _int([7, 7])
    block.compact(block.KVCache(kd, vd), _int([[0, 1], [2, 3]]), _int([3, 0]), _int(np.zeros((2, 0))), _int([0, 4]), new_len)
    assert torch.equal(kd.cpu(), k) and new_len.tolist() == [3, 0]


def test_compact_many_requests():
    """More units than one launch's work-groups would take in one round."""
    R = 65536
    k = torch.arange(2 * R, dtype=F32, device=DEV).view(R, 2, 1, 1).expand(R, 2, 40, 8).contiguous()
    v = k + 0.5
    block.compact(block.KVCache(k, v), torch.arange(R, dtype=torch.int32, device=DEV).view(R, 1), _int(np.zeros(R)),
                  _int(np.ones((R, 1))), _int(np.ones(R)))
    want = torch.arange(2 * R, dtype=F32, device=DEV).view(R, 2)[:, 1:].expand(R, 2)
    assert bool((k == want[:, :, None, None]).all()) and bool((v == want[:, :, None, None] + 0.5).all())


def test_compact_in_a_graph():
    """Drafts accepted step by step, captured once: each replay moves another path."""
    R, P, ps, W = 9, 6, 4, 5
    rng = np.random.default_rng(2)
    table = rng.permutation(R * P).reshape(R, P)
    k, v = _cache(R * P, ps, 2, 16, BF16, False)
    kd, vd = k.to(DEV), v.to(DEV)
    start_d, kept_d, n_d, table_d = _int(np.zeros(R)), _int(np.zeros((R, W))), _int(np.zeros(R)), _int(table)
    cache = block.KVCache(kd, vd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block.compact(cache, table_d, start_d, kept_d, n_d)
    for _ in range(6):
        start = rng.integers(0, 8, size=R)
        n = rng.integers(0, W + 1, size=R)
        kept = np.stack([a + np.sort(rng.permutation(P * ps - a)[:W]) for a in start])
        start_d.copy_(_int(start)), kept_d.copy_(_int(kept)), n_d.copy_(_int(n))
        g.replay()
        torch.cuda.synchronize()
        k, v = _compact_ref(k, table, start, kept, n, ps), _compact_ref(v, table, start, kept, n, ps)
        assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_one_workspace_for_forks_of_several_sizes():
    """A workspace zeroed once serves calls of other requests and pages in turn."""
    sizes = [(64, 9, 16, 7), (700, 40, 5, 900), (2500, 5, 16, 0), (1, 5, 4, 9000), (300, 60, 2, 5000), (4100, 3, 8, 1)]
    forks = [block.Fork(R, P, R * P + spare, DEV) for R, P, _, spare in sizes]
    one = torch.zeros(max(f._workspace.shape[0] for f in forks), dtype=torch.uint8, device=DEV)
    for f in forks:
        f.args.workspace, f.args.workspace_bytes = one.data_ptr(), one.shape[0]
    for i in (1, 2, 1, 4, 0, 3, 5, 4, 2, 3, 1, 5, 0, 4):
        (R, P, ps, spare), f = sizes[i], forks[i]
        length, parent, keep, table, ring, head, tail, n_pages = _case(R + P, R, P, ps, beams=4, spare=spare, share_free=0.3)
        want, ring_want = fork_ref(length, parent, keep, table, ring, head, tail, ps, n_pages)
        ring_d = _int(ring)
        block.fork_pages(_int(length), _int(parent), _int(table), ring_d, torch.tensor([head, tail], device=DEV), ps, f,
                         keep=_int(keep))
        torch.cuda.synchronize()
        for name, v in want.items():
            same = np.array_equal(getattr(f, name).cpu().numpy(), v)
            assert same, (i, name)
        same = np.array_equal(ring_d.cpu().numpy(), ring_want)
        assert same, i

"""The operators between a block's adapter layers (lora_normal_form_amd.block)
against plain implementations in 64 bits on the CPU, at the sizes and masks
where they can go wrong.

Tolerances count roundings: one to type t is off by at most u(t) =
finfo(t).eps / 2 relative to the value (bf16 2^-8, fp32 2^-24); an fp32 sum of
n terms by at most n u(fp32) of the sum of their magnitudes."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    err = torch.where(nan, 0.0, (got - want).abs() - tol)
    worst = float(err.max()) if err.numel() else 0.0
    assert worst <= 0.0, f"{what}: off by {worst:.3e} more than the bound at {int(err.argmax())}"


def _int(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


# ---- pages and slots ------------------------------------------------------------------------------

def _assign_ref(old, new, table, ring, head, tail, ps, max_tokens):
    """The step in plain loops."""
    table, ring = table.copy(), ring.copy()
    R, P = table.shape
    cap = len(ring)
    free = [int(ring[c % cap]) for c in range(head, tail)]
    rows = {"seq_len": np.zeros(R, np.int64), "cu_len": np.zeros(R + 1, np.int64), "slot": np.full(max_tokens, -1),
            "req": np.full(max_tokens, -1), "pos": np.zeros(max_tokens, np.int64), "len": np.zeros(max_tokens, np.int64)}
    want_so_far = placed = refused = t = 0
    taken = 0
    back = []
    for r in range(R):
        o, n = max(0, int(old[r])), int(new[r])
        held = -(-o // ps)
        rows["cu_len"][r] = t
        if n < 0:
            back += [int(p) for p in table[r, :min(held, P)]]
            continue
        upto = -(-(o + n) // ps)
        ok = upto <= P
        want = upto - held if ok else 0
        if want:
            ok = want_so_far + want <= len(free)
            if ok:
                table[r, held:upto] = free[want_so_far:want_so_far + want]
                taken = want_so_far + want
            want_so_far += want
        refused += not ok
        rows["seq_len"][r] = o + n if ok else o
        for i in range(n):
            if ok and t < max_tokens:
                p = o + i
                rows["slot"][t] = int(table[r, p // ps]) * ps + p % ps
                rows["req"][t], rows["pos"][t], rows["len"][t] = r, p, p + 1
            t += 1
        placed += n if ok else 0
    rows["cu_len"][R] = t
    for j, p in enumerate(back):
        ring[(tail + j) % cap] = p
    rows["cursor"] = np.array([head + taken, tail + len(back)])
    rows["counts"] = np.array([placed, taken, refused, len(back)])
    return table, ring, rows


def _assign_case(seed, R, P, ps, max_new, free_share=1.0, ended=0.1):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, P * ps + 1, size=R)
    old[rng.random(R) < 0.1] = 0
    new = rng.integers(0, max_new + 1, size=R)
    new[rng.random(R) < ended] = -1
    cap = max(1, R * P)
    pages = rng.permutation(cap)
    table = np.full((R, P), -7, np.int64)
    k = 0
    for r in range(R):
        h = -(-int(old[r]) // ps)
        table[r, :h] = pages[k:k + h]
        k += h
    free = int((cap - k) * free_share)
    head = int(rng.integers(0, 3 * cap))
    ring = np.full(cap, -9, np.int64)
    for j in range(free):
        ring[(head + j) % cap] = pages[k + j]
    return old, new, table, ring, head, head + free


@pytest.mark.parametrize("R, P, ps, max_new, cap_tokens, free_share", [
    (0, 1, 16, 1, 4, 1.0), (1, 1, 1, 1, 1, 1.0), (1, 40, 7, 250, 300, 1.0), (5, 6, 16, 0, 3, 1.0),
    (64, 9, 16, 1, 64, 1.0), (64, 9, 16, 1, 64, 0.02), (300, 12, 5, 40, 9000, 0.3), (300, 12, 5, 40, 2000, 1.0),
    (1023, 4, 16, 3, 3100, 0.5), (1024, 4, 16, 3, 3100, 1.0), (1025, 4, 16, 3, 3100, 0.1), (2500, 3, 128, 6, 9000, 0.4)])
def test_assign_matches_loops(R, P, ps, max_new, cap_tokens, free_share):
    old, new, table, ring, head, tail = _assign_case(R + P, R, P, ps, max_new, free_share)
    want = _assign_ref(old, new, table, ring, head, tail, ps, cap_tokens)
    wide = torch.full((R, P + 3), -5, dtype=torch.int32, device=DEV)
    wide[:, :P] = _int(table.reshape(R, P))
    ring_d, cur = _int(ring), torch.tensor([head, tail], device=DEV)
    rows = block.Rows(R, cap_tokens, DEV)
    old_d, new_d = _int(old), _int(new)
    for _ in range(2):  # the inputs stand, so a second call does the same
        block.assign_pages(old_d, new_d, wide[:, :P], ring_d, cur, ps, rows)
    torch.cuda.synchronize()
    assert np.array_equal(wide[:, :P].cpu().numpy(), want[0])
    assert bool((wide[:, P:] == -5).all())
    assert np.array_equal(ring_d.cpu().numpy(), want[1])
    for name, v in want[2].items():
        assert np.array_equal(getattr(rows, name).cpu().numpy(), v), name


def test_assign_steps_in_a_graph():
    """Three hundred captured steps that swap two Rows: requests grow, end and
    start again; no page is ever held twice."""
    R, P, ps, cap = 33, 6, 4, 120
    rng = np.random.default_rng(3)
    table = torch.full((R, P), -1, dtype=torch.int32, device=DEV)
    ring, new_d = torch.arange(cap, dtype=torch.int32, device=DEV), _int(np.zeros(R))
    a, b = block.Rows(R, 64, DEV), block.Rows(R, 64, DEV)
    a.cursor.copy_(torch.tensor([0, cap]))
    graphs = []
    s = torch.cuda.Stream()
    for src, dst in ((a, b), (b, a)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            block.assign_pages(src.seq_len, new_d, table, ring, src.cursor, ps, dst)
        graphs.append((g, src, dst))
    for step in range(60):
        g, src, dst = graphs[step % 2]
        new = rng.integers(0, 3, size=R)
        new[rng.random(R) < 0.15] = -1
        new_d.copy_(_int(new))
        old, tab, rg = src.seq_len.cpu().numpy(), table.cpu().numpy(), ring.cpu().numpy()
        head, tail = src.cursor.tolist()
        want = _assign_ref(old, new, tab, rg, head, tail, ps, 64)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(table.cpu().numpy(), want[0]) and np.array_equal(ring.cpu().numpy(), want[1])
        for name, v in want[2].items():
            assert np.array_equal(getattr(dst, name).cpu().numpy(), v), (step, name)
        n, tab = dst.seq_len.tolist(), table.tolist()
        held = [p for r in range(R) for p in tab[r][:-(-n[r] // ps)]]
        h, t = dst.cursor.tolist()
        assert sorted(held + [int(ring[c % cap]) for c in range(h, t)]) == list(range(cap))


# ---- rotary positions ---------------------------------------------------------------------------------

def _cache_tensors(n_pages, ps, heads, dim, dt, by_head=False, seed=0, fill=None):
    g = torch.Generator().manual_seed(seed)
    shape = (n_pages, heads, ps, dim) if by_head else (n_pages, ps, heads, dim)
    k, v = (torch.randn(shape, generator=g) if fill is None else torch.full(shape, fill) for _ in range(2))
    k, v = k.to(DEV, dt), v.to(DEV, dt)
    return (k.transpose(1, 2), v.transpose(1, 2)) if by_head else (k, v)


@pytest.mark.parametrize("T, Hq, Hk, D, rd, axes, inter, src, dt, by_head, odd", [
    (1, 32, 8, 128, 128, 1, False, F32, BF16, False, 0), (5, 4, 2, 64, 64, 3, False, F32, BF16, True, 0),
    (5, 4, 2, 64, 64, 3, True, F32, BF16, False, 0), (7, 3, 3, 40, 20, 2, False, F32, F32, False, 0),
    (7, 3, 1, 40, 22, 2, True, BF16, F32, False, 0), (7, 3, 1, 40, 22, 2, False, BF16, BF16, True, 0),
    (9, 2, 1, 256, 256, 4, True, BF16, BF16, False, 0), (9, 2, 1, 256, 2, 1, False, F32, BF16, False, 0),
    (4, 2, 1, 8, 0, 1, False, F32, BF16, False, 0), (6, 4, 2, 64, 64, 2, False, F32, BF16, False, 1),
    (6, 4, 2, 64, 32, 1, True, BF16, F32, False, 3), (1300, 2, 1, 16, 8, 8, False, F32, BF16, False, 0)])
def test_rotary_and_store(T, Hq, Hk, D, rd, axes, inter, src, dt, by_head, odd):
    g = torch.Generator().manual_seed(T + D + rd)
    ps, n_pages = 5, T // 5 + 3
    wide = (Hq + 2 * Hk) * D
    # odd: rows start and lie off 16 bytes (one element an access)
    buf = torch.randn((T, wide + 4 + odd), generator=g).to(DEV, src)
    y = buf[:, odd:odd + wide]
    q, k, v = (t.unflatten(1, (-1, D)) for t in torch.split(y, [Hq * D, Hk * D, Hk * D], dim=1))
    n = rd // 2
    freq = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(1, n))
    axis = torch.randint(0, axes, (n,), generator=g, dtype=torch.int32)
    pos = torch.randint(-1000, 1 << 30, (axes, T), generator=g, dtype=torch.int32)
    kc, vc = _cache_tensors(n_pages, ps, Hk, D, dt, by_head)
    slot = torch.randperm(n_pages * ps, generator=g)[:T]
    if T > 3:
        slot[1], slot[3] = -1, n_pages * ps
    k0, v0 = kc.cpu().clone(), vc.cpu().clone()
    q_buf = torch.full((T + 1, Hq, D), 77.0, dtype=dt, device=DEV)
    cache = block.KVCache(kc, vc)
    ro = block.Rotary(freq.to(DEV), D, axis=axis.to(DEV) if axes > 1 else None, n_axes=axes, interleaved=inter)
    ro.store(q, k, v, pos.to(DEV) if axes > 1 else pos[0].to(DEV), slot.to(DEV), cache, q_buf[:T])
    torch.cuda.synchronize()
    ang = pos.double()[axis.long() if axes > 1 else torch.zeros(n, dtype=torch.long)].T * freq

    def turned(z):
        z = z.cpu().double()
        a, b = (2 * torch.arange(n), 2 * torch.arange(n) + 1) if inter else (torch.arange(n), torch.arange(n) + n)
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        out, mag = z.clone(), torch.zeros_like(z)
        out[..., a], out[..., b] = z[..., a] * c - z[..., b] * s, z[..., a] * s + z[..., b] * c
        mag[..., a] = mag[..., b] = z[..., a].abs() + z[..., b].abs()
        # the angle: in turns at most 2^30 / 6, known to 2^27.4 2^-52 of a turn (two fp64 roundings), its fraction
        # rounded to fp32 (2^-25 turns), then sincospi (under 2 ulp, 2^-23) and three fp32 roundings
        off = 2 * math.pi * (2.0 ** -25 + 2.0 ** -23) + 2.0 ** -22 + 3 * U[F32]
        return out, off * mag + U[dt] * (out.abs() + off * mag)

    want, tol = turned(q)
    _close(q_buf[:T], want, tol, "q")
    assert bool((q_buf[T] == 77.0).all())
    kw, kt = turned(k)
    ref_k, tol_k = k0.double(), torch.zeros_like(k0, dtype=torch.float64)
    ref_v, tol_v = v0.double(), torch.zeros_like(tol_k)
    for t in range(T):
        s = int(slot[t])
        if 0 <= s < n_pages * ps:
            ref_k[s // ps, s % ps], tol_k[s // ps, s % ps] = kw[t], kt[t]
            ref_v[s // ps, s % ps], tol_v[s // ps, s % ps] = v[t].cpu().double(), U[dt] * v[t].cpu().double().abs()
    _close(kc, ref_k, tol_k, "k")
    _close(vc, ref_v, tol_v, "v")


def test_rotary_no_tokens():
    kc, vc = _cache_tensors(2, 4, 1, 8, BF16)
    ro = block.Rotary(torch.ones(4, dtype=torch.float64, device=DEV), 8)
    z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    ro.store(z(0, 2, 8), z(0, 1, 8), z(0, 1, 8), _int(np.zeros(0)), z(0).long(), block.KVCache(kc, vc),
             z(0, 2, 8).to(BF16))
    torch.cuda.synchronize()


# ---- attention ------------------------------------------------------------------------------------------

def _attend_ref(q, kc, vc, table, lens, req, window, scale):
    """(out, its bound) in 64 bits; positions whose page is not in the cache are not seen."""
    q, kc, vc, table = q.cpu().double(), kc.cpu(), vc.cpu(), table.cpu()
    dt = kc.dtype
    N, H, D = q.shape
    n_pages, ps, Hk, _ = kc.shape
    R, P = table.shape
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(N):
        r = int(req[i])
        n = min(int(lens[i]), P * ps) if 0 <= r < R else 0
        t = torch.arange(max(0, n - window) if window else 0, max(0, n))
        page = table[r, t // ps].long() if len(t) else t
        ok = (page >= 0) & (page < n_pages)
        t, page = t[ok], page[ok]
        if not len(t):
            continue
        K, V = kc[page, t % ps].double(), vc[page, t % ps].double()
        for h in range(H):
            g = h // (H // Hk)
            s = K[:, g] @ q[i, h] * scale
            p = torch.softmax(s, 0)
            out[i, h] = p @ V[:, g]
            # a score is off by D + 3 fp32 roundings of its terms' magnitudes (and the exponent's argument by as
            # much as the running maximum's again), exp2 by 2 ulp, the sums by n roundings; a weight is the sum of
            # two bf16 (off by 2^-8 2^-8) for a bf16 cache, and the output is rounded once
            off = float((K[:, g].abs() @ q[i, h].abs()).max()) * abs(scale) * (D + 3) * U[F32]
            rel = 2 * 2 * off + (2 * len(t) + 16) * U[F32]
            mag = p @ V[:, g].abs()
            tol[i, h] = (rel + (U[dt] ** 2 if dt == BF16 else 0.0)) * mag + U[dt] * (out[i, h].abs() + 2 * rel * mag)
    return out, tol


def _attend_case(seed, lens, P, ps, Hq, Hk, D, dt, by_head=False, spare=3):
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    kc, vc = _cache_tensors(R * P + spare, ps, Hk, D, dt, by_head, seed)
    table = torch.randperm(R * P + spare, generator=g)[:R * P].view(R, P).int().to(DEV)
    q = torch.randn((R, Hq, D), generator=g).to(DEV, dt)
    return kc, vc, table, q


def _run_attend(kc, vc, table, q, lens, req=None, window=0, scale=None):
    cache = block.KVCache(kc, vc)
    att = block.PagedAttention(cache, q.shape[1], window=window, scale=scale)
    buf = torch.full((q.shape[0] + 1, q.shape[1], q.shape[2]), 55.0, dtype=q.dtype, device=DEV)
    out = att.forward(q, table, _int(lens), buf[:-1], row_req=None if req is None else _int(req))
    torch.cuda.synchronize()
    assert bool((buf[-1] == 55.0).all())
    ref, tol = _attend_ref(q, kc, vc, table, lens, range(len(lens)) if req is None else req, window,
                           1 / math.sqrt(q.shape[2]) if scale is None else scale)
    _close(out, ref, tol, "out")
    return att, out


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D, Hq, Hk, ps, by_head", [
    (128, 32, 8, 16, False), (128, 32, 8, 16, True), (64, 8, 8, 32, False), (256, 4, 2, 16, False),
    (8, 5, 1, 16, False), (80, 12, 4, 5, False), (72, 6, 2, 1, True), (96, 17, 1, 48, False), (136, 40, 2, 7, False),
    (192, 3, 1, 64, True), (248, 2, 2, 100, False),
    (128, 32, 1, 16, False), (64, 33, 1, 16, True), (256, 100, 2, 6, False), (40, 64, 1, 1, False)])
def test_attention_shapes(dt, D, Hq, Hk, ps, by_head):
    lens = [1, 0, 2, 15, 16, 17, 31, 32, 33, 64, 65, 130]
    kc, vc, table, q = _attend_case(D + Hq, lens, -(-130 // ps), ps, Hq, Hk, D, dt, by_head)
    _run_attend(kc, vc, table, q, lens)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 5000])
def test_attention_window(dt, window):
    lens = [1, 3, 40, 100, 101, 500, 0]
    kc, vc, table, q = _attend_case(window, lens, 32, 16, 4, 2, 64, dt)
    _run_attend(kc, vc, table, q, lens, window=window)


@pytest.mark.parametrize("dt, Hq, Hk, D, lens", [
    (BF16, 8, 2, 128, [5000]), (BF16, 1, 1, 64, [9000, 1]), (F32, 4, 1, 128, [3000, 0, 2999]),
    (BF16, 16, 1, 256, [4097]), (BF16, 20, 1, 64, [2048] * 3),
    (BF16, 80, 2, 128, [6000, 17, 4001]), (F32, 71, 1, 256, [2500, 600])])
def test_attention_long(dt, Hq, Hk, D, lens):
    """A few rows over long contexts: the work is split over the length."""
    kc, vc, table, q = _attend_case(len(lens), lens, -(-max(lens) // 16), 16, Hq, Hk, D, dt)
    _run_attend(kc, vc, table, q, lens)


@pytest.mark.parametrize("ps", [16, 6])
def test_attention_many_rows(ps):
    """More rows than a work-group has threads, most of them short; the rows of
    one request are its new tokens."""
    rng = np.random.default_rng(ps)
    R, N = 7, 700
    kc, vc, table, _ = _attend_case(1, [0] * R, 200 // ps + 1, ps, 4, 2, 64, BF16)
    lens, req = rng.integers(0, 200, size=N), rng.integers(-1, R + 1, size=N)
    req[:40] = 3
    lens[:40] = np.arange(100, 140)
    q = torch.randn((N, 4, 64), generator=torch.Generator().manual_seed(2)).to(DEV, BF16)
    _run_attend(kc, vc, table, q, lens.tolist(), req=req.tolist())


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("ps", [16, 32, 5])
def test_attention_masked_places_hold_anything(dt, ps):
    """Infinities and NaN behind a row's length, before its window, in pages
    of no request and in bad pages' place change nothing; neither do lengths
    past the table."""
    P = -(-96 // ps)
    lens = [33, 96, 1, 50, P * ps + 1000]
    kc, vc, table, q = _attend_case(5, lens, P, ps, 4, 2, 64, dt)
    table[3, 1] = -1
    table[3, 2] = kc.shape[0]
    table[1, 0] = 1 << 30
    window = 40
    seen = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for r, n in enumerate(lens):
        for t in range(max(0, min(n, P * ps) - window) if n <= P * ps else P * ps - window, min(n, P * ps)):
            page = int(table[r, t // ps])
            if 0 <= page < kc.shape[0]:
                seen[page, t % ps] = True
    for i, bad in enumerate((float("nan"), float("inf"), float("-inf"))):
        for c in (kc, vc):
            c[(~seen).to(DEV)] = bad
        cache = block.KVCache(kc, vc)
        out = torch.empty_like(q)
        block.PagedAttention(cache, 4, window=window).forward(q, table, _int(lens), out)
        torch.cuda.synchronize()
        ref, tol = _attend_ref(q, kc, vc, table, lens, range(len(lens)), window, 1 / 8)
        assert bool(torch.isfinite(ref).all())
        _close(out, ref, tol, f"masked {bad}")


@pytest.mark.parametrize("dt, Hq, Hk, D, ps, window", [
    (BF16, 4, 4, 128, 16, 0), (BF16, 4, 2, 64, 16, 0), (BF16, 8, 2, 128, 32, 0), (BF16, 6, 2, 80, 5, 0),
    (BF16, 10, 2, 128, 16, 20), (BF16, 16, 2, 64, 16, 7), (BF16, 9, 1, 64, 16, 0), (F32, 6, 2, 80, 5, 30),
    (F32, 4, 1, 256, 16, 0), (BF16, 8, 2, 256, 48, 33), (BF16, 16, 2, 128, 16, 0), (BF16, 5, 1, 96, 16, 40),
    (F32, 7, 1, 128, 6, 0), (BF16, 33, 3, 64, 16, 0), (F32, 16, 1, 72, 16, 25), (BF16, 24, 1, 128, 16, 0),
    (BF16, 20, 1, 256, 16, 0), (BF16, 6, 1, 256, 16, 0)])
def test_attention_rows_of_one_request(dt, Hq, Hk, D, ps, window):
    """Rows of one request share the reads of its cache: runs of one to seven
    rows, with lengths that rise, fall, repeat and vanish, rows of no request
    between them; a NaN that only the longest row of a run sees stays with it."""
    req = [0, 0, 0, 0, 0, 1, 1, 2, 3, 3, 3, -1, -1, 4, 4, 9, 4, 4, 5, 5, 5, 5, 5, 5, 5]
    lens = [100, 101, 102, 103, 104, 33, 32, 64, 0, 1, 2, 50, 0, 130, 7, 9, 70, 70, 60, 61, 62, 63, 64, 65, 66]
    kc, vc, table, _ = _attend_case(D + ps, [0] * 6, -(-140 // ps), ps, Hq, Hk, D, dt)
    q = torch.randn((len(req), Hq, D), generator=torch.Generator().manual_seed(1)).to(DEV, dt)
    _run_attend(kc, vc, table, q, lens, req=req, window=window)
    for r, n in ((0, 104), (5, 66), (4, 130)):
        page, at = int(table[r, (n - 1) // ps]), (n - 1) % ps
        vc[page, at, :, 3:5] = torch.tensor([float("nan"), float("inf")], device=DEV)
        kc[page, at, 0, 1] = float("nan")
    cache = block.KVCache(kc, vc)
    out = block.PagedAttention(cache, Hq, window=window).forward(q, table, _int(lens), torch.empty_like(q),
                                                                 row_req=_int(req))
    torch.cuda.synchronize()
    ref, tol = _attend_ref(q, kc, vc, table, lens, req, window, 1 / math.sqrt(D))
    clean = [i for i in range(len(req)) if i not in (4, 13, 24)]
    assert bool(torch.isfinite(ref[clean]).all()) and bool(torch.isfinite(out[clean]).all())
    _close(out[clean], ref[clean], tol[clean], "rows that do not see the NaN")
    for i in (4, 13, 24):
        assert bool(torch.isnan(out[i, :Hq // Hk]).all()) and bool(torch.isnan(out[i, :, 3]).all())


def test_attention_extreme_scores():
    """Scores far apart (no overflow, the far ones vanish), equal scores, and
    values of the type's lowest in a seen place (the score is then -inf or
    far below: its weight is 0)."""
    lens = [70, 70, 70]
    kc, vc, table, q = _attend_case(9, lens, 5, 16, 2, 1, 64, F32)
    q[0] *= 300.0
    q[1] = 0.0
    page = int(table[2, 1])
    kc[page, 3] = torch.finfo(F32).min / 1e5 * q[2, 0].sign().view(1, -1)
    q[2, 1] = q[2, 0]
    ref = torch.zeros(3, 2, 64, dtype=torch.float64)
    for i in range(3):
        t = torch.arange(70)
        K = kc[table[i, (t // 16).to(DEV)].long(), (t % 16).to(DEV), 0].cpu().double()
        V = vc[table[i, (t // 16).to(DEV)].long(), (t % 16).to(DEV), 0].cpu().double()
        ref[i] = torch.softmax(q[i].cpu().double() @ K.T / 8, 1) @ V
    out = block.PagedAttention(block.KVCache(kc, vc), 2).forward(q, table, _int(lens), torch.empty_like(q))
    torch.cuda.synchronize()
    # scores up to 300 |q.k| / 8 ~ 3000: 67 fp32 roundings of them give 4e-2 relative to a weight at most
    assert float((out[0].cpu().double() - ref[0]).abs().max()) <= 4e-2 * 8
    _close(out[1:], ref[1:], torch.full_like(ref[1:], 2e-5), "equal and lowest")


def test_attention_nan_in_a_seen_place():
    lens = [40, 40]
    kc, vc, table, q = _attend_case(11, lens, 3, 16, 2, 2, 64, BF16)
    kc[int(table[0, 1]), 2, 0, 5] = float("nan")
    out = block.PagedAttention(block.KVCache(kc, vc), 2).forward(q, table, _int(lens), torch.empty_like(q))
    assert bool(torch.isnan(out[0, 0]).all()) and bool(torch.isfinite(out[0, 1]).all())
    assert bool(torch.isfinite(out[1]).all())


def test_attention_strided_rows_and_padded_table():
    """q, out and the table as views of wider buffers."""
    lens = [20, 300, 7]
    kc, vc, table, _ = _attend_case(13, lens, 19, 16, 4, 2, 64, BF16)
    wide_t = torch.full((3, 30), 1 << 29, dtype=torch.int32, device=DEV)
    wide_t[:, :19] = table
    buf = torch.randn((3, 10, 64), generator=torch.Generator().manual_seed(1)).to(DEV, BF16)
    obuf = torch.full((3, 7, 64), 9.0, dtype=BF16, device=DEV)
    q = buf[:, 2:6]
    block.PagedAttention(block.KVCache(kc, vc), 4).forward(q, wide_t[:, :19], _int(lens), obuf[:, 1:5])
    torch.cuda.synchronize()
    ref, tol = _attend_ref(q, kc, vc, table, lens, range(3), 0, 1 / 8)
    _close(obuf[:, 1:5], ref, tol, "out")
    assert bool((obuf[:, 0] == 9.0).all()) and bool((obuf[:, 5:] == 9.0).all())


def test_attention_offsets_past_32_bits():
    """Pages that lie more than 2^32 bytes (and 2^31 elements) into the cache."""
    ps, Hk, D = 64, 8, 128
    n_pages = (1 << 31) // (ps * Hk * D) + 40
    kc = torch.empty((n_pages, ps, Hk, D), dtype=BF16, device=DEV)
    vc = torch.empty_like(kc)
    lens = [130, 200]
    table = torch.tensor([[n_pages - 1, 0, n_pages - 7, 3], [n_pages - 2, n_pages - 3, 5, n_pages - 11]],
                         dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(4)
    for p in table.flatten().tolist():
        kc[p], vc[p] = torch.randn((ps, Hk, D), generator=g).to(DEV), torch.randn((ps, Hk, D), generator=g).to(DEV)
    # the newest position of each request is written by the rotary store (no rotation: two pairs of angle 0)
    cache = block.KVCache(kc, vc)
    ro = block.Rotary(torch.zeros(2, dtype=torch.float64, device=DEV), D)
    new = torch.randn((2, (16 + 2 * Hk) * D), generator=g).to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in torch.split(new, [16 * D, Hk * D, Hk * D], dim=1))
    slot = torch.tensor([(n_pages - 7) * ps + 129 - 128, (n_pages - 11) * ps + 199 - 192], device=DEV)
    qo = torch.empty((2, 16, D), dtype=BF16, device=DEV)
    ro.store(q, k, v, _int([129, 199]), slot, cache, qo)
    assert torch.equal(kc[n_pages - 7, 1], k[0].to(BF16)) and torch.equal(vc[n_pages - 11, 7], v[1].to(BF16))
    out = block.PagedAttention(cache, 16).forward(qo, table, _int(lens), torch.empty_like(qo))
    torch.cuda.synchronize()
    pages, inv = torch.unique(table, return_inverse=True)
    small_k, small_v = kc[pages.long()], vc[pages.long()]
    ref, tol = _attend_ref(qo, small_k, small_v, inv.int(), lens, range(2), 0, 1 / math.sqrt(D))
    _close(out, ref, tol, "out")


def test_attention_repeats_the_same_bits_and_graphs():
    """The same call gives the same bits; a captured call, replayed between
    eager ones, follows its inputs, lengths and pages; two handles run side by
    side on two streams."""
    lens = [1000, 3, 700, 0, 64]
    kc, vc, table, q = _attend_case(17, lens, 64, 16, 8, 2, 128, BF16)
    n = _int(lens)
    cache = block.KVCache(kc, vc)
    att, att2 = block.PagedAttention(cache, 8), block.PagedAttention(cache, 8)
    first = att.forward(q, table, n, torch.empty_like(q)).clone()
    out, eager, out2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        att.forward(q, table, n, out)
    s2 = torch.cuda.Stream()
    for step in range(4):
        if step:
            q.copy_(torch.randn(q.shape, device=DEV).to(BF16))
            n.copy_(_int(np.random.default_rng(step).integers(0, 1025, size=5)))
            table.copy_(torch.randperm(kc.shape[0], device=DEV)[:table.numel()].view_as(table).int())
        torch.cuda.synchronize()
        g.replay()
        att2.forward(q, table, n, out2, stream=s2)
        torch.cuda.synchronize()
        att.forward(q, table, n, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(out2, eager)
        if step == 0:
            assert torch.equal(out, first)
    ref, tol = _attend_ref(q, kc, vc, table, n.tolist(), range(5), 0, 1 / math.sqrt(128))
    _close(out, ref, tol, "after the replays")
    assert int(att.workspace.view(torch.int32)[:64].abs().sum()) == 0  # (the counters are left zero)


def test_attention_refusals_with_tensors():
    kc, vc, table, q = _attend_case(1, [5, 5], 2, 16, 4, 2, 64, BF16)
    cache = block.KVCache(kc, vc)
    att = block.PagedAttention(cache, 4)
    n, out = _int([5, 5]), torch.empty_like(q)
    for args, kw in (((q.float(), table, n, out), {}), ((q, table.long(), n, out), {}), ((q, table, n.long(), out), {}),
                     ((q[:, :2], table, n, out), {}), ((q, table, n[:1], out), {}), ((q, table[:1], n, out), {}),
                     ((q, table, n, out), dict(row_req=n[:1])), ((q, table.cpu(), n, out), {}),
                     ((q.transpose(0, 1).contiguous().transpose(0, 1), table, n, out), {})):
        with pytest.raises(ValueError):
            att.forward(*args, **kw)
    with pytest.raises(scute.ScuteError):  # (in place)
        att.forward(q, table, n, q)
    with pytest.raises(ValueError):
        block.PagedAttention(cache, 3)
    att.workspace = att.workspace[:16]
    with pytest.raises(scute.ScuteError):
        att.forward(q, table, n, out)
    none = att.forward(q[:0], table, n[:0], out[:0])  # no rows: nothing to do
    assert none.shape[0] == 0


def test_attention_row_limit():
    kc, vc, table, q = _attend_case(1, [5, 5], 2, 16, 4, 2, 64, BF16)
    att = block.PagedAttention(block.KVCache(kc, vc), 4, max_rows=1)
    att.forward(q[:1], table, _int([5]), torch.empty_like(q[:1]))
    with pytest.raises(ValueError):
        att.forward(q, table, _int([5, 5]), torch.empty_like(q))
    torch.cuda.synchronize()


def test_handles_are_ready_on_every_stream():
    """A handle made behind a stream's work is zeroed by the time it is there."""
    kc, vc, table, q = _attend_case(1, [5, 5], 2, 16, 4, 2, 64, BF16)
    busy = torch.randn((4096, 4096), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = torch.mm(busy, busy).clamp_(-1, 1)
        rows = block.Rows(64, 1000, DEV)
        for _ in range(20):
            busy = torch.mm(busy, busy).clamp_(-1, 1)
        att = block.PagedAttention(block.KVCache(kc, vc), 4)
    rows.slot.fill_(7)
    att.workspace[:64].fill_(7)
    torch.cuda.synchronize()
    assert bool((rows.slot == 7).all()) and bool((att.workspace[:64] == 7).all())


# ---- the norms around the residual ----------------------------------------------------------------------

def _norm_ref(z, e, kind, w, b, eps):
    """N(z) in 64 bits, and its bound for a z known to e: each fp32 step rounds once, the sums are trees of depth
    under 64 (at most 32 terms a thread, 64 lanes, 16 waves), so 256 roundings of the terms' magnitudes cover it."""
    mu = z.mean(1, keepdim=True) if kind == "layer" else torch.zeros(z.shape[0], 1, dtype=torch.float64)
    c = z - mu
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    w = torch.ones(z.shape[1], dtype=torch.float64) if w is None else w.cpu().double()
    b = torch.zeros(z.shape[1], dtype=torch.float64) if b is None else b.cpu().double()
    e_c = e + e.mean(1, keepdim=True) + 256 * U[F32] * (z.abs() + z.abs().mean(1, keepdim=True))
    e_r = torch.sqrt((e_c * e_c).mean(1, keepdim=True)) * r + 256 * U[F32]
    out = c * r * w + b
    return out, (w * r).abs() * (e_c + c.abs() * e_r) + 4 * U[F32] * (out.abs() + (c * r * w).abs())


@pytest.mark.parametrize("T, d, kind, post, affine, gate, y_dt, h_dt, x_dt, pre, off", [
    (1, 4096, "rms", True, True, None, F32, BF16, BF16, True, 0), (3, 4096, "layer", True, True, "token", F32, F32, BF16, True, 0),
    (2, 1, "rms", True, True, None, F32, F32, F32, True, 0), (2, 1, "layer", True, True, "channel", F32, F32, F32, True, 0),
    (5, 7, "layer", False, True, "channel", BF16, BF16, F32, True, 0), (5, 1001, "rms", True, False, "token", BF16, F32, BF16, True, 0),
    (2, 32768, "layer", True, True, None, F32, BF16, BF16, True, 0), (2, 32767, "layer", True, True, "token", F32, BF16, BF16, True, 0),
    (4, 256, "rms", False, True, None, F32, BF16, BF16, True, 0), (4, 260, "rms", True, True, "channel", F32, BF16, BF16, False, 0),
    (4, 512, "layer", True, True, "token", BF16, BF16, BF16, True, 1), (3, 10000, "rms", True, True, None, BF16, F32, F32, True, 0)])
def test_residual_norm(T, d, kind, post, affine, gate, y_dt, h_dt, x_dt, pre, off):
    g = torch.Generator().manual_seed(T * d)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731

    def rows(dt, scale, shift):  # (off: rows that start off 16 bytes)
        return (scale * rnd(T, d + 2 * off) + shift).to(DEV, dt)[:, off:off + d]

    y, h = rows(y_dt, 3.0, 5.0), rows(h_dt, 2.0, -1.0)
    vec = lambda m, on: (m + 0.2 * rnd(d)).to(DEV) if on else None  # noqa: E731
    pw, pb = vec(1.0, post and affine), vec(0.0, post and affine)
    ew, eb = vec(1.0, pre and affine), vec(0.0, pre and affine)
    gt = {None: None, "channel": vec(0.0, True), "token": rows(F32, 1.0, 0.0)}[gate]
    a, c, eps = 0.9, -1.3, 1e-5
    norm = block.ResidualNorm(d, kind, post=post, post_weight=pw, post_bias=pb, pre=pre, pre_weight=ew, pre_bias=eb,
                              h_scale=a, y_scale=c, eps=eps, device=DEV)
    ho = torch.full((T + 1, d), 5.0, dtype=h_dt, device=DEV)
    xo = torch.full((T + 1, d), 5.0, dtype=x_dt, device=DEV) if pre else None
    norm.forward(y, h, ho[:T], xo[:T] if pre else None, gate=gt)
    torch.cuda.synchronize()
    z = y.cpu().double()
    e = torch.zeros_like(z)
    if post:
        z, e = _norm_ref(z, e, kind, pw, pb, eps)
    gd = 1.0 if gt is None else gt.cpu().double()
    a32, c32 = float(np.float32(a)), float(np.float32(c))
    hp = a32 * h.cpu().double() + c32 * z * gd
    e = abs(c32) * e * (gd.abs() if gt is not None else 1.0) + \
        4 * U[F32] * ((a32 * h.cpu().double()).abs() + (c32 * z * gd).abs())
    _close(ho[:T], hp, e + U[h_dt] * (hp.abs() + e), "h")
    assert bool((ho[T] == 5.0).all())
    if pre:
        want, ex = _norm_ref(hp, e, kind, ew, eb, eps)
        _close(xo[:T], want, ex + U[x_dt] * (want.abs() + ex), "x")
        assert bool((xo[T] == 5.0).all())


def test_residual_norm_forms():
    """In place, without y, without h_out; no rows."""
    g = torch.Generator().manual_seed(1)
    y, h = torch.randn((6, 64), generator=g).to(DEV), torch.randn((6, 64), generator=g).to(DEV)
    norm = block.ResidualNorm(64, device=DEV)
    x, x2 = torch.empty_like(h), torch.empty_like(h)
    out, _ = norm.forward(y, h, torch.empty_like(h), x)
    norm.forward(y, h, None, x2)
    hh = h.clone()
    norm.forward(y, hh, hh, torch.empty_like(h))
    torch.cuda.synchronize()
    assert torch.equal(x, x2) and torch.equal(hh, out) and torch.equal(out, h + y)
    norm.forward(None, out, None, x2)
    torch.cuda.synchronize()
    assert torch.equal(x, x2)
    norm.forward(y[:0], h[:0], None, x[:0])
    for args, kw in (((y, h, h.to(BF16), x), {}), ((y, h, None, None), {}), ((y[:, :32], h, None, x), {}),
                     ((y, h, None, x), dict(gate=y.to(BF16))), ((None, h, None, x), dict(gate=y)),
                     ((y.cpu(), h, None, x), {}), ((y.half(), h, None, x), {})):
        with pytest.raises(ValueError):
            norm.forward(*args, **kw)
    with pytest.raises(scute.ScuteError):
        norm.forward(y, h, None, h)


def test_residual_norm_large_mean_and_zeros():
    """A mean far above the spread (the variance is summed about the mean) and
    rows of zeros (eps alone)."""
    g = torch.Generator().manual_seed(2)
    h = (1000.0 + torch.randn((3, 4096), generator=g)).to(DEV)
    h[1] = 0.0
    x = torch.empty_like(h)
    block.ResidualNorm(4096, "layer", device=DEV).forward(None, h, None, x)
    torch.cuda.synchronize()
    want, tol = _norm_ref(h.cpu().double(), torch.zeros(3, 4096, dtype=torch.float64), "layer", None, None, 1e-5)
    _close(x, want, tol, "x")
    assert bool((x[1] == 0.0).all())

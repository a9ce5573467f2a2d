"""The operators between a block's adapter layers at their edges: values,
sizes and orders of calls that the documentation allows, against plain
implementations in 64 bits (tests/test_block_gpu.py, whose bounds hold here)."""

import dataclasses
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402
from test_block_step_gpu import D, H, N, _bar, _step  # noqa: E402
from test_block_gpu import (BF16, DEV, F32, U, _assign_case, _attend_case, _attend_ref, _close, _int,  # noqa: E402
                            _norm_ref, _run_attend, test_residual_norm as _check_norm)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---- attention: values that are not finite -------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D, Hq, Hk, ps, lens, req, window", [
    (128, 32, 8, 16, [1, 700, 33, 0, 3000], None, 0), (64, 3, 1, 5, [2, 40], None, 7),
    (72, 40, 1, 16, [1, 900], None, 0), (256, 24, 1, 16, [1, 300], None, 0), (248, 8, 2, 16, [1, 130, 500], None, 0),
    (128, 8, 2, 16, [100, 101, 102, 103, 64, 65], [0, 0, 0, 0, 1, 1], 0),
    (80, 4, 1, 6, [50, 51, 52, 53, 54], [0, 0, 0, 0, 0], 20), (256, 6, 1, 16, [200, 199, 7], [0, 0, 0], 0)])
def test_attention_infinite_v(dt, D, Hq, Hk, ps, lens, req, window):
    """An infinity in the V that a row sees is the output's (a weight is
    positive), two of other signs or a NaN give NaN, and the other elements
    and rows are what they are without it."""
    kc, vc, table, q = _attend_case(D + Hq, lens, -(-max(lens) // ps), ps, Hq, Hk, D, dt)
    q *= 0.3  # (no weight vanishes in fp32)
    req = list(range(len(lens))) if req is None else req
    clean_k, clean_v = kc.clone(), vc.clone()
    inf, nan = float("inf"), float("nan")
    odd = torch.zeros(len(lens), Hq, D, dtype=torch.float64)  # the sum of what is not finite

    def plant(row, t, dim, value):
        """Into V of request req[row], position t, and into the rows that see it."""
        vc[int(table[req[row], t // ps]), t % ps, :, dim] = value
        for i, n in enumerate(lens):
            if req[i] == req[row] and (max(0, n - window) if window else 0) <= t < n:
                odd[i, :, dim] += value

    for row, n in enumerate(lens):
        if n == 0 or req[row] in req[:row]:
            continue
        plant(row, n - 1, 0, inf)
        plant(row, n - 1, D - 1, -inf)
        plant(row, max(0, n - 2), 5, inf)
        plant(row, max(0, n - 7), 5, -inf if n > 6 else inf)
        plant(row, n // 2, 9, -inf)
        plant(row, max(0, n - 3), 11, nan)
    cache, hit = block.KVCache(kc, vc), odd != 0
    ref, tol = _attend_ref(q, clean_k, clean_v, table, lens, req, window, 1 / math.sqrt(D))
    assert bool(hit.any()) and not bool(hit.all())
    orders = [_int(req)] + ([None] if req == list(range(len(lens))) else [])
    for rows in orders:
        got = block.PagedAttention(cache, Hq, window=window).forward(q, table, _int(lens), torch.empty_like(q),
                                                                     row_req=rows).cpu().double()
        assert torch.equal(torch.nan_to_num(got[hit], nan=7.0, posinf=8.0, neginf=9.0),
                           torch.nan_to_num(odd[hit], nan=7.0, posinf=8.0, neginf=9.0))
        zero = torch.zeros_like(got)
        _close(torch.where(hit, zero, got), torch.where(hit, zero, ref), tol, "elsewhere")


# ---- attention: every way the work is cut ------------------------------------------------------------------

def _counters(att):
    """The workspace's counters: the queue's two, and the arrivals at eight
    places a compute unit, for groups and for all."""
    units = torch.cuda.get_device_properties(0).multi_processor_count
    return att.workspace[:4 * (64 + 2 * 8 * units)].view(torch.int32)


def _long_ref(q, kc, vc, table, lens, req, window, chain):
    """(out, bound) on the GPU in 64 bits, all heads of a key head at once. The
    bound: scores as in _attend_ref; sums whose longest chain has `chain` roundings."""
    N, H, D = q.shape
    n_pages, ps, Hk, _ = kc.shape
    G, out, tol, dt = H // Hk, torch.zeros(q.shape, dtype=torch.float64, device=DEV), [], kc.dtype
    for i, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        tol.append(torch.zeros((H, D), dtype=torch.float64, device=DEV))
        if n <= lo:
            continue
        pages = table[req[i], :-(-n // ps)].long()
        for g in range(Hk):
            K, V = (c[pages, :, g].flatten(0, 1)[lo:n].double() for c in (kc, vc))
            qh = q[i, g * G:(g + 1) * G].double() / math.sqrt(D)
            p = torch.softmax(torch.mm(qh, K.T.contiguous()), 1)
            out[i, g * G:(g + 1) * G] = o = torch.mm(p, V)
            off = float(torch.mm(qh.abs(), K.abs().T.contiguous()).max()) * (D + 3) * U[F32]
            rel, mag = 4 * off + chain * U[F32], torch.mm(p, V.abs())
            tol[-1][g * G:(g + 1) * G] = (rel + (U[dt] ** 2 if dt == BF16 else 0.0)) * mag + U[dt] * (o.abs() + 2 * rel * mag)
    return out.cpu(), torch.stack(tol).cpu()


@pytest.mark.parametrize("dt, each, rows, Hq, Hk, D, ps, run, window", [
    (BF16, 70, 8, 4, 1, 64, 64, 0, 0),      # a tail of a 16th of the units
    (BF16, 140, 5, 4, 1, 64, 64, 0, 0),     # of an 8th
    (BF16, 70, 3, 40, 1, 64, 16, 0, 0),     # two query tiles at once
    (BF16, 70, 20, 4, 1, 64, 32, 4, 0),     # rows of one request
    (BF16, 75, 90, 2, 2, 64, 16, 0, 0),     # more than 64 rows
    (BF16, 72, 300, 2, 1, 64, 16, 0, 0),    # more pieces than work-groups
    (BF16, 68, 8, 6, 1, 64, 13, 0, 290000),  # pages of any size, a window
    (F32, 70, 7, 2, 1, 64, 16, 0, 0), (F32, 130, 3, 24, 1, 40, 16, 0, 0)])
def test_attention_long_work(dt, each, rows, Hq, Hk, D, ps, run, window):
    """Work enough for the tail of short slices that work-groups take from a
    counter: values that follow the position, so that no slice can be left out,
    taken twice or mixed up; the counters are left zero, and the bits repeat."""
    units = torch.cuda.get_device_properties(0).multi_processor_count
    per = each * units * (128 if dt == BF16 else 64) // (Hk * max(1, rows // max(1, run)))  # positions a request
    rng = np.random.default_rng(rows)
    R = rows // run if run else rows
    total = (per * (0.8 + 0.4 * rng.random(R))).astype(int)
    total[-1] += R * per - total.sum()  # (the work asked for, whatever the shares)
    P = -(-int(total.max()) // ps)
    g = torch.Generator(device=DEV).manual_seed(each)
    n_pages = int(sum(-(-int(n) // ps) for n in total)) + 3
    free = torch.randperm(n_pages, generator=g, device=DEV)
    kc = torch.randn((n_pages, ps, Hk, D), generator=g, device=DEV, dtype=dt)
    vc = torch.empty_like(kc)
    table = torch.full((R, P), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(total.tolist()):
        m = -(-n // ps)
        mine = free[at:at + m]
        table[r, :m] = mine.int()
        at += m
        t = torch.arange(m * ps, device=DEV, dtype=F32)
        wave = torch.cos(t[:, None] * (2 * math.pi / n) * (1 + torch.arange(D, device=DEV) % 29) + r)
        vc[mine] = wave.view(m, ps, 1, D).to(dt)
    q = (0.2 * torch.randn((rows, Hq, D), generator=g, device=DEV)).to(dt)
    req = np.repeat(np.arange(R), run) if run else np.arange(R)
    lens = [int(total[r]) - (run - 1 - i % run if run else 0) for i, r in enumerate(req)]
    att = block.PagedAttention(block.KVCache(kc, vc), Hq, window=window)
    call = lambda: att.forward(q, table, _int(lens), torch.full_like(q, 9.0), row_req=_int(req) if run else None)  # noqa: E731
    out = call()
    torch.cuda.synchronize()
    assert int(_counters(att).abs().sum()) == 0
    # a slice has at most 144 units, a tile of each a wave: 40 roundings a tile (32 products and their sums, in two
    # parts, the running maximum's factor), and as many again for the joins
    ref, tol = _long_ref(q, kc, vc, table, lens, req, window, 2 * 40 * 144)
    _close(out, ref, tol, "out")
    assert torch.equal(call(), out)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows", [65, 257, 600])
@pytest.mark.parametrize("Hq, Hk, D, ps", [(4, 2, 64, 16), (18, 1, 72, 5), (2, 2, 136, 16)])
def test_attention_row_a_request(dt, rows, Hq, Hk, D, ps):
    """More rows than lanes, and than threads, each of a request of its own."""
    lens = np.random.default_rng(rows).integers(0, 70, size=rows)
    lens[:5] = [0, 1, 200, 64, 65]
    kc, vc, table, q = _attend_case(rows + D, lens.tolist(), -(-200 // ps), ps, Hq, Hk, D, dt)
    att, _ = _run_attend(kc, vc, table, q, lens.tolist())
    assert int(_counters(att).abs().sum()) == 0


@pytest.mark.parametrize("by_request", [False, True])
def test_attention_in_several_launches(by_request):
    """A table so wide that the rows go through several launches: later
    launches read their own rows, requests and lengths."""
    Hk, D, ps, P = 8, 16, 32, 1 << 24
    rows = 150 if by_request else 70
    R = 3 if by_request else rows
    table = torch.empty((R, P), dtype=torch.int32, device=DEV)
    table[:, :7] = torch.arange(R * 7, device=DEV).view(R, 7)
    kc, vc = (torch.randn((R * 7, ps, Hk, D), generator=torch.Generator().manual_seed(s)).to(DEV, BF16) for s in (1, 2))
    q = torch.randn((rows, 8, D), generator=torch.Generator().manual_seed(3)).to(DEV, BF16)
    lens = np.random.default_rng(1).integers(0, 200, size=rows)
    req = np.sort(np.random.default_rng(2).integers(0, R, size=rows)) if by_request else np.arange(rows)
    out = block.PagedAttention(block.KVCache(kc, vc), 8).forward(
        q, table, _int(lens), torch.full_like(q, 5.0), row_req=_int(req) if by_request else None)
    torch.cuda.synchronize()
    ref, tol = _attend_ref(q, kc, vc, table[:, :7], lens.tolist(), req.tolist(), 0, 1 / math.sqrt(D))
    _close(out, ref, tol, "out")


# ---- the norms: rows by the hundred, and one element an access ------------------------------------------------

@pytest.mark.parametrize("T, d, kind, gate, off", [
    (600, 4096, "rms", None, 0), (513, 8192, "layer", "token", 0), (520, 16384, "rms", "channel", 0),
    (513, 1500, "layer", "token", 1), (520, 4001, "rms", "channel", 0), (3, 2500, "layer", None, 1),
    (2, 6000, "rms", "token", 1), (513, 9000, "layer", None, 1), (700, 64, "rms", None, 0)])
def test_norm_many_rows(T, d, kind, gate, off):
    _check_norm(T, d, kind, True, True, gate, F32, BF16 if off else F32, BF16, True, off)


# ---- inputs and outputs in one buffer ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 6])
def test_columns_of_one_buffer(rows):
    """Column ranges of one buffer are no overlap, a row's outputs may follow
    its inputs, and q may be turned where it lies: the same bits as apart."""
    g = torch.Generator().manual_seed(rows)
    kc, vc, table, _ = _attend_case(3, [20] * rows, 2, 16, 4, 2, 64, BF16)
    cache, lens = block.KVCache(kc, vc), _int([20 - i for i in range(rows)])
    att = block.PagedAttention(cache, 4)
    wide = torch.randn((rows, 12, 64), generator=g).to(DEV, BF16)
    apart = att.forward(wide[:, 4:8].contiguous(), table, lens, torch.empty((rows, 4, 64), dtype=BF16, device=DEV))
    for at in (0, 8):
        att.forward(wide[:, 4:8], table, lens, wide[:, at:at + 4])
        torch.cuda.synchronize()
        assert torch.equal(wide[:, at:at + 4], apart)
    # rotary: q, k, v and q_out in one buffer, then in place
    y = torch.randn((rows, 12, 64), generator=g).to(DEV, BF16)
    q, k, v, out = y[:, :4], y[:, 4:6], y[:, 6:8], y[:, 8:12]
    ro = block.Rotary(torch.tensor([0.7 ** i for i in range(32)], dtype=torch.float64, device=DEV), 64)
    pos, slot = _int(range(5, 5 + rows)), torch.arange(rows, device=DEV)
    apart = ro.store(q.contiguous(), k, v, pos, slot, cache, torch.empty((rows, 4, 64), dtype=BF16, device=DEV))
    ro.store(q, k, v, pos, slot, cache, out)
    ro.store(q, k, v, pos, slot, cache, q)
    torch.cuda.synchronize()
    assert torch.equal(out, apart) and torch.equal(q, apart)
    # norms: h, h' and x as columns of one buffer
    b = torch.randn((rows, 3 * 64), generator=g).to(DEV)
    norm = block.ResidualNorm(64, device=DEV)
    y = torch.randn((rows, 64), generator=g).to(DEV)
    want = norm.forward(y, b[:, 64:128].contiguous(), torch.empty((rows, 64), device=DEV), torch.empty((rows, 64), device=DEV))
    norm.forward(y, b[:, 64:128], b[:, :64], b[:, 128:])
    torch.cuda.synchronize()
    assert torch.equal(b[:, :64], want[0]) and torch.equal(b[:, 128:], want[1])


# ---- pages and slots ----------------------------------------------------------------------------------------

def _assign_flags_ref(old, new, table, ring, head, tail, ps, max_tokens, fit, one_each=False):
    """The step in plain loops, request by request."""
    table, ring = table.copy(), ring.copy()
    (R, P), cap = table.shape, len(ring)
    rows = {"seq_len": np.zeros(R, np.int64), "cu_len": np.zeros(R + 1, np.int64), "slot": np.full(max_tokens, -1),
            "req": np.full(max_tokens, -1), "pos": np.zeros(max_tokens, np.int64), "len": np.zeros(max_tokens, np.int64)}
    free = [int(ring[c % cap]) for c in range(head, tail)]
    wanted = taken = placed = refused = t = 0
    back = []
    for r in range(R):
        o, n = max(0, int(old[r])), int(new[r])
        held = -(-o // ps)
        rows["cu_len"][r] = first = t
        t += 1 if one_each else max(0, n)
        if n < 0:
            back += [int(p) for p in table[r, :min(held, P)]]
            continue
        want = -(-(o + n) // ps) - held
        ok = held + want <= P and not (fit and n and first + n > max_tokens) and not (one_each and n > 1)
        if ok and want:
            wanted += want
            ok = wanted <= len(free)
            if ok:
                table[r, held:held + want] = free[wanted - want:wanted]
                taken = wanted
        refused += not ok
        rows["seq_len"][r] = o + n if ok else o
        placed += n if ok else 0
        for i in range(min(n, max_tokens - first) if ok else 0):
            rows["slot"][first + i] = int(table[r, (o + i) // ps]) * ps + (o + i) % ps
            rows["req"][first + i], rows["pos"][first + i], rows["len"][first + i] = r, o + i, o + i + 1
    rows["cu_len"][R] = t
    for j, p in enumerate(back):
        ring[(tail + j) % cap] = p
    rows["cursor"] = np.array([head + taken, tail + len(back)])
    rows["counts"] = np.array([placed, taken, refused, len(back)])
    return table, ring, rows


@pytest.mark.parametrize("R, P, ps, max_new, rows, free_share, fit", [
    (300, 12, 5, 40, 2000, 1.0, True), (300, 12, 5, 40, 2000, 1.0, False), (300, 12, 5, 40, 0, 1.0, True),
    (64, 9, 16, 3, 40, 0.05, True), (2500, 3, 8, 6, 3000, 0.6, True), (40000, 2, 4, 2, 20000, 0.5, True),
    (65536, 1, 16, 1, 65536, 1.0, True), (5, 4, 16, 7, 1, 1.0, True)])
def test_assign_fits_rows(R, P, ps, max_new, rows, free_share, fit):
    """A request whose tokens pass the last row is refused (with fit_rows):
    what seq_len counts has a row, so it can be stored."""
    old, new, table, ring, head, tail = _assign_case(R + rows, R, P, ps, max_new, free_share)
    want = _assign_flags_ref(old, new, table, ring, head, tail, ps, rows, fit)
    got = block.Rows(R, rows, DEV)
    tab, ring_d = _int(table), _int(ring)
    old_d = _int(old)
    block.assign_pages(old_d, _int(new), tab, ring_d, torch.tensor([head, tail], device=DEV), ps, got, fit_rows=fit)
    torch.cuda.synchronize()
    assert np.array_equal(tab.cpu().numpy(), want[0]) and np.array_equal(ring_d.cpu().numpy(), want[1])
    for name, v in want[2].items():
        assert np.array_equal(getattr(got, name).cpu().numpy(), v), name
    if fit:
        grown = (got.seq_len - old_d.clamp(min=0)).clamp(min=0)
        here = got.req[got.req >= 0].long()
        assert torch.equal(torch.bincount(here, minlength=R), grown.long())


@pytest.mark.parametrize("R, P, ps, max_new, spare, free_share", [
    (1, 3, 4, 1, 0, 1.0), (7, 3, 1, 3, 2, 1.0), (128, 30, 16, 1, 0, 1.0), (1025, 4, 4, 2, 5, 0.1), (3000, 3, 4, 1, 0, 0.5)])
def test_assign_a_row_each(R, P, ps, max_new, spare, free_share):
    """Row r stays request r's, whoever ended, brought nothing or was refused."""
    old, new, table, ring, head, tail = _assign_case(R, R, P, ps, max_new, free_share, ended=0.2)
    want = _assign_flags_ref(old, new, table, ring, head, tail, ps, R + spare, True, one_each=True)
    got = block.Rows(R, R + spare, DEV)
    tab, ring_d = _int(table), _int(ring)
    block.assign_pages(_int(old), _int(new), tab, ring_d, torch.tensor([head, tail], device=DEV), ps, got, fit_rows=True,
                       one_each=True)
    torch.cuda.synchronize()
    assert np.array_equal(tab.cpu().numpy(), want[0]) and np.array_equal(ring_d.cpu().numpy(), want[1])
    for name, v in want[2].items():
        assert np.array_equal(getattr(got, name).cpu().numpy(), v), name
    assert bool(((got.req[:R] == -1) | (got.req[:R] == torch.arange(R, device=DEV))).all())


# ---- more rows than one launch has threads for ------------------------------------------------------------

def test_rotary_more_tokens_than_a_launch():
    """2^24 + 5 tokens (a launch has fewer than 2^32 threads): every token of
    every launch is turned, and stored where its slot says."""
    T, D = (1 << 24) + 5, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    y = torch.randn((T, 3 * D), generator=g, device=DEV, dtype=F32).to(BF16)
    q, k, v = (t.unflatten(1, (1, D)) for t in y.split(D, dim=1))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    slot = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    kept = [0, 3, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, T - 1]
    slot[torch.tensor(kept, device=DEV)] = torch.arange(len(kept), device=DEV)
    kc, vc = torch.zeros((2, 4, 1, D), dtype=BF16, device=DEV), torch.zeros((2, 4, 1, D), dtype=BF16, device=DEV)
    out = torch.zeros((T + 1, 1, D), dtype=BF16, device=DEV)
    freq = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64, device=DEV)
    block.Rotary(freq, D).store(q, k, v, pos, slot, block.KVCache(kc, vc), out[:T])
    torch.cuda.synchronize()
    ang = pos.double()[:, None] * freq
    c, s = torch.cos(ang).float(), torch.sin(ang).float()

    def worst(z, got, rows=slice(None)):
        a, b = z[rows, 0, :4].float(), z[rows, 0, 4:].float()
        want = torch.cat([a * c[rows] - b * s[rows], a * s[rows] + b * c[rows]], 1)
        # one rounding to bf16; angle, sine and products in fp32 (the bound of the smaller sizes: under 1e-5)
        tol = U[BF16] * want.abs() + 1e-5 * (a.abs() + b.abs()).repeat(1, 2)
        return float(((got[:, 0].float() - want).abs() - tol).max())

    assert worst(q, out[:T]) <= 0 and bool((out[T] == 0).all())
    at = torch.tensor(kept, device=DEV)
    assert worst(k, kc.view(8, 1, D)[:6], at) <= 0 and torch.equal(vc.view(8, 1, D)[:6], v[at])
    assert bool((kc.view(8, D)[6:] == 0).all())


def test_norm_more_rows_than_a_launch():
    """2^26 + 7 rows of one element: 64 threads a row pass 2^32."""
    T = (1 << 26) + 7
    g = torch.Generator(device=DEV).manual_seed(1)
    h, y = torch.randn((T, 1), generator=g, device=DEV), torch.randn((T, 1), generator=g, device=DEV)
    gate = torch.rand((T, 1), generator=g, device=DEV) + 0.5
    h_out, x = torch.full((T + 1, 1), 5.0, device=DEV), torch.full((T + 1, 1), 5.0, device=DEV)
    block.ResidualNorm(1, eps=0.25, device=DEV).forward(y, h, h_out[:T], x[:T], gate=gate)
    torch.cuda.synchronize()
    hp = h.double() + y.double() * gate
    # h': a product and a sum, a rounding each; x: under 16 more roundings of its own size
    assert bool(((h_out[:T] - hp).abs() <= 2 * U[F32] * (h.abs() + (y * gate).abs())).all())
    hp = h_out[:T].double()
    want = hp / torch.sqrt(hp * hp + 0.25)
    assert bool(((x[:T] - want).abs() <= 16 * U[F32] * want.abs()).all())
    assert float(h_out[T]) == 5.0 and float(x[T]) == 5.0


# ---- the attention step -----------------------------------------------------------------------------------

def test_timed_step_rows():
    """The timing of the attention step runs its steps on tensors that stay."""
    from lora_normal_form_amd import multiproj
    got = multiproj.attention_rows(torch, 40, n=8, heads=4, kv_heads=2, head_dim=64, page_size=16)
    assert [r["route"] for r in got] == ["attention step", "norm + pages + rotary", "attention over the cache",
                                         "residual + norm"]
    assert all(r["us"] > 0 for r in got)


def test_step_refuses_tokens_past_its_rows():
    """A request whose tokens do not all have rows keeps its length; when it
    comes again it is placed."""
    st, *_ = _step(91)
    h = torch.zeros((N, H * D), device=DEV)
    h_out, x_out = torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)
    for new, lens in (([9, 7, 4, 8, 0], [9, 7, 4, 0, 0]), ([1, 1, 0, 8, 20], [10, 8, 4, 8, 0]),
                      ([0, 0, 1, 0, 20], [10, 8, 5, 8, 20])):
        st.forward(h, _int(new), h_out, x_out)
        assert st.rows.seq_len.tolist() == lens, new
    st.close()
    st.qkv.close()


def _request_step(seed, n_requests, n_pages, n=N, **kw):
    """An attention step of n rows for n_requests requests of up to 9 pages of 4."""
    from lora_normal_form_amd import multiproj
    from synth import AdapterSpec, WorkloadSpec, make_workload
    d, lora, dora, ia3 = H * D, AdapterSpec("lora", rank=16, bias=True), AdapterSpec("dora", rank=16), AdapterSpec("ia3")
    ten = [(lora, lora, lora), (None, ia3, ia3), (dora, None, lora)]
    wls, tt = multiproj.projection_workloads(ten, n, d, (d, 2 * D, 2 * D), seed=seed)
    wl_out = make_workload(WorkloadSpec("out", "bf16", d, d, n, [lora, dora], assign="explicit",
                                        token_adapter=np.asarray(tt) % 3 - 1, seed=seed + 9))
    qkv = multiproj.QKVFused(wls, tt, len(ten))
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) / (D // 2))
    st = multiproj.AttentionStep(qkv, wl_out, H, 2, D, n_requests, 9, 4, n_pages, freq, **kw)
    return st, wls, wl_out


def _oracle_attention(st, q, k, v, seen):
    """Attention of each row over what its request has stored (lists of k and
    v rows, in the cache's type), in 64 bits: (out, bound) by _attend_ref."""
    kc = torch.zeros((N, 64, st.cache.n_kv_heads, D), dtype=BF16)
    vc = torch.zeros_like(kc)
    lens = []
    for i, r in enumerate(seen):
        lens.append(len(k[r]) if r >= 0 else 0)
        for t in range(lens[-1]):
            kc[i, t], vc[i, t] = k[r][t], v[r][t]
    table = torch.arange(N, dtype=torch.int32)[:, None]
    return _attend_ref(q, kc, vc, table, lens, range(N), 0, 1 / math.sqrt(D))


@pytest.mark.parametrize("one_each, captured", [(False, False), (True, False), (False, True), (True, True)])
def test_step_reads_its_own_request(one_each, captured):
    """Every row's attention is over what its own request stored, whatever
    requests before it ended, rested or found no page (a record of each
    request's keys and values is kept here, by request and not by row)."""
    st, *_ = _request_step(93, N, 40, one_each=one_each)
    g = torch.Generator().manual_seed(3)
    k, v, held = [[] for _ in range(N)], [[] for _ in range(N)], 0
    rng = np.random.default_rng(4)
    h, new_d = torch.zeros((N, H * D), device=DEV), _int(np.zeros(N))
    h_out, x_out = torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)
    if captured:
        st.forward(h, new_d, h_out, x_out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st.forward(h, new_d, h_out, x_out)
    for step in range(9):
        new = np.where(rng.random(N) < 0.25, np.where(rng.random(N) < 0.5, -1, 0), 1) if step else np.ones(N, int)
        h.copy_(torch.randn((N, H * D), generator=g))
        new_d.copy_(_int(new))
        if captured and step % 4 != 2:
            graph.replay()
        else:
            st.forward(h, new_d, h_out, x_out)
        torch.cuda.synchronize()
        seen, slot = st.rows.req.tolist(), st.rows.slot.tolist()
        for r in range(N):
            if new[r] < 0:
                k[r], v[r] = [], []
        for i, r in enumerate(seen):
            if r < 0:
                continue
            assert new[r] == 1 and (not one_each or i == r)
            at = divmod(slot[i], st.cache.page_size)
            k[r].append(st.cache.k[at].cpu())
            v[r].append(st.cache.v[at].cpu())
        assert [len(x) for x in k] == st.rows.seq_len.tolist()
        assert [len(x) for x in k] != [step + 1] * N or step == 0
        ref, tol = _oracle_attention(st, st.q_rot, k, v, seen)
        _close(st.a, ref, tol, f"attention, step {step}")
    st.close()
    st.qkv.close()


def test_step_refused_on_its_way_may_come_again():
    """A call that is turned away by a later operator's checks has not moved
    the requests on."""
    st, *_ = _request_step(95, 5, 30)
    h = torch.randn((N, H * D), generator=torch.Generator().manual_seed(1)).to(DEV)
    good, x_out = torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)
    st.forward(h, _int([3, 4, 0, 5, 1]), good, x_out)
    for args, kw in (((good.to(BF16), x_out), {}), ((good, x_out[:5]), {}), ((good, None), {}),
                     ((good, x_out), dict(gate=h.to(BF16))), ((good, x_out), dict(pos=torch.zeros(3, N, device=DEV)))):
        with pytest.raises(ValueError):
            st.forward(h, _int([2, -1, 6, 1, 0]), *args, **kw)
    st.forward(h, _int([2, -1, 6, 1, 0]), good, x_out)
    assert st.rows.seq_len.tolist() == [5, 0, 6, 6, 1]
    # 5 pages were taken, then 3 and one given back
    assert st.rows.cursor.tolist() == [5 + 3, 30 + 1], st.rows.cursor.tolist()
    st.close()
    st.qkv.close()


@pytest.mark.parametrize("how", ["tenants", "captured", "plans"])
def test_step_runs_rows_under_their_requests_adapters(how):
    """With `tenants`, or plans made for the step, a row's adapters are its
    request's, whichever row it is: requests that rest, end, bring prompts, and
    one that changes hands."""
    ids = np.array([[0, 1, 2, 4, -1], [0, 2, -1, 1, 1]])
    st, wls, wl_out, *_ = _step(97, **({} if how == "plans" else dict(tenants=_int(ids))))
    g = torch.Generator().manual_seed(9)
    h, new_d = torch.zeros((N, H * D), device=DEV), _int(np.zeros(5))
    h_out, x_out = torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)
    st.forward(h, new_d, h_out, x_out)
    graph = torch.cuda.CUDAGraph()
    if how == "captured":
        with torch.cuda.graph(graph):
            st.forward(h, new_d, h_out, x_out)
    for step, new in enumerate(([9, 0, 1, 2, 5], [0, 6, 1, 0, 1], [1, -1, 0, 1, 1], [-1, 3, 1, 12, 2], [4, 1, 1, 1, 1])):
        if step == 3:
            ids[:, 1] = (3, 0)
            if how != "plans":
                st.tenants[:, 1] = _int(ids[:, 1])
        h.copy_(torch.randn((N, H * D), generator=g))
        new_d.copy_(_int(new))
        want = np.repeat(np.arange(5), np.maximum(0, new))
        ten = np.concatenate([ids[:, want], np.full((2, N - len(want)), -1)], 1)
        if how == "plans":
            plans = st.qkv.layer.plan(ten[0]), st.out.layer.plan(ten[1])
            st.forward(h, new_d, h_out, x_out, plans=plans)
        elif how == "captured" and step != 2:
            graph.replay()
        else:
            st.forward(h, new_d, h_out, x_out)
        torch.cuda.synchronize()
        req = st.rows.req.cpu().numpy()
        assert np.array_equal(req[req >= 0], want)
        c0 = 0
        for wl, of in wls:
            wl = dataclasses.replace(wl, token_adapter=np.array([of.get(t, -1) for t in ten[0].tolist()]))
            _bar(wl, st.qkv.x.cpu().double().numpy(), st.qkv.y[:, c0:c0 + wl.d_out].cpu().double().numpy())
            c0 += wl.d_out
        _bar(dataclasses.replace(wl_out, token_adapter=ten[1]), st.out.x.cpu().double().numpy(),
             st.out.y.cpu().double().numpy())
    short = st.qkv.layer.plan(ten[0][:5]), st.out.layer.plan(ten[1])
    lens = st.rows.seq_len.tolist()
    with pytest.raises(ValueError, match="plans"):
        st.forward(h, new_d, h_out, x_out, plans=short)
    with pytest.raises(scute.ScuteError):  # (each plan belongs to its layer)
        st.forward(h, new_d, h_out, x_out, plans=(st.out.batch, st.qkv.batch))
    st.forward(h, _int([0] * 5), h_out, x_out)
    assert st.rows.seq_len.tolist() == lens
    with pytest.raises(ValueError, match="tenants"):
        _step(97, tenants=_int(ids[:, :4]))
    st.close()
    st.qkv.close()


def test_steps_take_turns_on_one_cache():
    """A step with rows for prompts and a one_each step on the same requests:
    each goes on from what the other stored."""
    prompts, *_ = _request_step(101, 5, 40)
    decode, *_ = _request_step(103, 5, 40, n=5, one_each=True, like=prompts)
    g, lens = torch.Generator().manual_seed(2), np.zeros(5, int)
    graph, h5, new5 = torch.cuda.CUDAGraph(), torch.zeros((5, H * D), device=DEV), _int(np.zeros(5))
    outs = torch.empty_like(h5), torch.empty((5, H * D), dtype=BF16, device=DEV)
    decode.forward(h5, new5, *outs)
    with torch.cuda.graph(graph):
        decode.forward(h5, new5, *outs)
    for st, new in ((prompts, [9, 7, 0, 8, 0]), (decode, [1, 1, 0, 1, 0]), (decode, [1, -1, 0, 1, 0]),
                    (prompts, [0, 12, 6, 1, 0]), (decode, [1, 1, 1, 1, 1]), (decode, [0, 1, -1, 1, 1]),
                    (prompts, [1, 1, 20, 0, 1]), (decode, [1, 1, 1, 1, 1])):
        n = st.q_rot.shape[0]
        h = torch.randn((n, H * D), generator=g).to(DEV)
        if st is decode:
            h5.copy_(h)
            new5.copy_(_int(new))
            graph.replay()
        else:
            st.forward(h, _int(new), torch.empty_like(h), torch.empty((n, H * D), dtype=BF16, device=DEV))
        torch.cuda.synchronize()
        rows = [(r, lens[r] + i + 1) for r in range(5) for i in range(new[r])]
        if st is decode:
            rows = [(r, lens[r] + 1 if new[r] == 1 else 0) for r in range(5)]
        lens = np.where(np.array(new) < 0, 0, lens + np.maximum(0, new))
        assert st.rows.seq_len.tolist() == lens.tolist()
        rows += [(-1, 0)] * (n - len(rows))
        ref, tol = _attend_ref(st.q_rot, st.cache.k, st.cache.v, st.table, [x for _, x in rows], [r for r, _ in rows], 0,
                               1 / math.sqrt(D))
        _close(st.a, ref, tol, "attention")
        # (the newest key of every row is the one that the step just turned: in its place, not another's)
        for i, (r, x) in enumerate(rows):
            if x:
                at = divmod(x - 1, 4)
                k = st.cache.k[int(st.table[r, at[0]]), at[1]]
                v = st.cache.v[int(st.table[r, at[0]]), at[1]]
                assert torch.equal(v, st.v[i].to(BF16)) and bool(torch.isfinite(k.float()).all())
    with pytest.raises(ValueError, match="like"):
        _request_step(103, 5, 41, n=5, one_each=True, like=prompts)
    for st in (decode, prompts):
        st.close()
        st.qkv.close()


def test_step_is_ready_on_every_stream(monkeypatch):
    """What a step made behind a stream's work keeps is there by the time the
    step is: its requests' adapters, lengths and pages."""
    ids = np.array([[0, 1, 2, 4, -1], [0, 2, -1, 1, 1]])
    side, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    made = block.ResidualNorm

    def behind_work(*a, **kw):
        nonlocal busy
        for _ in range(20):
            busy = torch.mm(busy, busy).clamp_(-1, 1)
        return made(*a, **kw)

    monkeypatch.setattr(block, "ResidualNorm", behind_work)
    with torch.cuda.stream(side):
        st, *_ = _step(105, tenants=torch.tensor(ids, dtype=torch.int32))
    got = st.tenants.cpu(), st._ids[:, 0].cpu(), st.state.cpu(), st.ring.cpu()
    assert np.array_equal(got[0].numpy(), ids) and bool((got[1] == -1).all())
    assert got[2].tolist() == [0, 30, 0, 0, 0] and got[3].tolist() == list(range(30))
    torch.cuda.synchronize()
    st.close()
    st.qkv.close()

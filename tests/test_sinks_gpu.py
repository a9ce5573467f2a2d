"""Attention with a window and first positions that stay visible
(PagedAttention(window=, sinks=)) against the formula in 64 bits. Tolerances are
those of test_block_gpu: roundings, counted."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402
from test_block_gpu import BF16, DEV, F32, U, _attend_case, _close, _int  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def attend_ref(q, kc, vc, table, lens, req, seen, scale, weight=U[BF16] ** 2):
    """(out, its bound) in 64 bits; seen(i, n): the positions of row i, of length
    n; those whose page is not in the cache are not seen. The bound is that of
    test_block_gpu._attend_ref; weight: how far off a weight of a bf16 cache is."""
    q, kc, vc, table = q.cpu().double(), kc.cpu(), vc.cpu(), table.cpu()
    dt = kc.dtype
    N, H, D = q.shape
    n_pages, ps, Hk, _ = kc.shape
    R, P = table.shape
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(N):
        r = int(req[i])
        n = min(int(lens[i]), P * ps) if 0 <= r < R else 0
        t = seen(i, n) if n > 0 else torch.zeros(0, dtype=torch.int64)
        page = table[r, t // ps].long() if len(t) else t
        ok = (page >= 0) & (page < n_pages)
        t, page = t[ok], page[ok]
        if not len(t):
            continue
        K = kc[page, t % ps].double().transpose(0, 1).contiguous()  # [Hk][n][D]
        V = vc[page, t % ps].double().transpose(0, 1).contiguous()
        qi = q[i].view(Hk, H // Hk, D)
        p = torch.softmax((qi @ K.transpose(1, 2)) * scale, -1)
        o, mag = p @ V, p @ V.abs()
        off = (qi.abs() @ K.transpose(1, 2).abs()).amax(-1, keepdim=True) * abs(scale) * (D + 3) * U[F32]
        rel = 4 * off + (2 * len(t) + 16) * U[F32]
        b = (rel + (weight if dt == BF16 else 0.0)) * mag + U[dt] * (o.abs() + 2 * rel * mag)
        out[i], tol[i] = o.reshape(H, D), b.reshape(H, D)
    return out, tol


def close(got, want, tol, what):
    """_close, infinities equal where the formula has them."""
    inf = torch.isinf(want)
    assert torch.equal(got.cpu().double()[inf], want[inf]), what
    _close(torch.where(inf.to(got.device), 0.0, got), torch.where(inf, 0.0, want), torch.where(inf, 0.0, tol), what)


def visible(window, sinks):
    def seen(i, n):
        t = torch.arange(n)
        return t[(t < sinks) | (t >= n - window)] if window > 0 else t
    return seen


def run(kc, vc, table, q, lens, window, sinks, req=None):
    att = block.PagedAttention(block.KVCache(kc, vc), q.shape[1], window=window, sinks=sinks)
    buf = torch.full((q.shape[0] + 1, q.shape[1], q.shape[2]), 55.0, dtype=q.dtype, device=DEV)
    out = att.forward(q, table, _int(lens), buf[:-1], row_req=None if req is None else _int(req))
    torch.cuda.synchronize()
    assert bool((buf[-1] == 55.0).all())
    ref, tol = attend_ref(q, kc, vc, table, lens, range(len(lens)) if req is None else req, visible(window, sinks),
                          1 / math.sqrt(q.shape[2]))
    close(out, ref, tol, "out")
    return out


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("window, sinks", [(1, 1), (7, 4), (31, 33), (64, 1), (100, 16), (100, 50), (5000, 4), (40, 5000),
                                           (128, 200), (3, 96), (0, 4), (50, 0)])
@pytest.mark.parametrize("ps", [16, 5])
def test_windows_and_sinks(dt, window, sinks, ps):
    lens = [1, 3, 4, 5, 40, 100, 101, 135, 500, 0, 511, 64, 96, 300]
    kc, vc, table, q = _attend_case(window + sinks, lens, -(-512 // ps), ps, 4, 2, 64, dt)
    run(kc, vc, table, q, lens, window, sinks)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D, Hq, Hk, ps, by_head", [
    (128, 32, 8, 16, False), (128, 32, 8, 16, True), (256, 4, 2, 16, False), (8, 5, 1, 16, False), (80, 12, 4, 5, False),
    (72, 6, 2, 1, True), (96, 17, 1, 48, False), (136, 40, 2, 7, False), (192, 3, 1, 64, True), (248, 2, 2, 100, False),
    (128, 32, 1, 16, False), (64, 33, 1, 16, True), (256, 100, 2, 6, False)])
def test_shapes(dt, D, Hq, Hk, ps, by_head):
    lens = [1, 0, 2, 17, 31, 64, 65, 130, 400, 333]
    kc, vc, table, q = _attend_case(D + Hq, lens, -(-400 // ps), ps, Hq, Hk, D, dt, by_head)
    run(kc, vc, table, q, lens, 70, 9)


@pytest.mark.parametrize("dt, Hq, Hk, D, lens, window, sinks", [
    (BF16, 8, 2, 128, [5000], 3000, 700), (BF16, 1, 1, 64, [9000, 1], 4000, 4), (F32, 4, 1, 128, [3000, 0, 2999], 1500, 64),
    (BF16, 16, 1, 256, [4097], 2500, 1000), (BF16, 20, 1, 64, [2048] * 3, 900, 5), (BF16, 80, 2, 128, [6000, 17, 4001], 3500, 40)])
def test_long(dt, Hq, Hk, D, lens, window, sinks):
    """A few rows over long windows: the work is split over the length."""
    kc, vc, table, q = _attend_case(len(lens), lens, -(-max(lens) // 16), 16, Hq, Hk, D, dt)
    run(kc, vc, table, q, lens, window, sinks)


@pytest.mark.parametrize("dt, Hq, Hk, D, ps, window, sinks", [
    (BF16, 4, 4, 128, 16, 30, 4), (BF16, 4, 2, 64, 16, 17, 33), (BF16, 6, 2, 80, 5, 20, 7), (F32, 6, 2, 80, 5, 30, 16),
    (F32, 4, 1, 256, 16, 9, 40), (BF16, 8, 2, 256, 48, 33, 2), (BF16, 33, 3, 64, 16, 20, 5), (BF16, 5, 1, 96, 16, 40, 3)])
def test_rows_of_one_request(dt, Hq, Hk, D, ps, window, sinks):
    """Runs of one to seven rows; a NaN that only the longest row of a run sees
    stays with it, one between the sinks and every window with none."""
    req = [0, 0, 0, 0, 0, 1, 1, 2, 3, 3, 3, -1, -1, 4, 4, 9, 4, 4, 5, 5, 5, 5, 5, 5, 5]
    lens = [100, 101, 102, 103, 104, 33, 32, 64, 0, 1, 2, 50, 0, 130, 7, 9, 70, 70, 60, 61, 62, 63, 64, 65, 66]
    kc, vc, table, _ = _attend_case(D + ps, [0] * 6, -(-140 // ps), ps, Hq, Hk, D, dt)
    q = torch.randn((len(req), Hq, D), generator=torch.Generator().manual_seed(1)).to(DEV, dt)
    run(kc, vc, table, q, lens, window, sinks, req=req)
    for r, n in ((0, 104), (5, 66), (4, 130)):
        page, at = int(table[r, (n - 1) // ps]), (n - 1) % ps
        vc[page, at, :, 3:5] = torch.tensor([float("nan"), float("inf")], device=DEV)
        kc[page, at, 0, 1] = float("nan")
    at = 50  # below every window of request 0, past its sinks
    vc[int(table[0, at // ps]), at % ps] = float("nan")
    out = run(kc, vc, table, q, lens, window, sinks, req=req)
    assert bool(torch.isfinite(out[:4]).all()) and bool(torch.isnan(out[4, 0]).any())


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("ps", [16, 32, 5])
@pytest.mark.parametrize("dropped", [False, True])
def test_between_sinks_and_window_may_be_anything(dt, ps, dropped):
    """Infinities and NaN between them, behind the length and in pages of no
    request; or those pages are not there."""
    lens, window, sinks = [200, 150, 90, 201, 77], 60, 13
    P = -(-210 // ps)
    kc, vc, table, q = _attend_case(ps, lens, P, ps, 6, 2, 64, dt)
    used = torch.zeros((kc.shape[0], ps), dtype=torch.bool)
    tab = table.cpu()
    for r, n in enumerate(lens):
        t = visible(window, sinks)(r, n)
        used[tab[r, t // ps].long(), t % ps] = True
        if dropped:
            low = n - window
            c = torch.arange(P)
            tab[r, (c * ps >= sinks) & ((c + 1) * ps <= low)] = -1
    table = tab.to(DEV)
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        k2, v2 = kc.clone(), vc.clone()
        k2[~used.to(DEV)] = bad
        v2[~used.to(DEV)] = bad
        out = run(k2, v2, table, q, lens, window, sinks)
        assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("place", [2, 12, 150, 199])
@pytest.mark.parametrize("Hq", [4, 24])
def test_infinities_that_are_seen_stay(place, Hq):
    """An infinite V at a sink or in the window gives infinities, not NaN."""
    kc, vc, table, q = _attend_case(3, [200], 13, 16, Hq, 1, 128, BF16)
    vc[int(table[0, place // 16]), place % 16, 0, 7] = float("inf")
    vc[int(table[0, place // 16]), place % 16, 0, 9] = -float("inf")
    out = run(kc, vc, table, q, [200], 60, 13)
    assert bool((out[0, :, 7] == float("inf")).all()) and bool((out[0, :, 9] == -float("inf")).all())
    assert int((~torch.isfinite(out)).sum()) == 2 * Hq


def test_scores_that_are_masked_keep_nothing_of_the_type_s_lowest():
    """Scores as low as fp32 goes (large K and q of opposite sign) are still seen."""
    kc, vc, table, q = _attend_case(4, [100], 7, 16, 2, 1, 64, F32)
    kc.fill_(-1e17), q.fill_(1e17)
    run(kc, vc, table, q, [100], 20, 5)


def test_many_rows_and_repeats_bit_by_bit():
    rng = np.random.default_rng(6)
    N, R, ps = 700, 7, 16
    kc, vc, table, _ = _attend_case(1, [0] * R, 60, ps, 4, 2, 64, BF16)
    lens, req = rng.integers(0, 900, size=N), np.sort(rng.integers(-1, R + 1, size=N))
    q = torch.randn((N, 4, 64), generator=torch.Generator().manual_seed(2)).to(DEV, BF16)
    a = run(kc, vc, table, q, lens.tolist(), 100, 20, req=req.tolist()).clone()
    att = block.PagedAttention(block.KVCache(kc, vc), 4, window=100, sinks=20)
    for _ in range(3):
        assert torch.equal(att.forward(q, table, _int(lens), torch.empty_like(q), row_req=_int(req)), a)


def test_captured_and_on_another_stream():
    ps, R = 16, 5
    kc, vc, table, q = _attend_case(9, [0] * R, 20, ps, 8, 2, 128, BF16)
    att = block.PagedAttention(block.KVCache(kc, vc), 8, window=50, sinks=4)
    lens, out, s, g = _int([0] * R), torch.empty_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        att.forward(q, table, lens, out)
    for step in range(4):
        n = [int(x) for x in np.random.default_rng(step).integers(0, 320, size=R)]
        lens.copy_(_int(n))
        q.normal_()
        g.replay()
        torch.cuda.synchronize()
        ref, tol = attend_ref(q, kc, vc, table, n, range(R), visible(50, 4), 1 / math.sqrt(128))
        _close(out, ref, tol, f"replay {step}")
        other = torch.empty_like(out)
        att.forward(q, table, lens, other, stream=s)
        s.synchronize()
        assert torch.equal(out, other)


def test_refusals():
    kc, vc, table, q = _attend_case(1, [4], 2, 4, 2, 1, 8, F32)
    with pytest.raises(ValueError):
        block.PagedAttention(block.KVCache(kc, vc), 2, window=4, sinks=-1)
    att = block.PagedAttention(block.KVCache(kc, vc), 2, window=4, sinks=1)
    att.sinks = -1
    with pytest.raises(scute.ScuteError) as e:
        att.forward(q, table, _int([4]), torch.empty_like(q))
    assert e.value.code == scute.E_SHAPE


@pytest.mark.parametrize("dt, D, ps", [(BF16, 128, 16), (F32, 64, 16), (BF16, 40, 5)])
def test_prompts(dt, D, ps):
    """Hundreds of new tokens a request, from its first on and behind others."""
    g, P = torch.Generator().manual_seed(D), -(-1100 // ps)
    kc, vc = (torch.randn((2 * P, ps, 2, D), generator=g).to(DEV, dt) for _ in range(2))
    table = torch.randperm(2 * P, generator=g).view(2, P)
    req = np.repeat([0, 1], 400)
    lens = np.concatenate([1 + np.arange(400), 700 + np.arange(400)])
    q = torch.randn((800, 8, D), generator=g).to(DEV, dt)
    run(kc, vc, _int(table), q, lens, 130, 21, req=req)

"""Attention of rows whose contexts begin with the same positions
(block.SharedAttention) against the formula in 64 bits.

Tolerances are those of test_block_gpu, roundings counted, but for a bf16 cache's
weights over shared positions: the first of their two parts is cut off after 8
bits (2^-7 of the weight at most), the second is what remains, rounded (2^-8 of
it), and 2^-20 of the weight: 2^-15 + 2^-20 in all."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block  # noqa: E402
from test_block_gpu import BF16, DEV, F32, _cache_tensors, _int  # noqa: E402
from test_sinks_gpu import attend_ref, close  # noqa: E402

pytestmark = pytest.mark.gpu
WEIGHT = 2.0 ** -15 + 2.0 ** -20


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def everything(i, n):
    return torch.arange(n)


def make(seed, groups, ps, Hq, Hk, D, dt, by_head=False, outside=0, suffix=40):
    """groups: (requests, shared positions) each. Requests of a group share the
    pages of its positions (a last page that is not full with them, too: then
    their own positions there are the same as well, until they leave it), the
    `outside` last requests share nothing. Returns the tensors and the requests'
    lengths."""
    rng = np.random.default_rng(seed)
    R = sum(n for n, _ in groups) + outside
    P = -(-(max([s for _, s in groups] + [1]) + suffix) // ps) + 1
    pages = iter(rng.permutation(R * P + 5))
    table = np.full((R, P), -1)
    lens, r = np.zeros(R, np.int64), 0
    for n, shared in list(groups) + [(1, 0)] * outside:
        first = [next(pages) for _ in range(-(-shared // ps))]
        for _ in range(n):
            own = int(rng.integers(0, suffix + 1))
            lens[r] = shared + own if shared % ps == 0 else shared + min(own, ps - shared % ps)
            held = -(-int(lens[r]) // ps)
            table[r, :len(first)] = first
            table[r, len(first):held] = [next(pages) for _ in range(max(0, held - len(first)))]
            r += 1
    kc, vc = _cache_tensors(R * P + 5, ps, Hk, D, dt, by_head, seed)
    q = torch.randn((R, Hq, D), generator=torch.Generator().manual_seed(seed)).to(DEV, dt)
    return kc, vc, table, q, lens


def run(kc, vc, table, q, lens, offsets, shared, req=None, scale=None, again=True, always=True):
    att = block.SharedAttention(block.KVCache(kc, vc), q.shape[1], q.shape[0], max(1, len(shared)), scale=scale,
                                always=always)
    buf = torch.full((q.shape[0] + 1, q.shape[1], q.shape[2]), 55.0, dtype=q.dtype, device=DEV)
    tab, rl = _int(table), _int(lens)
    rr = None if req is None else _int(req)
    out = att.forward(q, tab, rl, _int(offsets), _int(shared), buf[:-1], row_req=rr)
    torch.cuda.synchronize()
    assert bool((buf[-1] == 55.0).all())
    ref, tol = attend_ref(q, kc, vc, tab, lens, range(len(lens)) if req is None else req, everything,
                          1 / math.sqrt(q.shape[2]) if scale is None else scale, weight=WEIGHT)
    close(out, ref, tol, "out")
    if again:  # the workspace is as it was: the same bits again
        two = att.forward(q, tab, rl, _int(offsets), _int(shared), torch.empty_like(q), row_req=rr)
        assert torch.equal(out.view(torch.int16 if out.dtype == BF16 else torch.int32),
                           two.view(torch.int16 if out.dtype == BF16 else torch.int32))
    return out


def offsets_of(groups):
    return np.concatenate([[0], np.cumsum([n for n, _ in groups])])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D, Hq, Hk, ps, by_head", [
    (128, 32, 8, 16, False), (128, 32, 8, 16, True), (64, 8, 8, 32, False), (256, 4, 2, 16, False), (8, 5, 1, 16, False),
    (80, 12, 4, 5, False), (72, 6, 2, 1, True), (96, 17, 1, 48, False), (136, 40, 2, 7, False), (192, 3, 1, 64, True),
    (248, 2, 2, 100, False), (128, 32, 1, 16, False), (64, 33, 1, 16, True), (256, 100, 2, 6, False), (40, 150, 1, 1, False)])
def test_shapes(dt, D, Hq, Hk, ps, by_head):
    groups = [(3, 4 * ps), (1, 70 // ps * ps), (0, 9), (6, 3), (2, 0), (5, 2 * ps + ps // 2)]
    kc, vc, table, q, lens = make(D + Hq, groups, ps, Hq, Hk, D, dt, by_head, outside=2)
    run(kc, vc, table, q, lens, offsets_of(groups), [n for _, n in groups])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows, shared", [(1, 1), (1, 5000), (2, 3000), (33, 1600), (130, 512), (64, 4096), (7, 63), (7, 65)])
def test_one_group(dt, rows, shared):
    """Prefixes cut over many work-groups, or one unit of them."""
    groups = [(rows, shared // 16 * 16 if shared > 100 else shared)]
    kc, vc, table, q, lens = make(rows, groups, 16, 8, 2, 64, dt)
    run(kc, vc, table, q, lens, [0, rows], [groups[0][1]])


@pytest.mark.parametrize("n_groups", [255, 257, 700])
def test_many_groups(n_groups):
    """More groups than a work-group has threads; some without rows."""
    rng = np.random.default_rng(n_groups)
    groups = [(int(rng.integers(0, 3)), 4 * int(rng.integers(0, 30))) for _ in range(n_groups)]
    kc, vc, table, q, lens = make(n_groups, groups, 4, 2, 1, 16, BF16, outside=3)
    run(kc, vc, table, q, lens, offsets_of(groups), [n for _, n in groups])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("Hq, Hk, D, ps", [(8, 2, 64, 16), (6, 3, 128, 5), (20, 1, 96, 16)])
def test_rows_that_see_less(dt, Hq, Hk, D, ps):
    """Several rows of a request, rows of no request, empty ones, rows that end
    inside the shared positions, and rows of no group before and after them."""
    groups = [(4, 40 * ps // ps // ps * ps), (5, 130 // ps * ps)]
    kc, vc, table, _, lens_r = make(D + ps, groups, ps, Hq, Hk, D, dt, outside=2)
    req = [9, 0, 0, 0, 1, 2, 2, -1, 3, 4, 4, 5, -1, 6, 7, 7, 7, 8, 8, 10, 10, 99]
    lens = [lens_r[r] - j if 0 <= r < len(lens_r) else 50 for j, r in zip([0, 2, 1, 0, 0, 1, 0, 0, 0, 1, 0, 0, 0, 0, 2, 1, 0, 0, 0, 1, 0, 0], req)]
    lens[8], lens[11], lens[13], lens[17] = 17, 0, 33, 1
    q = torch.randn((len(req), Hq, D), generator=torch.Generator().manual_seed(4)).to(DEV, dt)
    offsets = [1, 9, 19]
    run(kc, vc, table, q, np.maximum(lens, 0), offsets, [n for _, n in groups], req=req)
    # rows of a group none of which sees anything
    none = np.array(lens)
    none[1:9] = 0
    run(kc, vc, table, q, none, offsets, [n for _, n in groups], req=req)
    # and what only the longer rows of a group see is not finite
    page, at = int(table[6, 100 // ps]), 100 % ps
    vc[page, at, :, 3:5] = torch.tensor([float("nan"), float("inf")], device=DEV)
    kc[page, at, 0, 1] = float("nan")
    out = run(kc, vc, table, q, np.maximum(lens, 0), offsets, [n for _, n in groups], req=req)
    assert bool(torch.isfinite(out[13]).all()) and bool(torch.isnan(out[14]).any())


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("ps", [16, 5])
def test_what_nobody_sees_may_be_anything(dt, ps):
    groups = [(5, 20 * ps), (3, 6 * ps)]
    kc, vc, table, q, lens = make(ps, groups, ps, 6, 2, 64, dt, outside=1)
    used = torch.zeros((kc.shape[0], ps), dtype=torch.bool)
    for r, n in enumerate(lens):
        t = torch.arange(int(n))
        used[torch.tensor(table[r])[t // ps], t % ps] = True
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        k2, v2 = kc.clone(), vc.clone()
        k2[~used.to(DEV)] = bad
        v2[~used.to(DEV)] = bad
        out = run(k2, v2, table, q, lens, [0, 5, 8], [20 * ps, 6 * ps])
        assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("dt", [BF16, F32])
def test_pages_that_are_not_there(dt):
    """Shared positions whose page is outside the cache are not seen."""
    kc, vc, table, q, lens = make(3, [(9, 200)], 8, 4, 1, 64, dt)
    for c, bad in ((3, -1), (7, kc.shape[0]), (24, 1 << 30)):
        table[:, c] = bad
    run(kc, vc, table, q, lens, [0, 9], [200])
    table[:, :25] = -1  # none of them
    run(kc, vc, table, q, lens, [0, 9], [200])


@pytest.mark.parametrize("place", [0, 40, 1999, 2003])
def test_infinities_that_are_seen_stay(place):
    kc, vc, table, q, lens = make(3, [(6, 2000)], 16, 4, 1, 128, BF16)
    lens[:] = 2010
    table[:, 125] = table[0, 125] if table[0, 125] >= 0 else 0
    page = int(table[0, place // 16])
    vc[page, place % 16, 0, 7], vc[page, place % 16, 0, 9] = float("inf"), -float("inf")
    out = run(kc, vc, table, q, lens, [0, 6], [2000])
    assert bool((out[:, :, 7] == float("inf")).all()) and bool((out[:, :, 9] == -float("inf")).all())
    assert int((~torch.isfinite(out)).sum()) == 2 * 24


def test_scales_of_any_sign_and_large_scores():
    kc, vc, table, q, lens = make(5, [(9, 320)], 16, 4, 2, 64, BF16)
    for scale in (-0.3, 0.0, 2.0):
        run(kc, vc, table, q, lens, [0, 9], [320], scale=scale)


def test_lengths_past_the_table():
    kc, vc, table, q, lens = make(5, [(4, 64)], 16, 4, 2, 64, F32, suffix=20)
    P = table.shape[1]
    table[:, 4:] = table[0, 0]
    lens[:] = [P * 16 + 9, 1 << 30, 64, P * 16]
    run(kc, vc, table, q, lens, [0, 4], [1 << 30])
    run(kc, vc, table, q, lens, [0, 4], [64])


@pytest.mark.parametrize("offsets", [[0, 12, 0, 12, 0, 12], [5, 3, 20, -4, 12, 1 << 30], [12, 12, 12, 12, 12, 12], [-9] * 6])
def test_offsets_that_do_not_ascend_stay_in_bounds(offsets):
    """What such rows give is not said; nothing else is written, and the next
    call is right."""
    kc, vc, table, q, lens = make(6, [(12, 400)], 8, 8, 2, 64, BF16)
    att = block.SharedAttention(block.KVCache(kc, vc), 8, 12, 5, always=True)
    n = att.workspace.shape[0]
    wide = torch.full((n + (1 << 20),), 77, dtype=torch.uint8, device=DEV)
    wide[:n] = 0
    assert wide.data_ptr() % 256 == 0
    att.workspace = wide[:n]
    buf = torch.full((14, 8, 64), 55.0, dtype=BF16, device=DEV)
    k0, v0 = kc.clone(), vc.clone()
    att.forward(q, _int(table), _int(lens), _int(offsets), _int([400] * 5), buf[1:13])
    torch.cuda.synchronize()
    assert bool((wide[n:] == 77).all()) and bool((buf[0] == 55.0).all()) and bool((buf[13] == 55.0).all())
    assert torch.equal(k0, kc) and torch.equal(v0, vc)
    out = att.forward(q, _int(table), _int(lens), _int([0, 12]), _int([400]), torch.empty_like(q))
    ref, tol = attend_ref(q, kc, vc, _int(table), lens, range(12), everything, 1 / 8, weight=WEIGHT)
    close(out, ref, tol, "after")


def test_captured_steps():
    """One captured call: lengths, groups and queries change between replays."""
    ps, N = 16, 24
    kc, vc, table, q, _ = make(7, [(24, 320)], ps, 8, 2, 128, BF16, suffix=60)
    table = table.copy()
    rng = np.random.default_rng(1)
    free = np.setdiff1d(np.arange(kc.shape[0]), table)
    table[:, 20:] = rng.choice(free, size=table[:, 20:].shape)
    att = block.SharedAttention(block.KVCache(kc, vc), 8, N, 3, always=True)
    tab, lens, offs, shared = _int(table), _int(np.zeros(N)), _int([0] * 4), _int([0] * 3)
    out, s, g = torch.empty_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        att.forward(q, tab, lens, offs, shared, out)
    for step in range(6):
        n = rng.integers(0, 380, size=N)
        o = np.sort(rng.integers(0, N + 1, size=4))
        sh = rng.integers(0, 21, size=3) * ps
        lens.copy_(_int(n)), offs.copy_(_int(o)), shared.copy_(_int(sh)), q.normal_()
        g.replay()
        torch.cuda.synchronize()
        ref, tol = attend_ref(q, kc, vc, tab, n, range(N), everything, 1 / math.sqrt(128), weight=WEIGHT)
        close(out, ref, tol, f"replay {step}")
        other = torch.empty_like(out)
        att.forward(q, tab, lens, offs, shared, other, stream=s)
        s.synchronize()
        assert torch.equal(out, other)


def test_without_groups_nothing_is_shared():
    kc, vc, table, q, lens = make(8, [(5, 96)], 16, 8, 2, 64, BF16)
    outs = [run(kc, vc, table, q, lens, offs, shared) for offs, shared in (([0], []), ([0, 5], [0]), ([0, 5], [-7]), ([2, 2], [96]))]
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_calls_that_share_little():
    """Without `always` the rows are read one by one: paged attention's bits. Calls
    of both kinds may follow each other with one workspace."""
    kc, vc, table, q, lens = make(9, [(30, 160)], 16, 8, 2, 64, BF16)
    paged = block.PagedAttention(block.KVCache(kc, vc), 8).forward(q, _int(table), _int(lens), torch.empty_like(q))
    assert torch.equal(run(kc, vc, table, q, lens, [0, 30], [160], always=False), paged)
    att = block.SharedAttention(block.KVCache(kc, vc), 8, 30, 1)
    outs = []
    for flags in (0, 1, 0, 1, 1, 0):
        att.flags = flags
        outs.append(att.forward(q, _int(table), _int(lens), _int([0, 30]), _int([160]), torch.empty_like(q)))
    assert torch.equal(outs[2], paged) and torch.equal(outs[5], paged)
    assert torch.equal(outs[1], outs[3]) and torch.equal(outs[1], outs[4])


def test_a_table_wide_enough_shares():
    """The rule itself takes the shared path: a wide table, 60 rows past one a group."""
    kc, vc, table, q, lens = make(10, [(61, 480)], 16, 8, 2, 64, BF16)
    wide = np.full((61, 560), -1)
    wide[:, :table.shape[1]] = table
    assert 60 * 560 * 16 * 2 * 2 * 64 * 2 > 256 << 20
    shares = run(kc, vc, wide, q, lens, [0, 61], [480], always=False)
    assert torch.equal(shares, run(kc, vc, wide, q, lens, [0, 61], [480]))


def test_refusals():
    kc, vc, table, q, lens = make(8, [(5, 96)], 16, 8, 2, 64, BF16)
    cache = block.KVCache(kc, vc)
    att = block.SharedAttention(cache, 8, 5, 1)
    ok = dict(q=q, table=_int(table), row_len=_int(lens), group=_int([0, 5]), shared_len=_int([96]), out=torch.empty_like(q))
    for kw in (dict(group=_int([0, 2, 5]), shared_len=_int([96, 96])), dict(group=_int([0])), dict(shared_len=torch.zeros(1, device=DEV)),
               dict(q=q.float()), dict(out=torch.empty_like(q).float()), dict(table=_int(table)[:3]), dict(row_len=_int(lens[:4])),
               dict(group=torch.tensor([0, 5], dtype=torch.int32)), dict(row_req=_int([0] * 4))):
        with pytest.raises(ValueError):
            att.forward(**{**ok, **kw})
    with pytest.raises(ValueError):
        block.SharedAttention(cache, 7, 5, 1)
    with pytest.raises(ValueError):
        small = block.SharedAttention(cache, 8, 4, 1)
        small.forward(**ok)


@pytest.mark.parametrize("dt, D, ps", [(BF16, 128, 16), (F32, 64, 16), (BF16, 40, 5)])
def test_prompts_behind_what_they_share(dt, D, ps):
    """Hundreds of new tokens a request, part of a prompt each."""
    kc, vc, table, _, lens_r = make(D, [(3, 40 * ps)], ps, 8, 2, D, dt, suffix=260)
    req = np.repeat([0, 1, 2], 250)
    lens = np.concatenate([np.maximum(0, n - 249 + np.arange(250)) for n in lens_r])
    q = torch.randn((750, 8, D), generator=torch.Generator().manual_seed(4)).to(DEV, dt)
    run(kc, vc, table, q, lens, [0, 750], [40 * ps], req=req)

"""Workspaces of attention over shared positions: one for caches of several head
sizes, paged calls between."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block  # noqa: E402
from test_block_gpu import BF16, DEV, F32, _int  # noqa: E402
from test_shared_gpu import WEIGHT  # noqa: E402
from test_sinks_gpu import attend_ref, close  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == BF16 else torch.int32), b.view(torch.int16 if b.dtype == BF16 else torch.int32))


def _workspace(n):
    w = torch.zeros(n, dtype=torch.uint8, device=DEV)
    assert w.data_ptr() % 256 == 0
    return w


def test_one_workspace_for_heads_of_several_sizes():
    """A workspace zeroed once serves caches of 64, 128 and 256 elements and paged
    calls in turn: the bits of handles of their own. The rows' own positions are
    more chunks than waves, so the counter of chunks is used."""
    N, H, Hq, L, ps = 64, 8, 128, 6000, 16
    g = torch.Generator().manual_seed(5)
    rng = np.random.default_rng(5)
    P = -(-L // ps) + 4
    table = _int(rng.integers(0, 300, size=(N, P)))  # (read only: pages may repeat)
    lens, none = _int(rng.integers(L - 200, L + 1, size=N)), _int([0, 3])
    calls = {}
    for D, dt in ((64, BF16), (128, BF16), (256, BF16), (64, F32), (256, F32)):
        kc, vc = (torch.randn((300, ps, H, D), generator=g).to(DEV, dt) for _ in range(2))
        q = torch.randn((N, Hq, D), generator=g).to(DEV, dt)
        cache = block.KVCache(kc, vc)
        shared, paged = block.SharedAttention(cache, Hq, N, 1, always=True), block.PagedAttention(cache, Hq)
        args = (q, table, lens, none, _int([32]))
        want = shared.forward(*args, torch.empty_like(q)), paged.forward(q, table, lens, torch.empty_like(q))
        calls[D, dt] = shared, paged, args, want
    torch.cuda.synchronize()
    one = _workspace(max(h.workspace.shape[0] for c in calls.values() for h in c[:2]))
    for shared, paged, *_ in calls.values():
        shared.workspace = paged.workspace = one
    keys = list(calls)
    for i in range(40):
        key = keys[int(rng.integers(0, len(keys)))]
        shared, paged, args, want = calls[key]
        q = args[0]
        if i % 3 == 2:
            same = _same(paged.forward(q, table, lens, torch.full_like(q, math.nan)), want[1])
        else:
            same = _same(shared.forward(*args, torch.full_like(q, math.nan)), want[0])
        assert same, (i, key)


def test_more_rows_and_heads_than_the_join_has_threads():
    """4500 rows of 64 heads of 256: the join's work-groups take several each."""
    N, H, D, ps = 4500, 64, 256, 16
    g = torch.Generator().manual_seed(6)
    rng = np.random.default_rng(6)
    kc, vc = (torch.randn((200, ps, 1, D), generator=g).to(DEV, BF16) for _ in range(2))
    q = torch.randn((N, H, D), device=DEV).to(BF16)
    table = rng.integers(0, 200, size=(N, 4))
    table[:, :2] = table[0, :2]
    lens = rng.integers(0, 65, size=N)
    att = block.SharedAttention(block.KVCache(kc, vc), H, N, 2, always=True)
    out = att.forward(q, _int(table), _int(lens), _int([0, 2000, N - 3]), _int([32, 30]), torch.full_like(q, math.nan))
    some = np.unique(np.concatenate([rng.integers(0, N, size=200), [0, 1999, 2000, N - 4, N - 3, N - 1]]))
    ref, tol = attend_ref(q[some], kc, vc, _int(table[some]), lens[some], range(len(some)), lambda i, n: torch.arange(n),
                          1 / math.sqrt(D), weight=WEIGHT)
    close(out[some], ref, tol, "rows")
    assert not bool(torch.isnan(out).any())


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("ps", [16, 5])
@pytest.mark.parametrize("by_request", [False, True])
def test_calls_smaller_than_their_handle(dt, ps, by_request):
    """One handle for 512 rows in 64 groups, in turn for calls of fewer, whose waves
    stand in other ways; nothing behind its workspace is written."""
    H, Hk, D = 8, 2, 64
    g = torch.Generator().manual_seed(ps)
    rng = np.random.default_rng(ps)
    kc, vc = (torch.randn((900, ps, Hk, D), generator=g).to(DEV, dt) for _ in range(2))
    att = block.SharedAttention(block.KVCache(kc, vc), H, 512, 64, always=True)
    n = att.workspace.shape[0]
    wide = torch.full((n + (1 << 20),), 77, dtype=torch.uint8, device=DEV)
    wide[:n] = 0
    assert wide.data_ptr() % 256 == 0
    att.workspace = wide[:n]
    for rows, groups in ((512, 1), (512, 64), (7, 1), (33, 20), (1, 64), (512, 3), (40, 1), (3, 0), (512, 64)):
        offsets = np.sort(np.concatenate([[0], rng.integers(0, rows + 1, size=groups)]))
        table = rng.integers(0, 900, size=(rows, 70))
        shared = rng.integers(0, 50, size=groups) * ps
        for x in range(groups):
            table[offsets[x]:offsets[x + 1], :50] = table[offsets[x] if offsets[x] < rows else 0, :50]
        lens = rng.integers(0, 70 * ps + 1, size=rows) if rows < 100 else rng.integers(0, 20 * ps, size=rows)
        req = rng.permutation(rows) if by_request else np.arange(rows)
        q = torch.randn((rows, H, D), generator=g).to(DEV, dt)
        tab = np.empty_like(table)
        tab[req] = table
        out = att.forward(q, _int(tab), _int(lens), _int(offsets), _int(shared), torch.full_like(q, math.nan),
                          row_req=_int(req) if by_request else None)
        torch.cuda.synchronize()
        some = np.arange(rows) if rows < 100 else np.sort(rng.permutation(rows)[:60])
        ref, tol = attend_ref(q[some], kc, vc, _int(table[some]), lens[some], range(len(some)), lambda i, n: torch.arange(n),
                              1 / math.sqrt(D), weight=WEIGHT)
        close(out[some], ref, tol, f"{rows} rows in {groups}")
        assert not bool(torch.isnan(out).any()) and bool((wide[n:] == 77).all()), (rows, groups)

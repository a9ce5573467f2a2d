"""The operators between a block's adapter layers at their edges: values,
sizes and orders of calls that the documentation allows, against plain
implementations in 64 bits (tests/test_block_gpu.py, whose bounds hold here)."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block  # noqa: E402
from test_block_gpu import BF16, DEV, F32, _attend_case, _attend_ref, _close, _int  # noqa: E402

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


# ---- the attention step -----------------------------------------------------------------------------------

def test_timed_step_rows():
    """The timing of the attention step runs its steps on tensors that stay."""
    from lora_normal_form_amd import multiproj
    got = multiproj.attention_rows(torch, 40, n=8, heads=4, kv_heads=2, head_dim=64, page_size=16)
    assert [r["route"] for r in got] == ["attention step", "norm + pages + rotary", "attention over the cache",
                                         "residual + norm"]
    assert all(r["us"] > 0 for r in got)

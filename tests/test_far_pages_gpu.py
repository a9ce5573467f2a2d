"""Caches of more than 2^32 elements: what the operators over pages do there has
the bits of what they do in a small cache, whose odd pages lie behind the
2^32nd element here."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block  # noqa: E402
from test_block_gpu import BF16, DEV, _int  # noqa: E402
from test_shared_gpu import make, offsets_of  # noqa: E402

pytestmark = pytest.mark.gpu

PS, HK, D = 16, 8, 128
FAR = (1 << 32) // (PS * HK * D) + 3


@pytest.fixture(scope="module")
def far():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kv = [torch.empty((FAR + 1000, PS, HK, D), dtype=BF16, device=DEV) for _ in range(2)]
    yield kv
    del kv[:]
    torch.cuda.empty_cache()


def _moved(p):
    p = np.asarray(p)
    return np.where((p >= 0) & (p % 2 == 1), p + FAR, p)


def _spread(far, small):
    at = torch.as_tensor(_moved(np.arange(small[0].shape[0])), device=DEV)
    for big, z in zip(far, small):
        big[at] = z
    return at


def test_attention(far):
    groups = [(6, 150), (5, 33)]
    kc, vc, table, q, lens = make(7, groups, PS, 32, HK, D, BF16, outside=2)
    _spread(far, (kc, vc))
    outs = []
    for k, v, tab in ((kc, vc, table), (*far, _moved(table))):
        c, tab = block.KVCache(k, v), _int(tab)
        for att, extra in ((block.SharedAttention(c, 32, len(lens), 2, always=True), True),
                           (block.PagedAttention(c, 32, window=40, sinks=9), False)):
            args = (_int(offsets_of(groups)), _int([150, 33])) if extra else ()
            outs.append(att.forward(q, tab, _int(lens), *args, torch.empty_like(q)))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert bool(outs[0].isfinite().all()) and bool((outs[0] != 0).any())


def test_copies_compaction_and_stores(far):
    g, rng = torch.Generator().manual_seed(9), np.random.default_rng(9)
    R, P = 5, 12
    small = [torch.randn((R * P + 10, PS, HK, D), generator=g).to(DEV, BF16) for _ in range(2)]
    at = _spread(far, small)
    table = rng.permutation(R * P).reshape(R, P)
    kept = np.full((R, 60), 0)
    for r in range(R):
        kept[r] = np.sort(rng.choice(np.arange(20, P * PS), 60, replace=False))
    src, dst = table[:, 3], R * P + np.arange(R)
    T = 40
    qkv = [torch.randn((T, h, D), generator=g).to(DEV) for h in (32, HK, HK)]
    slot = np.sort(rng.choice(R * P * PS, T, replace=False))
    rot = block.Rotary(torch.ones(D // 2, dtype=torch.float64, device=DEV), D)
    outs = []
    for (k, v), move in ((small, np.asarray), (far, _moved)):
        c = block.KVCache(k, v)
        block.copy_pages(c, _int(move(src)), _int(move(dst)), _int([16, 1, 7, 15, 3]))
        block.compact(c, _int(move(table)), _int([20] * R), _int(kept), _int([60, 0, 59, 1, 60]))
        slots = torch.as_tensor(move(slot // PS) * PS + slot % PS, device=DEV)
        outs.append(rot.store(*qkv, torch.arange(T, dtype=torch.int32, device=DEV), slots, c,
                              torch.empty((T, 32, D), dtype=BF16, device=DEV), norm=block.HeadNorm(D)))
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    for big, z in zip(far, small):
        same = torch.equal(big[at], z)
        assert same

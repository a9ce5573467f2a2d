"""The rotary store with norms of the heads against the formulas in 64 bits.

Tolerances count roundings: u = 2^-24 is half a step of fp32, and an fp32 sum of
n terms is off by at most n u of the sum of their magnitudes."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block  # noqa: E402
from test_block_gpu import BF16, DEV, F32, U, _cache_tensors, _close, _int  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def norm_ref(z, kind, w, b, eps):
    """z [T][H][D] in 64 bits; its norm, and how far the fp32 one may be off."""
    d, u = z.shape[-1], U[F32]
    mu = z.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(z[..., :1])
    c = z - mu
    # the mean: a sum of d terms, and one product
    e_mu = (d + 2) * u * z.abs().mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(mu)
    e_c = e_mu + u * c.abs()
    var = (c * c).mean(-1, keepdim=True) + eps
    # squares and their sum; rsqrt halves a relative error, its own is 2 u
    e_var = (2 * c.abs() * e_c + e_c * e_c).mean(-1, keepdim=True) + (d + 4) * u * var
    r = var.rsqrt()
    # (an error that may be as large as the variance itself has no first order)
    e_r = torch.where(e_var < 0.5 * var, r * (e_var / var + 3 * u), torch.full_like(r, float("inf")))
    w = torch.ones(d, dtype=torch.float64) if w is None else w.cpu().double()
    b = torch.zeros(d, dtype=torch.float64) if b is None else b.cpu().double()
    out = c * r * w + b
    tol = (c.abs() * e_r + e_c * r) * w.abs() + 3 * u * (c * r * w).abs() + u * out.abs()
    return out, tol


def turned(z, tol, ang, n, inter):
    """z with its pairs rotated, and the tolerance with the turn's own roundings: the
    angle is reduced in 64 bits and rounded to fp32 (at most pi u), cos and sin are
    within 2 u of theirs, then two products and a sum."""
    u = U[F32]
    i = torch.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + n)
    out, t = z.clone(), tol.clone()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = z[..., ia], z[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size = a.abs() + b.abs()
    t[..., ia] = tol[..., ia] * c.abs() + tol[..., ib] * s.abs() + 10 * u * size
    t[..., ib] = tol[..., ia] * s.abs() + tol[..., ib] * c.abs() + 10 * u * size
    return out, t


CASES = [  # T, Hq, Hk, D, rot, axes, adjacent, kind, own weights, biases, src, cache, by head, off
    (1, 32, 8, 128, 128, 1, False, "rms", False, False, F32, BF16, False, 0),
    (5, 4, 2, 64, 64, 3, False, "layer", True, True, F32, BF16, True, 0),
    (5, 4, 2, 64, 64, 3, True, "rms", True, True, F32, BF16, False, 0),
    (7, 3, 3, 40, 20, 2, False, "rms", False, False, F32, F32, False, 0),
    (7, 3, 1, 40, 24, 2, False, "layer", False, True, F32, F32, False, 0),
    (7, 3, 1, 40, 22, 2, True, "rms", True, False, BF16, F32, False, 0),
    (7, 3, 1, 40, 22, 2, False, "layer", True, True, BF16, BF16, True, 0),
    (9, 2, 1, 256, 256, 4, True, "rms", False, False, BF16, BF16, False, 0),
    (9, 2, 1, 256, 256, 1, False, "layer", False, False, F32, BF16, False, 0),
    (9, 2, 1, 256, 2, 1, False, "rms", False, True, F32, BF16, False, 0),
    (9, 5, 5, 256, 0, 1, False, "layer", True, True, F32, F32, False, 0),
    (4, 2, 1, 8, 0, 1, False, "rms", False, False, F32, BF16, False, 0),
    (4, 40, 20, 8, 8, 1, False, "rms", True, False, F32, F32, False, 0),
    (4, 40, 20, 8, 8, 1, True, "layer", False, False, BF16, F32, False, 0),
    (6, 4, 2, 64, 64, 2, False, "rms", False, False, F32, BF16, False, 1),
    (6, 4, 2, 64, 32, 1, True, "layer", True, True, BF16, F32, False, 3),
    (1300, 6, 2, 48, 32, 8, False, "rms", True, False, F32, BF16, False, 0),
    (1300, 6, 2, 96, 96, 2, True, "rms", False, False, BF16, BF16, False, 0)]


@pytest.mark.parametrize("T, Hq, Hk, D, rd, axes, inter, kind, own, bias, src, dt, by_head, off", CASES)
def test_norm_rotary_store(T, Hq, Hk, D, rd, axes, inter, kind, own, bias, src, dt, by_head, off):
    g = torch.Generator().manual_seed(T + D + rd)
    ps, n_pages, eps = 5, T // 5 + 3, 1e-5
    wide = (Hq + 2 * Hk) * D
    buf = (2.0 * torch.randn((T, wide + 4 + off), generator=g) + 0.5).to(DEV, src)
    buf[:, off:off + D] = 0.0  # a head without anything: eps alone
    q, k, v = (t.unflatten(1, (-1, D)) for t in torch.split(buf[:, off:off + wide], [Hq * D, Hk * D, Hk * D], dim=1))
    n = rd // 2
    freq = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(1, n))
    axis = torch.randint(0, axes, (n,), generator=g, dtype=torch.int32)
    pos = torch.randint(-1000, 1 << 30, (axes, T), generator=g, dtype=torch.int32)
    kc, vc = _cache_tensors(n_pages, ps, Hk, D, dt, by_head)
    k0, v0 = kc.cpu().clone(), vc.cpu().clone()
    slot = torch.randperm(n_pages * ps, generator=g)[:T]
    if T > 3:
        slot[1], slot[2] = -1, n_pages * ps
    vecs = [torch.randn((h, D) if own else (D,), generator=g).to(DEV) for h in (Hq, Hk, Hq, Hk)]
    qb, kb = vecs[2:] if bias else (None, None)
    norm = block.HeadNorm(D, kind, vecs[0], vecs[1], qb, kb, eps=eps)
    rot = block.Rotary(freq.to(DEV), D, axis=axis.to(DEV), n_axes=axes, interleaved=inter)
    out = torch.full((T, Hq, D), 7.0, device=DEV, dtype=dt)
    rot.store(q, k, v, pos.to(DEV), slot.to(DEV), block.KVCache(kc, vc), out, norm=norm)
    ang = pos.double()[axis.long()].T * freq if n else torch.zeros((T, 0), dtype=torch.float64)
    ang = torch.remainder(ang, 2 * np.pi)  # (exact to 64 bits' own rounding, 2^30 2^-52)
    got = []
    for z, w, b in ((q, vecs[0], qb), (k, vecs[1], kb)):
        x, tol = norm_ref(z.cpu().double(), kind, w, b, eps)
        x, tol = turned(x, tol, ang, n, inter)
        tol = tol + 2.0 ** -20 * x.abs().amax(-1, keepdim=True) * 2.0 ** -4  # (the reference's angles)
        got.append((x, tol + U[dt] * (x.abs() + tol)))
    _close(out, *got[0], "q")
    live = (slot >= 0) & (slot < n_pages * ps)
    want_k, tol_k, want_v = k0.double(), torch.zeros_like(k0, dtype=torch.float64), v0.clone()
    at = slot[live]
    want_k[at // ps, at % ps], tol_k[at // ps, at % ps] = got[1][0][live], got[1][1][live]
    want_v[at // ps, at % ps] = v.cpu().to(dt)[live]
    _close(kc, want_k, tol_k, "k")
    assert torch.equal(vc.cpu(), want_v)


def test_in_place_and_without_weights():
    g = torch.Generator().manual_seed(2)
    T, H, D = 33, 4, 64
    q0 = torch.randn((T, H, D), generator=g)
    k, v = (torch.randn((T, 1, D), generator=g).to(DEV) for _ in range(2))
    kc, vc = (torch.zeros((40, 1, 1, D), device=DEV) for _ in range(2))
    rot = block.Rotary(torch.ones(D // 2, dtype=torch.float64, device=DEV), D)
    pos, slot = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    q, out = q0.to(DEV), torch.empty((T, H, D), device=DEV)
    norm = block.HeadNorm(D)
    rot.store(q, k, v, pos, slot, block.KVCache(kc, vc), out, norm=norm)
    rot.store(q, k, v, pos, slot, block.KVCache(kc, vc), q, norm=norm)
    assert torch.equal(q, out)
    x, tol = norm_ref(q0.double(), "rms", None, None, 1e-6)
    x, tol = turned(x, tol, pos.cpu().double()[:, None].expand(T, D // 2), D // 2, False)
    _close(out, x, tol + U[F32] * x.abs(), "q")


def test_values_that_are_not_finite_stay_in_their_head():
    """One head with an infinity and one with a NaN: the others are as without."""
    T, H, D = 6, 4, 128
    q = torch.randn((T, H, D), device=DEV)
    k, v = torch.randn((T, 2, D), device=DEV), torch.randn((T, 2, D), device=DEV)
    rot = block.Rotary(torch.ones(D // 2, dtype=torch.float64, device=DEV), D)
    pos, slot = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    outs = []
    for bad in (False, True):
        z = q.clone()
        if bad:
            z[1, 2, 5], z[3, 0, 9] = float("inf"), float("nan")
        kc, vc = (torch.zeros((T, 1, 2, D), device=DEV) for _ in range(2))
        out = torch.empty_like(q)
        rot.store(z, k, v, pos, slot, block.KVCache(kc, vc), out, norm=block.HeadNorm(D))
        outs.append((out, kc))
    keep = torch.ones((T, H), dtype=torch.bool, device=DEV)
    keep[1, 2] = keep[3, 0] = False
    assert torch.equal(outs[0][0][keep], outs[1][0][keep]) and torch.equal(outs[0][1], outs[1][1])
    assert not bool(torch.isfinite(outs[1][0][1, 2, 5]))
    assert bool(torch.isnan(outs[1][0][3, 0]).all())


def test_captured_and_on_another_stream():
    T, H, D = 20, 4, 64
    q, k, v = (torch.randn((T, h, D), device=DEV) for h in (H, 2, 2))
    rot = block.Rotary(torch.ones(D // 2, dtype=torch.float64, device=DEV), D)
    pos, slot = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    kc, vc = (torch.zeros((T, 1, 2, D), device=DEV, dtype=BF16) for _ in range(2))
    cache, norm = block.KVCache(kc, vc), block.HeadNorm(D, "layer")
    out, s, g = torch.empty((T, H, D), device=DEV, dtype=BF16), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rot.store(q, k, v, pos, slot, cache, out, norm=norm)
    for step in range(3):
        q.normal_(), k.normal_(), pos.copy_(_int(np.arange(T) * step))
        g.replay()
        want, kw = torch.empty_like(out), torch.zeros_like(kc)
        torch.cuda.synchronize()
        rot.store(q, k, v, pos, slot, block.KVCache(kw, torch.zeros_like(kc)), want, norm=norm, stream=s)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(kc, kw)


def test_norms_of_other_heads_refused():
    T, H, D = 3, 4, 64
    q, k = torch.zeros((T, H, D), device=DEV), torch.zeros((T, 2, D), device=DEV)
    kc = torch.zeros((4, 1, 2, D), device=DEV)
    rot = block.Rotary(torch.ones(D // 2, dtype=torch.float64, device=DEV), D)
    pos, slot = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    for norm in (block.HeadNorm(32), block.HeadNorm(D, "rms", torch.ones((3, D), device=DEV)),
                 block.HeadNorm(D, "rms", None, torch.ones((4, D), device=DEV))):
        with pytest.raises(ValueError):
            rot.store(q, k, k, pos, slot, block.KVCache(kc, kc.clone()), torch.empty_like(q), norm=norm)


PROMPTS = [  # (as CASES) two tokens a work-group, the last one odd or not: every pair of types and size of head
    (4096, 3, 1, 64, 64, 2, False, "rms", False, False, F32, BF16, False, 0),
    (4097, 3, 2, 64, 32, 1, True, "layer", True, True, BF16, F32, False, 0),
    (8191, 2, 1, 64, 64, 1, False, "layer", False, True, BF16, BF16, True, 0),
    (4097, 5, 1, 32, 16, 1, False, "rms", True, False, F32, F32, False, 0),
    (4096, 3, 1, 128, 64, 3, False, "layer", True, True, F32, BF16, False, 0),
    (8191, 2, 2, 128, 128, 1, True, "rms", False, True, BF16, BF16, False, 0),
    (4097, 2, 1, 96, 96, 2, False, "rms", True, False, F32, F32, True, 0),
    (4097, 2, 1, 104, 40, 2, False, "layer", False, False, BF16, F32, False, 0),
    (4097, 2, 1, 256, 256, 1, False, "rms", True, True, F32, BF16, False, 0),
    (4096, 1, 1, 256, 100, 2, True, "layer", False, False, F32, F32, False, 0),
    (8191, 1, 1, 200, 0, 1, False, "layer", True, True, BF16, BF16, False, 0),
    (4097, 3, 1, 136, 64, 4, False, "rms", False, False, BF16, F32, False, 0),
    (4097, 3, 1, 136, 66, 1, False, "rms", True, True, F32, BF16, False, 1)]  # (one element an access)


@pytest.mark.parametrize("T, Hq, Hk, D, rd, axes, inter, kind, own, bias, src, dt, by_head, off", PROMPTS)
def test_prompts(T, Hq, Hk, D, rd, axes, inter, kind, own, bias, src, dt, by_head, off):
    test_norm_rotary_store(T, Hq, Hk, D, rd, axes, inter, kind, own, bias, src, dt, by_head, off)


def test_prompts_in_place():
    """q rotated where it lies: what the two tokens of a work-group ask for early is not what it writes."""
    g = torch.Generator().manual_seed(3)
    T, H, D = 4097, 6, 128
    q = torch.randn((T, H, D), generator=g).to(DEV)
    k, v = (torch.randn((T, 1, D), generator=g).to(DEV) for _ in range(2))
    kc, vc = (torch.zeros((T, 1, 1, D), device=DEV) for _ in range(2))
    rot = block.Rotary(torch.ones(D // 2, dtype=torch.float64, device=DEV), D)
    pos, slot = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    norm, out = block.HeadNorm(D), torch.empty_like(q)
    rot.store(q, k, v, pos, slot, block.KVCache(kc, vc), out, norm=norm)
    k0 = kc.clone()
    rot.store(q, k, v, pos, slot, block.KVCache(kc, vc), q, norm=norm)
    assert torch.equal(q, out) and torch.equal(kc, k0)

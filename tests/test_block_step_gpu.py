"""The attention step (multiproj.AttentionStep): its operators and the adapter
layers run together over prompts, decode steps, requests that end and rows
that stay empty. Every stage is checked on what the stages before it left on
the GPU: the layers against the fp64 oracle at the bf16 bar, the operators
against 64 bits at the bounds of test_block_gpu."""

import dataclasses
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from synth import AdapterSpec, WorkloadSpec, make_workload  # noqa: E402
from test_block_gpu import BF16, DEV, F32, U, _assign_ref, _attend_ref, _close, _int, _norm_ref  # noqa: E402

pytestmark = pytest.mark.gpu

L, Dr, I3 = AdapterSpec("lora", rank=16, bias=True), AdapterSpec("dora", rank=16), AdapterSpec("ia3")
O, V = AdapterSpec("oft", blk=32), AdapterSpec("vera")
H, HK, D, N, R, PS, P = 8, 2, 64, 24, 5, 4, 9


def _step(seed, **kw):
    from lora_normal_form_amd import multiproj
    d = H * D
    ten = [(L, L, L), (O, O, O), (V, V, V), (None, I3, I3), (Dr, None, L)]
    wls, tt = multiproj.projection_workloads(ten, N, d, (d, HK * D, HK * D), seed=seed, vera_rank=64)
    wl_out = make_workload(WorkloadSpec("out", "bf16", d, d, N, [L, Dr, V], vera_rank=64, assign="explicit",
                                        token_adapter=np.asarray(tt) % 4 - 1, seed=seed + 9))
    qkv = multiproj.QKVFused(wls, tt, len(ten))
    g = torch.Generator().manual_seed(seed)
    w = [(1.0 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(3)]
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) / (D // 2))
    st = multiproj.AttentionStep(qkv, wl_out, H, HK, D, R, P, PS, 30, freq, norm_in=w[0], norm_post=w[1],
                                 norm_out=w[2], **kw)
    return st, wls, wl_out, w, freq


def _bar(wl, x, y):
    ref = oracle.forward(dataclasses.replace(wl, x=x))
    err = np.max(np.abs(y - ref)) / np.max(np.abs(ref))
    assert err <= 1e-2, (wl.name, err)


@pytest.mark.parametrize("axes", [1, 3])
def test_steps_run_together(axes):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    kw = dict(n_axes=axes, axis=(torch.arange(D // 2, device=DEV) % axes).int()) if axes > 1 else {}
    st, wls, wl_out, w, freq = _step(31 + axes, **kw)
    g = torch.Generator().manual_seed(5)
    table, ring = st.table.cpu().numpy().astype(np.int64), st.ring.cpu().numpy().astype(np.int64)
    lens, cursor = np.zeros(R, np.int64), (0, 30)
    for step, new in enumerate(([9, 7, 0, 8, 0], [1, 1, 5, 1, 16], [1, 1, 1, 1, 1], [-1, 1, 1, -1, 20], [6, 1, 1, 3, 1],
                                [1, 1, 1, 1, 1])):
        print(f"[gpu] step {step}: new lengths {new}", flush=True)
        h = torch.randn((N, H * D), generator=g).to(DEV)
        pos = torch.randint(0, 5000, (axes, N), generator=g, dtype=torch.int32).to(DEV) if axes > 1 else None
        h_out, x_out = torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)
        k0, v0 = st.cache.k.cpu().double(), st.cache.v.cpu().double()
        st.forward(h, _int(new), h_out, x_out, pos=pos)
        torch.cuda.synchronize()
        # pages and slots
        table, ring, rows = _assign_ref(lens, new, table, ring, *cursor, PS, N)
        assert np.array_equal(st.table.cpu().numpy(), table)
        for name, v in rows.items():
            assert np.array_equal(getattr(st.rows, name).cpu().numpy(), v), (step, name)
        lens, cursor = rows["seq_len"], rows["cursor"]
        # the norm before, and the q / k / v layer
        zero = torch.zeros((N, H * D), dtype=torch.float64)
        want, tol = _norm_ref(h.cpu().double(), zero, "rms", w[0], None, 1e-5)
        _close(st.qkv.x, want, tol + U[BF16] * (want.abs() + tol), "x")
        x, y = st.qkv.x.cpu().double().numpy(), st.qkv.y.cpu().double()
        c0 = 0
        for wl, _ in wls:
            _bar(wl, x, y[:, c0:c0 + wl.d_out].numpy())
            c0 += wl.d_out
        # rotary and the cache
        p = torch.as_tensor(rows["pos"])[None].double() if pos is None else pos.cpu().double()
        ang = p[torch.arange(D // 2) % axes].T * freq.cpu()
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

        def turned(z):
            z = z.unflatten(1, (-1, D))
            a, b = z[..., :D // 2], z[..., D // 2:]
            mag = 2e-6 * (a.abs() + b.abs())  # (angle 2 pi 2^-25, sincospi 2^-22, four roundings)
            out = torch.cat([a * c - b * s, a * s + b * c], -1)
            return out, torch.cat([mag, mag], -1) + U[BF16] * (out.abs() + 1e-5)

        _close(st.q_rot, *turned(y[:, :H * D]), "q")
        kt, k_tol = turned(y[:, H * D:(H + HK) * D])
        vt = y[:, (H + HK) * D:].unflatten(1, (-1, D))
        tol_k, tol_v = torch.zeros_like(k0), torch.zeros_like(v0)
        for t in range(N):
            if rows["slot"][t] >= 0:
                at = divmod(int(rows["slot"][t]), PS)
                k0[at], tol_k[at], v0[at], tol_v[at] = kt[t], k_tol[t], vt[t], U[BF16] * vt[t].abs()
        _close(st.cache.k, k0, tol_k, "k")
        _close(st.cache.v, v0, tol_v, "v")
        # attention, the output projection, residual and next norm
        ref, tol = _attend_ref(st.q_rot, st.cache.k, st.cache.v, st.table, rows["len"], rows["req"], 0, 1 / math.sqrt(D))
        _close(st.a, ref, tol, "attention")
        _bar(wl_out, st.out.x.cpu().double().numpy(), st.out.y.cpu().double().numpy())
        z, e = _norm_ref(st.out.y.cpu().double(), zero, "rms", w[1], None, 1e-5)
        hp = h.cpu().double() + z
        e = e + 4 * U[F32] * (h.cpu().double().abs() + z.abs())
        _close(h_out, hp, e + U[F32] * (hp.abs() + e), "h'")
        want, ex = _norm_ref(hp, e, "rms", w[2], None, 1e-5)
        _close(x_out, want, ex + U[BF16] * (want.abs() + ex), "x'")
    st.close()
    st.qkv.close()


def test_one_token_each_matches_rows_with_requests():
    """one_each (row i is request i) gives what the rows' requests give."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lora_normal_form_amd import block
    st, *_ = _step(77)
    h = torch.randn((N, H * D), generator=torch.Generator().manual_seed(1)).to(DEV)
    h_out, x_out = torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)
    st.forward(h, _int([9, 7, 1, 3, 4]), h_out, x_out)
    st.forward(h, _int([1] * R), h_out, x_out)
    out = torch.empty((R, H, D), dtype=BF16, device=DEV)
    block.PagedAttention(st.cache, H).forward(st.q_rot[:R], st.table, st.rows.len[:R], out)
    torch.cuda.synchronize()
    ref, tol = _attend_ref(st.q_rot[:R], st.cache.k, st.cache.v, st.table, st.rows.len[:R].tolist(), range(R), 0,
                           1 / math.sqrt(D))
    _close(out, ref, tol, "one each")
    _close(st.a[:R], ref, tol, "by request")
    st.close()
    st.qkv.close()


def test_step_refuses():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lora_normal_form_amd import multiproj
    st, wls, wl_out, w, freq = _step(78)
    with pytest.raises(ValueError, match="heads wide"):
        multiproj.AttentionStep(st.qkv, wl_out, H, 1, D, R, P, PS, 30, freq)
    with pytest.raises(ValueError, match="layer's width"):
        multiproj.AttentionStep(st.qkv, wls[1][0], H, HK, D, R, P, PS, 30, freq)
    with pytest.raises(ValueError, match="one_each"):
        multiproj.AttentionStep(st.qkv, wl_out, H, HK, D, R, P, PS, 30, freq, one_each=True)
    st.close()
    st.qkv.close()

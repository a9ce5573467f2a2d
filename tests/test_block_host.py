"""Refusals of the operators between a block's adapter layers, without a GPU:
every call below is turned away by its argument checks before anything touches
a device, so the pointers handed in are made-up addresses."""

import math

import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402

FAKE = 1 << 20  # an address that no check may follow


def _raises(code, fn, *args):
    with pytest.raises(scute.ScuteError) as e:
        fn(*args)
    assert e.value.code == code, e.value
    return str(e.value)


def _cache(**kw):
    d = dict(device=0, dtype=scute.BF16, page_size=16, n_kv_heads=2, head_dim=64, reserved=0, n_pages=10,
             page_stride=16 * 128, token_stride=128, head_stride=64, k=FAKE, v=FAKE)
    d.update(kw)
    return scute.KVCacheDesc(**d)


BAD_CACHES = [
    (dict(device=-1), scute.E_INVALID), (dict(dtype=scute.F64), scute.E_INVALID),
    (dict(page_size=0), scute.E_SHAPE), (dict(page_size=65537), scute.E_SHAPE),
    (dict(n_kv_heads=0), scute.E_SHAPE), (dict(head_dim=0), scute.E_SHAPE), (dict(head_dim=12), scute.E_SHAPE),
    (dict(head_dim=264), scute.E_SHAPE), (dict(n_pages=0), scute.E_SHAPE), (dict(n_pages=1 << 31), scute.E_SHAPE),
    (dict(page_stride=0), scute.E_SHAPE), (dict(token_stride=-128), scute.E_SHAPE),
    (dict(token_stride=1 << 24), scute.E_SHAPE), (dict(head_stride=12), scute.E_SHAPE),
    (dict(page_stride=(1 << 40) + 8), scute.E_SHAPE),
    (dict(k=None), scute.E_INVALID), (dict(v=FAKE + 8), scute.E_INVALID)]


# ---- scute_cache_assign ------------------------------------------------------------------------

def _assign(**kw):
    d = dict(device=0, n_requests=4, table_width=8, page_size=16, ring_size=100, max_tokens=32, table_stride=8)
    ptrs = ("old_len", "new_len", "table", "ring", "cursor", "cursor_out", "seq_len", "cu_len", "slot", "req",
            "pos", "len", "counts")
    d.update({p: FAKE + 4096 * i for i, p in enumerate(ptrs)})
    d.update(kw)
    return scute.CacheAssignArgs(**d)


@pytest.mark.parametrize("kw, code", [
    (dict(device=-1), scute.E_INVALID),
    (dict(n_requests=-1), scute.E_SHAPE), (dict(n_requests=65537), scute.E_SHAPE),
    (dict(page_size=0), scute.E_SHAPE), (dict(page_size=65537), scute.E_SHAPE),
    (dict(table_width=0), scute.E_SHAPE), (dict(table_stride=7), scute.E_SHAPE),
    (dict(ring_size=0), scute.E_SHAPE), (dict(ring_size=(1 << 30) + 1), scute.E_SHAPE),
    (dict(max_tokens=-1), scute.E_SHAPE), (dict(max_tokens=(1 << 30) + 1), scute.E_SHAPE),
    (dict(ring=None), scute.E_INVALID), (dict(cursor=None), scute.E_INVALID), (dict(counts=None), scute.E_INVALID),
    (dict(cu_len=None), scute.E_INVALID), (dict(old_len=None), scute.E_INVALID), (dict(slot=None), scute.E_INVALID),
    (dict(table=FAKE + 2), scute.E_INVALID), (dict(slot=FAKE + 4), scute.E_INVALID),
    (dict(cursor=FAKE + 4), scute.E_INVALID), (dict(cursor_out=FAKE + 4096 * 4), scute.E_INVALID),
    (dict(seq_len=FAKE), scute.E_INVALID)])
def test_assign_refuses(kw, code):
    assert "scute_cache_assign" in _raises(code, scute.scute_cache_assign, _assign(**kw), 0)


# ---- scute_rotary_store ------------------------------------------------------------------------

def _rotary(rot=None, cache=None, **kw):
    d = dict(q=FAKE, q_stride=512, k=FAKE, k_stride=128, v=FAKE, v_stride=128, src_dtype=scute.F32, pos=FAKE,
             pos_stride=7, slot=FAKE, n_tokens=7, n_heads=8, q_out=FAKE, q_out_stride=512)
    d.update(kw)
    r = dict(head_dim=64, rot_dim=64, n_axes=1, interleaved=0, freq=FAKE, axis=None)
    r.update(rot or {})
    scute.scute_rotary_store(scute.RotaryDesc(**r), _cache(**(cache or {})), *d.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(rot=dict(head_dim=32)), scute.E_SHAPE), (dict(rot=dict(rot_dim=66)), scute.E_SHAPE),
    (dict(rot=dict(rot_dim=31)), scute.E_SHAPE), (dict(rot=dict(rot_dim=-2)), scute.E_SHAPE),
    (dict(rot=dict(n_axes=0)), scute.E_SHAPE), (dict(rot=dict(n_axes=9)), scute.E_SHAPE),
    (dict(rot=dict(interleaved=2)), scute.E_INVALID), (dict(rot=dict(freq=None)), scute.E_INVALID),
    (dict(rot=dict(freq=FAKE + 4)), scute.E_INVALID), (dict(src_dtype=scute.F64), scute.E_INVALID),
    (dict(n_tokens=-1), scute.E_SHAPE), (dict(n_heads=0), scute.E_SHAPE), (dict(q_stride=-1), scute.E_SHAPE),
    (dict(q_out_stride=511), scute.E_SHAPE), (dict(q=None), scute.E_INVALID), (dict(slot=None), scute.E_INVALID),
    (dict(pos=None), scute.E_INVALID), (dict(q=FAKE + 2), scute.E_INVALID), (dict(slot=FAKE + 4), scute.E_INVALID),
    (dict(q_out=FAKE + 1), scute.E_INVALID)])
def test_rotary_refuses(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _rotary(**kw)
    assert e.value.code == code, e.value


@pytest.mark.parametrize("kw, code", BAD_CACHES)
def test_caches_refused(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _rotary(cache=kw)
    assert e.value.code == code, e.value
    with pytest.raises(scute.ScuteError) as e:
        _attend(cache=kw)
    assert e.value.code == code, e.value


# ---- scute_paged_attention -----------------------------------------------------------------------

def _attend(cache=None, **kw):
    d = dict(q=FAKE, q_stride=512, n_heads=8, table=FAKE, table_stride=8, n_requests=5, table_width=8, len=FAKE,
             req=None, n_rows=5, scale=0.125, window=0, out=FAKE + 4096, out_stride=512, workspace=FAKE,
             workspace_bytes=1 << 30)
    d.update(kw)
    scute.scute_paged_attention(_cache(**(cache or {})), *d.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(n_heads=0), scute.E_SHAPE), (dict(n_heads=7), scute.E_SHAPE), (dict(n_rows=-1), scute.E_SHAPE),
    (dict(n_rows=6), scute.E_SHAPE), (dict(n_rows=(1 << 20) + 1, req=FAKE), scute.E_SHAPE),
    (dict(n_requests=-1, req=FAKE), scute.E_SHAPE), (dict(table_width=0), scute.E_SHAPE),
    (dict(table_stride=7), scute.E_SHAPE), (dict(window=-1), scute.E_SHAPE),
    (dict(scale=math.inf), scute.E_INVALID), (dict(scale=math.nan), scute.E_INVALID),
    (dict(q_stride=516), scute.E_SHAPE), (dict(out_stride=504), scute.E_SHAPE), (dict(q=None), scute.E_INVALID),
    (dict(len=None), scute.E_INVALID), (dict(q=FAKE + 8), scute.E_INVALID), (dict(len=FAKE + 2), scute.E_INVALID),
    (dict(workspace=None), scute.E_INVALID), (dict(workspace=FAKE + 64), scute.E_INVALID),
    (dict(out=FAKE), scute.E_INVALID)])
def test_attention_refuses(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _attend(**kw)
    assert e.value.code == code, e.value


@pytest.mark.parametrize("dev, dim, code", [(-1, 64, scute.E_INVALID), (0, 4, scute.E_SHAPE), (0, 257, scute.E_SHAPE)])
def test_attention_workspace_refuses(dev, dim, code):
    _raises(code, scute.scute_paged_attention_workspace, dev, dim)


# ---- scute_residual_norm ---------------------------------------------------------------------------

def _norm(desc=None, **kw):
    d = dict(y=FAKE, y_dtype=scute.F32, y_stride=64, h=FAKE + 4096, h_dtype=scute.BF16, h_stride=64, gate=None,
             gate_stride=0, h_out=FAKE + 8192, h_out_stride=64, x=FAKE + 12288, x_dtype=scute.BF16, x_stride=64,
             n_rows=3)
    d.update(kw)
    n = dict(device=0, kind=0, d=64, post=1, eps=1e-5, h_scale=1.0, y_scale=1.0)
    n.update(desc or {})
    scute.scute_residual_norm(scute.NormDesc(**n), *d.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(desc=dict(device=-1)), scute.E_INVALID), (dict(desc=dict(kind=2)), scute.E_INVALID),
    (dict(desc=dict(d=0)), scute.E_SHAPE), (dict(desc=dict(d=32769)), scute.E_SHAPE),
    (dict(desc=dict(pre_w=FAKE + 2)), scute.E_INVALID), (dict(n_rows=-1), scute.E_SHAPE),
    (dict(h_dtype=scute.F64), scute.E_INVALID), (dict(y_dtype=7), scute.E_INVALID), (dict(x_dtype=-1), scute.E_INVALID),
    (dict(h_out=None, x=None), scute.E_INVALID), (dict(y_stride=-1), scute.E_SHAPE), (dict(x_stride=63), scute.E_SHAPE),
    (dict(h_out_stride=0), scute.E_SHAPE), (dict(h=None), scute.E_INVALID), (dict(x=FAKE + 4096), scute.E_INVALID),
    (dict(h_out=FAKE), scute.E_INVALID), (dict(h_out=FAKE + 4096, h_out_stride=128), scute.E_INVALID),
    (dict(y=FAKE + 2), scute.E_INVALID), (dict(gate=FAKE + 2), scute.E_INVALID)])
def test_norm_refuses(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _norm(**kw)
    assert e.value.code == code, e.value


# ---- what the tensor functions refuse -----------------------------------------------------------

def test_tensors_refused():
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        block.KVCache(z(4, 16, 2, 64), z(4, 16, 2, 64))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        block.KVCache(z(4, 16, 2, 64).half(), z(4, 16, 2, 64).half())
    with pytest.raises(ValueError, match="n_pages"):
        block.KVCache(z(4, 16, 128), z(4, 16, 128))
    with pytest.raises(ValueError, match="strides"):
        block.KVCache(z(4, 16, 2, 64), z(4, 2, 16, 64).transpose(1, 2))
    with pytest.raises(ValueError, match="last axis"):
        block.KVCache(z(4, 16, 64, 2).transpose(2, 3), z(4, 16, 64, 2).transpose(2, 3))
    with pytest.raises(ValueError, match="pairs"):
        block.Rotary(z(33, dtype=torch.float64), 64)
    with pytest.raises(ValueError, match="freq"):
        block.Rotary(z(32), 64)
    with pytest.raises(ValueError, match="n_axes"):
        block.Rotary(z(32, dtype=torch.float64), 64, n_axes=9)
    with pytest.raises(ValueError, match="kind"):
        block.ResidualNorm(64, kind="batch", device="cpu")
    with pytest.raises(ValueError, match="without post"):
        block.ResidualNorm(64, post_weight=z(64), device="cpu")
    with pytest.raises(ValueError, match="without pre"):
        block.ResidualNorm(64, pre=False, pre_bias=z(64), device="cpu")
    with pytest.raises(ValueError, match="pre_weight"):
        block.ResidualNorm(64, pre_weight=z(63), device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        block.ResidualNorm(64, pre_weight=z(64))
    rows = block.Rows(2, 4, device="cpu")
    i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    cur = z(2, dtype=torch.int64)
    for bad in ((i(3), i(2), i(2, 5), i(9), cur), (i(2), i(2).long(), i(2, 5), i(9), cur),
                (i(2), i(2), i(3, 5), i(9), cur), (i(2), i(2), i(5, 2).T, i(9), cur),
                (i(2), i(2), i(2, 5), i(18)[::2], cur), (i(2), i(2), i(2, 5), i(9), i(2))):
        with pytest.raises(ValueError, match="must be"):
            block.assign_pages(*bad, 16, rows)
    with pytest.raises(ValueError, match="GPU"):
        block.assign_pages(i(2), i(2), i(2, 5), i(9), cur, 16, rows)

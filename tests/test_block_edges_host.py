"""What the operators between a block's adapter layers refuse at their edges,
without a GPU: handles are stood in for, so every call below has to be turned
away by its argument checks."""

from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402

F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def _handle(cls, **attrs):
    """A handle of `cls` that no constructor has seen."""
    h = cls.__new__(cls)
    h.__dict__.update(attrs)
    return h


# ---- rotary positions ------------------------------------------------------------------------------

@pytest.mark.parametrize("q_dim, k_dim, cache_dim, rot_dim", [
    (64, 64, 128, 128), (128, 128, 64, 64), (64, 64, 64, 128), (64, 128, 128, 128)])
def test_rotary_refuses_heads_of_another_size(q_dim, k_dim, cache_dim, rot_dim):
    """The kernel strides by the cache's head size: q, k, v, q_out and the
    rotary's heads have to be of that size."""
    cache = SimpleNamespace(device=torch.device("cpu"), index=0, dtype=BF16, n_kv_heads=2, head_dim=cache_dim,
                            page_size=16, desc=None)
    ro = _handle(block.Rotary, freq=torch.ones(4, dtype=torch.float64), axis=None, n_axes=1, head_dim=rot_dim,
                 device=torch.device("cpu"), desc=None)
    q, k, v = torch.zeros(3, 4, q_dim), torch.zeros(3, 2, k_dim), torch.zeros(3, 2, k_dim)
    with pytest.raises(ValueError, match="head_dim"):
        ro.store(q, k, v, torch.zeros(3, dtype=I32), torch.zeros(3, dtype=I64), cache,
                 torch.zeros(3, 4, q_dim, dtype=BF16))


# ---- pages and slots -------------------------------------------------------------------------------

def test_rows_keep_what_their_descriptor_points_to():
    """assign_pages writes to the addresses in `args`, so the tensors behind
    them cannot be replaced (the first would be freed, and then written)."""
    rows = block.Rows(3, 5, device="cpu")
    shapes = {"seq_len": 3, "cu_len": 4, "slot": 5, "req": 5, "pos": 5, "len": 5, "cursor": 2, "counts": 4}
    for name, n in shapes.items():
        t = getattr(rows, name)
        assert t.shape == (n,) and t.dtype == (I64 if name in ("slot", "cursor") else I32)
        assert t.data_ptr() == getattr(rows.args, "cursor_out" if name == "cursor" else name)
        with pytest.raises(AttributeError):
            setattr(rows, name, t.clone())
        assert getattr(rows, name) is t


def _assign_args(**kw):
    a = scute.CacheAssignArgs()
    a.n_requests, a.table_width, a.page_size, a.ring_size, a.max_tokens, a.table_stride = 4, 8, 16, 100, 32, 8
    for i, name in enumerate(("old_len", "new_len", "table", "ring", "cursor", "cursor_out", "seq_len", "cu_len", "slot",
                              "req", "pos", "len", "counts")):
        setattr(a, name, (1 << 20) + 4096 * i)  # addresses that no check may follow
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def test_assign_refuses_unknown_flags():
    with pytest.raises(scute.ScuteError, match="flag") as e:
        scute.scute_cache_assign(_assign_args(flags=1 << 16), 0)
    assert e.value.code == scute.E_INVALID


def test_assign_refuses_fewer_rows_than_requests():
    with pytest.raises(scute.ScuteError, match="a row for each") as e:
        scute.scute_cache_assign(_assign_args(flags=scute.ASSIGN_ONE_EACH, max_tokens=3), 0)
    assert e.value.code == scute.E_SHAPE


# ---- the attention step ----------------------------------------------------------------------------

def test_step_runs_on_the_stream_of_its_tensors_device(monkeypatch):
    """The layers and the operators between them run on one stream, that of the
    device of the step's tensors, whichever device is current."""
    from lora_normal_form_amd import multiproj
    streams = []

    class Part:
        def __getattr__(self, name):
            return lambda *a, stream=None, **kw: streams.append((name, stream))

    layer = lambda: SimpleNamespace(layer=Part(), batch=0, x=0, W=0, y=0)  # noqa: E731
    rows = block.Rows(2, 3, device="cpu")
    st = _handle(multiproj.AttentionStep, qkv=layer(), out=layer(), one_each=False, tenants=None, rows=rows, state=rows.state.clone(),
                 table=0, ring=0, cache=SimpleNamespace(index=1, page_size=4), rotary=SimpleNamespace(n_axes=1, store=Part().store),
                 attention=Part(), norm_in=Part(), norm_out=Part(), q=0, k=0, v=0, q_rot=0, a=0)
    monkeypatch.setattr(block, "current_stream", lambda index: 1000 + index)
    monkeypatch.setattr(block, "assign_pages", Part().assign_pages)
    st.forward(0, 0, 0, 0)
    assert streams == [(name, 1001) for name in ("assign_pages", "forward", "forward", "store", "forward", "forward",
                                                 "forward")]


# ---- attention -------------------------------------------------------------------------------------

@pytest.mark.parametrize("scale, ok", [(2.4e38, False), (-3.0e38, False), (2.3e38, True)])
def test_attention_refuses_a_scale_past_fp32(scale, ok):
    """The scores are taken times scale log2(e): an infinite product would make
    NaN of equal scores. (What passes the check is turned away for its q.)"""
    addr = 1 << 20
    cache = scute.KVCacheDesc(0, scute.BF16, 16, 2, 64, 0, 10, 16 * 128, 128, 64, addr, addr)
    with pytest.raises(scute.ScuteError, match="null" if ok else "scale"):
        scute.scute_paged_attention(cache, None, 512, 8, addr, 8, 5, 8, addr, None, 5, scale, 0, addr + 4096, 512, addr,
                                    1 << 30, 0)


# ---- outputs that overlap inputs -------------------------------------------------------------------

A0 = 1 << 20  # an address that no check may follow


def _cache_desc(dtype=scute.BF16):
    return scute.KVCacheDesc(0, dtype, 16, 2, 64, 0, 10, 16 * 128, 128, 64, 1 << 30, 1 << 31)


@pytest.mark.parametrize("output, other, by", [
    ("cu_len", "old_len", -16), ("seq_len", "old_len", 12), ("seq_len", "new_len", -12), ("pos", "new_len", 0),
    ("cursor_out", "cursor", 8), ("cursor_out", "seq_len", -8), ("counts", "cursor", 8), ("slot", "cursor", -248),
    ("req", "pos", -124), ("len", "cu_len", 16), ("ring", "counts", -396), ("ring", "old_len", 12)])
def test_assign_refuses_overlaps(output, other, by):
    """Four requests, 32 rows, a ring of 100: one output `by` bytes from another
    array, of which they share the first or the last element."""
    a = _assign_args()
    setattr(a, output, getattr(a, other) + by)
    with pytest.raises(scute.ScuteError, match="output") as e:
        scute.scute_cache_assign(a, 0)
    assert e.value.code == scute.E_INVALID


@pytest.mark.parametrize("src, q, q_stride, k, v, out, out_stride, tokens", [
    (scute.F32, 0, 768, 2048, 2560, 0, 768, 5),            # q_out over a wider q
    (scute.BF16, 0, 768, 1024, 1280, 0, 1024, 5),          # the same place, another stride
    (scute.BF16, 0, 768, 1024, 1280, 512, 768, 5),         # a column range that reaches into q's and k's
    (scute.BF16, 0, 768, 1024, 1280, 768 * 2 * 4 + 16, 768, 5),  # the last row's
    (scute.BF16, 1 << 14, 512, 0, 1 << 16, 128, 512, 1), (scute.BF16, 1 << 14, 512, 1 << 17, 0, -256, 512, 1)])
def test_rotary_refuses_overlaps(src, q, q_stride, k, v, out, out_stride, tokens):
    ro = scute.RotaryDesc(64, 64, 1, 0, 1 << 32, None)
    with pytest.raises(scute.ScuteError, match="overlaps") as e:
        scute.scute_rotary_store(ro, _cache_desc(), A0 + q, q_stride, A0 + k, q_stride, A0 + v, q_stride, src, 1 << 33, 0,
                                 1 << 34, tokens, 8, A0 + out, out_stride, 0)
    assert e.value.code == scute.E_INVALID


@pytest.mark.parametrize("out, q_stride, out_stride, rows", [
    (0, 512, 512, 5), (16, 512, 512, 1), (-1008, 512, 512, 1), (1024 * 4, 512, 512, 5), (-1024 * 4, 512, 512, 5),
    (512, 1024, 1024, 5), (2048 * 4 - 16, 1024, 1024, 5)])
def test_attention_refuses_overlaps(out, q_stride, out_stride, rows):
    with pytest.raises(scute.ScuteError, match="also q") as e:
        scute.scute_paged_attention(_cache_desc(), A0 + 8192, q_stride, 8, A0, 8, 5, 8, A0, None, rows, 0.1, 0, A0 + 8192 + out,
                                    out_stride, 1 << 32, 1 << 30, 0)
    assert e.value.code == scute.E_INVALID


@pytest.mark.parametrize("h_out, x, gate, rows", [
    (256, 1 << 16, None, 3), (-256, 1 << 16, None, 3), (1 << 16, 512, None, 3), (1 << 16, (1 << 16) + 4, None, 1),
    (1 << 16, 1 << 17, 1 << 16, 3), (1 << 16, 1 << 17, (1 << 17) + 8, 1), (1 << 15, 1 << 16, None, 3)])
def test_norm_refuses_overlaps(h_out, x, gate, rows):
    """h (fp32, 64 elements a row) at 0, y at 2^15."""
    n = scute.NormDesc(device=0, kind=0, d=64, post=1, eps=1e-5, h_scale=1.0, y_scale=1.0)
    with pytest.raises(scute.ScuteError, match="is also") as e:
        scute.scute_residual_norm(n, A0 + (1 << 15), scute.F32, 64, A0, scute.F32, 64, None if gate is None else A0 + gate, 64,
                                  A0 + h_out, 64, A0 + x, scute.F32, 64, rows, 0)
    assert e.value.code == scute.E_INVALID

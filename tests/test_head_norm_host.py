"""Refusals of the rotary store with norms of the heads, without a GPU."""

import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402
from test_block_host import BAD_CACHES, FAKE, _cache  # noqa: E402


def _call(rot=None, cache=None, norm=None, **kw):
    d = dict(q=FAKE, q_stride=512, k=FAKE, k_stride=128, v=FAKE, v_stride=128, src_dtype=scute.F32, pos=FAKE,
             pos_stride=7, slot=FAKE, n_tokens=7, n_heads=8, q_out=FAKE + (1 << 18), q_out_stride=512)
    d.update(kw)
    r = dict(head_dim=64, rot_dim=64, n_axes=1, interleaved=0, freq=FAKE, axis=None)
    r.update(rot or {})
    n = dict(kind=0, eps=1e-6, q_w=FAKE, q_b=None, k_w=FAKE, k_b=None, q_stride=0, k_stride=64)
    n.update(norm or {})
    scute.scute_norm_rotary_store(scute.RotaryDesc(**r), scute.HeadNormDesc(**n), _cache(**(cache or {})), *d.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(norm=dict(kind=2)), scute.E_INVALID), (dict(norm=dict(kind=-1)), scute.E_INVALID),
    (dict(norm=dict(q_w=FAKE + 2)), scute.E_INVALID), (dict(norm=dict(k_b=FAKE + 1)), scute.E_INVALID),
    (dict(norm=dict(q_stride=63)), scute.E_SHAPE), (dict(norm=dict(k_stride=-64)), scute.E_SHAPE),
    (dict(norm=dict(k_stride=(1 << 20) + 4)), scute.E_SHAPE), (dict(rot=dict(head_dim=32)), scute.E_SHAPE),
    (dict(rot=dict(rot_dim=66)), scute.E_SHAPE), (dict(rot=dict(n_axes=9)), scute.E_SHAPE),
    (dict(rot=dict(interleaved=2)), scute.E_INVALID), (dict(src_dtype=scute.F64), scute.E_INVALID),
    (dict(n_tokens=-1), scute.E_SHAPE), (dict(n_heads=0), scute.E_SHAPE), (dict(q_out_stride=511), scute.E_SHAPE),
    (dict(q=None), scute.E_INVALID), (dict(slot=FAKE + 4), scute.E_INVALID), (dict(q_out=FAKE), scute.E_INVALID)])
def test_refuses(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _call(**kw)
    assert e.value.code == code and "scute_norm_rotary_store" in str(e.value), e.value


@pytest.mark.parametrize("kw, code", BAD_CACHES)
def test_caches_refused(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _call(cache=kw)
    assert e.value.code == code, e.value


def test_no_norm():
    with pytest.raises(scute.ScuteError) as e:
        scute._check(scute.lib.scute_norm_rotary_store(None, None, None, *[0] * 6, 0, 0, 0, 0, 1, 1, 0, 0, 0))
    assert e.value.code == scute.E_INVALID


def test_handles_refuse():
    v, w = torch.ones(64), torch.ones(8, 64)
    for a in ((64, "mean"), (32, "rms", v), (64, "rms", w, None, v), (64, "rms", v.double()), (64, "rms", v.view(1, 1, 64)),
              (64, "layer", torch.ones(64, 8).T), (64, "rms", v)):  # (the last: not on a GPU)
        with pytest.raises(ValueError):
            block.HeadNorm(*a)
    assert block.HeadNorm(64).device is None

"""Refusals of attention over shared positions, without a GPU."""

import math

import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import scute  # noqa: E402
from test_block_host import BAD_CACHES, FAKE, _cache  # noqa: E402


def _attend(cache=None, **kw):
    d = dict(q=FAKE, q_stride=512, n_heads=8, table=FAKE, table_stride=8, n_requests=5, table_width=8, len=FAKE,
             req=None, n_rows=5, group=FAKE, shared_len=FAKE, n_groups=2, scale=0.125, out=FAKE + (1 << 14),
             out_stride=512, workspace=FAKE, workspace_bytes=1 << 30, flags=0)
    d.update(kw)
    scute.scute_shared_attention(_cache(**(cache or {})), *d.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(flags=2), scute.E_INVALID), (dict(n_groups=-1), scute.E_SHAPE), (dict(n_groups=65537), scute.E_SHAPE), (dict(group=None), scute.E_INVALID),
    (dict(shared_len=None), scute.E_INVALID), (dict(group=FAKE + 1), scute.E_INVALID), (dict(shared_len=FAKE + 2), scute.E_INVALID),
    (dict(n_heads=7), scute.E_SHAPE), (dict(n_rows=6), scute.E_SHAPE), (dict(n_rows=-1), scute.E_SHAPE),
    (dict(table_width=0), scute.E_SHAPE), (dict(table_stride=7), scute.E_SHAPE), (dict(scale=math.inf), scute.E_INVALID),
    (dict(q_stride=516), scute.E_SHAPE), (dict(out_stride=504), scute.E_SHAPE), (dict(q=None), scute.E_INVALID),
    (dict(len=FAKE + 2), scute.E_INVALID), (dict(workspace=FAKE + 64), scute.E_INVALID), (dict(out=FAKE), scute.E_INVALID)])
def test_refuses(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _attend(**kw)
    assert e.value.code == code and "scute_shared_attention" in str(e.value), e.value


@pytest.mark.parametrize("kw, code", BAD_CACHES)
def test_caches_refused(kw, code):
    with pytest.raises(scute.ScuteError) as e:
        _attend(cache=kw)
    assert e.value.code == code, e.value


def test_no_rows():
    _attend(n_rows=0, q=None, len=None, out=None, workspace=None, group=None, shared_len=None)


@pytest.mark.parametrize("args, code", [
    ((-1, scute.BF16, 64, 8, 2, 5, 1), scute.E_INVALID), ((0, scute.F64, 64, 8, 2, 5, 1), scute.E_INVALID),
    ((0, scute.BF16, 60, 8, 2, 5, 1), scute.E_SHAPE), ((0, scute.BF16, 264, 8, 2, 5, 1), scute.E_SHAPE),
    ((0, scute.BF16, 64, 7, 2, 5, 1), scute.E_SHAPE), ((0, scute.BF16, 64, 8, 0, 5, 1), scute.E_SHAPE),
    ((0, scute.BF16, 64, 8, 2, -1, 1), scute.E_SHAPE), ((0, scute.BF16, 64, 8, 2, (1 << 20) + 1, 1), scute.E_SHAPE),
    ((0, scute.BF16, 64, 8, 2, 5, -1), scute.E_SHAPE), ((0, scute.BF16, 64, 8, 2, 5, 65537), scute.E_SHAPE)])
def test_workspace_refuses(args, code):
    with pytest.raises(scute.ScuteError) as e:
        scute.scute_shared_attention_workspace(*args)
    assert e.value.code == code, e.value

"""Refusals of the operators on shared pages, without a GPU: every call below is
turned away by its argument checks before anything touches a device, so the
pointers handed in are made-up addresses."""

import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402
from test_block_host import BAD_CACHES, FAKE, _cache  # noqa: E402


def _code(code, fn, *args):
    with pytest.raises(scute.ScuteError) as e:
        fn(*args)
    assert e.value.code == code, e.value


def _fork(**kw):
    d = dict(device=0, n_requests=4, table_width=8, page_size=16, ring_size=100, n_pages=100, window=0, sinks=0,
             table_stride=8, table_out_stride=8, workspace_bytes=1 << 20)
    ptrs = ("len", "parent", "keep", "table", "ring", "cursor", "cursor_out", "table_out", "seq_len", "src", "dst",
            "n", "counts", "workspace")
    d.update({p: FAKE + 4096 * i for i, p in enumerate(ptrs)})
    d.update(kw)
    return scute.CacheForkArgs(**d)


@pytest.mark.parametrize("kw, code", [
    (dict(device=-1), scute.E_INVALID), (dict(n_requests=-1), scute.E_SHAPE), (dict(n_requests=65537), scute.E_SHAPE),
    (dict(page_size=0), scute.E_SHAPE), (dict(page_size=65537), scute.E_SHAPE), (dict(table_width=0), scute.E_SHAPE),
    (dict(table_width=(1 << 24) + 1, table_stride=1 << 25, table_out_stride=1 << 25), scute.E_SHAPE),
    (dict(table_stride=7), scute.E_SHAPE), (dict(table_out_stride=7), scute.E_SHAPE),
    (dict(ring_size=0), scute.E_SHAPE), (dict(ring_size=(1 << 30) + 1), scute.E_SHAPE),
    (dict(n_pages=0), scute.E_SHAPE), (dict(n_pages=(1 << 24) + 1), scute.E_SHAPE), (dict(window=-1), scute.E_SHAPE),
    (dict(sinks=-1), scute.E_SHAPE), (dict(len=None), scute.E_INVALID), (dict(parent=None), scute.E_INVALID),
    (dict(table=None), scute.E_INVALID), (dict(table_out=None), scute.E_INVALID), (dict(ring=None), scute.E_INVALID),
    (dict(cursor=None), scute.E_INVALID), (dict(counts=None), scute.E_INVALID), (dict(dst=None), scute.E_INVALID),
    (dict(workspace=None), scute.E_INVALID), (dict(workspace=FAKE + 13 * 4096 + 64), scute.E_INVALID),
    (dict(workspace_bytes=100), scute.E_INVALID), (dict(keep=FAKE + 2), scute.E_INVALID),
    (dict(cursor=FAKE + 4), scute.E_INVALID), (dict(table_out=FAKE + 3 * 4096), scute.E_INVALID),
    (dict(table_out=FAKE + 3 * 4096 + 124), scute.E_INVALID), (dict(seq_len=FAKE), scute.E_INVALID),
    (dict(src=FAKE + 10 * 4096), scute.E_INVALID), (dict(cursor_out=FAKE + 5 * 4096), scute.E_INVALID),
    (dict(ring=FAKE + 3 * 4096 + 64), scute.E_INVALID)])
def test_fork_refuses(kw, code):
    _code(code, scute.scute_cache_fork, _fork(**kw), 0)


def test_fork_workspace_refuses():
    for R, n in ((-1, 1), (65537, 1), (1, 0), (1, (1 << 24) + 1)):
        _code(scute.E_SHAPE, scute.scute_cache_fork_workspace, R, n)
    assert scute.scute_cache_fork_workspace(0, 1) > 0
    assert scute.scute_cache_fork_workspace(65536, 1 << 24) >= 6 << 24


@pytest.mark.parametrize("kw, code", [
    (dict(n_copies=-1), scute.E_SHAPE), (dict(n_copies=(1 << 20) + 1), scute.E_SHAPE), (dict(src=None), scute.E_INVALID),
    (dict(dst=None), scute.E_INVALID), (dict(n=None), scute.E_INVALID), (dict(n=FAKE + 2), scute.E_INVALID)])
def test_copy_refuses(kw, code):
    d = dict(src=FAKE, dst=FAKE, n=FAKE, n_copies=3)
    d.update(kw)
    _code(code, scute.scute_cache_copy, _cache(), *d.values(), 0)


def _compact(cache=None, **kw):
    d = dict(table=FAKE, table_stride=8, n_requests=4, table_width=8, start=FAKE + 4096, kept=FAKE + 8192, kept_stride=9,
             kept_width=9, n_kept=FAKE + 12288, new_len=FAKE + 16384)
    d.update(kw)
    scute.scute_cache_compact(cache or _cache(), *d.values(), 0)


@pytest.mark.parametrize("kw, code", [
    (dict(n_requests=-1), scute.E_SHAPE), (dict(n_requests=65537), scute.E_SHAPE), (dict(table_width=0), scute.E_SHAPE),
    (dict(table_stride=7), scute.E_SHAPE), (dict(kept_width=-1), scute.E_SHAPE), (dict(kept_stride=8), scute.E_SHAPE),
    (dict(kept_width=(1 << 29) + 1, kept_stride=1 << 30), scute.E_SHAPE), (dict(table=None), scute.E_INVALID),
    (dict(start=None), scute.E_INVALID), (dict(kept=None), scute.E_INVALID), (dict(n_kept=None), scute.E_INVALID),
    (dict(start=FAKE + 4097), scute.E_INVALID), (dict(new_len=FAKE + 4096), scute.E_INVALID),
    (dict(new_len=FAKE + 8192 + 64), scute.E_INVALID), (dict(new_len=FAKE + 100), scute.E_INVALID)])
def test_compact_refuses(kw, code):
    _code(code, lambda: _compact(**kw))


@pytest.mark.parametrize("kw, code", BAD_CACHES)
def test_caches_refused(kw, code):
    _code(code, scute.scute_cache_copy, _cache(**kw), FAKE, FAKE, FAKE, 3, 0)
    _code(code, lambda: _compact(cache=_cache(**kw)))


def test_nothing_to_do():
    scute.scute_cache_copy(_cache(), None, None, None, 0, 0)
    _compact(n_requests=0, table=None, start=None, kept=None, n_kept=None, new_len=None)


def test_torch_checks():
    i32 = dict(dtype=torch.int32)
    c = object.__new__(block.KVCache)
    c.device, c.index, c.desc = torch.device("cpu"), 0, _cache()
    with pytest.raises(ValueError):
        block.copy_pages(c, torch.zeros(3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    with pytest.raises(ValueError):
        block.copy_pages(c, torch.zeros(3), torch.zeros(3, **i32), torch.zeros(3, **i32))
    good = dict(table=torch.zeros((2, 5), **i32), start=torch.zeros(2, **i32), kept=torch.zeros((2, 4), **i32),
                n_kept=torch.zeros(2, **i32))
    for kw in (dict(table=torch.zeros((3, 5), **i32)), dict(table=torch.zeros((2, 10), **i32)[:, ::2]),
               dict(start=torch.zeros(3, **i32)), dict(kept=torch.zeros((2, 4))), dict(kept=torch.zeros(8, **i32)),
               dict(kept=torch.zeros((2, 8), **i32)[:, ::2]), dict(n_kept=torch.zeros((2, 1), **i32)),
               dict(new_len=torch.zeros(3, **i32)), {}):  # (the last: not on a GPU)
        with pytest.raises(ValueError):
            block.compact(c, **{**good, **kw})

"""What runs between the adapter layers of a decoder block, on torch tensors:
the steps from the q / k / v layer's output to the output projection's input,
and the norms around the residual.

  assign_pages    pages and slots of a step's tokens from the requests'
                  lengths, on the GPU (scute_cache_assign)
  fork_pages      requests that go on from others, are cut back, end or lose
                  the pages behind a window (scute_cache_fork); copy_pages
                  copies what it says in each layer's cache (scute_cache_copy)
  compact         positions of a request that stay, moved together
                  (scute_cache_compact)
  Rotary.store    rotary positions with several axes; k and v into the paged
                  cache (scute_rotary_store), with norms of the heads (HeadNorm)
                  in the same pass (scute_norm_rotary_store)
  PagedAttention  attention of new tokens over the paged cache
                  (scute_paged_attention; with a window and first positions
                  that stay visible scute_sink_attention)
  SharedAttention the same for rows whose contexts begin with the same
                  positions, read once (scute_shared_attention)
  ResidualNorm    the norms after and before a block, with its gate and
                  residual scale (scute_residual_norm)

The functions check shapes, types, strides and devices (ValueError) and hand
pointers to the library, whose own checks raise ScuteError. Every launch goes
to ``stream``, by default torch's current stream of the tensors' device, which
need not be the current device. Nothing is allocated or synchronised after a
handle is made, so the calls may be captured into a graph; the caller keeps the
tensors until the stream has run them. A decode step
(``multiproj.AttentionStep`` is one)::

    rows = assign_pages(seq_len, new_len, table, ring, cursor, 16, rows)
    rotary.store(q, k, v, rows.pos, rows.slot, cache, q_out)
    attention.forward(q_out, table, rows.len, out, row_req=rows.req)
"""

from __future__ import annotations

import ctypes as C
import math

import torch

from . import scute

_DTYPES = {torch.float32: scute.F32, torch.bfloat16: scute.BF16}
_F32, _BF16, _I32, _I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def _bad(what):
    raise ValueError(what)


# torch's current stream of a device as an address (its accessor without the
# Stream object, which costs more than a launch's other checks together)
current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream, index):
    if stream is None:
        return current_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _gpu(device, *tensors):
    """Every tensor (None passes) on `device`, a GPU."""
    if device.type != "cuda":
        _bad(f"the tensors must be on a GPU, got {device}")
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            _bad(f"tensors on {t.device} and {device} in one call")


def settle(device):
    """Waits for what a new handle is filled with, so that its first call may be
    on any stream."""
    if device.type == "cuda":
        with torch.cuda.device(device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(device).synchronize()


def _vector(t, n, dtype, name):
    """A contiguous one-dimensional tensor of n elements; its address."""
    if t.dtype != dtype or t.shape != (n,) or not t.is_contiguous():
        _bad(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    return t.data_ptr()


def _heads(t, n, heads, dim, name):
    """[n][heads][dim] with the heads of a row contiguous; its row stride."""
    if t.shape != (n, heads, dim):
        _bad(f"{name} must be [{n}][{heads}][{dim}], got {tuple(t.shape)}")
    a, b, c = t.stride()
    if c != 1 or (b != dim and heads > 1):
        _bad(f"{name}: the heads of a row must be contiguous")
    return a


# ---- the cache -----------------------------------------------------------------------------------

class KVCache:
    """A paged key-value cache over the caller's tensors k and v
    [n_pages][page_size][n_kv_heads][head_dim] (float32 or bfloat16; a
    transposed view of [n_pages][n_kv_heads][page_size][head_dim] is served
    too). The tensors stay the caller's; the handle keeps them alive."""

    def __init__(self, k, v):
        if k.dtype not in _DTYPES or v.dtype != k.dtype:
            _bad("k and v must both be float32 or bfloat16")
        if k.dim() != 4 or v.shape != k.shape:
            _bad("k and v must both be [n_pages][page_size][n_kv_heads][head_dim]")
        n_pages, ps, heads, dim = k.shape
        # (the stride of an axis of one element says nothing)
        strides = [s if n > 1 else dim for s, n in zip(k.stride()[:3], k.shape[:3])]
        if strides != [s if n > 1 else dim for s, n in zip(v.stride()[:3], v.shape[:3])]:
            _bad("k and v must have the same strides")
        if dim > 1 and (k.stride(3) != 1 or v.stride(3) != 1):
            _bad("the last axis of k and v must be contiguous")
        _gpu(k.device, v)
        self.k, self.v = k, v
        self.device, self.index = k.device, k.device.index
        self.dtype, self.page_size, self.n_kv_heads, self.head_dim = k.dtype, ps, heads, dim
        self.desc = scute.KVCacheDesc(k.device.index, _DTYPES[k.dtype], ps, heads, dim, 0, n_pages,
                                      *strides, k.data_ptr(), v.data_ptr())


# ---- pages and slots ----------------------------------------------------------------------------

def split_state(state, n_requests):
    """(cursor, seq_len) of a Rows' state buffer, or of another laid out like it."""
    return state[:2], state[2:].view(_I32)[:n_requests]


class Rows:
    """What assign_pages fills in for a step of at most n_requests requests
    and max_tokens tokens: seq_len [n_requests], cu_len [n_requests + 1], and
    for each token slot (int64), req, pos, len [max_tokens] (rows past the last
    token: -1, -1, 0, 0); cursor [2] (int64) and counts [4] (tokens placed,
    pages taken, requests refused, pages returned). The tensors stay the
    handle's, whose descriptor holds their addresses: their elements may be
    written, the attributes not set. cursor and seq_len, which the next step
    begins with, are parts of one buffer, `state` (int64)."""

    def __init__(self, n_requests, max_tokens, device=None):
        dev = torch.device("cuda" if device is None else device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.n_requests, self.max_tokens, self.device = int(n_requests), int(max_tokens), dev
        a = self.args = scute.CacheAssignArgs()
        a.device = dev.index if dev.type == "cuda" else -1
        a.n_requests, a.max_tokens = n_requests, max_tokens
        self._state = torch.zeros(2 + (n_requests + 1) // 2, dtype=_I64, device=dev)
        self._filled = dict(zip(("cursor", "seq_len"), split_state(self._state, n_requests)))
        for name, n, dt in (("cu_len", n_requests + 1, _I32), ("slot", max_tokens, _I64), ("req", max_tokens, _I32),
                            ("pos", max_tokens, _I32), ("len", max_tokens, _I32), ("counts", 4, _I32)):
            self._filled[name] = torch.zeros(n, dtype=dt, device=dev)
        for name, t in self._filled.items():
            setattr(a, "cursor_out" if name == "cursor" else name, t.data_ptr())
        settle(dev)

    seq_len, cu_len, slot, req, pos, len, cursor, counts = (
        property(lambda self, name=name: self._filled[name])
        for name in ("seq_len", "cu_len", "slot", "req", "pos", "len", "cursor", "counts"))
    state = property(lambda self: self._state)


def assign_pages(old_len, new_len, table, ring, cursor, page_size, rows, stream=None, fit_rows=False,
                 one_each=False):
    """One step's pages and slots (scute_cache_assign): requests hold old_len
    [R] positions and bring new_len [R] tokens (negative: the request ends and
    its pages go back). table [R][P] and ring are updated; everything else goes
    into rows, which is returned. The next step takes rows.seq_len and
    rows.cursor as old_len and cursor and another Rows (inputs and outputs may
    not be the same tensors). fit_rows: requests with tokens past rows.max_tokens
    are refused; without it they are placed, although those tokens have no row
    (rows.cu_len[R] says how many tokens there are). one_each: row r is request
    r's one token, or empty where it brings none, ends or is refused (as with
    more than one token); rows then need no request to say whose they are."""
    R = rows.n_requests
    a = rows.args
    a.old_len, a.new_len = _vector(old_len, R, _I32, "old_len"), _vector(new_len, R, _I32, "new_len")
    if table.dtype != _I32 or table.dim() != 2 or table.shape[0] != R:
        _bad(f"table must be int32 [{R}][pages] with contiguous rows")
    P, (ts, tc) = table.shape[1], table.stride()
    if tc != 1 and P > 1:
        _bad(f"table must be int32 [{R}][pages] with contiguous rows")
    a.ring_size = size = ring.shape[0]
    a.ring, a.cursor = _vector(ring, size, _I32, "ring"), _vector(cursor, 2, _I64, "cursor")
    _gpu(rows.device, old_len, new_len, table, ring, cursor)
    a.flags = (scute.ASSIGN_FIT_ROWS if fit_rows else 0) | (scute.ASSIGN_ONE_EACH if one_each else 0)
    a.table_width, a.page_size, a.table_stride, a.table = P, page_size, ts if R > 1 else P, table.data_ptr()
    scute._check(scute.lib.scute_cache_assign(a, _stream(stream, rows.device.index)))
    return rows


# ---- requests that share pages --------------------------------------------------------------------

class Fork:
    """What fork_pages fills in for n_requests requests of up to `pages` pages
    each over a cache of n_pages: table [n_requests][pages], seq_len, and for
    each request the page to copy, where to, and its positions (src, dst, n
    [n_requests]; -1, -1, 0: none); cursor [2] (int64) and counts [4] (requests
    that hold positions, pages taken, requests refused, pages returned). The
    tensors stay the handle's, as those of Rows; cursor and seq_len are parts of
    `state`, laid out like a Rows'. The handle owns the workspace of one call at
    a time: calls that may overlap need handles of their own."""

    def __init__(self, n_requests, pages, n_pages, device=None):
        dev = torch.device("cuda" if device is None else device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.n_requests, self.pages, self.n_pages, self.device = int(n_requests), int(pages), int(n_pages), dev
        nbytes = scute.scute_cache_fork_workspace(n_requests, n_pages)
        a = self.args = scute.CacheForkArgs()
        a.device = dev.index if dev.type == "cuda" else -1
        a.n_requests, a.table_width, a.n_pages, a.table_out_stride = n_requests, pages, n_pages, pages
        self._state = torch.zeros(2 + (n_requests + 1) // 2, dtype=_I64, device=dev)
        self._filled = dict(zip(("cursor", "seq_len"), split_state(self._state, n_requests)))
        self._filled["table"] = torch.full((n_requests, pages), -1, dtype=_I32, device=dev)
        for name, m in (("src", n_requests), ("dst", n_requests), ("n", n_requests), ("counts", 4)):
            self._filled[name] = torch.zeros(m, dtype=_I32, device=dev)
        for name, t in self._filled.items():
            setattr(a, {"cursor": "cursor_out", "table": "table_out"}.get(name, name), t.data_ptr())
        self._workspace = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        a.workspace, a.workspace_bytes = self._workspace.data_ptr(), nbytes
        settle(dev)

    table, seq_len, src, dst, n, cursor, counts = (
        property(lambda self, name=name: self._filled[name])
        for name in ("table", "seq_len", "src", "dst", "n", "cursor", "counts"))
    state = property(lambda self: self._state)


def fork_pages(seq_len, parent, table, ring, cursor, page_size, fork, keep=None, window=0, sinks=0, stream=None):
    """Requests that go on from others (scute_cache_fork): request r then holds
    the first keep[r] (None: all) positions of request parent[r] (itself,
    another, or outside the requests: it ends). Whole pages are shared; a last
    page that others hold too is to be copied (copy_pages, in each layer's
    cache); pages that nobody holds any more go back to the ring; window > 0
    drops the pages between sinks and the last `window` positions (of a request
    that is refused, too: where the window is not whole pages its next rows may
    see one of them, so it is ended or read again). seq_len,
    parent, keep int32 [R]; table [R][P] is left as it is, the new one is
    fork.table. Everything but the ring goes into fork, which is returned."""
    R, P, a = fork.n_requests, fork.pages, fork.args
    a.len, a.parent = _vector(seq_len, R, _I32, "seq_len"), _vector(parent, R, _I32, "parent")
    a.keep = None if keep is None else _vector(keep, R, _I32, "keep")
    if table.dtype != _I32 or table.shape != (R, P) or (table.stride(1) != 1 and P > 1):
        _bad(f"table must be int32 [{R}][{P}] with contiguous rows")
    a.ring_size = size = ring.shape[0]
    a.ring, a.cursor = _vector(ring, size, _I32, "ring"), _vector(cursor, 2, _I64, "cursor")
    _gpu(fork.device, seq_len, parent, keep, table, ring, cursor)
    a.table, a.table_stride, a.page_size = table.data_ptr(), table.stride(0) if R > 1 else P, page_size
    a.window, a.sinks = window, sinks
    scute._check(scute.lib.scute_cache_fork(a, _stream(stream, fork.device.index)))
    return fork


def copy_pages(cache, src, dst, n, stream=None):
    """The first n[i] positions of page src[i] to page dst[i] of a KVCache
    (scute_cache_copy), int32 [m] each: a Fork's src, dst and n."""
    m = src.shape[0]
    sp, dp, np_ = _vector(src, m, _I32, "src"), _vector(dst, m, _I32, "dst"), _vector(n, m, _I32, "n")
    _gpu(cache.device, src, dst, n)
    scute._check(scute.lib.scute_cache_copy(cache.desc, sp, dp, np_, m, _stream(stream, cache.index)))


def compact(cache, table, start, kept, n_kept, new_len=None, stream=None):
    """Positions that stay, moved together (scute_cache_compact): place
    start[r] + j of request r gets what position kept[r][j] held, for
    j < n_kept[r]. kept int32 [R][places], ascending; new_len int32 [R] gets
    start + n_kept (the keep of fork_pages, which gives back the pages behind)."""
    if kept.dim() != 2 or kept.dtype != _I32 or (kept.stride(1) != 1 and kept.shape[1] > 1):
        _bad("kept must be int32 [n_requests][places] with contiguous rows")
    R, W = kept.shape
    if table.dtype != _I32 or table.dim() != 2 or table.shape[0] != R or (table.stride(1) != 1 and table.shape[1] > 1):
        _bad(f"table must be int32 [{R}][pages] with contiguous rows")
    P = table.shape[1]
    sp, kp = _vector(start, R, _I32, "start"), _vector(n_kept, R, _I32, "n_kept")
    lp = None if new_len is None else _vector(new_len, R, _I32, "new_len")
    _gpu(cache.device, table, start, kept, n_kept, new_len)
    scute._check(scute.lib.scute_cache_compact(
        cache.desc, table.data_ptr(), table.stride(0) if R > 1 else P, R, P, sp, kept.data_ptr(),
        kept.stride(0) if R > 1 else W, W, kp, lp, _stream(stream, cache.index)))


# ---- rotary positions ------------------------------------------------------------------------------

class HeadNorm:
    """Norms of q's and k's heads, each over a head's head_dim elements, before
    the rotation (Rotary.store). kind "rms" or "layer"; weights and biases
    float32 [head_dim], or [n_heads][head_dim] ([n_kv_heads][head_dim] for k's)
    for each head its own, on the GPU (None: ones, zeros)."""

    def __init__(self, head_dim, kind="rms", q_weight=None, k_weight=None, q_bias=None, k_bias=None, eps=1e-6):
        if kind not in ("rms", "layer"):
            _bad("kind must be 'rms' or 'layer'")
        self.head_dim, self._vecs, self.heads, ptrs = int(head_dim), (q_weight, q_bias, k_weight, k_bias), [], []
        for pair, name in (((q_weight, q_bias), "q"), ((k_weight, k_bias), "k")):
            heads = None
            for t in pair:
                if t is not None and (t.dtype != _F32 or t.dim() not in (1, 2) or t.shape[-1] != head_dim or
                                      not t.is_contiguous()):
                    _bad(f"{name}'s vectors must be contiguous float32 [{head_dim}] or [heads][{head_dim}]")
                ptrs.append(None if t is None else t.data_ptr())
                if t is not None:
                    own = t.shape[0] if t.dim() == 2 else 0
                    if heads not in (None, own):
                        _bad(f"{name}'s weight and bias must be of the same heads")
                    heads = own
            self.heads.append(heads or 0)
        self.device = next((t.device for t in self._vecs if t is not None), None)
        if self.device is not None:
            _gpu(self.device, *self._vecs)
        self.desc = scute.HeadNormDesc(scute.NORM_RMS if kind == "rms" else scute.NORM_LAYER, eps, *ptrs,
                                       *(head_dim if h else 0 for h in self.heads))


class Rotary:
    """Rotary positions of heads of head_dim elements: pair i of the first
    2 len(freq) elements is turned by pos[axis[i]] * freq[i] radians. freq
    float64 [rot_dim / 2] on the GPU; axis int32 [rot_dim / 2] (None: one axis
    for all); interleaved: pairs are (2i, 2i + 1) instead of
    (i, i + rot_dim / 2)."""

    def __init__(self, freq, head_dim, axis=None, n_axes=1, interleaved=False):
        n = freq.shape[0]
        _vector(freq, n, torch.float64, "freq")
        if axis is not None:
            _vector(axis, n, _I32, "axis")
        if not 0 <= 2 * n <= head_dim:
            _bad("freq holds more than head_dim / 2 pairs")
        if not 1 <= n_axes <= 8:
            _bad("n_axes must be in [1, 8]")
        _gpu(freq.device, axis)
        self.freq, self.axis, self.n_axes, self.device = freq, axis, int(n_axes), freq.device
        self.head_dim = int(head_dim)
        self.desc = scute.RotaryDesc(head_dim, 2 * n, n_axes, 1 if interleaved else 0, freq.data_ptr(),
                                     None if axis is None else axis.data_ptr())

    def store(self, q, k, v, pos, slot, cache, q_out, stream=None, norm=None):
        """q [T][n_heads][head_dim] rotated into q_out (the cache's type), k
        [T][n_kv_heads][head_dim] rotated and v as it is into the cache at slot
        [T] (int64; negative: not stored). q, k, v float32 or bfloat16, e.g.
        column ranges of one layer's output; pos int32 [n_axes][T] ([T] with
        one axis). norm: a HeadNorm that q's and k's heads go through first."""
        if q.dim() != 3:
            _bad("q must be [tokens][n_heads][head_dim]")
        T, H, D = q.shape
        if D != cache.head_dim or D != self.head_dim:
            _bad(f"q's heads, the cache's and the rotary's must have one head_dim, got {D}, {cache.head_dim} and "
                 f"{self.head_dim}")
        dt = q.dtype
        if dt not in _DTYPES or k.dtype != dt or v.dtype != dt:
            _bad("q, k and v must all be float32 or all bfloat16")
        if q_out.dtype != cache.dtype:
            _bad("q_out must have the cache's type")
        qs, ks = _heads(q, T, H, D, "q"), _heads(k, T, cache.n_kv_heads, D, "k")
        vs, os = _heads(v, T, cache.n_kv_heads, D, "v"), _heads(q_out, T, H, D, "q_out")
        sp = _vector(slot, T, _I64, "slot")
        if pos.dim() == 2:
            ok, (ps, pc) = pos.shape == (self.n_axes, T), pos.stride()
        else:
            ok, ps, pc = pos.shape == (T,) and self.n_axes == 1, 0, 1 if pos.is_contiguous() else 0
        if not ok or pos.dtype != _I32 or (pc != 1 and T > 1):
            _bad(f"pos must be int32 [{self.n_axes}][{T}] with contiguous rows")
        _gpu(cache.device, self.freq, q, k, v, pos, slot, q_out)
        call, desc = scute.lib.scute_rotary_store, (self.desc,)
        if norm is not None:
            if norm.head_dim != D or norm.heads[0] not in (0, H) or norm.heads[1] not in (0, cache.n_kv_heads):
                _bad(f"the norm's vectors must be of {D} elements, and of all heads or of {H} and {cache.n_kv_heads}")
            if norm.device is not None and norm.device != cache.device:
                _bad(f"tensors on {norm.device} and {cache.device} in one call")
            call, desc = scute.lib.scute_norm_rotary_store, (self.desc, norm.desc)
        scute._check(call(
            *desc, cache.desc, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPES[dt],
            pos.data_ptr(), ps, sp, T, H, q_out.data_ptr(), os, _stream(stream, cache.index)))
        return q_out


# ---- attention -----------------------------------------------------------------------------------

class PagedAttention:
    """Attention of new tokens over a KVCache with n_heads query heads
    (n_heads / n_kv_heads of them share a key head). scale: 1 / sqrt(head_dim)
    by default; window: a row sees its last `window` positions (0: all);
    sinks: and the first `sinks`, which stay visible. max_rows: calls of more rows are refused (None: up to 2^20).

    The handle owns the workspace of one call at a time: calls that may
    overlap (other streams, graphs replayed side by side) need handles of their
    own."""

    def __init__(self, cache, n_heads, max_rows=None, scale=None, window=0, sinks=0):
        if n_heads < 1 or n_heads % cache.n_kv_heads:
            _bad("n_heads must be a multiple of the cache's n_kv_heads")
        if window < 0:
            _bad("window must be >= 0")
        if sinks < 0:
            _bad("sinks must be >= 0")
        self.cache, self.n_heads, self.window, self.sinks = cache, int(n_heads), int(window), int(sinks)
        self.scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else float(scale)
        nbytes = scute.scute_paged_attention_workspace(cache.device.index, cache.head_dim)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=cache.device)
        self.max_rows = None if max_rows is None else int(max_rows)
        settle(cache.device)

    def forward(self, q, table, row_len, out, row_req=None, stream=None):
        """q, out [rows][n_heads][head_dim] (the cache's type); table int32
        [n_requests][pages]; row_len int32 [rows]: row i sees positions below
        row_len[i] of request row_req[i] (None: request i). Rows that see
        nothing give zeros."""
        c = self.cache
        N, D, H = q.shape[0], c.head_dim, self.n_heads
        qs, os = _heads(q, N, H, D, "q"), _heads(out, N, H, D, "out")
        if self.max_rows is not None and N > self.max_rows:
            _bad(f"{N} rows: the handle takes up to {self.max_rows}")
        if q.dtype != c.dtype or out.dtype != c.dtype:
            _bad("q and out must have the cache's type")
        if table.dtype != _I32 or table.dim() != 2:
            _bad("table must be int32 [n_requests][pages] with contiguous rows")
        (R, P), (ts, tc) = table.shape, table.stride()
        if tc != 1 and P > 1:
            _bad("table must be int32 [n_requests][pages] with contiguous rows")
        lp, rp = _vector(row_len, N, _I32, "row_len"), None
        if row_req is not None:
            rp = _vector(row_req, N, _I32, "row_req")
        elif N > R:
            _bad("more rows than requests: row_req says whose they are")
        _gpu(c.device, q, table, row_len, out, row_req)
        ws = self.workspace
        call, seen = scute.lib.scute_paged_attention, (self.window,)
        if self.sinks:
            call, seen = scute.lib.scute_sink_attention, (self.window, self.sinks)
        scute._check(call(
            c.desc, q.data_ptr(), qs if N > 1 else 0, H, table.data_ptr(), ts if R > 1 else P, R, P, lp, rp, N,
            self.scale, *seen, out.data_ptr(), os if N > 1 else 0, ws.data_ptr(), ws.shape[0],
            _stream(stream, c.index)))
        return out


class SharedAttention:
    """Attention over a KVCache of rows whose contexts begin with the same
    positions (samples of a prompt, users of a system prompt): those are read
    once for all rows of a group. Up to max_rows rows in up to max_groups groups
    a call; scale as in PagedAttention, and as there the handle owns the
    workspace of one call at a time (for 32 query and 8 key heads of 128
    227 MB for 4 rows of one group, 240 for 128 rows). Calls that sharing could not save the reads of
    256 MiB, if all rows past one a group shared the table's whole width, are
    PagedAttention's (the library's rule: the shared lengths are on the GPU), with
    `always` none. So with a table much wider than what is shared (AttentionStep's
    is as wide as its requests may get) rows that share little take longer than
    PagedAttention's."""

    def __init__(self, cache, n_heads, max_rows, max_groups, scale=None, always=False):
        if n_heads < 1 or n_heads % cache.n_kv_heads:
            _bad("n_heads must be a multiple of the cache's n_kv_heads")
        self.cache, self.n_heads = cache, int(n_heads)
        self.max_rows, self.max_groups = int(max_rows), int(max_groups)
        self.flags = scute.SHARED_ALWAYS if always else 0
        self.scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else float(scale)
        nbytes = scute.scute_shared_attention_workspace(cache.device.index, _DTYPES[cache.dtype], cache.head_dim,
                                                        self.n_heads, cache.n_kv_heads, max_rows, max_groups)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=cache.device)
        settle(cache.device)

    def forward(self, q, table, row_len, group, shared_len, out, row_req=None, stream=None):
        """q, table, row_len, out, row_req as in PagedAttention.forward. group
        int32 [n_groups + 1]: rows group[g] .. group[g + 1] - 1 hold the first
        shared_len[g] (int32 [n_groups]) positions of their requests in the
        same pages."""
        c = self.cache
        N, D, H = q.shape[0], c.head_dim, self.n_heads
        qs, os = _heads(q, N, H, D, "q"), _heads(out, N, H, D, "out")
        n_groups = shared_len.shape[0]
        if N > self.max_rows or n_groups > self.max_groups:
            _bad(f"{N} rows in {n_groups} groups: the handle takes up to {self.max_rows} in {self.max_groups}")
        if q.dtype != c.dtype or out.dtype != c.dtype:
            _bad("q and out must have the cache's type")
        if table.dtype != _I32 or table.dim() != 2:
            _bad("table must be int32 [n_requests][pages] with contiguous rows")
        (R, P), (ts, tc) = table.shape, table.stride()
        if tc != 1 and P > 1:
            _bad("table must be int32 [n_requests][pages] with contiguous rows")
        lp, rp = _vector(row_len, N, _I32, "row_len"), None
        if row_req is not None:
            rp = _vector(row_req, N, _I32, "row_req")
        elif N > R:
            _bad("more rows than requests: row_req says whose they are")
        gp, sp = _vector(group, n_groups + 1, _I32, "group"), _vector(shared_len, n_groups, _I32, "shared_len")
        _gpu(c.device, q, table, row_len, group, shared_len, out, row_req)
        ws = self.workspace
        scute._check(scute.lib.scute_shared_attention(
            c.desc, q.data_ptr(), qs if N > 1 else 0, H, table.data_ptr(), ts if R > 1 else P, R, P, lp, rp, N, gp, sp,
            n_groups, self.scale, out.data_ptr(), os if N > 1 else 0, ws.data_ptr(), ws.shape[0], self.flags,
            _stream(stream, c.index)))
        return out


# ---- the norms around the residual ---------------------------------------------------------------

class ResidualNorm:
    """h' = h_scale h + y_scale (gate (.) N_post(y)), x = N_pre(h') for rows of
    d elements. kind "rms" or "layer"; post: whether y goes through N_post; the
    weights and biases are float32 [d] (None: ones, zeros)."""

    def __init__(self, d, kind="rms", post=False, post_weight=None, post_bias=None, pre=True, pre_weight=None,
                 pre_bias=None, h_scale=1.0, y_scale=1.0, eps=1e-5, device=None):
        if kind not in ("rms", "layer"):
            _bad("kind must be 'rms' or 'layer'")
        vecs = (post_weight, post_bias, pre_weight, pre_bias)
        if not post and (post_weight is not None or post_bias is not None):
            _bad("post weights without post")
        if not pre and (pre_weight is not None or pre_bias is not None):
            _bad("pre weights without pre")
        for t, name in zip(vecs, ("post_weight", "post_bias", "pre_weight", "pre_bias")):
            if t is not None:
                _vector(t, d, _F32, name)
        dev = next((t.device for t in vecs if t is not None), torch.device("cuda" if device is None else device))
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        _gpu(dev, *vecs)
        self.d, self.pre, self.device, self._vecs = int(d), bool(pre), dev, vecs
        self.desc = scute.NormDesc(dev.index, scute.NORM_RMS if kind == "rms" else scute.NORM_LAYER, d,
                                   1 if post else 0, eps, h_scale, y_scale, 0,
                                   *[None if t is None else t.data_ptr() for t in vecs])

    def _rows(self, t, n, name):
        if t.shape != (n, self.d):
            _bad(f"{name} must be [{n}][{self.d}]")
        a, b = t.stride()
        if b != 1 and self.d > 1:
            _bad(f"{name} must have contiguous rows")
        dt = _DTYPES.get(t.dtype)
        if dt is None:
            _bad(f"{name} must be float32 or bfloat16")
        return t.data_ptr(), dt, a if n > 1 else 0

    def forward(self, y, h, h_out, x=None, gate=None, stream=None):
        """y [T][d] (a layer's output; None: h' = h_scale h), h [T][d], gate
        float32 [d] or [T][d]; h_out [T][d] in h's type (None: not written; may
        be h), x [T][d] (with pre). Returns (h_out, x)."""
        n = h.shape[0]
        if self.pre != (x is not None):
            _bad("x is given exactly when the handle has a pre norm")
        hp = self._rows(h, n, "h")
        yp = (None, 0, 0) if y is None else self._rows(y, n, "y")
        op = (None, 0, 0) if h_out is None else self._rows(h_out, n, "h_out")
        xp = (None, 0, 0) if x is None else self._rows(x, n, "x")
        if h_out is not None and h_out.dtype != h.dtype:
            _bad("h_out must have h's type")
        gp, gs = None, 0
        if gate is not None:
            if gate.dim() == 1:
                gp = _vector(gate, self.d, _F32, "gate")
            else:
                gp, gt, gs = self._rows(gate, n, "gate")
                if gt != scute.F32:
                    _bad("gate must be float32")
            if y is None:
                _bad("a gate without y")
        _gpu(self.device, y, h, h_out, x, gate)
        scute._check(scute.lib.scute_residual_norm(
            self.desc, yp[0], yp[1], yp[2], hp[0], hp[1], hp[2], gp, gs, op[0], op[2], xp[0], xp[1], xp[2], n,
            _stream(stream, self.device.index)))
        return h_out, x

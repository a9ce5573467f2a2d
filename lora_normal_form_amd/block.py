"""What runs between the adapter layers of a decoder block, on torch tensors:
the steps from the q / k / v layer's output to the output projection's input,
and the norms around the residual.

  assign_pages    pages and slots of a step's tokens from the requests'
                  lengths, on the GPU (scute_cache_assign)
  Rotary.store    rotary positions with several axes; k and v into the paged
                  cache (scute_rotary_store)
  PagedAttention  attention of new tokens over the paged cache
                  (scute_paged_attention)
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


# ---- rotary positions ------------------------------------------------------------------------------

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

    def store(self, q, k, v, pos, slot, cache, q_out, stream=None):
        """q [T][n_heads][head_dim] rotated into q_out (the cache's type), k
        [T][n_kv_heads][head_dim] rotated and v as it is into the cache at slot
        [T] (int64; negative: not stored). q, k, v float32 or bfloat16, e.g.
        column ranges of one layer's output; pos int32 [n_axes][T] ([T] with
        one axis)."""
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
        scute._check(scute.lib.scute_rotary_store(
            self.desc, cache.desc, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPES[dt],
            pos.data_ptr(), ps, sp, T, H, q_out.data_ptr(), os, _stream(stream, cache.index)))
        return q_out


# ---- attention -----------------------------------------------------------------------------------

class PagedAttention:
    """Attention of new tokens over a KVCache with n_heads query heads
    (n_heads / n_kv_heads of them share a key head). scale: 1 / sqrt(head_dim)
    by default; window: a row sees its last `window` positions (0: all).
    max_rows: calls of more rows are refused (None: up to 2^20).

    The handle owns the workspace of one call at a time: calls that may
    overlap (other streams, graphs replayed side by side) need handles of their
    own."""

    def __init__(self, cache, n_heads, max_rows=None, scale=None, window=0):
        if n_heads < 1 or n_heads % cache.n_kv_heads:
            _bad("n_heads must be a multiple of the cache's n_kv_heads")
        if window < 0:
            _bad("window must be >= 0")
        self.cache, self.n_heads, self.window = cache, int(n_heads), int(window)
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
        scute._check(scute.lib.scute_paged_attention(
            c.desc, q.data_ptr(), qs if N > 1 else 0, H, table.data_ptr(), ts if R > 1 else P, R, P, lp, rp, N,
            self.scale, self.window, out.data_ptr(), os if N > 1 else 0, ws.data_ptr(), ws.shape[0],
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

"""The attention step with requests that go on from others: norms of heads,
shared attention or a window with first positions, forks and compaction run
together, each stage checked on what the stages before it left on the GPU, at
the bounds of the operators' own tests."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_normal_form_amd import block, scute  # noqa: E402
from test_block_gpu import BF16, DEV, U, _assign_ref, _close, _int  # noqa: E402
from test_block_step_gpu import D, H, HK, N, P, PS, R, _step  # noqa: E402
from test_head_norm_gpu import norm_ref, turned  # noqa: E402
from test_pages_gpu import _compact_ref, fork_ref  # noqa: E402
from test_shared_gpu import WEIGHT  # noqa: E402
from test_sinks_gpu import attend_ref, close, visible  # noqa: E402

pytestmark = pytest.mark.gpu

PAGES = 30


class Steps:
    """A step and what its requests hold, in plain loops."""

    def __init__(self, seed, window=0, sinks=0, **kw):
        if not torch.cuda.is_available():
            pytest.skip("no GPU")
        g = torch.Generator().manual_seed(seed)
        self.qw, self.kw = (1.0 + 0.2 * torch.randn(D, generator=g), 1.0 + 0.2 * torch.randn(HK, D, generator=g))
        norm = block.HeadNorm(D, "rms", self.qw.to(DEV), self.kw.to(DEV), eps=1e-5)
        self.st, *_, self.freq = _step(seed, head_norm=norm, window=window, sinks=sinks, forks=True, **kw)
        if self.st.group is not None:
            self.st.attention.flags = scute.SHARED_ALWAYS
        self.window, self.sinks, self.g = window, sinks, g
        self.table, self.ring = self.st.table.cpu().numpy().astype(np.int64), np.arange(PAGES)
        self.lens, self.cursor = np.zeros(R, np.int64), (0, PAGES)

    def same(self):
        st = self.st
        cursor, seq_len = block.split_state(st.state, R)
        assert seq_len.tolist() == list(self.lens) and cursor.tolist() == list(self.cursor)
        assert np.array_equal(st.ring.cpu().numpy(), self.ring)
        for r in range(R):  # (entries behind a request's pages hold anything)
            held = -(-int(self.lens[r]) // PS)
            assert np.array_equal(st.table[r, :held].cpu().numpy(), self.table[r, :held]), r

    def forward(self, new, group=(), shared=()):
        st = self.st
        h = torch.randn((N, H * D), generator=self.g).to(DEV)
        if st.group is not None:
            st.group.copy_(_int(list(group) + [group[-1] if group else 0] * (len(st.group) - len(group))))
            st.shared_len.copy_(_int(list(shared) + [0] * (len(st.shared_len) - len(shared))))
        k0, v0 = st.cache.k.cpu().double(), st.cache.v.cpu().double()
        st.forward(h, _int(new), torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV))
        torch.cuda.synchronize()
        self.table, self.ring, rows = _assign_ref(self.lens, np.maximum(0, new), self.table, self.ring, *self.cursor, PS,
                                                  N)
        for name, v in rows.items():
            assert np.array_equal(getattr(st.rows, name).cpu().numpy(), v), name
        self.lens, self.cursor = rows["seq_len"], tuple(rows["cursor"])
        self.same()
        # norms of heads, rotary and the cache
        y = st.qkv.y.cpu().double()
        ang = torch.as_tensor(rows["pos"]).double()[:, None] * self.freq.cpu()
        got = []
        for a, heads, w in ((0, H, self.qw), (H * D, HK, self.kw)):
            z = y[:, a:a + heads * D].unflatten(1, (heads, D))
            x, tol = turned(*norm_ref(z, "rms", w, None, 1e-5), ang, D // 2, False)
            got.append((x, tol + U[BF16] * (x.abs() + tol)))
        _close(st.q_rot, *got[0], "q")
        tol_k = torch.zeros_like(k0)
        for t in np.flatnonzero(rows["slot"] >= 0):
            at = divmod(int(rows["slot"][t]), PS)
            k0[at], tol_k[at], v0[at] = got[1][0][t], got[1][1][t], y[t, (H + HK) * D:].view(HK, D).to(BF16)
        _close(st.cache.k, k0, tol_k, "k")
        v_same = torch.equal(st.cache.v.cpu().double(), v0)
        assert v_same
        ref, tol = attend_ref(st.q_rot, st.cache.k, st.cache.v, st.table, rows["len"], rows["req"],
                              visible(self.window, self.sinks), 1 / math.sqrt(D),
                              **({} if st.group is None else dict(weight=WEIGHT)))
        close(st.a, ref, tol, "attention")

    def forked(self, f, parent, keep, drop, k, v):
        want, self.ring = fork_ref(self.lens, parent, keep, self.table, self.ring, *self.cursor, PS, PAGES,
                                   self.window if drop else 0, self.sinks)
        for name, z in want.items():
            assert np.array_equal(getattr(f, name).cpu().numpy(), z), name
        for a, b, n in zip(want["src"], want["dst"], want["n"]):
            if n:
                k[b, :n], v[b, :n] = k[a, :n].clone(), v[a, :n].clone()
        assert torch.equal(self.st.cache.k.cpu(), k) and torch.equal(self.st.cache.v.cpu(), v)
        self.table, self.lens, self.cursor = want["table"], want["seq_len"], tuple(want["cursor"])
        self.same()
        # no page is in the ring that a request holds, or twice anywhere
        free = [int(self.ring[c % PAGES]) for c in range(*self.cursor)]
        held = {int(e) for r in range(R) for e in self.table[r] if e >= 0}
        assert sorted(free + list(held)) == list(range(PAGES))

    def fork(self, parent, keep=None, drop=False):
        k, v = self.st.cache.k.cpu(), self.st.cache.v.cpu()
        f = self.st.fork(_int(parent), None if keep is None else _int(keep), drop=drop)
        self.forked(f, parent, keep, drop, k, v)

    def keep_only(self, start, kept, n_kept):
        k, v = (_compact_ref(z.cpu(), self.table, start, np.asarray(kept), n_kept, PS) for z in (self.st.cache.k, self.st.cache.v))
        f = self.st.keep_only(_int(start), _int(kept), _int(n_kept))
        self.forked(f, range(R), np.add(start, n_kept), False, k, v)

    def close(self):
        self.st.close()
        self.st.qkv.close()


def test_samples_of_a_prompt_run_together():
    s = Steps(41, groups=3)
    s.forward([18, 0, 0, 0, 5])
    s.fork([0, 0, 0, 0, 4])  # three more samples, and a request of its own
    s.forward([1, 1, 1, 1, 1], group=[0, 4], shared=[16])
    s.forward([3, 4, 3, 2, 2], group=[0, 12, 14], shared=[16, 4])  # drafts
    s.keep_only([19, 19, 19, 19, 6], [[20, 21, 0], [19, 22, 0], [19, 0, 0], [0, 0, 0], [6, 7, 0]], [2, 2, 1, 0, 2])
    s.forward([1, -1, 1, 1, 0], group=[0, 3], shared=[16])  # (a negative length: no tokens)
    s.fork([2, 1, 2, 9, 4], keep=[30, 17, 30, 30, 0])  # beams: the best twice, one cut back, two end
    s.forward([1, 1, 1, 0, 7], group=[0, 3], shared=[16])
    s.fork([4, 4, 4, 4, 4])  # the prompt's own pages go back
    s.forward([2, 2, 2, 2, 2], group=[0, 10], shared=[4])
    s.fork([-1] * 5)
    assert s.cursor[1] - s.cursor[0] == PAGES
    s.forward([0] * 5)
    s.close()


def test_a_window_over_forks():
    s = Steps(42, window=6, sinks=3)
    s.forward([19, 0, 0, 3, 0])
    s.fork([0, 0, 3, 3, 9], drop=True)
    for _ in range(3):
        s.forward([1, 2, 1, 2, 1])
        s.fork([0, 1, 2, 3, 4], drop=True)
    s.fork([1, 1, 0, 3, 4])
    s.forward([1, 1, 1, 4, 1])
    s.close()


def test_captured_steps_match_eager():
    """Each replay is another step, fork and compaction: what eager calls leave."""
    steps = [Steps(43, groups=2).st for _ in range(2)]
    h = torch.zeros((N, H * D), device=DEV)
    new, parent, start, n_kept = (_int(np.zeros(R)) for _ in range(4))
    kept = _int(np.zeros((R, 2)))
    outs = [(torch.empty_like(h), torch.empty((N, H * D), dtype=BF16, device=DEV)) for _ in steps]

    def one(st, out):
        st.forward(h, new, *out)
        st.keep_only(start, kept, n_kept)
        st.fork(parent)

    parent.copy_(_int(range(R)))
    for st, out in zip(steps, outs):
        one(st, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(steps[1], outs[1])
    g = torch.Generator().manual_seed(8)
    far = [50] * R
    for i, (n, par, a, kp, nk, grp, sh) in enumerate((
            ([17, 0, 0, 0, 3], [0, 0, 0, 0, 4], [17, 0, 0, 0, 3], [[0, 0]] * R, [0] * R, [0, 0, 0], [0, 0]),
            ([2, 2, 2, 2, 2], [0, 1, 2, 3, 4], [17, 17, 17, 17, 3], [[18, 0], [17, 18], [18, 0], [17, 0], [4, 0]],
             [1, 2, 1, 1, 1], [0, 8, 8], [16, 0]),
            ([1, 1, 1, 1, 1], [1, 1, 0, 3, 4], far, [[0, 0]] * R, [0] * R, [0, 4, 5], [16, 4]),
            ([1, 1, 1, 1, 1], [9, 1, 1, 9, 4], far, [[0, 0]] * R, [0] * R, [0, 4, 4], [16, 0]),
            ([0, 1, 1, 0, 1], [4, 4, 4, 4, 4], far, [[0, 0]] * R, [0] * R, [0, 2, 2], [16, 0]))):
        h.copy_(torch.randn((N, H * D), generator=g))
        for t, z in ((new, n), (parent, par), (start, a), (kept, kp), (n_kept, nk)):
            t.copy_(_int(z))
        for st in steps:
            st.group.copy_(_int(grp)), st.shared_len.copy_(_int(sh))
        one(steps[0], outs[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        x, y = steps
        for name in ("state", "table", "ring", "a", "q_rot"):
            assert torch.equal(getattr(x, name), getattr(y, name)), (i, name)
        assert torch.equal(x.cache.k, y.cache.k) and torch.equal(x.cache.v, y.cache.v) and torch.equal(*(o[1] for o in outs))
    assert min(block.split_state(steps[0].state, R)[1].tolist()) > 0
    for st in steps:
        st.close()
        st.qkv.close()


def test_steps_refuse():
    s = Steps(44)
    from lora_normal_form_amd import multiproj
    st = s.st
    with pytest.raises(ValueError, match="new_len"):
        st.forward(None, torch.ones(R - 1, dtype=torch.int32, device=DEV), None, None)
    plain, wls, wl_out, w, freq = _step(45)
    for call in (lambda: plain.fork(_int(range(R))), lambda: plain.keep_only(*[_int(range(R))] * 3)):
        with pytest.raises(ValueError, match="without forks"):
            call()
    with pytest.raises(ValueError, match="none"):
        multiproj.AttentionStep(plain.qkv, wl_out, H, HK, D, R, P, PS, PAGES, freq, like=plain, forks=True)
    with pytest.raises(ValueError, match="without a window"):
        multiproj.AttentionStep(plain.qkv, wl_out, H, HK, D, R, P, PS, PAGES, freq, window=4, groups=1)
    plain.close()
    plain.qkv.close()
    s.close()


def test_steps_that_share_a_cache_have_one_window():
    """fork(drop=True) gives back pages that its own window does not see, so another
    step on the same requests may not see more."""
    from lora_normal_form_amd import multiproj
    s = Steps(46, window=6, sinks=3)
    st = s.st
    same = _step(46, window=6, sinks=3, forks=True, like=st)[0]
    for window, sinks, groups in ((0, 0, 0), (7, 3, 0), (6, 2, 0), (0, 0, 2)):
        with pytest.raises(ValueError, match="window"):
            _step(46, window=window, sinks=sinks, groups=groups, forks=True, like=st)
    same.close()
    same.qkv.close()
    s.close()

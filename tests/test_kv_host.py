"""The paged cache's host side: the page pool against a plain model of it, the
entry points' refusals, and the oracle against dense formulas.  CPU only."""
import ctypes
import random

import numpy as np
import pytest
import torch

from oracle import ptl_oracle as O
from packed_sequence_transformer_b200 import build as B


@pytest.fixture(scope="module")
def P():
    B.build()
    from packed_sequence_transformer_b200 import ptl
    ptl.lib()
    return ptl


def _status(P, fn, *args):
    with pytest.raises(P.PtlError) as e:
        fn(*args)
    return e.value.name


# ------------------------------------------------------------------- pool
class Model:
    """Sequences as lists of owned tokens' page contents: what each page holds
    is the set of (sequence, page index) that refer to it."""

    def __init__(self, pages, seqs):
        self.free = set(range(pages))
        self.lists = [[] for _ in range(seqs)]
        self.lens = [0] * seqs

    def refs(self, p):
        return sum(lst.count(p) for lst in self.lists)

    def take(self):
        p = min(self.free)
        self.free.remove(p)
        return p

    def drop(self, p):
        if p >= 0 and self.refs(p) == 0:
            self.free.add(p)

    def reserve(self, seqs, lens):
        need = sum(-(-n // 64) - len(self.lists[s]) for s, n in zip(seqs, lens))
        if need > len(self.free):
            return False
        for s, n in zip(seqs, lens):
            while len(self.lists[s]) < -(-n // 64):
                self.lists[s].append(self.take())
            self.lens[s] = n
        return True

    def fork(self, src, dst):
        if sum(self.lens[s] % 64 != 0 for s in src) > len(self.free):
            return None
        out = []
        for s, d in zip(src, dst):
            self.lists[d] = list(self.lists[s][:self.lens[s] // 64])
            if self.lens[s] % 64:
                p = self.take()
                out.append((self.lists[s][-1], p))
                self.lists[d].append(p)
            self.lens[d] = self.lens[s]
        return out

    def release(self, s):
        old, self.lists[s], self.lens[s] = self.lists[s], [], 0
        for p in old:
            self.drop(p)

    def trim(self, s, window, sinks):
        for k, p in enumerate(self.lists[s]):
            seen = any(t < sinks or self.lens[s] - t < window for t in range(64 * k, 64 * k + 64))
            if not seen and p >= 0:
                self.lists[s][k] = -1
                self.drop(p)

    def compact(self):
        pages = {p for lst in self.lists for p in lst if p >= 0}
        n = len(pages)
        moves = list(zip(sorted(p for p in pages if p >= n), sorted(set(range(n)) - pages)))
        to = dict(moves)
        self.lists = [[to.get(p, p) for p in lst] for lst in self.lists]
        self.free = set(range(n, n + len(self.free)))
        return moves


@pytest.mark.parametrize("seed", range(6))
def test_pool_against_a_model(P, seed):
    rng = random.Random(seed)
    pages, seqs = rng.choice([5, 40, 200]), rng.choice([2, 9])
    pool, m = P.KvPool(pages, seqs), Model(pages, seqs)
    for _ in range(400):
        op = rng.choice(["reserve", "reserve", "reserve", "fork", "release", "trim", "compact"])
        some = rng.sample(range(seqs), rng.randint(1, seqs))
        if op == "reserve":
            lens = [m.lens[s] + rng.choice([0, 1, 3, 64, 200]) for s in some]
            if m.reserve(some, lens):
                pool.reserve(some, lens)
            else:
                assert _status(P, pool.reserve, some, lens) == "PTL_ERR_CACHE_FULL"
        elif op == "fork":
            dst = [s for s in some if not m.lists[s]]
            src = [rng.choice([s for s in range(seqs) if s not in dst] or [0]) for _ in dst]
            if any(s in dst for s in src):
                continue
            want = m.fork(src, dst)
            if want is None:
                assert _status(P, pool.fork, src, dst) == "PTL_ERR_CACHE_FULL"
            else:
                a, b = pool.fork(src, dst)
                assert list(zip(a.tolist(), b.tolist())) == want
        elif op == "release":
            pool.release(some[:2])
            for s in some[:2]:
                m.release(s)
        elif op == "trim":
            w, k, before = rng.choice([1, 2, 64, 65, 300]), rng.choice([0, 1, 64, 65, 200]), len(m.free)
            freed = pool.trim(some, w, k)
            for s in some:
                m.trim(s, w, k)
            assert freed == len(m.free) - before
        else:
            a, b = pool.compact()
            assert list(zip(a.tolist(), b.tolist())) == m.compact()
        assert pool.free_pages == len(m.free)
        width = max(1, max(len(x) for x in m.lists))
        assert pool.table(range(seqs), width).tolist() == [x + [-1] * (width - len(x)) for x in m.lists]
        assert [pool.length(s) for s in range(seqs)] == m.lens


def test_pool_refusals_change_nothing(P):
    pool = P.KvPool(10, 4)
    pool.reserve([0, 1], [100, 64])
    before = pool.table(range(4), 10).tolist(), pool.free_pages
    for args in [([0, 0], [101, 102]), ([4], [1]), ([-1], [1]), ([0], [99])]:
        assert _status(P, pool.reserve, *args) == "PTL_ERR_SHAPE"
    assert _status(P, pool.reserve, [2, 3], [200, 64 * 8]) == "PTL_ERR_CACHE_FULL"
    assert _status(P, pool.reserve, [2, 3], [2 ** 31 - 1, 2 ** 31 - 1]) == "PTL_ERR_CACHE_FULL"
    for args in [([0], [1]), ([0], [0]), ([2], [3, 3]), ([0, 0], [2, 2]), ([2], [2]), ([4], [2]), ([0], [-1]),
                 ([0, 2], [2, 3])]:
        with pytest.raises((P.PtlError, ValueError)):
            pool.fork(*args)
    for args in [([4],), ([0, -1],)]:
        assert _status(P, pool.release, *args) == "PTL_ERR_SHAPE"
    assert _status(P, pool.trim, [0], 0) == "PTL_ERR_BAD_MASK"
    assert _status(P, pool.trim, [0], 5, -1) == "PTL_ERR_BAD_MASK"
    assert _status(P, pool.trim, [9], 5) == "PTL_ERR_SHAPE"
    assert _status(P, pool.table, [0], 1) == "PTL_ERR_SHAPE"
    assert pool.length(4) == -1 and pool.length(-1) == -1
    assert (pool.table(range(4), 10).tolist(), pool.free_pages) == before
    with pytest.raises(P.PtlError):
        P.KvPool(0, 1)
    with pytest.raises(P.PtlError):
        P.KvPool(1, 0)
    L, n = P.lib(), ctypes.c_int32()
    assert L.ptl_kv_pool_create(1, 1, None) == P.STATUS_CODE["PTL_ERR_NULL"]
    assert L.ptl_kv_pool_reserve(None, None, None, 0) == P.STATUS_CODE["PTL_ERR_NULL"]
    assert L.ptl_kv_pool_compact(pool._p, 0, None, None, ctypes.byref(n)) == 0 and n.value == 0
    pool.release([0, 0, 0])  # the same sequence again: empty by then
    assert pool.free_pages == 9
    # too little room for the list of moves
    assert L.ptl_kv_pool_compact(pool._p, 0, None, None, ctypes.byref(n)) == P.STATUS_CODE["PTL_ERR_SHAPE"]
    assert n.value == 1 and pool.table([1], 1).tolist() == [[2]]
    L.ptl_kv_pool_destroy(None)


# ---------------------------------------------------------- entry points
FAKE = 0x10000  # aligned, never dereferenced: validation fails first


def test_entry_points_refuse(P):
    L, C = P.lib(), P.STATUS_CODE
    kv = P.KvPagesStruct(FAKE, FAKE, 4)
    wsb = L.ptl_attention_paged_workspace_size(64, 4, 1)
    assert wsb > 0
    for bad in [(-1, 1, 1), (2 ** 31, 1, 1), (1, 0, 1), (1, 1, 7)]:
        assert L.ptl_attention_paged_workspace_size(*bad) == 0

    def append(qkv=FAKE, cu=FAKE, U=2, T=10, dt=1, kv=kv, tab=FAKE, mp=3, past=FAKE, ws=FAKE, wsb=256):
        return L.ptl_kv_append(qkv, cu, U, T, dt, ctypes.byref(kv) if kv else None, tab, mp, past, ws, wsb, None)

    def attend(qkv=FAKE, out=FAKE, cu=FAKE, U=2, T=10, dt=1, kv=kv, tab=FAKE, mp=3, past=FAKE, win=0, sinks=0,
               ws=FAKE, wsb=wsb):
        return L.ptl_attention_paged(qkv, out, cu, U, T, dt, ctypes.byref(kv) if kv else None, tab, mp, past, win,
                                     sinks, ws, wsb, None)

    for call in (append, attend):
        assert call(dt=7) == C["PTL_ERR_DTYPE"]
        for over in [dict(U=0), dict(U=2 ** 30 + 1), dict(T=-1), dict(T=2 ** 31), dict(mp=0), dict(mp=2 ** 25), dict(mp=-4),
                     dict(kv=P.KvPagesStruct(FAKE, FAKE, 0))]:
            assert call(**over) == C["PTL_ERR_SHAPE"]
        for over in [dict(qkv=None), dict(cu=None), dict(tab=None), dict(past=None), dict(ws=None), dict(kv=None),
                     dict(kv=P.KvPagesStruct(None, FAKE, 4)), dict(kv=P.KvPagesStruct(FAKE, None, 4))]:
            assert call(**over) == C["PTL_ERR_NULL"]
        for over in [dict(qkv=FAKE + 8), dict(cu=FAKE + 2), dict(tab=FAKE + 2), dict(past=FAKE + 1),
                     dict(ws=FAKE + 128), dict(kv=P.KvPagesStruct(FAKE + 8, FAKE, 4)),
                     dict(kv=P.KvPagesStruct(FAKE, FAKE + 2, 4))]:
            assert call(**over) == C["PTL_ERR_ALIGN"]
        assert call(wsb=255) == C["PTL_ERR_WORKSPACE"]
        assert call(T=0, qkv=None, kv=None, tab=None) == C["PTL_OK"]
    assert attend(wsb=wsb - 1) == C["PTL_ERR_WORKSPACE"]
    assert attend(out=None) == C["PTL_ERR_NULL"] and attend(out=FAKE + 4) == C["PTL_ERR_ALIGN"]
    assert attend(sinks=-1) == C["PTL_ERR_BAD_MASK"]

    def copy(kv=kv, src=FAKE, dst=FAKE, n=3, ws=FAKE, wsb=256):
        return L.ptl_kv_copy_pages(ctypes.byref(kv) if kv else None, src, dst, n, ws, wsb, None)

    assert copy(n=0, src=None) == C["PTL_OK"]
    assert copy(n=-1) == C["PTL_ERR_SHAPE"] and copy(n=2 ** 31) == C["PTL_ERR_SHAPE"]
    assert copy(src=None) == C["PTL_ERR_NULL"] and copy(kv=None) == C["PTL_ERR_NULL"]
    assert copy(dst=FAKE + 2) == C["PTL_ERR_ALIGN"] and copy(ws=FAKE + 8) == C["PTL_ERR_ALIGN"]
    assert copy(wsb=0) == C["PTL_ERR_WORKSPACE"]


def test_binding_refuses(P):
    kv = P.KvPages(torch.zeros(3, 2, 8, 64, 64, dtype=torch.uint8), torch.ones(3, 2, 8))
    for codes, scales in [(torch.zeros(3, 2, 8, 64, 64), torch.ones(3, 2, 8)),
                          (torch.zeros(3, 2, 8, 64, 32, dtype=torch.uint8), torch.ones(3, 2, 8)),
                          (kv.codes, torch.ones(2, 2, 8)), (kv.codes, torch.ones(3, 2, 8, dtype=torch.float64)),
                          (kv.codes[:, :, :, :, ::2], kv.scales)]:
        with pytest.raises(ValueError):
            P.KvPages(codes, scales)
    i32 = dict(dtype=torch.int32)
    good = dict(qkv=torch.zeros(5, 1536), cu=torch.zeros(3, **i32), table=torch.zeros(2, 4, **i32),
                past=torch.zeros(2, **i32), ws=torch.zeros(256, dtype=torch.uint8), attn=torch.zeros(5, 512))
    for over in [dict(qkv=torch.zeros(5, 512)), dict(qkv=torch.zeros(5, 3, 512)), dict(cu=torch.zeros(4, **i32)),
                 dict(cu=torch.zeros(3, dtype=torch.int64)), dict(table=torch.zeros(3, 4, **i32)),
                 dict(table=torch.zeros(2, 4, dtype=torch.int64)), dict(past=torch.zeros(2, dtype=torch.int64)),
                 dict(attn=torch.zeros(5, 512, dtype=torch.bfloat16)), dict(attn=torch.zeros(4, 512)),
                 dict(table=torch.zeros(4, 2, **i32).t()), dict(qkv=torch.zeros(5, 1536, dtype=torch.float16))]:
        a = {**good, **over}
        with pytest.raises(ValueError):
            P.attention_paged(a["qkv"], a["attn"], a["cu"], kv, a["table"], a["past"], a["ws"], stream=0)
    pool = P.KvPool(4, 2)
    for window, sinks in [(2 ** 31, 0), (2 ** 32 + 5, 0), (-2 ** 31 - 1, 0), (5, 2 ** 31)]:
        with pytest.raises(ValueError):
            P.attention_paged(good["qkv"], good["attn"], good["cu"], kv, good["table"], good["past"], good["ws"],
                              window, sinks, stream=0)
        with pytest.raises(ValueError):
            pool.trim([0], window, sinks)
    with pytest.raises(ValueError):
        P.kv_copy_pages(kv, torch.zeros(2, **i32), torch.zeros(3, **i32), good["ws"], stream=0)
    with pytest.raises(ValueError):
        P.kv_copy_pages(kv, torch.zeros(2), torch.zeros(2), good["ws"], stream=0)
    with pytest.raises(ValueError):
        P.attention_paged_workspace(-1, 1, "bf16", device="cpu")
    with pytest.raises(ValueError):
        P.KvPool(4, 2).reserve([0, 1], [5])


# ---------------------------------------------------------------- oracle
def test_oracle_scale_is_the_smallest_that_fits():
    for amax in [1e-40, 1e-5, 0.3, 1.0, 1.75, 1.7500001, 447.9, 448.0, 448.1, 3e38]:
        s = O.kv_scale(amax)
        assert 448.0 * s >= amax and (s == 2.0 ** -100 or 448.0 * s / 2 < amax)
        assert np.frexp(s)[0] == 0.5
    assert O.kv_scale(0.0) == 2.0 ** -100


def test_oracle_append_holds_what_was_appended():
    """Whole prompts: every code is within half an e4m3 step of its token, and
    one append or several give the same where no scale rises."""
    rng = np.random.default_rng(0)
    kv = rng.standard_normal((130, 2, 8, 64))
    kv[0, :, :, 0] = 8.0  # the largest of the first page comes first
    kv[64, :, :, 0] = 8.0
    kv[128, :, :, 0] = 8.0
    table = [[2, 0, 1]]
    v1, s1 = O.kv_append(np.full((3, 2, 8, 64, 64), 7.0), np.ones((3, 2, 8)), kv, [0, 130], table, [0])
    k, v = O.paged_sequence(v1, s1, table[0], 130)
    for got, want in ((k, kv[:, 0]), (v, kv[:, 1])):
        assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10 * 8 / 256)).all()
    v2, s2 = np.full((3, 2, 8, 64, 64), 7.0), np.ones((3, 2, 8))
    for a, b in [(0, 1), (1, 40), (40, 100), (100, 130)]:
        O.kv_append(v2, s2, kv[a:b], [0, b - a], table, [a])
    assert np.array_equal(v1, v2) and np.array_equal(s1, s2)


def test_oracle_attention_against_dense():
    rng = np.random.default_rng(1)
    kv, q = rng.standard_normal((200, 2, 8, 64)), rng.standard_normal((60, 8, 64))
    vals, sc = O.kv_append(np.zeros((4, 2, 8, 64, 64)), np.ones((4, 2, 8)), kv, [0, 200], [[3, 1, 0, 2]], [0])
    k, v = O.paged_sequence(vals, sc, [3, 1, 0, 2], 200)
    for window, sinks in [(0, 0), (30, 0), (30, 5), (1, 0), (500, 3)]:
        got = O.attention_paged(q, vals, sc, [0, 60], [[3, 1, 0, 2]], [140], window, sinks)
        i, j = np.arange(140, 200)[:, None], np.arange(200)[None, :]
        vis = (j <= i) & ((window <= 0) | (i - j < window) | (j < sinks))
        s = np.where(vis[None], np.einsum("thd,jhd->htj", q, k) / 8, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        want = np.einsum("htj,jhd->thd", p / p.sum(-1, keepdims=True), v)
        np.testing.assert_allclose(got, want, rtol=0, atol=1e-12)


def test_binding_refuses_cpu_tensors(P, monkeypatch):
    """Before any library call: with a GPU in the machine the library would
    launch kernels on their addresses."""
    kv = P.KvPages(torch.zeros(3, 2, 8, 64, 64, dtype=torch.uint8), torch.ones(3, 2, 8))
    i32 = dict(dtype=torch.int32)
    cu, table, past = torch.tensor([0, 5], **i32), torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)

    def reached():
        raise AssertionError("the library was called")

    monkeypatch.setattr(P, "lib", reached)
    for stream in (None, 0):
        with pytest.raises(ValueError):
            P.kv_append(torch.zeros(5, 1536), cu, kv, table, past, ws, stream=stream)
        with pytest.raises(ValueError):
            P.attention_paged(torch.zeros(5, 1536), torch.zeros(5, 512), cu, kv, table, past, ws, stream=stream)
        with pytest.raises(ValueError):
            P.kv_copy_pages(kv, torch.zeros(2, **i32), torch.ones(2, **i32), ws, stream=stream)


def test_pool_numbers_are_not_cut(P):
    """Numbers that do not fit into 32 bits, or are no integers, are refused; none
    is taken for another."""
    pool = P.KvPool(4, 3)
    pool.reserve([0, 1], [100, 3])
    before = pool.table(range(3), 4).tolist(), pool.free_pages
    far = 2 ** 32
    for one in ([far], [far + 1], [-far], [2 ** 31], [2 ** 63], [2 ** 70], [0.0], [0.5], [True], torch.tensor([far]),
                np.array([far + 2]), np.array([2 ** 64 - far], np.uint64), torch.tensor([1.0]), torch.tensor([0.0, 1.0])):
        for call in (lambda x: pool.release(x), lambda x: pool.trim(x, 5), lambda x: pool.table(x, 4),
                     lambda x: pool.reserve(x, [101]), lambda x: pool.fork(x, [2]), lambda x: pool.fork([0], x)):
            with pytest.raises(ValueError):
                call(one)
    for length in ([far + 101], torch.tensor([far + 101]), [101.5]):
        with pytest.raises(ValueError):
            pool.reserve([0], length)
    for call in (lambda: pool.length(far), lambda: pool.table([0], far + 2), lambda: pool.trim([0], 1.5),
                 lambda: P.KvPool(far + 1, 1), lambda: P.KvPool(1, far + 1), lambda: P.KvPool(1.5, 1),
                 lambda: P.attention_paged_workspace(1, far + 1, "bf16", device="cpu")):
        with pytest.raises((ValueError, TypeError)):
            call()
    assert (pool.table(range(3), 4).tolist(), pool.free_pages) == before
    # what fits is taken in any integer type
    for seqs in (torch.tensor([0, 1]), np.array([0, 1], np.int64), np.array([0, 1], np.uint8), (0, 1), range(2),
                 [np.int64(0), 1], torch.tensor([0, 1], dtype=torch.int32)):
        assert pool.table(seqs, 4).tolist() == before[0][:2]
    pool.release([])
    assert pool.table([], 2).shape == (0, 2)


def test_wide_page_tables_are_not_cut(P):
    kv = P.KvPages(torch.zeros(3, 2, 8, 64, 64, dtype=torch.uint8), torch.ones(3, 2, 8))
    i32 = dict(dtype=torch.int32)
    qkv, out, ws = torch.zeros(5, 1536), torch.zeros(5, 512), torch.zeros(1 << 16, dtype=torch.uint8)
    meta = dict(dtype=torch.int32, device="meta")
    for cu, table, past in [(torch.zeros(2, **i32), torch.empty(1, 2 ** 32 + 1, **meta), torch.zeros(1, **i32)),
                            (torch.empty(2 ** 32 + 2, **meta), torch.empty(2 ** 32 + 1, 1, **meta),
                             torch.empty(2 ** 32 + 1, **meta))]:
        with pytest.raises(ValueError, match="32 bits"):
            P.attention_paged(qkv, out, cu, kv, table, past, ws, stream=0)
        with pytest.raises(ValueError, match="32 bits"):
            P.kv_append(qkv, cu, kv, table, past, ws, stream=0)

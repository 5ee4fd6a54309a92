"""Long histories over the paged cache in which each page can be told from the
others: value page p is not zero in one dim of each head only, so a page that is
lost, read twice or read in another's place moves that dim by a share that no
rounding reaches.  Outputs have a closed form; the bounds count the additions that
the kernels make."""
import math

import numpy as np
import pytest
import torch

from packed_sequence_transformer_b200 import ptl
from tests.gpu_util import dev, host, tdt

PAGE, HEADS, DH = 64, 8, 64
HEAVY = 5.5  # score of a heavy page's keys in the peaked cases; 0 elsewhere: weights e^5.5 = 245 to 1


class Long:
    """new tokens of each user behind its past ones.  flat: all weights alike;
    else 24 pages of each user, evenly spread, weigh 245 times what others do and
    together the greater part of all."""

    def __init__(self, name, dt, new, past, flat=True, window=0, sinks=0, beside=0):
        self.name, self.dt, self.new, self.past, self.flat = name, dt, new, past, flat
        self.window, self.sinks, self.beside = window, sinks, beside
        self.pages = [-(-(n + p) // PAGE) for n, p in zip(new, past)]

    def __repr__(self):
        return self.name

    def first_page(self, u):
        return sum(self.pages[:u])

    def dims(self, ids):
        """[pages, heads]: where page number `ids` of the pool holds its values."""
        return (ids[:, None] * (2 * np.arange(HEADS) + 1) + ids[:, None] // DH * np.arange(HEADS)) % DH

    def values(self, ids):
        """Values of page number `ids`: 1 to 1.875 in steps of e4m3."""
        return 1.0 + (ids * 5 % 8) / 8.0

    def heavy(self, u):
        """Which pages of user u weigh more."""
        k = np.arange(self.pages[u])
        every = max(1, self.pages[u] // 24)
        return (k % every == every // 2) & (not self.flat)

    def weights(self, u):
        """[queries, pages]: the sum of exp(score) over the tokens of each page that each query sees."""
        pos = self.past[u] + np.arange(self.new[u])[:, None]
        base = PAGE * np.arange(self.pages[u])[None, :]

        def upto(x):  # tokens of the page below position x
            return np.clip(x - base, 0, PAGE)

        seen = upto(pos + 1)
        if self.window > 0:
            lo = np.maximum(pos + 1 - self.window, 0)
            seen = seen - upto(lo) + upto(np.minimum(lo, self.sinks))
        return seen * np.where(self.heavy(u), math.exp(HEAVY), 1.0)

    def terms(self, u):
        """[queries, pages] weights, [pages, heads] dims, [pages] values of user u."""
        ids = self.first_page(u) + np.arange(self.pages[u])
        return self.weights(u), self.dims(ids), self.values(ids)

    def exact(self, u):
        w, dim, val = self.terms(u)
        out = np.zeros((w.shape[0], HEADS, DH))
        for h in range(HEADS):
            part = np.zeros((DH, w.shape[1]))
            part[dim[:, h], np.arange(w.shape[1])] = val
            out[:, h] = w @ part.T
        return out / w.sum(axis=1)[:, None, None]

    def tolerance(self, u):
        """Relative: all terms are positive.  Scores are multiples of 2^-5 below
        2^6, exact, and 2^x of them and the factor log2 e are off by 2^-22 and
        5.5 * 2^-22 at most, in the sum and in the normaliser; a weight in fp16
        2^-11 (bf16), in two halves 2^-22 (fp32).  Additions: a lane of the first
        kernel adds 8 weights a page, the second 18; the tensor cores take 64
        products a page, each off by 2^-23 (their additions truncate); a block
        has at most all pages of its unit, which for one query are cut into
        4 sqrt(pages) parts and for several into 1.5 sqrt(pages) (the smaller
        number counts here; calls with many new tokens count as not cut), and
        parts are added in a row.  Output: half a step."""
        half, prob = (2.0 ** -8, 2.0 ** -11) if self.dt == "bf16" else (2.0 ** -24, 2.0 ** -22)
        k = self.pages[u]
        parts = max(1, int(math.sqrt(k) * 1.5)) if sum(self.new) < 100 and not self.beside else 1
        held = -(-k // parts) + 1
        return half + prob + 2 * 6.5 * 2.0 ** -22 + (18 * held + k) * 2.0 ** -24 + (64 + held + k) * 2.0 ** -23


CASES = [
    # one token: one history over most of a call's blocks, and over few
    Long("one_20000", "bf16", [1], [20000]),
    Long("one_20000_peaked", "bf16", [1], [20000], False),
    Long("one_20000_fp32", "fp32", [1], [20000]),
    Long("one_20000_fp32_peaked", "fp32", [1], [20000], False),
    Long("one_360000", "bf16", [1], [360000]),
    Long("one_360000_peaked", "bf16", [1], [360000], False),
    Long("one_360000_fp32_peaked", "fp32", [1], [360000], False),
    Long("four_users", "bf16", [2, 1, 9, 1], [9000, 10, 4000, 12345]),
    Long("four_users_fp32", "fp32", [2, 1, 9, 1], [9000, 10, 4000, 12345]),
    Long("window", "bf16", [1, 1], [15000, 15000], window=9000, sinks=70),
    # more new tokens, first kernel and tcgen05 kernel
    Long("forty_12000", "bf16", [40], [12000]),
    Long("forty_12000_fp32", "fp32", [40], [12000]),
    Long("forty_12000_beside", "bf16", [40], [12000], beside=16000),
    Long("forty_12000_beside_peaked", "bf16", [40], [12000], False, beside=16000),
    # units of the tcgen05 kernel over many blocks each: one tile, two tiles, a tile of one row
    Long("hundred_60000", "bf16", [100], [60000]),
    Long("hundred_60000_peaked", "bf16", [100], [60000], False),
    Long("block_40000", "bf16", [256], [40000]),
    Long("block_40000_peaked", "bf16", [256], [40000], False),
    Long("row_30000", "bf16", [129], [30000]),
    Long("blocks_window", "bf16", [300, 140], [12000, 9000], window=7000, sinks=100),
]


@pytest.mark.parametrize("case", CASES, ids=repr)
def test_each_page_can_be_told(case):
    """In each case, a page left out of any one query's sums, or counted twice,
    takes some output out of its bound (a heavy page where weights differ: the
    others are too light to be told); one left out of the normaliser alone does in
    the cases with heavy pages and in fp32."""
    for u in range(len(case.new)):
        w, dim, val = case.terms(u)
        tol = case.tolerance(u)
        for i in sorted({0, case.new[u] // 2, case.new[u] - 1}):
            row, heavy = w[i], case.heavy(u)
            pages = (heavy if heavy.any() else True) & (row >= PAGE)
            sums = np.zeros((HEADS, DH))
            for h in range(HEADS):
                np.add.at(sums[h], dim[:, h], row * val)
            share = (row * val)[pages, None] / sums[np.arange(HEADS), dim[pages]]  # [pages, heads] of the dim's sum
            of_all = (row / row.sum())[pages]
            for sign in (-1.0, 1.0):
                off = np.abs((1 + sign * share) / (1 + sign * of_all)[:, None] - 1)
                assert (off.max(axis=1, initial=0.0)[of_all < 1] > tol).all(), (u, i, sign)
            if heavy.any() or case.dt == "fp32":
                assert (of_all > tol).all(), (u, i, of_all.min(), tol)
        assert np.abs(case.exact(u).sum(axis=2) - (w @ val / w.sum(axis=1))[:, None]).max() < 1e-12


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=repr)
def test_long_histories(case):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    users, total = len(case.new), sum(case.pages)
    ids = np.arange(total)
    order = np.random.default_rng(total).permutation(total)  # page number -> place in the pool
    codes = torch.zeros(total + 1, 2, HEADS, PAGE, DH, dtype=torch.uint8, device="cuda")
    place, dim = dev(order, torch.int64), dev(case.dims(ids), torch.int64)
    value = dev(0x38 + ids * 5 % 8, torch.uint8)  # 1 to 1.875
    for h in range(HEADS):
        codes[place, 1, h, dim[:, h]] = value[:, None].expand(-1, PAGE)
    heavy = np.concatenate([case.heavy(u) for u in range(users)])
    codes[place[dev(heavy, torch.bool)], 0] = 0x33  # 0.6875: a score of 64 * 0.6875 / 8 = HEAVY
    kv = ptl.KvPages(codes, torch.ones(total + 1, 2, HEADS, device="cuda"))
    new, past, width = list(case.new), list(case.past), max(case.pages + [-(-case.beside // PAGE)])
    if case.beside:  # a user whose output is not looked at, all of whose pages are one
        new, past = new + [case.beside], past + [0]
    table = np.full((len(new), width), -1, np.int32)
    for u in range(users):
        table[u, :case.pages[u]] = order[case.first_page(u):case.first_page(u) + case.pages[u]]
    if case.beside:
        table[-1] = total
    cu = np.concatenate([[0], np.cumsum(new)])
    qkv = torch.ones(cu[-1], 1536, dtype=tdt(case.dt), device="cuda")
    out = torch.full((int(cu[-1]), 512), float("nan"), dtype=tdt(case.dt), device="cuda")
    ws = ptl.attention_paged_workspace(int(cu[-1]), len(new), case.dt)
    ptl.attention_paged(qkv, out, dev(cu, torch.int32), kv, dev(table, torch.int32), dev(np.array(past), torch.int32),
                        ws, window=case.window, sinks=case.sinks)
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    for u in range(users):
        got = host(out[cu[u]:cu[u + 1]]).reshape(-1, HEADS, DH)
        want = case.exact(u)
        off = np.abs(got - want) - case.tolerance(u) * want
        assert (off <= 0).all(), (u, np.argwhere(~(off <= 0))[:3].tolist(), np.nanmax(off / np.maximum(want, 1e-30)))

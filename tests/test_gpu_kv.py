"""The 8-bit paged key/value cache on the GPU: the append's codes and scales
bit for bit against the oracle, the attention over the pages elementwise
within the bound that its roundings allow, the page copy, and all of them
together as a served layer uses them."""
import numpy as np
import pytest
import torch

from oracle import ptl_oracle as O
from packed_sequence_transformer_b200 import ptl
from packed_sequence_transformer_b200 import synthetic as S
from tests.gpu_util import dev, host, tdt
from tests.kv_util import Call, make_pages, value_of_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ptl.lib()


def _expect_append(c):
    return O.kv_append(value_of_codes(torch.from_numpy(c.codes)), c.scales.astype(np.float64),
                       c.qkv[:, 512:].reshape(c.T, 2, 8, 64), c.cu, c.table, c.past)


def _check_append(c, want):
    ws = c.append()
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    np.testing.assert_array_equal(host(c.kv.scales), want[1])
    np.testing.assert_array_equal(value_of_codes(c.kv.codes), want[0])


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("new,past", [
    ([1], [0]), ([1], [63]), ([1], [64]), ([2], [63]), ([64], [0]), ([65], [0]), ([130], [31]),
    ([0, 1, 0, 5, 70, 0], [3, 9, 0, 62, 1, 0]),
    ([1] * 40, list(range(25, 65))),
    ([33, 31, 32, 0, 200], [32, 33, 31, 7, 0]),
])
def test_append_codes_and_scales(dt, new, past):
    c = Call(len(new) * 100 + new[-1], new, past, dt)
    _check_append(c, _expect_append(c))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_append_raises_scales_step_by_step(dt):
    """One token at a time, each larger than all before it: every step raises
    the scale and rounds the kept codes again."""
    steps = 70
    c = Call(3, [1, 1], [0, 0], dt, num_pages=5)
    c.table = np.array([[4, 1], [0, 2]], np.int32)
    vals, sc = value_of_codes(torch.from_numpy(c.codes)), c.scales.astype(np.float64)
    c.upload()
    base = c.rng.standard_normal((steps, 2, 1536)).astype(np.float32)
    for k in range(steps):
        c.qkv_d = dev(base[k] * np.float32(1.3 ** k), tdt(dt))
        c.qkv, c.past = host(c.qkv_d), [k, k]
        c.past_d = dev(np.array(c.past), torch.int32)
        ws = c.append()
        O.kv_append(vals, sc, c.qkv[:, 512:].reshape(2, 2, 8, 64), c.cu, c.table, c.past)
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    np.testing.assert_array_equal(host(c.kv.scales), sc)
    np.testing.assert_array_equal(value_of_codes(c.kv.codes), vals)


def test_append_extremes():
    """Zeros, the smallest and largest numbers, exact borders of the scale, and
    what is no number."""
    c = Call(5, [8, 4], [0, 60], "fp32")
    x = c.qkv.copy().astype(np.float32).reshape(12, 3, 8, 64)
    x[:8, 1:, 0] = 0.0
    x[:8, 1:, 1] = 1e-45
    x[:8, 1:, 2] = 448.0 * 2.0 ** 5
    x[:8, 1:, 3] = np.nextafter(np.float32(448.0 * 2.0 ** 5), np.float32(np.inf))
    x[:8, 1:, 4] = np.finfo(np.float32).max
    x[3, 1, 5, 7], x[4, 2, 5, 9], x[5, 2, 5, 63] = np.nan, np.inf, -np.inf
    x[:8, 1:, 6] = np.nan
    x[9, 1, 7, 0] = 2.0 ** 100
    c.qkv_d = dev(x.reshape(12, 1536), torch.float32)
    c.upload()
    want = _expect_append(c)
    _check_append(c, want)
    assert np.isnan(want[0]).any()


def test_append_again_after_taking_tokens_back():
    c = Call(6, [5, 9], [62, 3])
    c.append()
    torch.cuda.synchronize()
    c.codes, c.scales = c.kv.codes.cpu().numpy(), c.kv.scales.cpu().numpy()
    c.qkv_d = dev(c.rng.standard_normal((14, 1536)).astype(np.float32), torch.bfloat16)
    c.upload()
    _check_append(c, _expect_append(c))


def test_append_reports_and_leaves_the_rest():
    # a page number out of range: that page is skipped, the other is written
    c = Call(7, [10, 10], [0, 0])
    good = c.table.copy()
    for bad in (-1, c.num_pages, 2 ** 31 - 1, -2 ** 31):
        c.table = good.copy()
        c.table[0, 0] = bad
        c.upload()
        ws = c.append()
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == ptl.STATUS_CODE["PTL_ERR_BAD_PAGE"]
        got = c.kv.codes.cpu().numpy()
        changed = [p for p in range(c.num_pages) if not np.array_equal(got[p], c.codes[p])]
        assert changed == [good[1, 0]]
    # positions or offsets that do not fit: nothing is written
    for cu, past, err in [([0, 10, 20], [60, 0], "PTL_ERR_BAD_PAGE"), ([0, 10, 20], [-1, 0], "PTL_ERR_BAD_PAGE"),
                          ([0, 10, 20], [2 ** 31 - 1, 0], "PTL_ERR_BAD_PAGE"),
                          ([0, 10, 19], [0, 0], "PTL_ERR_BAD_OFFSETS"), ([1, 10, 20], [0, 0], "PTL_ERR_BAD_OFFSETS"),
                          ([0, 21, 20], [0, 0], "PTL_ERR_BAD_OFFSETS"), ([0, -5, 20], [0, 0], "PTL_ERR_BAD_OFFSETS")]:
        c.table = good
        c.upload()
        c.cu_d, c.past_d = dev(np.array(cu), torch.int32), dev(np.array(past), torch.int32)
        ws = c.append()
        out, ws2 = c.attend()
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == ptl.STATUS_CODE[err]
        assert ptl.last_device_error(ws2) == ptl.STATUS_CODE[err]
        assert np.array_equal(c.kv.codes.cpu().numpy(), c.codes)
        assert np.array_equal(c.kv.scales.cpu().numpy(), c.scales)
        assert torch.isnan(out).all()


# ------------------------------------------------------------- attention
# (dtype, new tokens of a user beside the others': Call)
KINDS = [("bf16", 0), ("bf16", 16000), ("fp32", 0)]
SHAPES = [
    ([1], [0]), ([1], [1]), ([1], [62]), ([1], [63]), ([1], [64]), ([1], [500]),
    ([3], [0]), ([8], [120]), ([9], [120]), ([17], [55]), ([70], [0]), ([200], [0]), ([129], [131]),
    ([0, 1, 0, 2, 90, 0], [77, 0, 0, 130, 10, 5]),
    ([1] * 33, [7 * i for i in range(33)]), ([33], [0]), ([256], [64]), ([257], [300]), ([600, 40], [1500, 61]),
]


@pytest.mark.parametrize("dt,beside", KINDS)
@pytest.mark.parametrize("new,past", SHAPES)
def test_attention_against_the_oracle(dt, beside, new, past):
    Call(new[0] * 7 + past[0] + len(new), new, past, dt, beside=beside).check()


@pytest.mark.parametrize("window,sinks", [(63, 0), (64, 64), (65, 65), (100, 3), (128, 200), (300, 1000),
                                          (2 ** 31 - 1, 0), (0, 7), (900, 130)])
def test_attention_window_and_sinks_of_many_new_tokens(window, sinks):
    Call(window % 1000 + sinks % 1000, [1, 5, 200, 0, 1, 130], [700, 64, 90, 9, 0, 319], beside=40000).check(window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (63, 0), (5, 2 ** 31 - 1), (64, 64), (-4, 0)])
def test_attention_small_windows_of_a_long_prompt(window, sinks):
    Call(window % 1000 + 1, [140, 1100, 3, 33], [77, 0, 200, 640]).check(window, sinks)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (63, 0), (64, 64), (65, 65), (100, 3), (128, 200),
                                          (5, 2 ** 31 - 1), (2 ** 31 - 1, 0), (300, 1000), (0, 7), (-4, 0)])
def test_attention_window_and_sinks(dt, window, sinks):
    Call(window % 1000 + sinks % 1000, [1, 5, 200, 0, 1, 130], [700, 64, 90, 9, 0, 319], dt).check(window, sinks)


@pytest.mark.parametrize("dt,beside", KINDS)
def test_attention_many_parts(dt, beside):
    """One history over more blocks than the grid has, and users whose pages end
    inside a block's range."""
    Call(11, [1], [20000], dt, beside=beside).check()
    Call(12, [2, 1, 9, 1], [9000, 10, 4000, 12345], dt, beside=beside).check()
    Call(13, [1, 1], [15000, 15000], dt, beside=beside).check(window=9000, sinks=70)
    Call(31, [40], [12000], dt, beside=beside).check()
    Call(32, [50, 140, 33], [5000, 3000, 0], dt, beside=beside).check(window=2900, sinks=100)


def test_attention_many_users():
    """More users than a block has threads."""
    rng = np.random.default_rng(14)
    Call(14, rng.integers(0, 3, 700).tolist(), rng.integers(0, 150, 700).tolist()).check()


@pytest.mark.parametrize("dt,beside", KINDS)
@pytest.mark.parametrize("new", [[16, 6], [150, 40]])
def test_attention_magnitudes(dt, beside, new):
    """Rows of q from tiny to huge, scales far apart from page to page."""
    c = Call(15, new, [200, 300], dt, beside=beside)
    x = host(c.qkv_d).astype(np.float32)
    x[:, :512] *= (10.0 ** np.linspace(-30, 1, c.T))[:, None].astype(np.float32)
    x[3, :512] = 0.0
    c.qkv_d = dev(x, tdt(dt))
    c.scales[:, 1] *= (2.0 ** c.rng.integers(-30, 20, (c.num_pages, 8))).astype(np.float32)
    c.upload()
    c.check()


@pytest.mark.parametrize("beside", [0, 16000])
@pytest.mark.parametrize("new,past,window,sinks", [
    ([50, 140, 33], [5000, 3000, 0], 2900, 100), ([140, 60, 200, 40, 300], [10, 700, 0, 300, 100], 0, 0),
    ([129, 128, 257, 33, 512] * 4, [0, 64, 3, 500, 0] * 4, 0, 0)])
def test_attention_same_bits_every_time(beside, new, past, window, sinks):
    """Blocks that go from users with one tile of queries to users with two and
    back: whoever is ahead waits for the others, call after call."""
    c = Call(34, new, past, beside=beside)
    first = c.check(window, sinks)
    ws = ptl.attention_paged_workspace(c.T, len(c.new), "bf16")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    other = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            other.fill_(i & 255)
        out, _ = c.attend(window, sinks, ws=ws)
        differ += (out[:c.rows].view(torch.int16) != first[:c.rows].view(torch.int16)).any()
    assert differ.item() == 0
    assert ptl.last_device_error(ws) == 0


@pytest.mark.parametrize("dt,beside", KINDS)
@pytest.mark.parametrize("new", [[4], [40], [300]])
@pytest.mark.parametrize("big", [0, 7, 14])
def test_pages_of_very_small_values_keep_their_weight(dt, beside, new, big):
    """Equal scores; one page's values are 2^30, the others' zero with the
    smallest scale: those weigh nothing in the sum of the values and as much as
    any in the normaliser."""
    c = Call(17, new, [1000], dt, q_std=0.0, beside=beside)
    c.codes[:, 1] = 0
    c.scales[:, 1] = 2.0 ** -100
    c.codes[c.table[0, big], 1] = 0x38  # 1.0
    c.scales[c.table[0, big], 1] = 2.0 ** 30
    c.upload()
    c.check()


@pytest.mark.parametrize("dt,beside", KINDS)
@pytest.mark.parametrize("new", [[4], [40], [300]])
def test_many_small_weights_beside_a_large_one(dt, beside, new):
    """Token 0 outweighs each other by e^18, about 2^26, and its value is zero:
    the output is the sum of thousands of small weights.  Their errors: the
    exponent's as in Call.bound for sums of |q k| / 8 up to 18; a weight 2^26
    below the largest is held to 2^-11 in the first kernel, where the largest is
    2^15, and to 2^-10 where the largest may be 2^11 and this one, 2^-15, lies
    in fp16's subnormals (a step of 2^-24, half of it lost); in the fp32 build
    the second half of a weight 2^-11 does, 2^-25 of it lost, 2^-14 relative; the
    output's rounding."""
    c = Call(18, new, [4096], dt, beside=beside)
    qkv = c.qkv.copy()
    qkv[:, :512] = 1.0
    c.qkv_d = dev(qkv.astype(np.float32), tdt(dt))
    c.codes[:] = 0
    c.codes[:, 1] = 0x38  # 1.0
    c.scales[:] = 1.0
    first = c.table[0, 0]
    c.codes[first, 0, :, 0, 0] = 0x71  # 144
    c.codes[first, 1, :, :, 0] = 0
    c.upload()
    out, ws = c.attend()
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    others = (4096 + np.arange(c.rows)).astype(np.float64)
    ref = others * np.exp(-18.0) / (1 + others * np.exp(-18.0))
    half, prob = (2.0 ** -8, 2.0 ** -10) if dt == "bf16" else (2.0 ** -24, 2.0 ** -14)
    tol = half + prob + 2 * (67 * 2.0 ** -23 + 2.0 ** -22) * 18 + 2 * 2.0 ** -22 + 3 * 4400 * 2.0 ** -24
    off = np.abs(host(out[:c.rows]) / ref[:, None] - 1)
    assert off.max() <= tol, (off.max(), tol)


@pytest.mark.parametrize("dt,beside", KINDS)
@pytest.mark.parametrize("new,past", [([3, 1], [100, 700]), ([150, 40], [100, 700])])
def test_masked_places_have_no_effect(dt, beside, new, past):
    """NaN codes behind the last token, before the window, and in front of
    later queries; visible ones reach the queries that see them."""
    c = Call(16, new, past, dt, beside=beside)
    nan = np.uint8(0x7F)
    # behind the end
    for u in range(2):
        end = new[u] + past[u]
        page = c.table[u, (end - 1) // 64]
        c.codes[page, 0, :, end % 64 or 64:], c.codes[page, 1, :, :, end % 64 or 64:] = nan, np.uint8(0xFF)
    c.upload()
    c.check()
    # user 1: a key and a value that some queries see through the window and others do not
    at = past[1] - 20
    page = c.table[1, at // 64]
    c.codes[page, 1, 2, 5, at % 64] = nan
    c.codes[page, 1, 3, 40, at % 64] = np.uint8(0xFF)
    c.codes[page, 0, 6, at % 64, 11] = nan
    c.upload()
    c.check(window=30, sinks=1)
    c.check(window=21, sinks=1)
    c.check(window=20, sinks=1)
    c.check()
    # the same for longer windows
    at = past[1] - 140
    page = c.table[1, at // 64]
    c.codes[page, 1, 5, 7, at % 64] = nan
    c.codes[page, 0, 4, at % 64, 63] = nan
    c.upload()
    for window in (151, 141, 140):
        c.check(window=window, sinks=1)
    # in a row of the call itself: later queries see it, earlier ones do not
    at = past[0] + new[0] - 2
    page = c.table[0, at // 64]
    c.codes[page, 1, 0, 0, at % 64] = nan
    c.upload()
    out = c.check()
    assert torch.isnan(out[new[0] - 2:new[0], 0]).all() and torch.isfinite(out[:new[0] - 2, 0]).all()


@pytest.mark.parametrize("beside", [0, 16000])
def test_infinite_queries_stay_in_their_rows(beside):
    n = 40 if beside else 4
    c = Call(17, [n, 1], [90, 90], beside=beside)
    c.qkv_d[1, 70] = float("inf")
    c.qkv_d[2, 3] = float("nan")
    c.upload()
    out, ws = c.attend()
    torch.cuda.synchronize()
    bad = torch.isnan(out[:n + 1].view(n + 1, 8, 64)).all(-1).cpu().numpy()
    want = np.zeros((n + 1, 8), bool)
    want[1, 1] = want[2, 0] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("beside", [0, 16000])
def test_attention_bad_page_is_reported(beside):
    c = Call(18, [40 if beside else 1, 2], [300, 10], beside=beside)
    good = c.table.copy()
    for bad in (-1, c.num_pages, 2 ** 31 - 1, -2 ** 31):
        c.table = good.copy()
        c.table[0, 2] = bad
        c.upload()
        _, ws = c.attend()
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == ptl.STATUS_CODE["PTL_ERR_BAD_PAGE"]
        # outside the window it is not needed
        out, ws = c.attend(window=70, sinks=20)
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == 0 and torch.isfinite(out).all()


def test_two_users_of_a_call_share_pages():
    c = Call(19, [3, 3], [200, 200])
    c.table[1] = c.table[0]
    c.qkv_d[3:] = c.qkv_d[:3]
    c.upload()
    out = c.check()
    assert torch.equal(out[:3], out[3:])


# ------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("dt,beside", KINDS)
def test_same_bits_on_other_streams_and_in_graphs(dt, beside):
    """Two calls under way at once, each with its workspace; two graphs that
    share one, replayed in turn, on new inputs."""
    a, b = (Call(20, [1, 7, 90], [4000, 50, 0], dt, beside=beside),
            Call(21, [2, 1, 33], [10, 9000, 200], dt, beside=beside))
    want = [c.check().clone() for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [ptl.attention_paged_workspace(c.T, 3, dt) for c in (a, b)]
    outs = [torch.zeros(c.T, 512, dtype=tdt(dt), device="cuda") for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, ws, o in zip((a, b), streams, wss, outs):
            c.attend(ws=ws, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for c, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.append(ws=small)
            c.attend(ws=wss[0], out=o)
        graphs.append(g)
    for _ in range(3):
        for c in (a, b):
            c.qkv_d.normal_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, o in zip((a, b), outs):
            got = o.clone()
            c.qkv = host(c.qkv_d)
            assert torch.equal(got, c.check())
    assert ptl.last_device_error(wss[0]) == 0 and ptl.last_device_error(small) == 0


@pytest.mark.parametrize("dt,beside", KINDS)
def test_pages_beyond_32_bits_of_bytes(dt, beside):
    """The same call at the far end of a cache of 4.6 GB: the same bits."""
    total = 70000
    c = Call(35, [3, 70, 1], [100, 700, 64], dt, beside=beside)
    want = c.check().clone()
    small = c.kv
    kv = ptl.alloc_kv_pages(total)
    kv.codes[total - c.num_pages:] = small.codes
    kv.scales[total - c.num_pages:] = small.scales
    table, c.kv = c.table_d, kv
    c.table_d = torch.where(table < 0, table, table + (total - c.num_pages))
    out, ws = c.attend()
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    assert torch.equal(out[:c.rows], want[:c.rows])
    if beside:
        return  # (its one page would be written many times at once)
    assert ptl.last_device_error(c.append()) == 0
    c.kv, far, c.table_d = small, kv, table
    assert ptl.last_device_error(c.append()) == 0
    assert torch.equal(far.codes[total - c.num_pages:], small.codes)
    assert torch.equal(far.scales[total - c.num_pages:], small.scales)
    assert not far.codes[:total - c.num_pages].any()
    # and copied down
    src = torch.arange(total - c.num_pages, total, dtype=torch.int32, device="cuda")
    dst = src - 40000
    ptl.kv_copy_pages(far, src, dst, ws)
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    assert torch.equal(far.codes[dst.long()], small.codes) and torch.equal(far.scales[dst.long()], small.scales)


# ------------------------------------------------------------- page copy
@pytest.mark.parametrize("pairs", [[(0, 1)], [(3, 0), (3, 5), (4, 1)], [(i, 39 - i) for i in range(20)]])
def test_copy_pages(pairs):
    rng = np.random.default_rng(len(pairs))
    codes, scales = make_pages(rng, 40)
    kv = ptl.KvPages(dev(codes, torch.uint8), dev(scales, torch.float32))
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    src, dst = (dev(np.array(x), torch.int32) for x in zip(*pairs))
    ptl.kv_copy_pages(kv, src, dst, ws)
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    for s, d in pairs:
        codes[d], scales[d] = codes[s], scales[s]
    assert np.array_equal(kv.codes.cpu().numpy(), codes) and np.array_equal(kv.scales.cpu().numpy(), scales)


def test_copy_skips_and_reports_bad_pages():
    rng = np.random.default_rng(1)
    codes, scales = make_pages(rng, 4)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for s, d in [(-1, 1), (4, 1), (0, -1), (0, 4), (2 ** 31 - 1, -2 ** 31)]:
        kv = ptl.KvPages(dev(codes, torch.uint8), dev(scales, torch.float32))
        ptl.kv_copy_pages(kv, dev(np.array([s, 2]), torch.int32), dev(np.array([d, 3]), torch.int32), ws)
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == ptl.STATUS_CODE["PTL_ERR_BAD_PAGE"]
        want = codes.copy()
        want[3] = codes[2]
        assert np.array_equal(kv.codes.cpu().numpy(), want)


# ------------------------------------------------------------- together
def test_served_sequences_fork_trim_and_compact():
    """Prompts, single tokens, forks that go different ways, a window with
    pages given up, released sequences and a compaction: the attention of each
    step against the oracle on what the append holds for each sequence alone."""
    rng = np.random.default_rng(30)
    pool, kv = ptl.KvPool(64, 12), ptl.alloc_kv_pages(64)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ws = ptl.attention_paged_workspace(2000, 12, "bf16")
    # the same sequences, each in pages of its own that are never shared or moved
    own_v, own_s = np.zeros((12 * 20, 2, 8, 64, 64)), np.zeros((12 * 20, 2, 8))
    own_table = np.arange(12 * 20).reshape(12, 20)

    def step(seqs, new, window=0, sinks=0):
        past = [pool.length(q) for q in seqs]
        pool.reserve(seqs, [p + n for p, n in zip(past, new)])
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        qkv = dev(rng.standard_normal((int(cu[-1]), 1536)).astype(np.float32), torch.bfloat16)
        table = pool.table(seqs).cuda()
        cu_d, past_d = dev(cu, torch.int32), dev(np.array(past), torch.int32)
        out = torch.empty(int(cu[-1]), 512, dtype=torch.bfloat16, device="cuda")
        ptl.kv_append(qkv, cu_d, kv, table, past_d, small)
        ptl.attention_paged(qkv, out, cu_d, kv, table, past_d, ws, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert ptl.last_device_error(small) == 0 and ptl.last_device_error(ws) == 0
        x = host(qkv)
        O.kv_append(own_v, own_s, x[:, 512:].reshape(-1, 2, 8, 64), cu, own_table[seqs], past)
        ref, mag, smax, count = O.attention_paged(x[:, :512].reshape(-1, 8, 64), own_v, own_s, cu, own_table[seqs],
                                                  past, window, sinks, details=True)
        c = Call.__new__(Call)
        c.dt, c.kv = "bf16", kv
        off = np.abs(host(out).reshape(ref.shape) - ref) - c.bound(ref, mag, smax, count)
        assert (off <= 0).all(), float(off.max())

    def copy(lists):
        src, dst = lists
        ptl.kv_copy_pages(kv, src.cuda(), dst.cuda(), small)

    step([0, 1, 2], [200, 64, 37])
    step([2, 0, 1], [1, 1, 1])
    src, dst = pool.fork([0, 0, 1, 2], [3, 4, 5, 6])
    assert len(src) == 4
    copy((src, dst))
    for s, d in zip([0, 0, 1, 2], [3, 4, 5, 6]):
        own_v[own_table[d]], own_s[own_table[d]] = own_v[own_table[s]], own_s[own_table[s]]
    step([0, 3, 4, 5, 6], [1, 5, 80, 1, 30])
    step([0, 1, 2, 3, 4, 5, 6], [1] * 7)
    pool.release([1, 4])
    free = pool.free_pages
    assert pool.trim([0, 3], 70, 10) > 0 and pool.free_pages > free
    copy(pool.compact())
    used = 64 - pool.free_pages
    assert int(pool.table([0, 2, 3, 5, 6], 20).max()) == used - 1
    step([0, 3], [3, 1], window=70, sinks=10)
    for q in (1, 4):
        own_v[own_table[q]], own_s[own_table[q]] = 0.0, 0.0
    step([2, 5, 6, 1], [1, 2, 100, 66])
    pool.release(range(12))
    assert pool.free_pages == 64


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_layer_over_the_cache(dt):
    """One encoder layer served from the cache, step entry point by step entry
    point: with a fresh cache its attention differs from the layer's own only
    by the keys' and values' rounding to e4m3; the rest of the layer is the
    same calls."""
    case = S.make_case(f"kv_{dt}", lengths=[70, 3, 0, 129], seed=4, dtype=dt, gate_std=0.1, random_bias=True)
    T, U = case.total_tokens, case.num_users
    td = tdt(dt)
    w = ptl.to_device_layer(case.layers[0], dt)
    x, cu = dev(case.x, td), dev(case.cu_seqlens, torch.int32)
    ws, pws = ptl.alloc_workspace(T, U, dt), ptl.attention_paged_workspace(T, U, dt)
    pool, kv = ptl.KvPool(8, U), ptl.alloc_kv_pages(8)
    pool.reserve(range(U), case.lengths.tolist())
    table, past = pool.table(range(U)).cuda(), torch.zeros(U, dtype=torch.int32, device="cuda")

    def layer(x, cu, table, past):
        t = x.shape[0]
        qkv, attn = torch.empty(t, 1536, dtype=td, device="cuda"), torch.empty(t, 512, dtype=td, device="cuda")
        x1, out = torch.empty(t, 512, device="cuda"), torch.empty(t, 512, dtype=td, device="cuda")
        xn2 = torch.empty(t, 512, dtype=td, device="cuda")
        idx = torch.empty(t, 2, dtype=torch.int32, device="cuda")
        tw = torch.empty(t, 2, device="cuda")
        ptl.qkv_projection(x, qkv, w, ws)
        ptl.kv_append(qkv, cu, kv, table, past, pws)
        ptl.attention_paged(qkv, attn, cu, kv, table, past, pws)
        ptl.out_projection(attn, x, x1, w, ws)
        ptl.gate(x1, xn2, idx, tw, w, ws)
        ptl.moe(xn2, idx, tw, x1, out, w, ws)
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == 0 and ptl.last_device_error(pws) == 0
        return qkv, attn, out

    qkv, attn, out = layer(x, cu, table, past)
    h = host(qkv)
    vals, sc = np.zeros((8, 2, 8, 64, 64)), np.ones((8, 2, 8))
    O.kv_append(vals, sc, h[:, 512:].reshape(T, 2, 8, 64), case.cu_seqlens, table.cpu().numpy(), [0] * U)
    ref, mag, smax, count = O.attention_paged(h[:, :512].reshape(T, 8, 64), vals, sc, case.cu_seqlens,
                                              table.cpu().numpy(), [0] * U, details=True)
    c = Call.__new__(Call)
    c.dt, c.kv = dt, kv
    assert (np.abs(host(attn).reshape(ref.shape) - ref) <= c.bound(ref, mag, smax, count)).all()
    assert torch.isfinite(out).all()
    # the last token of each user served as a step of its own: the same codes
    # already stand in the pages, so it is the row that the prompt gave
    users = [0, 1, 3]
    rows = [int(case.cu_seqlens[u + 1]) - 1 for u in users]
    one = layer(x[rows].contiguous(), torch.arange(4, dtype=torch.int32, device="cuda"),
                table[users].contiguous(), dev(np.array([case.lengths[u] - 1 for u in users]), torch.int32))
    b = c.bound(ref, mag, smax, count)[rows]
    assert (np.abs(host(one[1]).reshape(3, 8, 64) - ref[rows]) <= b).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_candidates_as_forks(dt):
    """Groups of candidates that do not see one another, as ptl_attention_masked
    has them, over the cache: a fork of the history for each group.  Against the
    masked oracle on what the pages hold; the histories' pages stay as they were."""
    rng = np.random.default_rng(41)
    lens, groups, size = [200, 75], 3, 2
    pool, kv = ptl.KvPool(24, 8), ptl.alloc_kv_pages(24)
    ws = ptl.attention_paged_workspace(300, 8, dt)

    def call(seqs, past, qkv, attend):
        new = [pool.length(s) - p for s, p in zip(seqs, past)]
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        args = (dev(cu, torch.int32), kv, pool.table(seqs).cuda(), dev(np.array(past), torch.int32), ws)
        ptl.kv_append(qkv, *args)
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == 0
        if not attend:
            return None
        out = torch.empty(len(qkv), 512, dtype=tdt(dt), device="cuda")
        ptl.attention_paged(qkv, out, *args)
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == 0
        return cu, out

    pool.reserve([0, 1], lens)
    hist = rng.standard_normal((sum(lens), 1536)).astype(np.float32)
    for first in (0, lens[0]):  # no candidate raises a page's scale: the forks hold the same history
        hist[first:first + (lens[0] if first == 0 else lens[1]):64, 512:] = 8.0
    call([0, 1], [0, 0], dev(hist, tdt(dt)), False)
    codes, scales, free = kv.codes.clone(), kv.scales.clone(), pool.free_pages
    held = pool.table([0, 1], 4)[pool.table([0, 1], 4) >= 0].long()

    forks, src = list(range(2, 2 + 2 * groups)), [0] * groups + [1] * groups
    ptl.kv_copy_pages(kv, *(x.cuda() for x in pool.fork(src, forks)), ws)
    past = [lens[s] for s in src]
    pool.reserve(forks, [p + size for p in past])
    cand = dev(rng.standard_normal((2 * groups * size, 1536)).astype(np.float32).clip(-4, 4), tdt(dt))
    cu, out = call(forks, past, cand, True)
    assert torch.equal(kv.codes[held.cuda()], codes[held.cuda()])
    assert torch.equal(kv.scales[held.cuda()], scales[held.cuda()])

    vals, sc, table = value_of_codes(kv.codes), host(kv.scales), pool.table(forks).numpy()
    q = host(cand)[:, :512].reshape(-1, 8, 64)
    seqs = [O.paged_sequence(vals, sc, [p for p in t if p >= 0], p0 + size) for t, p0 in zip(table, past)]
    keys, values, queries, at = [], [], [], []
    for u in range(2):
        mine = range(u * groups, (u + 1) * groups)
        n = lens[u]
        for f in mine:
            assert np.array_equal(seqs[f][0][:n], seqs[u * groups][0][:n])
            assert np.array_equal(seqs[f][1][:n], seqs[u * groups][1][:n])
        keys += [seqs[u * groups][0][:n]] + [seqs[f][0][n:] for f in mine]
        values += [seqs[u * groups][1][:n]] + [seqs[f][1][n:] for f in mine]
        at += list(range(sum(map(len, queries)) + n, sum(map(len, queries)) + n + groups * size))
        queries += [np.zeros((n, 8, 64)), q[u * groups * size:(u + 1) * groups * size]]
    total = [n + groups * size for n in lens]
    want = O.jagged_hstu_attention(np.concatenate(queries), np.concatenate(keys), np.concatenate(values),
                                   np.concatenate([[0], np.cumsum(total)]), num_targets=[groups * size] * 2,
                                   target_group_size=size)[at]
    ref, mag, smax, count = O.attention_paged(q, vals, sc, cu, table, past, details=True)
    np.testing.assert_allclose(ref, want, rtol=0, atol=1e-12)
    c = Call.__new__(Call)
    c.dt, c.kv = dt, kv
    assert (np.abs(host(out).reshape(want.shape) - want) <= c.bound(want, mag, smax, count)).all()
    pool.release(forks)
    assert pool.free_pages == free

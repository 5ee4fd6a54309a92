"""Attention over the paged cache where pages' value scales lie far apart or far
from one: long histories whose outputs have closed forms."""
import numpy as np
import pytest
import torch

from packed_sequence_transformer_b200 import ptl
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu
BF16_HALF, FP16_HALF = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ptl.lib()


def _attend(codes, scales, table, users, new, past):
    kv = ptl.KvPages(dev(codes, torch.uint8), dev(scales, torch.float32))
    qkv = torch.ones(users * new, 1536, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(0, users * new + 1, new, dtype=torch.int32, device="cuda")
    pasts = torch.full((users,), past, dtype=torch.int32, device="cuda")
    ws = ptl.attention_paged_workspace(users * new, users, "bf16")
    out = torch.full((users * new, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    ptl.attention_paged(qkv, out, cu, kv, dev(table, torch.int32), pasts, ws)
    torch.cuda.synchronize()
    assert ptl.last_device_error(ws) == 0
    return host(out).astype(np.float64).reshape(users, new, 512)


@pytest.mark.parametrize("new", [4, 100, 256])
@pytest.mark.parametrize("pages,first_key", [(508, 0.0), (4900, 0.34375)])
@pytest.mark.parametrize("exp", [0, 100])
def test_many_pages_of_zeros_before_an_ordinary_one(new, pages, first_key, exp):
    """16 users; all values zero, with the smallest scale, but for the last page
    of the history.  The zeros weigh nothing in the values' sum and all but a
    thousandth in the normaliser, page after page; in half the cases the first
    two pages score 2^4 below the others.

    Tolerance, relative: the output's rounding 2^-8; a weight in fp16 2^-11;
    exponents: the scores are exact sums, the offsets up to 128 in magnitude are
    rounded a few times, 3 * 2^-18 each for numerator and normaliser, and 2^x
    itself 2^-22; the normaliser's additions, at most 8 a page in one lane of the
    first kernel and 18 a page in the second, of `pages` pages: 18 * 4900 * 2^-24."""
    c, users = 0.34375, 16
    codes = np.zeros((3, 2, 8, 64, 64), np.uint8)
    scales = np.ones((3, 2, 8), np.float32)
    scales[:, 1] = 2.0 ** -100
    codes[0, 0] = 0x2B if first_key else 0
    codes[1:, 0] = 0x2B  # 0.34375
    codes[2, 1], scales[2, 1] = 0x38, 2.0 ** exp  # 1.0
    past = 64 * pages
    table = np.ones((users, pages + -(-new // 64)), np.int32)
    table[:, :2], table[:, pages - 1] = 0, 2
    got = _attend(codes, scales, table, users, new, past)
    e, low = np.exp(8 * c), np.exp(8 * first_key)
    count = past + 1 + np.arange(new)
    ref = 64 * e / (128 * low + (count - 128) * e) * 2.0 ** exp
    tol = BF16_HALF + FP16_HALF + 2 * (3 * 2.0 ** -18 + 2.0 ** -22) + 18 * 4900 * 2.0 ** -24
    off = np.abs(got / ref[None, :, None] - 1)
    assert (off <= tol).all(), (np.nanmax(off), got.min(), got.max(), ref[0])


@pytest.mark.parametrize("new", [4, 100, 300])
@pytest.mark.parametrize("exp", [-100, -60, 60, 100])
def test_values_all_of_one_size(new, exp):
    """All values the same number 2^exp: whatever the weights are, so is the
    output.  Scores differ from page to page by up to 2^8 and users have up to
    2,000 tokens.  Tolerance: the output's and the weights' roundings, 18 additions
    a page in the normaliser and a product's 64 steps of 2^-23 a page, 40 pages."""
    users, pages = 40, 31
    codes = np.zeros((36, 2, 8, 64, 64), np.uint8)
    scales = np.ones((36, 2, 8), np.float32)
    for p in range(36):
        codes[p, 0] = [0x2B, 0xAB, 0x10, 0x28, 0x00][p % 5]  # +- 0.34375, 2^-5, 0.25, 0
    codes[:, 1], scales[:, 1] = 0x38, 2.0 ** exp
    table = np.stack([np.random.default_rng(u).permutation(36) for u in range(users)]).astype(np.int32)
    got = _attend(codes, scales, table[:, :pages + -(-new // 64)], users, new, 64 * pages)
    tol = BF16_HALF + FP16_HALF + 40 * (18 * 2.0 ** -24 + 64 * 2.0 ** -23)
    off = np.abs(got * 2.0 ** -exp - 1)
    assert (off <= tol).all(), (np.nanmax(off), got.min(), got.max())


@pytest.mark.parametrize("new", [100, 300])
@pytest.mark.parametrize("up", [True, False])
def test_scores_against_values(new, up):
    """Pages whose scores rise (or fall) by up to 2^45 while their values fall (or
    rise) by as much: each page weighs about alike in the values' sum, a few all
    in the normaliser.  (In the kernel for many new tokens: the other one holds
    weights relative to the largest score and loses the light ones.)

    Tolerance, relative: the output's and the weights' roundings; exponents, sums of
    numbers below 2^7 rounded a few times, 4 * 2^-18 for numerator and normaliser
    each, and 2^x 2^-22; 52 pages of 18 additions and 64 products."""
    users, pages = 40, 50
    total = pages + -(-new // 64)
    key = torch.linspace(0.0, 4.0, total) if up else torch.linspace(4.0, 0.0, total)  # scores 8 * key
    key = key.to(torch.float8_e4m3fn)
    codes = np.zeros((total, 2, 8, 64, 64), np.uint8)
    codes[:, 0] = key.view(torch.uint8).numpy()[:, None, None, None]
    codes[:, 1] = 0x38  # 1.0
    score = 8 * key.double().numpy()
    exps = np.round(-score / np.log(2))
    scales = np.ones((total, 2, 8), np.float32)
    scales[:, 1] = (2.0 ** exps)[:, None]
    got = _attend(codes, scales, np.tile(np.arange(total, dtype=np.int32), (users, 1)), users, new, 64 * pages)
    pos = 64 * pages + np.arange(new)[:, None]
    seen = np.clip(pos + 1 - 64 * np.arange(total)[None, :], 0, 64)
    ref = (seen * np.exp(score) * 2.0 ** exps).sum(1) / (seen * np.exp(score)).sum(1)
    tol = BF16_HALF + FP16_HALF + 2 * (4 * 2.0 ** -18 + 2.0 ** -22) + 52 * (18 * 2.0 ** -24 + 64 * 2.0 ** -23)
    off = np.abs(got / ref[None, :, None] - 1)
    assert (off <= tol).all(), (np.nanmax(off), tol)

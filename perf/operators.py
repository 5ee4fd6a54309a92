"""The operators of the 8-bit paged key/value cache, as they are measured.

Three operators serve a user's history without computing it again: the append
quantises new tokens' keys and values into pages, the attention reads the
pages, and the page copy carries out what forking and compacting sequences
asks for.

A page holds 64 tokens of one sequence: codes uint8 [page][2][8][64][64]
(e4m3; 0 = keys as [head][token][dim], 1 = values as [head][dim][token]) and
scales float32 [page][2][8], one power of two per page, side and head.

Each case is a dict: ``op`` is "append", "attend" or "copy".  Lengths follow
from the case alone (quantiles of a lognormal, in an order of their own), so
that ``work`` can count them; values and page numbers follow from the seed.
"""
import math
import random

import torch

own = False

PAGE, HEADS, DH, D = 64, 8, 64, 512
QKV = 3 * D
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SMALLEST = -100  # exponent of the smallest scale


# ------------------------------------------------------------------ cases
def _attend(name, dtype, users, new, new_spread, past, past_spread, window=0, sinks=0):
    return {"name": name, "op": "attend", "dtype": dtype, "users": users, "new": new, "new_spread": new_spread,
            "past": past, "past_spread": past_spread, "window": window, "sinks": sinks}


def _append(name, dtype, users, new, new_spread, past, past_spread):
    return {"name": name, "op": "append", "dtype": dtype, "users": users, "new": new, "new_spread": new_spread,
            "past": past, "past_spread": past_spread}


def listed():
    return [
        # one user's next action scored on its own: latency is all there is
        _attend("attend_one", "bf16", 1, 1, 0.0, 1000, 0.0),
        # one action for each user of the framework's usual batch (60 users, 6823 tokens)
        _attend("attend_step60", "bf16", 60, 1, 0.0, 113, 1.0),
        # a full server of long histories, one token each: two gigabytes of pages
        _attend("attend_step_long", "bf16", 250, 1, 0.0, 8000, 0.3),
        # the same server with a sliding window and sinks
        _attend("attend_step_window", "bf16", 250, 1, 0.0, 8000, 0.3, window=1000, sinks=4),
        # candidates of 60 users against their histories
        _attend("attend_candidates", "bf16", 60, 100, 0.5, 2000, 0.7),
        # prompts of 44,000 tokens in all, in one piece, read back from the pages
        _attend("attend_prompt44k", "bf16", 31, 1419, 0.2, 0, 0.0),
        # the fp32 build: a few actions each
        _attend("attend_fp32", "fp32", 60, 5, 0.5, 700, 0.7),
        # one action for each user of the usual batch
        _append("append_step60", "bf16", 60, 1, 0.0, 113, 1.0),
        # the usual batch and the largest batch, prompts whole
        _append("append_6823", "fp32", 60, 113, 1.0, 50, 0.7),
        _append("append_44k", "bf16", 391, 112, 1.0, 50, 0.7),
        # beams of the usual batch: each fork copies its last, unfinished page
        {"name": "copy_fork", "op": "copy", "pages": 700, "moved": 240, "sources": 60},
        # holes of a long-running server closed
        {"name": "copy_compact", "op": "copy", "pages": 12000, "moved": 3333, "sources": 3333},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "copy"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "copy":
        moved = _log_int(rng, 1, 3000)
        sources = moved if rng.random() < 0.5 else max(1, moved // rng.randint(2, 8))
        return {"op": "copy", "pages": 2 * moved + rng.randint(0, 500), "moved": moved, "sources": sources}
    users = _log_int(rng, 1, 250)
    if op == "append":
        return {"op": "append", "dtype": dtype, "users": users, "new": _log_int(rng, 1, max(1, 40000 // users)),
                "new_spread": rng.choice([0.0, 0.5, 1.0]), "past": rng.choice([0, _log_int(rng, 1, 300)]),
                "past_spread": rng.choice([0.0, 0.7])}
    kind = rng.choice(["step", "few", "block"])
    most = {"step": 1600000, "few": 400000, "block": 60000}[kind]  # keys over all users
    past = rng.choice([0, _log_int(rng, 1, max(1, most // users))])
    past = min(past, 30000)
    new = {"step": 1, "few": rng.randint(2, 40), "block": _log_int(rng, 30, 900)}[kind]
    if kind == "block":
        new = max(1, min(new, 20000 // users))
    windowed = rng.random() < 0.4
    return {"op": "attend", "dtype": dtype if kind != "block" else "bf16", "users": users, "new": new,
            "new_spread": 0.0 if kind == "step" else rng.choice([0.0, 0.5]), "past": past,
            "past_spread": rng.choice([0.0, 0.5]), "window": _log_int(rng, 1, 2000) if windowed else 0,
            "sinks": rng.choice([0, 1, 4, 100]) if windowed else 0}


# ------------------------------------------------------------------ lengths
def _normal_quantile(p):
    """Inverse of the standard normal distribution by bisection on erf."""
    lo, hi = -8.0, 8.0
    for _ in range(60):
        mid = 0.5 * (lo + hi)
        lo, hi = (mid, hi) if 0.5 * (1 + math.erf(mid / math.sqrt(2))) < p else (lo, mid)
    return 0.5 * (lo + hi)


def _spread_lengths(users, mean, spread, least, salt):
    """`users` lengths of about the given mean: lognormal quantiles in a shuffled order."""
    if spread == 0.0 or mean == 0:
        return [mean] * users
    raw = [math.exp(spread * _normal_quantile((i + 0.5) / users) - 0.5 * spread * spread) for i in range(users)]
    out = [max(least, int(round(mean * r))) for r in raw]
    random.Random(salt * 1000003 + users * 101 + mean).shuffle(out)
    return out


def _lengths(case):
    new = _spread_lengths(case["users"], case["new"], case["new_spread"], 1, 1)
    if case["users"] >= 8 and case["new_spread"] > 0:
        new[case["users"] // 2] = 0  # a user of the batch without new tokens
    return new, _spread_lengths(case["users"], case["past"], case["past_spread"], 0, 2)


def _visible(case, p):
    """How many keys the query at position p sees."""
    w, s = case["window"], case["sinks"]
    if w <= 0 or p + 1 <= w:
        return p + 1
    return w + min(s, p + 1 - w)


def work(case):
    if case["op"] == "copy":
        page = PAGE * D * 2 + 2 * HEADS * 4
        return {"bytes": (case["sources"] + case["moved"]) * page, "flops": 0}
    new, past = _lengths(case)
    size = 2 if case["dtype"] == "bf16" else 4
    tokens = sum(new)
    if case["op"] == "append":
        pages = sum(-(-(p + n) // PAGE) - p // PAGE for n, p in zip(new, past) if n)
        return {"bytes": tokens * 2 * D * (size + 1) + pages * 2 * HEADS * 4, "flops": 0}
    keys = pairs = 0
    for n, p in zip(new, past):
        if n == 0:
            continue
        lo = max(0, p - case["window"] + 1) if case["window"] > 0 else 0
        keys += p + n - lo + min(case["sinks"], lo)
        pairs += sum(_visible(case, i) for i in range(p, p + n))
    return {"bytes": keys * 2 * D + (keys // PAGE) * 2 * HEADS * 4 + tokens * 2 * D * size, "flops": pairs * 4 * D}


# ------------------------------------------------------------------ inputs
def _power_scale(amax):
    """The smallest power of two s with amax <= 448 s (at least 2**SMALLEST), elementwise."""
    m, e = torch.frexp(amax)  # amax = m 2**e with m in [0.5, 1)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=SMALLEST)
    k = torch.where(amax > 0, k, torch.full_like(k, SMALLEST))
    return torch.ldexp(torch.ones_like(amax), k)


def _to_codes(x):
    """float32 values (already divided by their scale) as e4m3 codes, held as bytes."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _from_codes(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _pages(gen, count):
    """Pages of ordinary keys and values: some heads larger than others, quantised page by page."""
    codes = torch.empty(count, 2, HEADS, PAGE, DH, dtype=torch.uint8, device="cuda")
    scales = torch.empty(count, 2, HEADS, device="cuda")
    for a in range(0, count, 4096):
        b = min(count, a + 4096)
        x = torch.randn(b - a, 2, HEADS, PAGE, DH, generator=gen, device="cuda")
        x *= torch.exp(0.5 * torch.randn(b - a, 2, HEADS, 1, 1, generator=gen, device="cuda"))
        s = _power_scale(x.abs().amax(dim=(3, 4)))
        codes[a:b] = _to_codes(x / s[..., None, None])
        scales[a:b] = s
    return codes, scales


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "copy":
        codes, scales = _pages(gen, case["pages"])
        ids = torch.randperm(case["pages"], generator=gen, device="cuda").to(torch.int32)
        src, dst = ids[:case["sources"]], ids[case["sources"]:case["sources"] + case["moved"]]
        which = torch.arange(case["moved"], device="cuda") % case["sources"]
        return {"codes": codes, "scales": scales, "src": src[which].contiguous(), "dst": dst.contiguous()}
    new, past = _lengths(case)
    n_cpu, p_cpu = torch.tensor(new, dtype=torch.int64), torch.tensor(past, dtype=torch.int64)
    need = (n_cpu + p_cpu + PAGE - 1) // PAGE
    total, width = int(need.sum()), max(1, int(need.max()))
    count = total + total // 8 + 2  # other sequences hold the rest of the pool
    codes, scales = _pages(gen, count)
    ids = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width)[None, :] < need[:, None]
    table[held.cuda()] = ids[:total]
    qkv = torch.randn(int(n_cpu.sum()), QKV, generator=gen, device="cuda")
    qkv *= torch.exp(0.5 * torch.randn(1, QKV // DH, 1, generator=gen, device="cuda")).expand(1, -1, DH).reshape(1, QKV)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n_cpu.cumsum(0)])
    return {"codes": codes, "scales": scales, "table": table, "qkv": qkv.to(DT[case["dtype"]]),
            "cu": cu.to(torch.int32).cuda(), "past": p_cpu.to(torch.int32).cuda()}


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if case["op"] == "attend":
        new, past = _lengths(case)
        st["most"] = max(new)
        st["out"] = torch.zeros(sum(new), D, dtype=DT[case["dtype"]], device="cuda")
    if own:
        from packed_sequence_transformer_b200 import ptl
        st["kv"] = ptl.KvPages(st["codes"], st["scales"])
        if case["op"] == "attend":
            st["ws"] = ptl.attention_paged_workspace(st["qkv"].shape[0], case["users"], case["dtype"])
        else:
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _append_plain(st):
    codes, scales, table, cu = st["codes"], st["scales"], st["table"].long(), st["cu"].long()
    past, users, tokens = st["past"].long(), st["past"].numel(), st["qkv"].shape[0]
    n = cu[1:] - cu[:-1]
    user = torch.repeat_interleave(torch.arange(users, device="cuda"), n, output_size=tokens)
    pos = past[user] + torch.arange(tokens, device="cuda") - cu[user]
    page, at = table[user, pos // PAGE], pos % PAGE
    kv = st["qkv"][:, D:].float().view(tokens, 2, HEADS, DH)
    # the scale of each touched page: that of the tokens it keeps, raised to fit the new ones
    big = torch.zeros_like(scales).index_reduce_(0, page, kv.abs().amax(-1), "amax")
    first = table[torch.arange(users, device="cuda"), (past // PAGE).clamp(max=table.shape[1] - 1)]
    kept = torch.zeros(scales.shape[0], dtype=torch.int64, device="cuda")
    opened = (n > 0) & (past % PAGE > 0)
    kept.index_add_(0, first.clamp(min=0), torch.where(opened, past % PAGE, 0))
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    rows = touched.nonzero()[:, 0]
    keep = kept[rows]
    old = scales[rows]
    raised = _power_scale(big[rows])
    raised = torch.where(keep[:, None, None] > 0, torch.maximum(old, raised), raised)
    # tokens kept are held at the raised scale, a page begun by this call starts as zeros
    t = torch.arange(PAGE, device="cuda")
    stay = t[None, :] < keep[:, None]
    empty = (keep == 0)[:, None]
    held = codes[rows]
    value = _to_codes(_from_codes(held) * (old / raised)[..., None, None])
    stay_k, stay_v = stay[:, None, :, None], stay[:, None, None, :]
    fresh = empty[:, :, None, None]
    held[:, 0] = torch.where(stay_k, value[:, 0], torch.where(fresh, 0, held[:, 0]))
    held[:, 1] = torch.where(stay_v, value[:, 1], torch.where(fresh, 0, held[:, 1]))
    codes[rows] = held
    scales[rows] = raised
    new = _to_codes(kv / scales[page][..., None])
    codes[page, 0, :, at, :] = new[:, 0]
    codes[page, 1, :, :, at] = new[:, 1]
    return codes.view(torch.float8_e4m3fn), scales


def _attend_plain(st):
    case, table, cu = st["case"], st["table"].long(), st["cu"].long()
    users, width, tokens, most = table.shape[0], table.shape[1], st["qkv"].shape[0], st["most"]
    at = table.clamp(min=0)
    kv = _from_codes(st["codes"][at]) * st["scales"][at][..., None, None]
    keys = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(users, HEADS, width * PAGE, DH)
    values = kv[:, :, 1].permute(0, 2, 1, 4, 3).reshape(users, HEADS, width * PAGE, DH)
    n = cu[1:] - cu[:-1]
    i = torch.arange(most, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=tokens - 1)
    q = st["qkv"][row, :D].float().view(users, most, HEADS, DH).transpose(1, 2)
    pos = (st["past"].long()[:, None] + i)[:, :, None]
    j = torch.arange(width * PAGE, device="cuda")
    seen = j <= pos
    if case["window"] > 0:
        seen &= (pos - j < case["window"]) | (j < case["sinks"])
    seen = seen[:, None]
    s = torch.matmul(q, keys.transpose(2, 3)) * 0.125
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, values) / p.sum(-1, keepdim=True)
    o = o.transpose(1, 2).reshape(users * most, D)
    user = torch.repeat_interleave(torch.arange(users, device="cuda"), n, output_size=tokens)
    return o[user * most + torch.arange(tokens, device="cuda") - cu[user]].to(st["qkv"].dtype)


def _copy_plain(st):
    src, dst = st["src"].long(), st["dst"].long()
    st["codes"][dst] = st["codes"][src]
    st["scales"][dst] = st["scales"][src]
    return st["codes"].view(torch.float8_e4m3fn), st["scales"]


def run(st):
    op = st["case"]["op"]
    if own:
        from packed_sequence_transformer_b200 import ptl
        if op == "attend":
            return ptl.attention_paged(st["qkv"], st["out"], st["cu"], st["kv"], st["table"], st["past"], st["ws"],
                                       window=st["case"]["window"], sinks=st["case"]["sinks"])
        if op == "append":
            ptl.kv_append(st["qkv"], st["cu"], st["kv"], st["table"], st["past"], st["ws"])
        else:
            ptl.kv_copy_pages(st["kv"], st["src"], st["dst"], st["ws"])
        return st["codes"].view(torch.float8_e4m3fn), st["scales"]
    return {"attend": _attend_plain, "append": _append_plain, "copy": _copy_plain}[op](st)


# ------------------------------------------------------------------ from the definition, in 64 bits
def _value_of(byte):
    """The number an e4m3 byte stands for: 4 exponent bits (bias 7), 3 mantissa bits, 0x7F and 0xFF no number."""
    mag, sign = byte % 128, 1.0 if byte < 128 else -1.0
    if mag == 127:
        return math.nan
    e, m = mag // 8, mag % 8
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


def _decode64(codes):
    lut = torch.tensor([_value_of(b) for b in range(256)], dtype=torch.float64, device="cuda")
    return lut[codes.int()]


def _round64(x):
    """The nearest number of e4m3, ties to the even mantissa."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -30))
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _scale64(amax):
    k = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0)).clamp(min=SMALLEST)
    k = torch.where(448.0 * torch.exp2(k - 1) >= amax, (k - 1).clamp(min=SMALLEST), k)  # log2 may be a hair off
    return torch.exp2(k)


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "copy":
        value, scales = _decode64(st["codes"]), st["scales"].double()
        value[st["dst"].long()], scales[st["dst"].long()] = value[st["src"].long()], scales[st["src"].long()]
        return value, scales
    new, past = _lengths(case)
    table, qkv, row = st["table"].tolist(), st["qkv"].double(), 0
    scales = st["scales"].double()
    if case["op"] == "append":
        value = _decode64(st["codes"])
        for u, (n, p) in enumerate(zip(new, past)):
            done = 0
            while done < n:
                page, r = table[u][(p + done) // PAGE], (p + done) % PAGE
                m = min(PAGE - r, n - done)
                x = qkv[row + done:row + done + m, D:].view(m, 2, HEADS, DH)
                s = _scale64(x.abs().amax(dim=(0, 3)))
                if r:
                    s = torch.maximum(s, scales[page])
                    ratio = (scales[page] / s)[..., None, None]
                    value[page, 0, :, :r] = _round64(value[page, 0, :, :r] * ratio[0])
                    value[page, 1, :, :, :r] = _round64(value[page, 1, :, :, :r] * ratio[1])
                else:
                    value[page] = 0.0
                scales[page] = s
                c = _round64(x / s[None, :, :, None])
                value[page, 0, :, r:r + m] = c[:, 0].transpose(0, 1)
                value[page, 1, :, :, r:r + m] = c[:, 1].permute(1, 2, 0)
                done += m
            row += n
        return value, scales
    out = torch.empty(qkv.shape[0], D, dtype=torch.float64, device="cuda")
    for u, (n, p) in enumerate(zip(new, past)):
        if n == 0:
            continue
        ids = st["table"][u, :(p + n + PAGE - 1) // PAGE].long()
        kv = _decode64(st["codes"][ids]) * scales[ids][..., None, None]
        k = kv[:, 0].transpose(0, 1).reshape(HEADS, -1, DH)[:, :p + n]
        v = kv[:, 1].permute(1, 0, 3, 2).reshape(HEADS, -1, DH)[:, :p + n]
        q = qkv[row:row + n, :D].view(n, HEADS, DH).transpose(0, 1)
        i = torch.arange(p, p + n, device="cuda")[:, None]
        j = torch.arange(p + n, device="cuda")[None, :]
        hidden = j > i
        if case["window"] > 0:
            hidden = hidden | ((i - j >= case["window"]) & (j >= case["sinks"]))
        a = torch.softmax((q @ k.transpose(1, 2) / 8.0).masked_fill(hidden, -math.inf), dim=-1)
        out[row:row + n] = (a @ v).transpose(0, 1).reshape(n, D)
        row += n
    return out

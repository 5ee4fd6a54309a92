"""Inputs and tolerances shared by the tests of the paged key/value cache."""
import numpy as np
import torch

from oracle import ptl_oracle as O
from packed_sequence_transformer_b200 import ptl
from tests.gpu_util import dev, host, tdt


def value_of_codes(codes):
    """uint8 codes (any device) as float64 values, NaN codes as NaN."""
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()


def make_pages(rng, num_pages, spread=2.0):
    """Random valid codes and power-of-two scales on the host: (uint8, float32)."""
    codes = rng.integers(0, 127, (num_pages, 2, 8, 64, 64)).astype(np.uint8)
    # ordinary magnitudes: e4m3 codes around 0x40 stand for values near 2
    codes = np.clip(codes // 3 + 16, 0, 126).astype(np.uint8)
    codes |= (rng.integers(0, 2, codes.shape).astype(np.uint8) << 7)
    scales = (2.0 ** rng.integers(-int(spread), int(spread) + 1, (num_pages, 2, 8))).astype(np.float32) * 0.25
    return codes, scales


def make_table(rng, new, past, num_pages=None, width=None):
    """A page table of distinct random pages: (int32 [U, width], pages of the pool)."""
    need = [-(-(n + p) // 64) for n, p in zip(new, past)]
    total = sum(need)
    num_pages = total + 3 if num_pages is None else num_pages
    ids = rng.permutation(num_pages)[:total].astype(np.int32)
    table = np.full((len(new), max([1] + need) if width is None else width), -1, np.int32)
    i = 0
    for u, k in enumerate(need):
        table[u, :k] = ids[i:i + k]
        i += k
    return table, num_pages


class Call:
    """One call's inputs, on the host and on the device.  `beside`: a last user
    with that many new tokens, all of whose pages are one page, whose output is
    not looked at; many of them send the others' long queries through the
    kernel for many new tokens."""

    def __init__(self, seed, new, past, dt="bf16", q_std=1.0, num_pages=None, beside=0):
        rng = np.random.default_rng(seed)
        self.rng, self.dt, self.new, self.past = rng, dt, new, past
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1])
        self.table, self.num_pages = make_table(rng, new, past, num_pages)
        self.codes, self.scales = make_pages(rng, self.num_pages)
        qkv = rng.standard_normal((self.T, 1536))
        qkv[:, :512] *= q_std
        self.qkv_d = dev(qkv.astype(np.float32), tdt(dt))
        self.rows, self.users = self.T, len(new)
        if beside:
            self.T += beside
            self.new, self.past = list(new) + [beside], list(past) + [0]
            self.cu = np.append(self.cu, self.T).astype(np.int32)
            table = np.full((self.users + 1, max(self.table.shape[1], -(-beside // 64))), -1, np.int32)
            table[:-1, :self.table.shape[1]] = self.table
            table[-1] = self.num_pages - 1
            self.table = table
            rest = torch.randn(beside, 1536, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
            self.qkv_d = torch.cat([self.qkv_d, rest.to(self.qkv_d.dtype)])
        self.upload()

    def upload(self):
        self.qkv = host(self.qkv_d)  # what the kernel sees
        self.kv = ptl.KvPages(dev(self.codes, torch.uint8), dev(self.scales, torch.float32))
        self.cu_d, self.table_d = dev(self.cu, torch.int32), dev(self.table, torch.int32)
        self.past_d = dev(np.asarray(self.past), torch.int32)

    def append(self, ws=None, stream=None):
        ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        ptl.kv_append(self.qkv_d, self.cu_d, self.kv, self.table_d, self.past_d, ws, stream=stream)
        return ws

    def attend(self, window=0, sinks=0, ws=None, out=None, stream=None):
        if ws is None:
            ws = ptl.attention_paged_workspace(self.T, len(self.new), self.dt)
            ws.fill_(255)
        out = torch.full((self.T, 512), float("nan"), dtype=tdt(self.dt), device="cuda") if out is None else out
        ptl.attention_paged(self.qkv_d, out, self.cu_d, self.kv, self.table_d, self.past_d, ws, window=window,
                            sinks=sinks, stream=stream)
        return out, ws

    def oracle(self, window=0, sinks=0):
        U = self.users
        return O.attention_paged(self.qkv[:self.rows, :512].reshape(-1, 8, 64), value_of_codes(self.kv.codes),
                                 host(self.kv.scales), self.cu[:U + 1], self.table[:U], self.past[:U], window, sinks,
                                 details=True)

    def bound(self, ref, mag, smax, count):
        """How far an output may be from the exact one, elementwise.

        Each visible key's weight carries these relative errors: the product q k,
        64 terms summed in fp32 on the tensor cores (one step 2^-23 each, their
        additions truncate) and scaled twice: 66 * 2^-23 of sum |q k| / 8, which
        is an absolute error of the exponent; q held in 11 + 11 bits (fp32 build)
        another 2^-22 of it; 2^x itself 2^-22; p in half precision 2^-11 (bf16
        build, fp32 build 2^-22), and absolutely 2^-25 where it is subnormal, of
        the sum of all weights, which is at least one.  The normaliser repeats
        the exponent's errors.  Sums of `count` weights and products in fp32 add
        2^-24 a step (the products' truncate: 2^-23).  At last the output's own
        rounding, half a step."""
        half = 2.0 ** -8 if self.dt == "bf16" else 2.0 ** -24
        prob = 2.0 ** -11 if self.dt == "bf16" else 2.0 ** -22
        expo = 2 * (67 * 2.0 ** -23 + 2.0 ** -22) * smax + 2 * 2.0 ** -22
        rel = expo[:, :, None] + prob + (count[:, None, None] * 3) * 2.0 ** -24
        vmax = np.nanmax(np.abs(value_of_codes(self.kv.codes)), initial=0.0) * float(self.kv.scales.max())
        tiny = count[:, None, None] * 2.0 ** -25 * vmax * (1.0 if self.dt == "bf16" else 2.0 ** -11)
        return half * np.abs(ref) + rel * mag + tiny + 1e-30

    def check(self, window=0, sinks=0, **kw):
        out, ws = self.attend(window, sinks, **kw)
        torch.cuda.synchronize()
        assert ptl.last_device_error(ws) == 0
        ref, mag, smax, count = self.oracle(window, sinks)
        got = host(out[:self.rows]).reshape(ref.shape)
        off = np.abs(got - ref) - self.bound(ref, mag, smax, count)
        assert np.isfinite(got).all() == np.isfinite(ref).all()
        bad = ~((off <= 0) | (np.isnan(got) & np.isnan(ref)))
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(off)))
        return out

"""Plain definitions of the dense latent operators (include/dsa.h) in 64 bits, for the tests,
with bounds on what the kernels' roundings can add up to. CPU only, no framework code."""
import math

import numpy as np
import torch

PAGE, LATENT, ROPE, ROW = 64, 512, 64, 576
CODES, SCALES, ROPES, PAGE_BYTES = 0, PAGE * LATENT, PAGE * LATENT + PAGE * 16, PAGE * 656
HALF = 2.0 ** -8               # half a step of bf16, relative to the value
CODE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
QMAX = {"e4m3": 448.0, "i8": 127.0}


def planes(pages):
    """Codes [P, 64, 512] and scales [P, 64, 4] and rotated part [P, 64, 64] as views of record pages [P, 41984]."""
    P = pages.shape[0]
    code = pages.as_strided((P, PAGE, LATENT), (PAGE_BYTES, LATENT, 1))
    scale = pages.view(torch.float32).as_strided((P, PAGE, 4), (PAGE_BYTES // 4, 4, 1), SCALES // 4)
    rope = pages.view(torch.bfloat16).as_strided((P, PAGE, ROPE), (PAGE_BYTES // 2, ROPE, 1), ROPES // 2)
    return code, scale, rope


class Case:
    """A cache and a batch on the CPU: lens[b] cached tokens of which new[b] are queries."""

    def __init__(self, lens, new, H=16, kind="bf16", seed=0, pad=0, spare=3, max_len=None):
        g = self.gen = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.H, self.kind = list(lens), list(new), H, kind
        self.T = sum(new) + pad
        self.max_len = max_len or max(max(lens), 1)
        per = [-(-n // PAGE) for n in lens]
        self.P = sum(per) + spare
        order = torch.randperm(self.P, generator=g).int()
        self.block_table = torch.full((len(lens), -(-self.max_len // PAGE)), -7, dtype=torch.int32)   # unused entries are no pages
        at = 0
        for b, n in enumerate(per):
            self.block_table[b, :n] = order[at:at + n]
            at += n
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32)
        self.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        x = 0.5 * torch.randn(self.P, PAGE, ROW, generator=g)
        if kind == "bf16":
            self.cache = x.bfloat16()
        else:
            self.cache = torch.zeros(self.P, PAGE_BYTES, dtype=torch.uint8)
            code, scale, rope = planes(self.cache)
            y = (x[..., :LATENT] * (QMAX[kind] / 2)).clamp(-QMAX[kind], QMAX[kind])
            code.copy_((y.round() if kind == "i8" else y).to(CODE[kind]).view(torch.uint8))
            scale.copy_(torch.exp(0.7 * torch.randn(self.P, PAGE, 4, generator=g)) * (2 / QMAX[kind]))
            rope.copy_(x[..., LATENT:].bfloat16())
        self.q = torch.randn(self.T, H, ROW, generator=g).bfloat16()

    def slot(self, b, pos):
        return int(self.block_table[b, pos // PAGE]), pos % PAGE

    def rows(self, b, n=None):
        """fp64 rows of request b's first n positions (bad pages as NaN), and which lie on a page."""
        n = self.lens[b] if n is None else n
        pos = torch.arange(max(n, 0))
        page = self.block_table[b][pos // PAGE].long()
        good = (page >= 0) & (page < self.P)
        p, s = page.clamp(0, self.P - 1), pos % PAGE
        if self.kind == "bf16":
            x = self.cache[p, s].double()
        else:
            code, scale, rope = planes(self.cache)
            c = code[p, s].view(CODE[self.kind]).double().view(-1, 4, 128) * scale[p, s].double()[..., None]
            x = torch.cat([c.view(-1, LATENT), rope[p, s].double()], 1)
        return x, good

    def codes(self, b, n):
        """fp64 codes [n, 512] and scales [n, 4] of request b's first n positions (records)."""
        pos = torch.arange(n)
        p, s = self.block_table[b][pos // PAGE].long().clamp(0, self.P - 1), pos % PAGE
        code, scale, _ = planes(self.cache)
        return code[p, s].view(CODE[self.kind]).double().numpy(), scale[p, s].double().numpy()

    def tokens(self):
        """(t, b, pos) of every real token (pos may be negative)."""
        t = 0
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            for j in range(m):
                yield t, b, n - m + j
                t += 1


def soften(z, v, mag_z, width):
    """softmax(z) v [H, ...], log-sum-exp, and bounds of both; z [H, n], mag_z the sums of the
    products' magnitudes. Sums in fp32 over `width` products may lose 2^-23 of their
    magnitudes each; weights, weights times scales and outputs are rounded to bf16."""
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(1, keepdims=True)
    p = e / s
    out = p @ v
    dz = (width * 2.0 ** -23) * mag_z.max(1) + 2.0 ** -20 * np.maximum(np.abs(z).max(1), 1.0)
    bo = (HALF + 2.5 * dz + 2.0 ** -18)[:, None] * (p @ np.abs(v)) + 1.01 * HALF * np.abs(out) + 1e-30
    lse = (top + np.log(s))[:, 0]
    return out, lse, bo, dz + 2.0 ** -21 * np.abs(lse) + 2.0 ** -20


def attend(c, scale, ts=None):
    """{t: (out [H, 512], lse [H], bounds of both)} of the case's tokens (or those in ts)."""
    res, rows = {}, {}
    for t, b, pos in c.tokens():
        if ts is not None and t not in ts:
            continue
        if b not in rows:
            rows[b] = c.rows(b)
        x, good = rows[b]
        keep = good[:max(pos + 1, 0)].numpy()
        k = x[:max(pos + 1, 0)].numpy()[keep]
        if len(k) == 0:
            res[t] = (np.zeros((c.H, LATENT)), np.full(c.H, -math.inf), np.zeros((c.H, LATENT)), np.zeros(c.H))
            continue
        q = c.q[t].double().numpy()
        res[t] = soften(scale * (q @ k.T), k[:, :LATENT], scale * (np.abs(q) @ np.abs(k).T), ROW)
        if c.kind != "bf16":
            # Records' weights w = a e^z s (s: a scale of the key) may be held in f16 as long as the largest of a row
            # is 2^7 at least. Below 2^-14 f16's half step is 2^-25, whatever the weight: off by 2^-25 |code| / (a sum e^z)
            # for each key; and with m the key of the largest, a e^z_m s_m >= 2^7 makes 1 / (a sum e^z) <= 2^-7 p_m s_m.
            code, sc = c.codes(b, len(keep))
            code, sc = code[keep], sc[keep]
            z = scale * (q @ k.T)
            p = np.exp(z - res[t][1][:, None])
            res[t][2][...] += 2.0 ** -32 * (p * sc.max(1)).max(1)[:, None] * np.abs(code).sum(0)[None]
    return res


def expanded(q, k, v, rope, cu_q, cu_k, scale, ts=None):
    """The same of ragged keys and values by head: {t: (out [H, 128], lse [H], bounds)}."""
    res = {}
    for b in range(len(cu_q) - 1):
        n, m = cu_k[b + 1] - cu_k[b], cu_q[b + 1] - cu_q[b]
        for j in range(m):
            t, sees = cu_q[b] + j, n - m + j + 1
            if ts is not None and t not in ts:
                continue
            H = q.shape[1]
            if sees <= 0:
                res[t] = (np.zeros((H, 128)), np.full(H, -math.inf), np.zeros((H, 128)), np.zeros(H))
                continue
            sl = slice(cu_k[b], cu_k[b] + sees)
            parts = []
            for h in range(H):
                key = torch.cat([k[sl, h], rope[sl]], 1).double().numpy()
                x = q[t, h].double().numpy()[None]
                parts.append(soften(scale * (x @ key.T), v[sl, h].double().numpy(), scale * (np.abs(x) @ np.abs(key).T), 192))
            res[t] = tuple(np.concatenate([p[i] for p in parts]) for i in range(4))
    return res


def frequencies(dim, base, factor=1.0, original=0, fast=32.0, slow=1.0):
    f = []
    lo = hi = 0.0
    if original:
        at = lambda turns: dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), dim - 1)
    for i in range(dim // 2):
        r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) if original else 1.0
        f.append(base ** (-2 * i / dim) * (1 - r + r / factor))
    return np.array(f)


def rotate(x, pos, f, interleaved, scale=1.0):
    """x [..., 64] rotated at `pos`, and a bound: half a step of bf16, the angle (2^-31 of a turn
    and its rounding to fp32), sine, cosine, products and sum in fp32 (together below 2^-20 of |a| + |b|)."""
    r = len(f)
    x = np.asarray(x, dtype=np.float64)
    ia = np.arange(r) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else r)
    y, slack = x.copy(), np.zeros_like(x)
    c, s = scale * np.cos(pos * f), scale * np.sin(pos * f)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    slack[..., ia] = slack[..., ib] = 2.0 ** -20 * abs(scale) * (np.abs(a) + np.abs(b))
    return y, HALF * np.abs(y) * (y != x) + 1.01 * slack


def normed(x, gamma, eps):
    """y and what its fp32 steps may be off by, relative to it."""
    x = np.asarray(x, dtype=np.float64)
    return x / math.sqrt((x * x).mean() + eps) * gamma, 2.0 ** -22

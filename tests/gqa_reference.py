"""Plain definitions of the grouped-query operators (include/dsa.h), for the tests: the
append step by step in fp32 as it is defined (so that codes can be compared bit for bit),
attention in 64 bits, the selection in whole numbers. CPU only, no framework code."""
import math

import numpy as np
import torch

PAGE = 64
QMAX = {torch.float8_e4m3fn: np.float32(448), torch.int8: np.float32(127)}


class Case:
    """A cache and a batch on the CPU: lens[b] cached tokens of which new[b] are queries."""

    def __init__(self, lens, new, H, Hkv, D=128, dtype=torch.float8_e4m3fn, seed=0, pad=0, spare=3, max_len=None):
        g = torch.Generator().manual_seed(seed)
        self.gen, self.lens, self.new = g, list(lens), list(new)
        self.H, self.Hkv, self.D, self.dtype, self.G = H, Hkv, D, dtype, H // Hkv
        self.T = sum(new) + pad
        self.max_len = max_len or max(max(lens), 1)
        nb = -(-self.max_len // PAGE)
        per = [-(-n // PAGE) for n in lens]
        self.P = sum(per) + spare
        order = torch.randperm(self.P, generator=g).int()
        self.block_table = torch.full((len(lens), nb), -7, dtype=torch.int32)   # unused entries are no pages
        at = 0
        for b, n in enumerate(per):
            self.block_table[b, :n] = order[at:at + n]
            at += n
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32)
        self.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        qmax = float(QMAX[dtype])

        def codes():
            x = (torch.randn(self.P, Hkv, PAGE, D, generator=g) * (qmax / 4)).clamp(-qmax, qmax)
            return (x.round() if dtype == torch.int8 else x).to(dtype)

        self.k, self.v = codes(), codes()
        self.k_scale = torch.exp(0.3 * torch.randn(self.P, Hkv, generator=g)) * (4 / qmax)
        self.v_scale = torch.exp(0.3 * torch.randn(self.P, Hkv, generator=g)) * (4 / qmax)
        self.k_mean = torch.randint(-127, 128, (self.P, Hkv, D), generator=g, dtype=torch.int32).to(torch.int8)
        self.k_mean_scale = torch.rand(self.P, Hkv, generator=g) + 0.5
        self.q = (1.5 * torch.randn(self.T, H, D, generator=g)).bfloat16()

    def tokens(self):
        """(t, b, pos) of every real token (pos may be negative)."""
        t = 0
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            for j in range(m):
                yield t, b, n - m + j
                t += 1


def rotate(x, pos, rope, cos, sin):
    """fp32 rotation of x [heads, D] (numpy float32), every operation rounded."""
    if not rope:
        return x.copy()
    r = rope // 2
    y, c, s = x.copy(), cos[pos], sin[pos]
    a, b = x[:, :r], x[:, r:rope]
    y[:, :r] = a * c - b * s
    y[:, r:rope] = b * c + a * s
    return y


def encode(x, dtype):
    """Codes of x (numpy float32, already divided by the scale) as their values in fp32."""
    q = QMAX[dtype]
    if dtype == torch.int8:
        with np.errstate(invalid="ignore"):
            return np.where(np.isnan(x), np.float32(0), np.clip(np.rint(x), -q, q)).astype(np.float32)
    t = torch.from_numpy(np.where(np.isnan(x), np.float32(0), np.clip(x, -q, q)).astype(np.float32)).to(torch.float8_e4m3fn)
    return np.where(np.isnan(x), np.float32(np.nan), t.float().numpy()).astype(np.float32)


def append(case, k_new, v_new, q_in, rope, cos, sin, mean=True):
    """The state after the append: dict of code values (fp32), scales, means, q."""
    f = np.float32
    st = {"k": case.k.float().numpy().copy(), "v": case.v.float().numpy().copy(),
          "k_scale": case.k_scale.numpy().copy(), "v_scale": case.v_scale.numpy().copy(),
          "k_mean": case.k_mean.numpy().copy(), "k_mean_scale": case.k_mean_scale.numpy().copy()}
    q = None if q_in is None else np.zeros((case.T, case.H, case.D), f)
    qmax, t0 = QMAX[case.dtype], 0
    for b, (n, m) in enumerate(zip(case.lens, case.new)):
        start = max(0, n - m)
        for blk in range(start // PAGE, -(-n // PAGE) if start < n else 0):
            a, z = max(start, blk * PAGE), min(n, (blk + 1) * PAGE)
            page, was = int(case.block_table[b, blk]), max(start, blk * PAGE) - blk * PAGE
            toks = [t0 + m - n + p for p in range(a, z)]
            if q is not None:
                for p, t in zip(range(a, z), toks):
                    q[t] = rotate(q_in[t].float().numpy(), p, rope, cos, sin)
            if not 0 <= page < case.P:
                continue
            for name, x in (("k", k_new), ("v", v_new)):
                y = np.stack([rotate(x[t].float().numpy(), p, rope if name == "k" else 0, cos, sin)
                              for p, t in zip(range(a, z), toks)])                       # [tokens, Hkv, D]
                for h in range(case.Hkv):
                    yh = y[:, h]
                    fin = np.abs(yh[np.isfinite(yh)])
                    big = fin.max() if fin.size else f(0)
                    old = st[name + "_scale"][page, h] if was else f(0)
                    s = max(old, big / qmax, f(2.0 ** -100))
                    block = st[name][page, h]
                    if was and s > old:
                        block[:was] = encode(block[:was] * (old / s), case.dtype)
                    with np.errstate(over="ignore"):
                        block[was:was + z - a] = encode(yh / s, case.dtype)
                    st[name + "_scale"][page, h] = s
            if mean:
                cnt = was + z - a
                for h in range(case.Hkv):
                    c = st["k"][page, h, :cnt]
                    msum = np.where(np.isnan(c), f(0), c).sum(0, dtype=np.float64).astype(f)
                    u = np.abs(msum).max() / f(127)
                    st["k_mean"][page, h] = np.rint(msum / u).astype(np.int8) if u > 0 else 0
                    st["k_mean_scale"][page, h] = (u * st["k_scale"][page, h]) / f(cnt)
        t0 += m
    if q is not None:
        st["q"] = torch.from_numpy(q).bfloat16()
    return st


def attend(case, sm_scale, blocks=None):
    """Attention in 64 bits: out, lse, and for the tolerances the attention of |v|, the sum
    of weights relative to the largest, the largest |v| and sum |q k| a row meets."""
    T, H, D, G = case.T, case.H, case.D, case.G
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -math.inf)
    mag, mass, top, dots, keys = np.zeros((T, H, D)), np.ones((T, H)), np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    K = (case.k.double() * case.k_scale.double()[..., None, None]).numpy()
    V = (case.v.double() * case.v_scale.double()[..., None, None]).numpy()
    q = case.q.double().numpy()
    for t, b, pos in case.tokens():
        if pos < 0:
            continue
        for h in range(case.Hkv):
            listed = range(pos // PAGE + 1) if blocks is None else [c for c in blocks[t, h].tolist() if 0 <= c <= pos // PAGE]
            at = [(int(case.block_table[b, c]), s) for c in listed for s in range(min(PAGE, pos + 1 - c * PAGE))
                  if 0 <= int(case.block_table[b, c]) < case.P]
            if not at:
                continue
            pg, sl = np.array([a[0] for a in at]), np.array([a[1] for a in at])
            kk, vv = K[pg, h, sl], V[pg, h, sl]
            for hh in range(h * G, (h + 1) * G):
                z = sm_scale * (kk @ q[t, hh])
                m = z.max()
                p = np.exp(z - m)
                l = p.sum()
                out[t, hh], lse[t, hh] = (p @ vv) / l, m + math.log(l)
                mag[t, hh], mass[t, hh] = (p @ np.abs(vv)) / l, l
                top[t, hh] = np.abs(vv).max()
                dots[t, hh] = sm_scale * (np.abs(kk) @ np.abs(q[t, hh])).max()
                keys[t, hh] = len(at)
    return dict(out=out, lse=lse, mag=mag, mass=mass, top=top, dots=dots, keys=keys)


def attend_bounds(ref):
    """Elementwise bounds of out and lse. The score of a key may be off by the rounding of
    its D-term fp32 sum, D * 2^-24 of sum |q k| (D <= 128: 2^-17); a weight is off by that
    much relatively, by fp16's half step 2^-11, by the exponential's 2^-21, and by half of
    fp16's smallest step, 2^-25 of the largest weight; the output is rounded to bf16 (half a
    step: 2^-8). The sum of the weights and the logarithm add a few 2^-24."""
    z = 2.0 ** -17 * ref["dots"][..., None]
    small = ref["keys"] * 2.0 ** -25 / ref["mass"] * ref["top"]
    inner = ref["mag"] * (2 * z + 2.0 ** -11 + 2.0 ** -20) + small[..., None]
    out = np.abs(ref["out"]) * 2.0 ** -8 + inner * (1 + 2.0 ** -8) + 1e-38
    with np.errstate(invalid="ignore"):
        lse = z[..., 0] + 2.0 ** -20 + np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0) * 2.0 ** -22
    return out, lse


def select(case, n_sel, n_first, n_last):
    """The blocks of each (token, key head) as lists, from whole numbers and fp32 products."""
    f = np.float32
    got = np.full((case.T, case.Hkv, n_sel), -1, np.int32)
    km = case.k_mean.numpy().astype(np.int64)
    for t, b, pos in case.tokens():
        nv = pos // PAGE + 1 if pos >= 0 else 0
        if nv == 0:
            continue
        pg = case.block_table[b, :nv].numpy()
        for h in range(case.Hkv):
            qs = case.q[t, h * case.G].float().numpy()
            for hh in range(h * case.G + 1, (h + 1) * case.G):
                qs = qs + case.q[t, hh].float().numpy()
            mags = np.where(np.isnan(qs), f(0), np.abs(qs))
            u = mags.max() / f(127)
            with np.errstate(invalid="ignore"):
                a = np.rint(qs / u) if u > 0 else np.zeros_like(qs)
            a = np.where(np.isnan(a), 0, np.clip(a, -127, 127)).astype(np.int64)
            dot = (km[np.clip(pg, 0, case.P - 1), h] @ a)
            score = dot.astype(f) * case.k_mean_scale.numpy()[np.clip(pg, 0, case.P - 1), h]
            rank = []
            for c in range(nv):
                bad = not 0 <= pg[c] < case.P
                forced = c < n_first or c >= nv - n_last
                s = score[c]
                rank.append((0 if forced else 3 if bad else 2 if np.isnan(s) else 1,
                             0.0 if forced or bad or np.isnan(s) else -float(s), c))
            take = sorted(c for _, _, c in sorted(rank)[:n_sel])
            got[t, h, :len(take)] = take
    return got

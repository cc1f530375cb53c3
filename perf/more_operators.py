"""Cases of the operators of dense latent attention, with their plain forms.

The paged cache holds one row a token: 512 latent values, which are key and value at once,
and 64 rotated ones, which are key only (bf16 rows, or records of e4m3 or int8 codes with a
scale for each 128 latent values and the rotated part in bf16). Four operators work on it:

  append    norms new rows, rotates their key part and the queries' (interleaved or half
            layout, frequencies scaled for long contexts), and writes the rows into their pages
  attend    causal attention over the whole context in the absorbed form
  gather    rows of the pages, dequantised, one after another: what a projection expands
  expanded  causal attention over keys and values that were expanded by head, the rotated
            part of the key shared by all heads
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, ROW = 64, 512, 64, 576
NOPE, VDIM = 128, 128
PLANES = (0, PAGE * LATENT, PAGE * LATENT + PAGE * 16, PAGE * 656)     # codes, scales, rotated part, end of a page
SCALE = 192 ** -0.5
EPS = 1e-6
# rotations between which frequencies pass from unscaled to scaled, and the length they were made for
BETA_FAST, BETA_SLOW, ORIGINAL = 32.0, 1.0, 4096


def _case(name, op, B, nq, lo, hi, H=16, cache="bf16", ragged=False, interleaved=True, base=10000.0, factor=1.0,
          dim=ROPE, keep=False):
    return dict(name=name, op=op, B=B, nq=nq, lo=lo, hi=hi, H=H, cache=cache, ragged=ragged, interleaved=interleaved,
                base=base, factor=factor, dim=dim, keep=keep)


def listed():
    return [
        # two short requests get a token each: what a call costs at least
        _case("append_tiny", "append", 2, 1, 200, 256),
        # a chunk of a prompt of 16384 tokens, e4m3 records, positions scaled by 40, rows kept in bf16 for the projection too
        _case("append_prefill_e4m3", "append", 1, 2048, 16384, 16384, H=64, cache="e4m3", factor=40.0, keep=True),
        # two short requests decode a token
        _case("attend_tiny", "attend", 2, 1, 200, 256),
        # a decode batch over ragged contexts, 16 heads
        _case("attend_decode", "attend", 64, 1, 2048, 8192),
        # the same with all 128 heads on one card
        _case("attend_decode_h128", "attend", 64, 1, 2048, 8192, H=128),
        # verification of drafted tokens, 1 to 4 a request, int8 records
        _case("attend_verify_i8", "attend", 32, 4, 4096, 16384, cache="i8", ragged=True),
        # a few long contexts, e4m3 records, 64 heads
        _case("attend_long_e4m3", "attend", 8, 1, 131072, 131072, H=64, cache="e4m3"),
        # two short contexts brought out of bf16 pages
        _case("gather_short", "gather", 2, 1, 500, 1000),
        # the cached contexts of a batch of prompts, e4m3 records
        _case("gather_e4m3", "gather", 8, 1, 4096, 16384, cache="e4m3"),
        # two short prompts
        _case("expanded_tiny", "expanded", 2, 64, 64, 100, ragged=True),
        # a batch of whole prompts of many lengths
        _case("expanded_ragged", "expanded", 16, 3000, 64, 3000, ragged=True),
        # a chunk of 2048 tokens at the end of a context of 16384, 32 heads
        _case("expanded_chunk", "expanded", 1, 2048, 16384, 16384, H=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: 1 to 128 heads, one to thousands of new tokens, contexts up to
    131072, such that rows, pairs and bytes stay within the listed cases'."""
    op = rng.choice(["append", "attend", "attend", "gather", "expanded"])
    cache = rng.choice(["bf16", "e4m3", "i8"])
    H = rng.choice([1, 2, 3, 5, 8, 12, 16, 16, 20, 24, 32, 40, 64, 128])
    interleaved, factor, dim, base, keep = True, 1.0, ROPE, 10000.0, False
    ragged = rng.random() < 0.5
    if op == "append":
        interleaved, factor, dim = rng.random() < 0.5, rng.choice([1.0, 4.0, 40.0]), rng.choice([16, 32, 64, 64])
        base, keep = rng.choice([10000.0, 1000000.0]), rng.random() < 0.5
        H = min(H, 64)
        nq = rng.choice([1, rng.randint(2, 6), _log(rng, 8, 2048)])
        B = _log(rng, 1, max(1, min(96, 2048 // nq)))
        lo = _log(rng, nq, 16384)
        hi = max(lo, min(16384, lo + _log(rng, 1, 4096)))
    elif op == "gather":
        nq, B = 1, _log(rng, 1, 32)
        hi = _log(rng, 1, min(131072, 100000 // B))
        lo = rng.randint(1, hi)
    elif op == "attend":
        nq = rng.choice([1, 1, rng.randint(2, 6), _log(rng, 8, 300)])
        B = _log(rng, 1, max(1, 96 // nq))
        hi = _log(rng, max(8, nq), max(max(8, nq), min(131072, 524288 // B, 40000000 // (B * nq * H))))
        lo = rng.randint(nq, max(nq, hi))
    else:
        cache = "bf16"
        H = min(H, 32)
        nq = _log(rng, 1, 2048)
        B = _log(rng, 1, max(1, min(16, 8192 // nq)))
        hi = _log(rng, max(8, nq), max(max(8, nq), min(16384, 32768 // B, 500000000 // (B * nq * H))))
        lo = rng.randint(1, hi)
    c = _case("", op, B, nq, lo, hi, H, cache, ragged, interleaved, base, factor, dim, keep)
    del c["name"]
    return c


def _lens(case):
    """Context lengths (the new tokens included) and new tokens of each request."""
    B, nq, lo, hi = case["B"], case["nq"], case["lo"], case["hi"]
    lens = [hi if B == 1 else min(hi, lo + int((hi - lo + 1) * ((b * 0.6180339887498949 + 0.31) % 1.0))) for b in range(B)]
    new = [1 + (5 * b + nq - 1) % nq if case["ragged"] else nq for b in range(B)]
    return lens, [min(n, m) for n, m in zip(lens, new)]


def _starts(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    op, B, H = case["op"], case["B"], case["H"]
    lens, new = _lens(case)
    T, S = sum(new), sum(lens)
    s = dict(case=case, lens=lens, new=new, T=T, S=S, max_len=max(lens), cu_q=_ints(_starts(new)), seq_lens=_ints(lens))
    if op == "expanded":
        # one projection's output holds a token's keys and values by head; the rotated keys are part of the latent rows
        s["q"] = (1.2 * rnd(T, H, NOPE + ROPE)).bfloat16()
        s["kv"] = rnd(S, H, NOPE + VDIM).bfloat16()
        s["rows"] = rnd(S, ROW).bfloat16()
        s["cu_k"] = _ints(_starts(lens))
        return s
    per = [-(-n // PAGE) for n in lens]
    P = s["P"] = sum(per) + 3
    order = torch.randperm(P, device=dev, generator=gen).int()
    s["block_table"] = bt = torch.zeros(B, max(per), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = order[at:at + n]
        at += n
    # latents differ in size from group to group, so that records' scales do
    if case["cache"] == "bf16":
        s["cache"] = (0.5 * rnd(P, PAGE, ROW)).bfloat16()
    else:
        pages = s["cache"] = torch.empty(P, PLANES[3], dtype=torch.uint8, device=dev)
        for p in range(0, P, 2048):
            x = 0.5 * rnd(min(2048, P - p), PAGE, 4, 128) * torch.exp(0.2 * rnd(min(2048, P - p), PAGE, 4, 1))
            code, scale = _encode(x, case["cache"])
            part = pages[p:p + 2048]
            part[:, :PLANES[1]] = code.view(torch.uint8).reshape(len(x), -1)
            part[:, PLANES[1]:PLANES[2]] = scale.contiguous().view(torch.uint8).reshape(len(x), -1)
            part[:, PLANES[2]:] = rnd(len(x), PAGE, ROPE).bfloat16().view(torch.uint8).reshape(len(x), -1)
    if op == "append":
        s["kv"] = (1.5 * rnd(T, ROW)).bfloat16()
        s["gamma"] = 1 + 0.1 * rnd(LATENT)
        s["q"] = rnd(T, H, NOPE + ROPE).bfloat16()         # the last 64 of each head's 192 are rotated
    elif op == "attend":
        s["q"] = rnd(T, H, ROW).bfloat16()
    else:
        s["cu_k"] = _ints(_starts(lens))
        s["first"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- the plain forms

def _where(s):
    """Request and position of each new token."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    return b, (s["seq_lens"][b] - s["cu_q"][b + 1] + t).long()


def _encode(x, cache):
    """Codes of x [..., 128] and their scale."""
    top = 448.0 if cache == "e4m3" else 127.0
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, top), torch.ones_like(amax))
    y = (x / scale).clamp(-top, top)
    return (y.to(torch.float8_e4m3fn) if cache == "e4m3" else torch.round(y).to(torch.int8)), scale


def _planes(pages, cache):
    """Codes [P, 64, 4, 128], scales [P, 64, 4] and rotated part [P, 64, 64] of record pages."""
    P = pages.shape[0]
    dt = torch.float8_e4m3fn if cache == "e4m3" else torch.int8
    return (pages[:, :PLANES[1]].view(dt).view(P, PAGE, 4, 128), pages[:, PLANES[1]:PLANES[2]].view(torch.float32).view(P, PAGE, 4),
            pages[:, PLANES[2]:].view(torch.bfloat16).view(P, PAGE, ROPE))


def _values(s, pages):
    """fp32 rows [n, 64, 576] of the listed pages."""
    if s["case"]["cache"] == "bf16":
        return s["cache"][pages].float()
    code, scale, rope = _planes(s["cache"][pages], s["case"]["cache"])
    return torch.cat([(code.float() * scale[..., None]).flatten(2), rope.float()], -1)


def _frequencies(case):
    r, base, factor = case["dim"] // 2, case["base"], case["factor"]
    i = torch.arange(r, dtype=torch.float64, device="cuda")
    f = base ** (-i / r)
    if factor == 1.0:
        return f, 1.0
    at = lambda turns: case["dim"] * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(BETA_FAST)), 0), min(math.ceil(at(BETA_SLOW)), case["dim"] - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1


def _rotate(x, cos, sin, case):
    """x [T, heads, 64] in 32 bits, its first dim values rotated."""
    d = case["dim"]
    a, b = (x[..., 0:d:2], x[..., 1:d:2]) if case["interleaved"] else (x[..., :d // 2], x[..., d // 2:d])
    c, n = cos[:, None], sin[:, None]
    y = (a * c - b * n, b * c + a * n)
    y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
    return torch.cat([y, x[..., d:]], -1)


def _append(s):
    c = s["case"]
    b, pos = _where(s)
    x = s["kv"][:, :LATENT].float()
    mean = (x.double() * x.double()).sum(-1, keepdim=True) / LATENT
    y = x * (1.0 / torch.sqrt(mean + EPS)).float() * s["gamma"]
    f, attn = _frequencies(c)
    ang = pos[:, None].double() * f
    cos, sin = (ang.cos() * attn).float(), (ang.sin() * attn).float()
    k = _rotate(s["kv"][:, None, LATENT:].float(), cos, sin, c)[:, 0].bfloat16()
    out = {"q": _rotate(s["q"][..., NOPE:].float(), cos, sin, c).bfloat16()}
    page, slot = s["block_table"][b, pos // PAGE].long(), pos % PAGE
    row = torch.cat([y.bfloat16(), k], -1)
    if c["keep"]:
        out["rows"] = row
    if c["cache"] == "bf16":
        s["cache"][page, slot] = row
        return {**out, "cache": s["cache"]}
    code, scale = _encode(y.view(-1, 4, 128), c["cache"])
    planes = _planes_views(s)
    planes[0].view(torch.uint8)[page, slot] = code.view(torch.uint8)
    planes[1][page, slot] = scale[..., 0]
    planes[2][page, slot] = k
    return {**out, "codes": planes[0], "scales": planes[1], "rope": planes[2]}


def _planes_views(s):
    """The planes as views of the cache itself."""
    pages, P = s["cache"], s["P"]
    dt = torch.float8_e4m3fn if s["case"]["cache"] == "e4m3" else torch.int8
    code = pages.as_strided((P, PAGE, 4, 128), (PLANES[3], LATENT, 128, 1)).view(dt)
    words = pages.view(torch.int32)
    scale = words.view(torch.float32).as_strided((P, PAGE, 4), (PLANES[3] // 4, 4, 1), PLANES[1] // 4)
    rope = pages.view(torch.bfloat16).as_strided((P, PAGE, ROPE), (PLANES[3] // 2, ROPE, 1), PLANES[2] // 2)
    return code, scale, rope


def _attend(s):
    c = s["case"]
    H, at = c["H"], 0
    outs, lses = [], []
    for b, (n, m) in enumerate(zip(s["lens"], s["new"])):
        kv = _values(s, s["block_table"][b, :-(-n // PAGE)].long()).view(-1, ROW)[:n]
        q = s["q"][at:at + m].float().view(m * H, ROW)
        z = torch.matmul(q, kv.t()).mul_(SCALE).view(m, H, n)
        hidden = torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None]
        z = z.masked_fill_(hidden[:, None], -math.inf)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(top).exp_()
        l = p.sum(-1, keepdim=True)
        outs.append((torch.matmul(p.view(m * H, n), kv[:, :LATENT]).view(m, H, LATENT) / l).bfloat16())
        lses.append((top + l.log())[..., 0])
        at += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _gather(s):
    rows = [_values(s, s["block_table"][b, :-(-n // PAGE)].long()).view(-1, ROW)[:n] for b, n in enumerate(s["lens"])]
    return {"rows": torch.cat(rows).bfloat16()}


def _expanded(s):
    outs, lses, tq, tk = [], [], 0, 0
    for n, m in zip(s["lens"], s["new"]):
        q = s["q"][tq:tq + m].float().transpose(0, 1)                        # [H, m, 192]
        kv = s["kv"][tk:tk + n].float().transpose(0, 1)
        rope = s["rows"][tk:tk + n, LATENT:].float()
        z = torch.matmul(q[..., :NOPE], kv[..., :NOPE].transpose(1, 2)) + torch.matmul(q[..., NOPE:], rope.t())
        hidden = torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None]
        z = z.mul_(SCALE).masked_fill_(hidden, -math.inf)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(top).exp_()
        l = p.sum(-1, keepdim=True)
        outs.append((torch.matmul(p, kv[..., NOPE:]) / l).transpose(0, 1).bfloat16())
        lses.append((top + l.log())[..., 0].t())
        tq, tk = tq + m, tk + n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


# ---------------------------------------------------------------- one pass

def _handles(s):
    """What a program keeps beside its cache: geometry, frequencies, outputs and a workspace."""
    from dsa_sparse_attention_02_gb300 import _lib
    c, T, H = s["case"], s["T"], s["case"]["H"]
    h = dict(lib=_lib, kind={"bf16": _lib.DSA_BF16, "e4m3": _lib.DSA_E4M3, "i8": _lib.DSA_I8}[c["cache"]])
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "expanded":
        size = _lib.dsa_latent_attend_expanded_workspace_size(c["B"], T, s["S"], H)
        h.update(out=new(T, H, VDIM), lse=new(T, H, dtype=torch.float32))
    else:
        geom = h["geom"] = _lib.Geometry(s["seq_lens"], s["cu_q"], s["block_table"], s["P"], s["max_len"], T)
        if c["op"] == "append":
            f = c["factor"]
            scaled = dict(factor=f, original_len=ORIGINAL, beta_fast=BETA_FAST, beta_slow=BETA_SLOW,
                          attn_factor=0.1 * math.log(f) + 1) if f != 1.0 else {}
            h["rope"] = _lib.Rope(c["dim"], c["base"], interleaved=c["interleaved"], **scaled)
            h.update(q=new(T, H, ROPE), rows=new(T, ROW) if c["keep"] else None)
            size = _lib.dsa_latent_append_workspace_size(geom)
        elif c["op"] == "attend":
            h.update(out=new(T, H, LATENT), lse=new(T, H, dtype=torch.float32))
            size = _lib.dsa_latent_attend_workspace_size(geom, H)
        else:
            h["rows"] = new(s["S"], ROW)
            size = _lib.dsa_latent_gather_workspace_size(geom)
    h["ws"] = _lib.workspace(size, "cuda")
    return h


def _own(s):
    h = s.get("handles")
    if h is None:
        h = s["handles"] = _handles(s)
    c, lib = s["case"], h["lib"]
    if c["op"] == "append":
        lib.dsa_latent_append(h["geom"], h["kind"], s["kv"], s["cache"], h["rope"], gamma=s["gamma"], eps=EPS,
                              q_in=s["q"][..., NOPE:], q_out=h["q"], kv_out=h["rows"], ws=h["ws"])
        out = {"q": h["q"], **({"rows": h["rows"]} if c["keep"] else {})}
        if c["cache"] == "bf16":
            return {**out, "cache": s["cache"]}
        return {**out, **dict(zip(("codes", "scales", "rope"), _planes_views(s)))}
    if c["op"] == "attend":
        lib.dsa_latent_attend(h["geom"], h["kind"], s["q"], s["cache"], SCALE, h["out"], h["lse"], h["ws"])
        return {"out": h["out"], "lse": h["lse"]}
    if c["op"] == "gather":
        lib.dsa_latent_gather(h["geom"], h["kind"], s["cache"], s["first"], s["cu_k"], h["rows"], h["ws"])
        return {"rows": h["rows"]}
    lib.dsa_latent_attend_expanded(s["cu_q"], s["cu_k"], s["q"], s["kv"][..., :NOPE], s["kv"][..., NOPE:],
                                   s["rows"][:, LATENT:], SCALE, h["out"], h["lse"], h["ws"])
    return {"out": h["out"], "lse": h["lse"]}


def run(s):
    if own:
        return _own(s)
    return {"append": _append, "attend": _attend, "gather": _gather, "expanded": _expanded}[s["case"]["op"]](s)


def work(case):
    lens, new = _lens(case)
    H, T, S = case["H"], sum(new), sum(lens)
    row = ROW * 2 if case["cache"] == "bf16" else 656
    if case["op"] == "append":
        return {"bytes": T * (ROW * 2 + row + 2 * H * ROPE * 2 + (ROW * 2 if case["keep"] else 0)),
                "flops": T * (4 * LATENT + 3 * (H + 1) * case["dim"])}
    if case["op"] == "gather":
        return {"bytes": S * (row + ROW * 2), "flops": 0 if case["cache"] == "bf16" else S * LATENT}
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
    if case["op"] == "attend":
        return {"bytes": S * row + T * H * (ROW * 2 + LATENT * 2 + 4), "flops": 2 * pairs * H * (ROW + LATENT)}
    return {"bytes": S * (H * (NOPE + VDIM) + ROPE) * 2 + T * H * ((NOPE + ROPE + VDIM) * 2 + 4),
            "flops": 2 * pairs * H * (NOPE + ROPE + VDIM)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lens(case)
    f8, op, H = torch.float64, case["op"], case["H"]
    kind = case["cache"]

    def row_of(b, positions):
        """64-bit rows of request b."""
        page, slot = s["block_table"][b][positions // PAGE].long(), positions % PAGE
        if kind == "bf16":
            return s["cache"][page, slot].to(f8)
        code, scale, rope = _planes_views(s)
        raw = code.view(torch.uint8)[page, slot]
        latent = raw.view(torch.float8_e4m3fn if kind == "e4m3" else torch.int8).to(f8) * scale[page, slot].to(f8)[..., None]
        return torch.cat([latent.reshape(len(positions), LATENT), rope[page, slot].to(f8)], 1)

    if op == "gather":
        return {"rows": torch.cat([row_of(b, torch.arange(n, device="cuda")) for b, n in enumerate(lens)])}
    if op in ("attend", "expanded"):
        width = LATENT if op == "attend" else VDIM
        out = torch.empty(s["T"], H, width, dtype=f8, device="cuda")
        lse = torch.empty(s["T"], H, dtype=f8, device="cuda")
        tq = tk = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            rows = row_of(b, torch.arange(n, device="cuda")) if op == "attend" else s["rows"][tk:tk + n].to(f8)
            for h in range(H):
                if op == "attend":
                    keys, values = rows, rows[:, :LATENT]
                else:
                    keys = torch.cat([s["kv"][tk:tk + n, h, :NOPE].to(f8), rows[:, LATENT:]], 1)
                    values = s["kv"][tk:tk + n, h, NOPE:].to(f8)
                z = s["q"][tq:tq + m, h].to(f8) @ keys.t() / math.sqrt(192)
                i, j = torch.arange(m, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
                z = z.masked_fill(j - i > n - m, -math.inf)
                e = torch.logsumexp(z, 1)
                lse[tq:tq + m, h] = e
                out[tq:tq + m, h] = torch.exp(z - e[:, None]) @ values
            tq, tk = tq + m, tk + n
        return {"out": out, "lse": lse}
    # append: rows and queries, unrounded quotients in place of codes
    d, r = case["dim"], case["dim"] // 2
    lo, hi = 0, 0
    if case["factor"] != 1.0:
        lo, hi = (d * math.log(ORIGINAL / (x * 2 * math.pi)) / (2 * math.log(case["base"])) for x in (BETA_FAST, BETA_SLOW))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), d - 1)
    attn = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1
    freq = []
    for i in range(r):
        part = 0.0 if case["factor"] == 1.0 else min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        freq.append(case["base"] ** (-2 * i / d) * (1 - part + part / case["factor"]))
    freq = torch.tensor(freq, dtype=f8, device="cuda")
    ia = torch.arange(r, device="cuda") * (2 if case["interleaved"] else 1)
    ib = ia + (1 if case["interleaved"] else r)

    def turn(x, pos):
        w = torch.polar(torch.full((len(pos), r), attn, dtype=f8, device="cuda"), pos.to(f8)[:, None] * freq)
        y = x.to(f8).clone()
        v = torch.complex(y[..., ia], y[..., ib]) * (w if x.dim() == 2 else w[:, None])
        y[..., ia], y[..., ib] = v.real, v.imag
        return y

    pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, new)])
    req = torch.cat([torch.full((m,), b, device="cuda") for b, m in enumerate(new)])
    c = s["kv"][:, :LATENT].to(f8)
    y = c / torch.sqrt((c ** 2).mean(1, keepdim=True) + EPS) * s["gamma"].to(f8)
    k = turn(s["kv"][:, LATENT:], pos)
    page, slot = s["block_table"][req, pos // PAGE].long(), pos % PAGE
    out = {"q": turn(s["q"][..., NOPE:], pos)}
    if case["keep"]:
        out["rows"] = torch.cat([y, k], 1)
    if kind == "bf16":
        cache = s["cache"].to(f8)
        cache[page, slot] = torch.cat([y, k], 1)
        return {**out, "cache": cache}
    code, scale, rope = _planes_views(s)
    scale, rope = scale.to(f8), rope.to(f8)
    top = 448.0 if kind == "e4m3" else 127.0
    g = y.view(-1, 4, 128)
    amax = g.abs().amax(-1)
    scale[page, slot], rope[page, slot] = amax / top, k
    if kind != "e4m3":
        return {**out, "codes": None, "scales": scale, "rope": rope}            # whole numbers
    code = code.to(f8)
    code[page, slot] = g / (amax / top)[..., None]
    return {**out, "codes": code, "scales": scale, "rope": rope}

"""Cases of the grouped-query operators over an 8-bit paged cache, with their plain forms.

The cache holds keys and values by head in 64-token pages: codes [P, Hkv, 64, D] (e4m3 or
int8) with one fp32 scale for each (page, head), and for each such block of keys an int8
mean [P, Hkv, D] with its scale. Four operators work on it:

  append   rotates new keys (and queries), quantises keys and values into their blocks
           (a block's scale grows with its largest value and its older codes follow)
           and refreshes the blocks' means
  attend   causal grouped-query attention over the whole context
  select   scores the blocks by their means and lists the best ones of each query and head
  blocks   the attention over the listed blocks only
"""
import functools
import math

import torch

own = False

PAGE = 64
QMAX = {"e4m3": 448.0, "i8": 127.0}
SCALE_FLOOR = 2.0 ** -100


def _case(name, op, B, nq, lo, hi, H, Hkv, D=128, cache="e4m3", ragged=False, rope=0, n_sel=0, first=0, last=0):
    return dict(name=name, op=op, B=B, nq=nq, lo=lo, hi=hi, H=H, Hkv=Hkv, D=D, cache=cache, ragged=ragged,
                rope=rope, n_sel=n_sel, first=first, last=last)


def listed():
    return [
        # two short requests get a token each: what a call costs at least
        _case("append_tiny", "append", 2, 1, 200, 256, 16, 4, rope=64),
        # a speculative batch's up to 4 new tokens a request, five query heads to a key head, int8
        _case("append_verify_i8", "append", 32, 4, 500, 1000, 40, 8, cache="i8", ragged=True, rope=128),
        # a 2048-token chunk of a 16384-token prompt
        _case("append_prefill", "append", 1, 2048, 16384, 16384, 64, 8, rope=128),
        # two short requests decode a token, heads of 64, three query heads to a key head
        _case("attend_tiny", "attend", 2, 1, 200, 256, 12, 4, D=64),
        # a decode batch over ragged contexts
        _case("attend_decode", "attend", 64, 1, 2048, 8192, 64, 8),
        # verification of drafted tokens, 1 to 4 a request, int8, 5 query heads to a key head
        _case("attend_verify_i8", "attend", 32, 4, 4096, 16384, 40, 8, cache="i8", ragged=True),
        # a few long contexts
        _case("attend_long", "attend", 8, 1, 131072, 131072, 64, 8),
        # a chunk of a prompt over what is cached of it
        _case("attend_prefill", "attend", 1, 2048, 16384, 16384, 64, 8),
        # the blocks (2048 tokens' worth) of a decode step over long contexts
        _case("select_long", "select", 8, 1, 131072, 131072, 64, 8, n_sel=32, first=1, last=2),
        # the blocks of each token of a prompt's chunk
        _case("select_prefill", "select", 1, 2048, 16384, 16384, 64, 8, n_sel=32, first=1, last=2),
        # attention over the selected blocks: decode over long contexts
        _case("blocks_long", "blocks", 8, 1, 131072, 131072, 64, 8, n_sel=32, first=1, last=2),
        # and each token of a prompt's chunk over its own blocks
        _case("blocks_prefill", "blocks", 1, 2048, 16384, 16384, 64, 8, n_sel=32, first=1, last=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: any head layout, one to thousands of new tokens, contexts up to
    131072, such that tokens x heads, score counts and new rows stay within the listed cases'."""
    op = rng.choice(["append", "attend", "select", "blocks"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while Hkv * g > 64:
        g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    kind = rng.choice(["decode", "verify", "prefill"])
    if kind == "prefill":
        nq = _log(rng, 8, 2048)
        hi = _log(rng, nq, 16384)
        B = rng.randint(1, max(1, min(8, 2048 * 16384 // (nq * hi))))
    else:
        nq = 1 if kind == "decode" else rng.randint(2, 6)
        B = _log(rng, 1, 96)
        hi = _log(rng, max(8, nq), min(131072, 8 * 131072 // B, (2048 * 16384) // (B * nq)))
    if op == "append":
        hi = max(nq, min(hi, 16384, 262144 // B))
    if op == "select":              # contexts with more blocks than are taken
        hi = max(hi, _log(rng, 2048, 4096))
        B = max(1, min(B, 2048 * 16384 // (nq * hi)))
    lo = rng.randint(max(nq, 2048) if op == "select" else nq, hi)
    n_sel = first = last = 0
    if op in ("select", "blocks"):
        n_sel = rng.choice([8, 16, 24] if op == "select" else [2, 3, 8, 16, 24, 32])
        first = rng.randint(0, 1)
        last = rng.randint(1, min(3, n_sel - first))
    c = _case("", op, B, nq, lo, hi, Hkv * g, Hkv, D, rng.choice(["e4m3", "i8"]), rng.random() < 0.5,
              rng.choice([0, 32, D]) if op == "append" else 0, n_sel, first, last)
    del c["name"]
    return c


def _lens(case):
    """Context lengths (the new tokens included) and new tokens of each request."""
    B, nq, lo, hi = case["B"], case["nq"], case["lo"], case["hi"]
    lens = [hi if B == 1 else min(hi, lo + int((hi - lo + 1) * ((b * 0.6180339887498949 + 0.31) % 1.0))) for b in range(B)]
    new = [1 + (5 * b + nq - 1) % nq if case["ragged"] else nq for b in range(B)]
    return lens, new


def _mean(kc, k_scale, n, valid):
    """The int8 mean of each block's codes kc [..., 64, D] over its n valid tokens, and its scale."""
    m = torch.where(valid[..., None], kc.float(), kc.new_zeros((), dtype=torch.float32)).sum(-2)
    u = m.abs().amax(-1)
    u = u / torch.full_like(u, 127.0)
    code = torch.where(u[..., None] > 0, torch.round(m / u[..., None]), torch.zeros_like(m)).to(torch.int8)
    return code, u * k_scale / n


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    lens, new = _lens(case)
    T = sum(new)
    max_len = max(lens)
    per = [-(-n // PAGE) for n in lens]
    P = sum(per) + 3
    order = torch.randperm(P, device=dev, generator=gen).int()
    bt = torch.zeros(B, -(-max_len // PAGE), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = order[at:at + n]
        at += n
    s = dict(case=case, max_len=max_len, T=T, P=P, block_table=bt, max_new=max(new),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             cu_q=torch.tensor([0] + [sum(new[:i + 1]) for i in range(B)], dtype=torch.int32, device=dev))
    # keys have a part that their block shares (so that its mean says something), values do not;
    # scales differ from block to block
    qmax = QMAX[case["cache"]]
    dt = torch.float8_e4m3fn if case["cache"] == "e4m3" else torch.int8

    def codes(shared):
        x = rnd(P, Hkv, PAGE, D)
        if shared:
            x += 0.6 * rnd(P, Hkv, 1, D)
        x = (x * (qmax / 5)).clamp_(-qmax, qmax)
        return (x.round_() if dt == torch.int8 else x).to(dt)

    s["k"], s["v"] = codes(True), codes(False)
    s["k_scale"] = torch.exp(0.2 * rnd(P, Hkv)) * (5 / qmax)
    s["v_scale"] = torch.exp(0.2 * rnd(P, Hkv)) * (5 / qmax)
    held = torch.zeros(P, dtype=torch.float32, device=dev)
    held[order[:sum(per)].long()] = torch.tensor([min(PAGE, n - PAGE * i) for n in lens for i in range(-(-n // PAGE))],
                                                 dtype=torch.float32, device=dev)
    held = held.clamp_(min=1.0)
    valid = torch.arange(PAGE, device=dev) < held[:, None, None]
    s["k_mean"], s["k_mean_scale"] = _mean(s["k"], s["k_scale"], held[:, None], valid.expand(P, Hkv, PAGE))
    # one projection's output holds queries, keys and values side by side; attention reads the queries alone
    if case["op"] == "append":
        qkv = (1.3 * rnd(T, H + 2 * Hkv, D)).bfloat16()
        s["q"], s["k_new"], s["v_new"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        r = case["rope"] // 2
        if r:
            ang = torch.arange(max_len, dtype=torch.float64, device=dev)[:, None] * \
                (10000.0 ** (-torch.arange(r, dtype=torch.float64, device=dev) / r))[None]
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    else:
        s["q"] = (1.5 * rnd(T, H, D)).bfloat16()
    if case["op"] == "blocks":
        n, f, l = case["n_sel"], case["first"], case["last"]
        b = torch.searchsorted(s["cu_q"][1:].contiguous(), torch.arange(T, device=dev, dtype=torch.int32), right=True)
        pos = s["seq_lens"][b] - s["cu_q"][b + 1] + torch.arange(T, device=dev, dtype=torch.int32)
        vis = (pos // PAGE + 1)[:, None, None]
        c = torch.arange(bt.shape[1], device=dev)[None, None]
        key = torch.rand(T, Hkv, bt.shape[1], device=dev, generator=gen) + 2.0 * ((c < f) | (c >= vis - l))
        key = torch.where(c < vis, key, -1.0)
        if key.shape[2] < n:
            key = torch.nn.functional.pad(key, (0, n - key.shape[2]), value=-1.0)
        top, idx = key.topk(n, dim=2)
        idx = torch.where(top >= 0, idx, 1 << 30).sort(dim=2).values
        s["list"] = torch.where(idx < (1 << 30), idx, -1).int().contiguous()
    return s


# ---------------------------------------------------------------- the plain forms

def _where(s):
    """Request, index among its request's new tokens, and position of each new token."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    j = t - s["cu_q"][b]
    return b, j.long(), (s["seq_lens"][b] - s["cu_q"][b + 1] + t).long()


def _rotate(x, rope, cos, sin):
    """fp32 rotation of x [T, heads, D] by the positions' cos and sin [T, rope/2]."""
    if not rope:
        return x
    r = rope // 2
    a, b, c, d = x[..., :r], x[..., r:rope], cos[:, None], sin[:, None]
    return torch.cat([a * c - b * d, b * c + a * d, x[..., rope:]], -1)


def _encode(x, cache):
    q = QMAX[cache]
    return torch.round(x).clamp(-q, q).to(torch.int8) if cache == "i8" else x.clamp(-q, q).to(torch.float8_e4m3fn)


def _bytes(x):
    return x.view(torch.uint8)


def _append(s):
    c = s["case"]
    b, _, pos = _where(s)
    rope, cache, B = c["rope"], c["cache"], c["B"]
    cos, sin = (s["cos"][pos], s["sin"][pos]) if rope else (None, None)
    q_out = _rotate(s["q"].float(), rope, cos, sin).bfloat16()
    bt, T, Hkv, D = s["block_table"].long(), s["T"], c["Hkv"], c["D"]
    start = (s["seq_lens"] - s["cu_q"].diff()).long()                 # each request's first new position
    blk0 = start // PAGE
    width = (s["max_new"] + PAGE - 2) // PAGE + 1                     # blocks that a request's new tokens can touch
    i, slot = pos // PAGE - blk0[b], pos % PAGE
    blk = blk0[:, None] + torch.arange(width, device="cuda")
    page = bt.gather(1, blk.clamp(max=bt.shape[1] - 1))               # [B, width]
    tok = torch.arange(PAGE, device="cuda")
    old = (blk[..., None] * PAGE + tok < start[:, None, None])[:, :, None]   # [B, width, 1, 64]: held before
    held = old.any(-1)
    page_t = bt[b, pos // PAGE]
    for_all = {}
    for name, x in (("k", _rotate(s["k_new"].float(), rope, cos, sin)), ("v", s["v_new"].float())):
        y = torch.zeros(B, width, PAGE, Hkv, D, device="cuda")
        y[b, i, slot] = x
        y = y.transpose(2, 3)                                         # [B, width, Hkv, 64, D]
        amax = y.abs().amax((-1, -2))
        s_old = torch.where(held, s[name + "_scale"][page], torch.zeros_like(amax))
        s_new = torch.maximum(s_old, (amax / torch.full_like(amax, QMAX[cache])).clamp(min=SCALE_FLOOR))
        was = s[name][page]
        moved = _encode(was.float() * (s_old / s_new)[..., None, None], cache)
        fresh = _encode(y / s_new[..., None, None], cache)
        grown = old[..., None] & (s_new > s_old)[..., None, None]
        first = torch.where(grown, _bytes(moved), _bytes(was))[:, 0]
        _bytes(s[name])[page[:, 0]] = first                           # older codes follow their scale
        _bytes(s[name])[page_t, :, slot] = _bytes(fresh)[b, i, :, slot]
        s[name + "_scale"][page_t] = s_new[b, i]
        for_all[name] = s_new
    n = (s["seq_lens"].long()[:, None] - blk * PAGE).clamp(1, PAGE)
    valid = (tok < n[..., None])[:, :, None].expand(B, width, Hkv, PAGE)
    mean, scale = _mean(s["k"][page], for_all["k"], n[..., None].float(), valid)
    s["k_mean"][page_t] = mean[b, i]
    s["k_mean_scale"][page_t] = scale[b, i]
    return {"q": q_out, **{n: s[n] for n in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")}}


def _attend(s, blocks=None):
    c = s["case"]
    b, j, pos = _where(s)
    B, H, Hkv, D, n = c["B"], c["H"], c["Hkv"], c["D"], s["max_new"]
    g = H // Hkv
    bt = s["block_table"].long()
    L = bt.shape[1] * PAGE
    deq = lambda x, sc: (x[bt].float() * sc[bt][..., None, None]).transpose(1, 2).reshape(B, Hkv, L, D)  # noqa: E731
    q = torch.zeros(B, n, H, D, device="cuda")
    q[b, j] = s["q"].float()
    q = q.reshape(B, n, Hkv, g, D).transpose(1, 2).reshape(B, Hkv, n * g, D)
    z = torch.matmul(q, deq(s["k"], s["k_scale"]).transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, n, g, L)
    at = torch.full((B, n), -1, dtype=torch.int64, device="cuda")
    at[b, j] = pos
    hidden = (torch.arange(L, device="cuda") > at[..., None])[:, None, :, None]       # [B, 1, n, 1, L]
    if blocks is not None:
        seen = torch.zeros(B, n, Hkv, L // PAGE + 1, dtype=torch.bool, device="cuda")
        mine = torch.zeros(s["T"], Hkv, L // PAGE + 1, dtype=torch.bool, device="cuda")
        seen[b, j] = mine.scatter_(2, torch.where(blocks < 0, L // PAGE, blocks).long(), True)
        hidden = hidden | ~seen[..., :-1].repeat_interleave(PAGE, 3).transpose(1, 2)[:, :, :, None]
    z = z.masked_fill_(hidden, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, n * g, L), deq(s["v"], s["v_scale"])).view(B, Hkv, n, g, D) / l.clamp(min=1e-30)
    lse = (m + l.log()).squeeze(-1)
    return {"out": o.transpose(1, 2).reshape(B, n, H, D)[b, j].bfloat16(), "lse": lse.transpose(1, 2).reshape(B, n, H)[b, j]}


def _select(s):
    c = s["case"]
    b, j, pos = _where(s)
    B, H, Hkv, D, n = c["B"], c["H"], c["Hkv"], c["D"], s["max_new"]
    bt = s["block_table"].long()
    qs = functools.reduce(torch.add, s["q"].float().view(s["T"], Hkv, H // Hkv, D).unbind(2))
    u = qs.abs().amax(-1, keepdim=True)
    u = u / torch.full_like(u, 127.0)
    code = torch.where(u > 0, torch.round(qs / u), torch.zeros_like(qs))
    a = torch.zeros(B, n, Hkv, D, device="cuda")
    a[b, j] = code
    dot = torch.matmul(a.transpose(1, 2), s["k_mean"][bt].float().permute(0, 2, 3, 1))    # whole numbers below 2^24
    score = (dot * s["k_mean_scale"][bt].transpose(1, 2)[:, :, None]).transpose(1, 2)[b, j]    # [T, Hkv, blocks]
    blk = torch.arange(bt.shape[1], device="cuda")[None, None]
    seen = (pos // PAGE + 1)[:, None, None]
    score = score.masked_fill((blk < c["first"]) | (blk >= seen - c["last"]), math.inf).masked_fill(blk >= seen, -math.inf)
    if bt.shape[1] < c["n_sel"]:
        score = torch.nn.functional.pad(score, (0, c["n_sel"] - bt.shape[1]), value=-math.inf)
    top, idx = score.sort(dim=2, descending=True, stable=True)
    far = bt.shape[1] + c["n_sel"]
    idx = torch.where(top > -math.inf, idx, far)[..., :c["n_sel"]].sort(dim=2).values
    return {"blocks": torch.where(idx < far, idx, -1).int()}


# ---------------------------------------------------------------- one pass

def _handles(s):
    """What a program keeps beside its cache: the geometry, the cache's handle, outputs and a workspace."""
    from dsa_sparse_attention_02_gb300 import _lib
    c = s["case"]
    geom = _lib.Geometry(s["seq_lens"], s["cu_q"], s["block_table"], s["P"], s["max_len"], s["T"])
    cache = _lib.GqaCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_mean"], s["k_mean_scale"])
    size = {"append": lambda: _lib.dsa_gqa_append_workspace_size(geom, cache),
            "attend": lambda: _lib.dsa_gqa_attend_workspace_size(geom, cache, c["H"]),
            "select": lambda: _lib.dsa_block_select_workspace_size(geom, cache, c["n_sel"]),
            "blocks": lambda: _lib.dsa_gqa_attend_blocks_workspace_size(geom, cache, c["H"], c["n_sel"])}[c["op"]]()
    h = dict(lib=_lib, geom=geom, cache=cache, ws=_lib.workspace(size, "cuda"))
    if c["op"] == "select":
        h["blocks"] = torch.empty(s["T"], c["Hkv"], c["n_sel"], dtype=torch.int32, device="cuda")
    elif c["op"] == "append":
        h["q"] = torch.empty(s["T"], c["H"], c["D"], dtype=torch.bfloat16, device="cuda")
    else:
        h["out"] = torch.empty(s["T"], c["H"], c["D"], dtype=torch.bfloat16, device="cuda")
        h["lse"] = torch.empty(s["T"], c["H"], dtype=torch.float32, device="cuda")
    return h


def _own(s):
    h = s.get("handles")
    if h is None:
        h = s["handles"] = _handles(s)
    c, lib = s["case"], h["lib"]
    if c["op"] == "append":
        lib.dsa_gqa_append(h["geom"], h["cache"], s["k_new"], s["v_new"], s["q"], h["q"], c["rope"], s.get("cos"), s.get("sin"), h["ws"])
        return {"q": h["q"], **{n: s[n] for n in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")}}
    if c["op"] == "select":
        lib.dsa_block_select(h["geom"], h["cache"], s["q"], c["n_sel"], c["first"], c["last"], h["blocks"], h["ws"])
        return {"blocks": h["blocks"]}
    if c["op"] == "attend":
        lib.dsa_gqa_attend(h["geom"], h["cache"], s["q"], c["D"] ** -0.5, h["out"], h["lse"], h["ws"])
    else:
        lib.dsa_gqa_attend_blocks(h["geom"], h["cache"], s["q"], s["list"], c["D"] ** -0.5, h["out"], h["lse"], h["ws"])
    return {"out": h["out"], "lse": h["lse"]}


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "append":
        return _append(s)
    if op == "select":
        return _select(s)
    return _attend(s, s.get("list"))


def work(case):
    lens, new = _lens(case)
    H, Hkv, D, T = case["H"], case["Hkv"], case["D"], sum(new)
    blocks = sum(-(-n // PAGE) for n in lens)
    if case["op"] == "append":
        touched = sum((n - 1) // PAGE - (n - m) // PAGE + 1 for n, m in zip(lens, new))
        kept = sum(min((n - m) % PAGE, PAGE) for n, m in zip(lens, new))     # older tokens in the touched blocks
        moved = T * (H + 2 * Hkv) * D * 2 + T * H * D * 2 + T * 2 * Hkv * D + kept * Hkv * D
        return {"bytes": moved + touched * Hkv * (D + 12) + T * case["rope"] * 4, "flops": T * (6 * (H + Hkv) + 3 * Hkv) * D}
    if case["op"] == "select":
        pairs = sum((n - m + i) // PAGE + 1 for n, m in zip(lens, new) for i in range(m))
        return {"bytes": blocks * Hkv * (D + 4) + T * H * D * 2 + T * Hkv * case["n_sel"] * 4,
                "flops": 2 * pairs * Hkv * D}
    io = T * H * (4 * D + 4)
    if case["op"] == "attend":
        pairs = sum(n - m + i + 1 for n, m in zip(lens, new) for i in range(m))
        return {"bytes": sum(lens) * Hkv * 2 * D + blocks * Hkv * 8 + io, "flops": 4 * pairs * H * D}
    listed_ = [min(case["n_sel"], (n - m + i) // PAGE + 1) for n, m in zip(lens, new) for i in range(m)]
    pairs = sum(listed_) * PAGE
    return {"bytes": min(blocks, sum(listed_)) * Hkv * (PAGE * 2 * D + 8) + T * Hkv * case["n_sel"] * 4 + io,
            "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "select":
        return None                                                       # whole numbers
    s = prepare(case, seed)
    lens, new = _lens(case)
    f8, H, Hkv, D = torch.float64, case["H"], case["Hkv"], case["D"]
    g, qmax = H // Hkv, QMAX[case["cache"]]
    bt = s["block_table"].cpu()
    t0 = 0
    if case["op"] != "append":
        out = torch.zeros(s["T"], H, D, dtype=f8, device="cuda")
        lse = torch.full((s["T"], H), -math.inf, dtype=f8, device="cuda")
        for b, (n, m) in enumerate(zip(lens, new)):
            pages = bt[b, :-(-n // PAGE)].long().cuda()
            pos = torch.arange(n - m, n, device="cuda")
            for h in range(Hkv):
                kk = (s["k"][pages, h].to(f8) * s["k_scale"][pages, h].to(f8)[:, None, None]).reshape(-1, D)[:n]
                vv = (s["v"][pages, h].to(f8) * s["v_scale"][pages, h].to(f8)[:, None, None]).reshape(-1, D)[:n]
                for lo in range(0, m, 256):
                    hi = min(m, lo + 256)
                    z = torch.einsum("tgd,sd->tgs", s["q"][t0 + lo:t0 + hi, h * g:(h + 1) * g].to(f8), kk) / math.sqrt(D)
                    ok = torch.arange(n, device="cuda")[None] <= pos[lo:hi, None]
                    if "list" in s:
                        has = torch.zeros(hi - lo, len(pages) + 1, dtype=torch.bool, device="cuda")
                        li = s["list"][t0 + lo:t0 + hi, h].long()
                        has.scatter_(1, torch.where(li < 0, len(pages), li), True)
                        ok &= has[:, torch.arange(n, device="cuda") // PAGE]
                    z = z.masked_fill(~ok[:, None], -math.inf)
                    e = torch.logsumexp(z, -1)
                    lse[t0 + lo:t0 + hi, h * g:(h + 1) * g] = e
                    out[t0 + lo:t0 + hi, h * g:(h + 1) * g] = torch.einsum("tgs,sd->tgd", torch.exp(z - e[..., None]), vv)
            t0 += m
        return {"out": out, "lse": lse}
    # append: rotated queries, unrounded quotients in place of e4m3 codes, scales
    rope, r = case["rope"], case["rope"] // 2

    def turn(x, pos):
        x = x.to(f8).clone()
        if r:
            c, d = s["cos"][pos].to(f8)[:, None], s["sin"][pos].to(f8)[:, None]
            lo, hi = x[..., :r].clone(), x[..., r:rope].clone()
            x[..., :r], x[..., r:rope] = lo * c - hi * d, hi * c + lo * d
        return x

    q = torch.zeros(s["T"], H, D, dtype=f8, device="cuda")
    code = {n: s[n].to(f8) for n in ("k", "v")}
    sc = {n: s[n + "_scale"].to(f8) for n in ("k", "v")}
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n - m, n, device="cuda")
        q[t0:t0 + m] = turn(s["q"][t0:t0 + m], pos)
        for name, x in (("k", turn(s["k_new"][t0:t0 + m], pos)), ("v", s["v_new"][t0:t0 + m].to(f8))):
            for blk in range((n - m) // PAGE, (n - 1) // PAGE + 1):
                pg, a, z = int(bt[b, blk]), max(n - m, blk * PAGE), min(n, blk * PAGE + PAGE)
                y = x[a - (n - m):z - (n - m)].transpose(0, 1)            # [Hkv, tokens, D]
                was = a - blk * PAGE
                big = (y.abs().amax((1, 2)) / qmax).clamp(min=SCALE_FLOOR)
                if was:
                    big = torch.maximum(big, sc[name][pg])
                    code[name][pg, :, :was] *= (sc[name][pg] / big)[:, None, None]
                sc[name][pg] = big
                code[name][pg, :, was:z - blk * PAGE] = y / big[:, None, None]
        t0 += m
    e4 = case["cache"] == "e4m3"
    return {"q": q, "k": code["k"] if e4 else None, "v": code["v"] if e4 else None, "k_scale": sc["k"], "v_scale": sc["v"],
            "k_mean": None, "k_mean_scale": None}

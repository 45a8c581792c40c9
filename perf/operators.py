"""Measured cases of the cache operators: rotary positions, appending to a paged
cache, reading it back as bf16 rows, and attention over a cache held in 4 bits.

``run`` computes a case in its plain form (elementary torch operations) or,
with ``own`` set, through the library's entry points.  ``exact`` is the same
operator in 64 bits, written apart from both.

A cache page holds ``page`` rows per head ([pages, H, page, D], row ``o`` of
page ``page_table[b, p]`` is position ``p * page + o`` of sequence b):
  bf16   the values;
  e4m3   x ~ scale * E4M3, one fp32 scale a row and head: max|x| / 448
         (1 for a row of zeros);
  e2m1   x ~ tensor_scale * E4M3 scale * E2M1, one scale for 16 elements:
         max|x| / (6 * tensor_scale) rounded to E4M3; two codes a byte, the
         even element in the low half.
A new key is rotated, rounded once to fp32, then rounded to the cache's type.
``kv_len[b]`` counts the sequence's tokens, the new ones among them (0: an
unused place of a padded batch).
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the indexer's 64 query heads of one decoded token for each of 32
        # sequences at contexts up to 524,288: a launch's latency
        dict(name="rotary_step", op="rotary", N=32, H=64, D=128, rot=64, off=0, inter=False,
             dtype="bfloat16", scaling="none", far=524288, inverse=False, pad=0),
        # the queries of an 8,192-token prompt, interleaved pairs, frequencies
        # scaled for a long context
        dict(name="rotary_prompt", op="rotary", N=8192, H=64, D=128, rot=64, off=0, inter=True,
             dtype="bfloat16", scaling="yarn", far=131072, inverse=False, pad=0),
        # gradients of rotated heads: the last 64 of 192 elements, fp32, an odd
        # number of tokens, heads inside a wider fused projection
        dict(name="rotary_grad", op="rotary", N=4099, H=16, D=192, rot=64, off=128, inter=False,
             dtype="float32", scaling="linear", far=32768, inverse=True, pad=64),
        # one new indexer key a sequence into the contiguous E4M3 cache that the
        # indexer scores (one page a sequence)
        dict(name="append_step_e4m3", op="append", cache="e4m3", B=32, S=1, ragged=False, ctx=512, page=512,
             H=1, Dk=128, Dv=0, rot=64, off=64, inter=True, idle=2),
        # ragged prompts into a bf16 paged cache, 8 key/value heads
        dict(name="append_prompt_bf16", op="append", cache="bf16", B=9, S=4096, ragged=True, ctx=4500, page=64,
             H=8, Dk=128, Dv=128, rot=128, off=0, inter=False, idle=1),
        # ragged prompts into a 4-bit paged cache, and the rows back as bf16 for
        # an attention that reads contiguous rows
        dict(name="append_prompt_e2m1", op="append", cache="e2m1", B=13, S=2048, ragged=True, ctx=2304, page=16,
             H=4, Dk=128, Dv=128, rot=64, off=0, inter=False, idle=1),
        # a short E4M3 context read back: a call's latency
        dict(name="read_e4m3", op="read", cache="e4m3", B=3, T=1000, page=16, H=1, D=128),
        # the prefixes of 8 sequences read back from 4 bits for a long prefill
        dict(name="read_e2m1", op="read", cache="e2m1", B=8, T=32768, page=64, H=1, D=128),
        # one token of one short conversation, grouped heads: latency
        dict(name="attention_step_short", op="attention", B=1, S=1, HA=32, Hkv=8, Dk=128, Dv=128, ctx=777,
             page=16, topk=0, ragged=False, idle=0, lse=False),
        # one token for each of 32 sequences of very different lengths
        dict(name="attention_step_ragged", op="attention", B=32, S=1, HA=64, Hkv=8, Dk=128, Dv=128, ctx=32768,
             page=64, topk=0, ragged=True, idle=1, lse=True),
        # one token a sequence over the 2,048 keys that the indexer selected of
        # 131,072: 128 heads over one shared cache row a key
        dict(name="attention_step_selected", op="attention", B=32, S=1, HA=128, Hkv=1, Dk=128, Dv=128,
             ctx=131072, page=131072, topk=2048, ragged=False, idle=0, lse=False),
        # a chunk of a prompt, each query over its own selection
        dict(name="attention_prompt_selected", op="attention", B=1, S=1024, HA=64, Hkv=1, Dk=128, Dv=128,
             ctx=8192, page=64, topk=2048, ragged=False, idle=0, lse=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "read", "attention", "attention"])
    if op == "rotary":
        D = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([d for d in (16, 32, 64, 96, 128) if d <= D])
        H = rng.choice([1, 2, 3, 8, 16, 64, 128])
        return dict(op=op, N=_log(rng, 1, max(2, 60_000_000 // (H * D))), H=H, D=D, rot=rot,
                    off=rng.choice([0, D - rot]), inter=rng.random() < 0.5,
                    dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), far=_log(rng, 1000, 1_000_000),
                    inverse=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 64]))
    if op == "append":
        cache = rng.choice(["bf16", "e4m3", "e2m1"])
        D = rng.choice([64, 128, 192, 256])
        H, B = rng.choice([1, 1, 2, 4, 8]), _log(rng, 1, 64)
        S = 1 if rng.random() < 0.4 else _log(rng, 2, max(3, 16_000_000 // (B * H * D)))
        rot = rng.choice([r for r in (0, 32, 64, 128) if r <= D])
        ctx = S + _log(rng, 1, 600)
        return dict(op=op, cache=cache, B=B, S=S, ragged=S > 1 and rng.random() < 0.6, ctx=ctx,
                    page=rng.choice([16, 64, 24, ctx]), H=H, Dk=D, Dv=rng.choice([0, 64, 128]), rot=rot,
                    off=rng.choice([0, D - rot]), inter=rng.random() < 0.5, idle=rng.choice([0, 0, 1]))
    if op == "read":
        D, H, B = rng.choice([64, 128, 192, 256]), rng.choice([1, 1, 2, 8]), _log(rng, 1, 32)
        return dict(op=op, cache=rng.choice(["bf16", "e4m3", "e2m1"]), B=B,
                    T=_log(rng, 1, max(2, 30_000_000 // (B * H * D))), page=rng.choice([16, 64, 24]), H=H, D=D)
    Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128), (256, 256)])
    if rng.random() < 0.5:      # every key, one token or a few
        Hkv = rng.choice([1, 2, 4, 8])
        G, B, S = rng.choice([1, 4, 5, 8, 16]), _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 4])
        return dict(op=op, B=B, S=S, HA=Hkv * G, Hkv=Hkv, Dk=Dk, Dv=Dv,
                    ctx=_log(rng, S, max(S + 1, 2_000_000 // (B * Hkv))), page=rng.choice([16, 64, 24]), topk=0,
                    ragged=rng.random() < 0.6, idle=rng.choice([0, 0, 1]) if B > 1 else 0, lse=rng.random() < 0.5)
    B, S = (_log(rng, 1, 32), 1) if rng.random() < 0.6 else (1, _log(rng, 2, 300))
    topk = _log(rng, 1, 2048)
    return dict(op=op, B=B, S=S, HA=rng.choice([8, 16, 40, 64, 128]), Hkv=1, Dk=Dk, Dv=Dv,
                ctx=max(S, topk, _log(rng, 64, 32768)), page=rng.choice([16, 64, 24]), topk=topk,
                ragged=rng.random() < 0.4, idle=0, lse=rng.random() < 0.5)


def _lens(case):
    """kv_len of every sequence, and its new tokens (append): from the case alone."""
    rng = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    B, ctx = case["B"], case.get("ctx", case.get("T"))
    idle = set(range(B - case.get("idle", 0), B)) if B > case.get("idle", 0) else set()
    if case["op"] == "append":
        new = [rng.randint(1, case["S"]) if case["ragged"] else case["S"] for _ in range(B)]
        if case["ragged"]:
            new[0] = case["S"]
        lens = [0 if b in idle else rng.randint(new[b], ctx) for b in range(B)]
        return lens, new
    if case["op"] == "read":
        return [ctx if b == 0 else rng.randint(max(1, ctx // 2), ctx) for b in range(B)], None
    low = max(case["S"], ctx // 64)
    lens = [ctx if b == 0 or not case["ragged"] else rng.randint(low, ctx) for b in range(B)]
    return [0 if b in idle else n for b, n in enumerate(lens)], None


# ---------------------------------------------------------------- inputs

def _frequencies(rot, scaling):
    """Rotation frequencies in fp32 and the factor on cos and sin, base 10,000 (published formulas)."""
    base, factor, original = 10000.0, 16.0, 8192
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = base ** (-i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling != "yarn":
        return f.float(), 1.0
    edge = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), rot - 1)
    ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
    return (f / factor * ramp + f * (1 - ramp)).float(), 0.1 * math.log(factor) + 1.0


def _pages(case, lens, g):
    """A page table with the pages of each sequence's tokens in random order, -1 past them, and the number of pages."""
    page, B = case["page"], case["B"]
    ctx = case.get("ctx", case.get("T"))
    per = -(-ctx // page)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 1
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((B, per), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), total


def _fill(cache, pages, H, page, D, g):
    """A cache of `pages` pages holding random rows."""
    shape = (pages, H, page)
    if cache == "bf16":
        return {"data": torch.randn(shape + (D,), generator=g, device="cuda").to(torch.bfloat16), "scale": None}
    if cache == "e4m3":
        x = torch.randn(shape + (D,), generator=g, device="cuda")
        s = x.abs().amax(-1) / 448
        return {"data": (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), "scale": s}
    # codes as a normal distribution gives them: any byte, and scales around one
    data = torch.randint(0, 256, shape + (D // 2,), generator=g, device="cuda", dtype=torch.uint8)
    s = (0.2 + 0.4 * torch.rand(shape + (D // 16,), generator=g, device="cuda")).to(torch.float8_e4m3fn)
    return {"data": data, "scale": s.view(torch.uint8)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "rotary":
        N, H, D = case["N"], case["H"], case["D"]
        wide = torch.randn((N, H, D + case["pad"]), generator=g, device="cuda").to(getattr(torch, case["dtype"]))
        s["x"] = wide[..., :D]
        s["pos"] = torch.randint(0, case["far"], (N,), generator=g, device="cuda", dtype=torch.int32)
        f, s["m"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = f.cuda()
        return s
    lens, new = _lens(case)
    s["table"], pages = _pages(case, lens, g)
    s["len"] = torch.tensor(lens, dtype=torch.int32).cuda()
    if op == "read":
        s["c"] = _fill(case["cache"], pages, case["H"], case["page"], case["D"], g)
        return s
    if op == "append":
        H = case["H"]
        s["k_cache"] = _fill(case["cache"], pages, H, case["page"], case["Dk"], g)
        s["v_cache"] = _fill(case["cache"], pages, H, case["page"], case["Dv"], g) if case["Dv"] else None
        ends = [0]
        for n in new:
            ends.append(ends[-1] + n)
        if case["ragged"]:
            s["cu"] = torch.tensor(ends, dtype=torch.int32).cuda()
            lead = (ends[-1],)
        else:
            s["cu"] = None
            lead = (case["B"], case["S"])
        s["k"] = torch.randn(lead + (H, case["Dk"]), generator=g, device="cuda").to(torch.bfloat16)
        s["v"] = torch.randn(lead + (H, case["Dv"]), generator=g, device="cuda").to(torch.bfloat16) if case["Dv"] else None
        s["freq"] = _frequencies(case["rot"], "none")[0].cuda() if case["rot"] else None
        return s
    B, S, ctx = case["B"], case["S"], case["ctx"]
    s["k_cache"] = _fill("e2m1", pages, case["Hkv"], case["page"], case["Dk"], g)
    s["v_cache"] = _fill("e2m1", pages, case["Hkv"], case["page"], case["Dv"], g)
    s["q"] = torch.randn((B, S, case["HA"], case["Dk"]), generator=g, device="cuda").to(torch.bfloat16)
    s["idx"] = None
    if case["topk"]:
        # each query's selection, best first: visible keys in random order, -1 behind them
        score = torch.rand((B, S, ctx), generator=g, device="cuda")
        at = s["len"][:, None].long() - S + torch.arange(S, device="cuda")
        score.masked_fill_(torch.arange(ctx, device="cuda") > at[..., None], -1.0)
        best, idx = score.topk(case["topk"], dim=-1)
        s["idx"] = idx.to(torch.int32).masked_fill(best < 0, -1)
    return s


# ---------------------------------------------------------------- plain forms

def _rotated(x, cos, sin, off, inter, inverse):
    """x [..., H, D] with its pairs turned; cos and sin [..., 1, rot / 2]."""
    rot = 2 * cos.shape[-1]
    r = x[..., off:off + rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    sin = -sin if inverse else sin
    u, v = a * cos - b * sin, b * cos + a * sin
    t = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((x[..., :off], t, x[..., off + rot:]), -1)


def _angles(pos, freq):
    t = pos[..., None].double() * freq.double()
    return torch.cos(t)[..., None, :], torch.sin(t)[..., None, :]


def _codes(x, kind):
    """fp32 rows as the cache's bytes and scales (and, for e2m1, the codes unpacked)."""
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    if kind == "e4m3":
        m = x.abs().amax(-1)
        s = torch.where(m > 0, m / torch.full_like(m, 448), torch.ones_like(m))   # a true division
        return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s
    y = x.unflatten(-1, (-1, 16))
    m = y.abs().amax(-1)
    s8 = (m / torch.full_like(m, 6)).clamp(max=448).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    z = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y)).flatten(-2)
    a = z.abs()
    # nearest of the eight magnitudes, a tie to the even code
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5).int())
    c = c + 8 * (z < 0).int()
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), s8.view(torch.uint8)


def _rows(c, kind, page, off):
    """The cache rows at (page, off), [..., H, D] in fp32."""
    data = c["data"][page, :, off]
    if kind == "bf16":
        return data.float()
    if kind == "e4m3":
        return data.view(torch.float8_e4m3fn).float() * c["scale"][page, :, off][..., None]
    codes = torch.stack((data & 15, data >> 4), -1).flatten(-2).int()
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=data.device)
    s = c["scale"][page, :, off].view(torch.float8_e4m3fn).float()
    return (table[codes].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _places(table, pos, page):
    """(page, offset, whether there is one) of positions pos [B, n]."""
    per = table.shape[1]
    p = torch.gather(table, 1, (pos // page).clamp(0, per - 1).long()).long()
    ok = (pos >= 0) & (pos < per * page) & (p >= 0)
    return p.clamp(min=0), pos % page, ok


def _tokens(s):
    """Sequence and position of every new token."""
    case, n = s["case"], s["len"].long()
    if s["cu"] is None:
        S = case["S"]
        seq = torch.arange(case["B"], device=n.device).repeat_interleave(S)
        return seq, (n[:, None] - S + torch.arange(S, device=n.device)).flatten()
    cu = s["cu"].long()
    N = s["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(case["B"], device=n.device), cu.diff(), output_size=N)
    return seq, n[seq] - cu[seq + 1] + torch.arange(N, device=n.device)


def _plain_append(s):
    case = s["case"]
    kind = case["cache"]
    seq, pos = _tokens(s)
    page, off, ok = _places(s["table"][seq], pos[:, None], case["page"])
    keep = (ok[:, 0] & (s["len"][seq] > 0)).nonzero()[:, 0]
    page, off = page[keep, 0], off[keep, 0]
    for x, cache, freq in ((s["k"], s["k_cache"], s["freq"]), (s["v"], s["v_cache"], None)):
        if cache is None:
            continue
        r = x.reshape(-1, *x.shape[-2:])[keep].double()
        if freq is not None:
            r = _rotated(r, *_angles(pos[keep], freq), case["off"], case["inter"], False)
        data, scale = _codes(r.float(), kind)
        cache["data"][page, :, off] = data
        if scale is not None:
            cache["scale"][page, :, off] = scale


def _plain_read(c, kind, table, lens, T, page):
    pos = torch.arange(T, device=lens.device).expand(table.shape[0], T)
    p, off, ok = _places(table, pos, page)
    rows = _rows(c, kind, p, off)
    return torch.where((ok & (pos < lens[:, None]))[..., None, None], rows, 0.0).to(torch.bfloat16)


def _plain_attention(s):
    case = s["case"]
    B, S, HA, Hkv, Dk, Dv = (case[n] for n in ("B", "S", "HA", "Hkv", "Dk", "Dv"))
    G, n, dev = HA // Hkv, s["len"].long(), s["q"].device
    last = n[:, None] - S + torch.arange(S, device=dev)           # [B, S]: a query's own position
    if s["idx"] is not None:
        pos = s["idx"].long().reshape(B, -1)
    else:
        pos = torch.arange(case["ctx"], device=dev).expand(B, -1)
    page, off, ok = _places(s["table"], pos, case["page"])
    k, v = _rows(s["k_cache"], "e2m1", page, off), _rows(s["v_cache"], "e2m1", page, off)
    q = s["q"].float().reshape(B, S, Hkv, G, Dk)
    if s["idx"] is not None:                                      # a list of keys for each query
        k, v = k.reshape(B, S, -1, Hkv, Dk), v.reshape(B, S, -1, Hkv, Dv)
        see = ok.view(B, S, -1) & (pos.view(B, S, -1) <= last[..., None])
        logits = q @ k.permute(0, 1, 3, 4, 2)
        v = v.permute(0, 1, 3, 2, 4)
    else:                                                         # every key of the sequence
        see = ok[:, None] & (pos[:, None] <= last[..., None])
        logits = (q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, Dk) @ k.permute(0, 2, 3, 1))
        logits = logits.view(B, Hkv, S, G, -1).transpose(1, 2)    # [B, S, Hkv, G, L]
        v = v.permute(0, 2, 1, 3)[:, None]
    logits = (logits * Dk ** -0.5).masked_fill(~see[:, :, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    out = out.reshape(B, S, HA, Dv).to(torch.bfloat16)
    return (out, (top + torch.log(total)).reshape(B, S, HA)) if case["lse"] else out


# ---------------------------------------------------------------- one pass

def _values(c, kind):
    return (c["data"].view(torch.float8_e4m3fn), c["scale"]) if kind == "e4m3" else c["data"]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import lightning_indexer_top_02_b200 as L
    if op == "rotary":
        how = dict(rot_offset=case["off"], interleaved=case["inter"], inverse=case["inverse"])
        if own:
            return L.rotary(s["x"], s["pos"], s["freq"], scale=s["m"], **how)
        cos, sin = _angles(s["pos"], s["freq"])
        x = s["x"].float()
        return _rotated(x, (cos * s["m"]).float(), (sin * s["m"]).float(), case["off"], case["inter"],
                        case["inverse"]).to(s["x"].dtype)
    if op == "read":
        if own:
            return L.cache_read(L.Cache(case["cache"], s["c"]["data"], s["c"]["scale"]), s["table"], s["len"], case["T"])
        return _plain_read(s["c"], case["cache"], s["table"], s["len"], case["T"], case["page"])
    if op == "append":
        kind, kc, vc = case["cache"], s["k_cache"], s["v_cache"]
        if own:
            k = L.Cache(kind, kc["data"], kc["scale"])
            v = L.Cache(kind, vc["data"], vc["scale"]) if vc else None
            L.cache_append(s["k"], k, s["table"], s["len"], v=s["v"], cache_v=v, cu_tokens=s["cu"],
                           inv_freq=s["freq"], rot_offset=case["off"], interleaved=case["inter"])
        else:
            _plain_append(s)
        if kind != "e2m1":
            return [_values(c, kind) for c in (kc, vc) if c]
        # what is held in 4 bits comes back as the values it stands for
        if own:
            return [L.cache_read(c, s["table"], s["len"], case["ctx"]) for c in (k, v) if c]
        return [_plain_read(c, kind, s["table"], s["len"], case["ctx"], case["page"]) for c in (kc, vc) if c]
    if own:
        kc, vc = s["k_cache"], s["v_cache"]
        return L.cache_attention(s["q"], L.Cache("e2m1", kc["data"], kc["scale"]), L.Cache("e2m1", vc["data"], vc["scale"]),
                                 s["table"], s["len"], scale=case["Dk"] ** -0.5, idx=s["idx"], return_lse=case["lse"])
    return _plain_attention(s)


def _row_bytes(kind, D):
    return {"bf16": 2 * D, "e4m3": D + 4, "e2m1": D // 2 + D // 16}[kind]


def work(case):
    op = case["op"]
    if op == "rotary":
        e = {"bfloat16": 2, "float16": 2, "float32": 4}[case["dtype"]]
        return {"bytes": 2 * e * case["N"] * case["H"] * case["D"] + 4 * case["N"],
                "flops": 3 * case["N"] * case["H"] * case["rot"]}
    lens, new = _lens(case)
    if op == "read":
        rows = sum(lens) * case["H"]
        return {"bytes": rows * _row_bytes(case["cache"], case["D"]) + 2 * case["B"] * case["T"] * case["H"] * case["D"],
                "flops": rows * case["D"]}
    if op == "append":
        rows = sum(n for n, have in zip(new, lens) if have) * case["H"]
        D = case["Dk"] + case["Dv"]
        wide = _row_bytes(case["cache"], case["Dk"]) + (_row_bytes(case["cache"], case["Dv"]) if case["Dv"] else 0)
        moved = rows * (2 * D + wide)
        if case["cache"] == "e2m1":       # and the read back
            moved += sum(lens) * case["H"] * wide + 2 * case["B"] * case["ctx"] * case["H"] * D
        return {"bytes": moved, "flops": rows * (3 * case["rot"] + 2 * D)}
    S, HA, Hkv, Dk, Dv, topk = (case[n] for n in ("S", "HA", "Hkv", "Dk", "Dv", "topk"))
    wide = _row_bytes("e2m1", Dk) + _row_bytes("e2m1", Dv)
    seen = rows = 0
    for n in lens:
        per = [max(0, min(n - S + i + 1, topk or n)) for i in range(S)] if n else []
        seen += sum(per)
        rows += min(n, sum(per)) if topk else n
    moved = rows * Hkv * wide + 2 * case["B"] * S * HA * (Dk + Dv) + (4 * case["B"] * S * topk)
    moved += 4 * case["B"] * S * HA if case["lse"] else 0
    return {"bytes": moved, "flops": 2 * HA * (Dk + Dv) * seen}


# ---------------------------------------------------------------- 64 bits

def _turn64(x, pos, freq, m, off, inter, inverse):
    """Pairs as complex numbers times m * exp(+-i angle)."""
    rot = 2 * freq.numel()
    w = torch.polar(torch.full((pos.numel(), freq.numel()), float(m), dtype=torch.float64, device=x.device),
                    torch.outer(pos.double(), freq.double()) * (-1 if inverse else 1))[:, None]
    y = x.double().clone()
    part = y[..., off:off + rot]
    pairs = part.unflatten(-1, (rot // 2, 2)) if inter else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    y[..., off:off + rot] = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
    return y


def _nearest64(x, levels):
    """Index of the level nearest to |x|, a tie to the even index (levels ascend, len <= 8)."""
    best = torch.zeros_like(x, dtype=torch.int64)
    near = (x.abs() - levels[0]).abs()
    for i in range(1, len(levels)):
        d = (x.abs() - levels[i]).abs()
        better = (d < near) | ((d == near) & (i % 2 == 0))
        best, near = torch.where(better, i, best), torch.where(better, d, near)
    return best


def _stored64(r, kind):
    """What a cache row of that kind holds for r (fp32 values), as (values, scale or None) in 64 bits."""
    if kind == "bf16":
        return r.to(torch.bfloat16).double(), None
    if kind == "e4m3":
        peak = r.abs().max(-1).values
        s = torch.where(peak == 0, 1.0, (peak.double() / 448).float().double())
        return (r.double() / s[..., None]).float().to(torch.float8_e4m3fn).double(), s
    y = r.unflatten(-1, (-1, 16))
    s = (y.abs().max(-1).values.double() / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn).double()[..., None]
    z = (y.double() / s.masked_fill(s == 0, 1.0)).float().double() * (s != 0)
    mags = torch.tensor(E2M1, dtype=torch.float64, device=r.device)
    return (mags[_nearest64(z, E2M1)] * z.sign() * s).flatten(-2), None


def _held64(c, kind):
    """Every row of a cache in 64 bits, [pages, H, page, D]."""
    if kind == "bf16":
        return c["data"].double()
    if kind == "e4m3":
        return c["data"].view(torch.float8_e4m3fn).double() * c["scale"].double()[..., None]
    table = torch.tensor([m * s for s in (1, -1) for m in E2M1], dtype=torch.float64, device="cuda")
    codes = torch.empty(c["data"].shape[:-1] + (2 * c["data"].shape[-1],), dtype=torch.uint8, device="cuda")
    codes[..., 0::2], codes[..., 1::2] = c["data"] % 16, c["data"] // 16
    s = c["scale"].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return table[codes.long()] * s


def _sequence64(held, pages, n, page):
    """The first n rows of a sequence, [n, H, D]."""
    used = pages[:-(-n // page)].long()
    return held[used].transpose(1, 2).flatten(0, 1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _turn64(s["x"], s["pos"], s["freq"], s["m"], case["off"], case["inter"], case["inverse"])
    lens, new = _lens(case)
    page = case["page"]
    if op == "read":
        held = _held64(s["c"], case["cache"])
        out = torch.zeros((case["B"], case["T"], case["H"], case["D"]), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            out[b, :n] = _sequence64(held, s["table"][b], n, page)
        return out
    if op == "append":
        kind, table, got = case["cache"], s["table"].cpu(), []
        for x, c, freq in ((s["k"], s["k_cache"], s["freq"]), (s["v"], s["v_cache"], None)):
            if c is None:
                continue
            x = x.reshape(-1, *x.shape[-2:])
            held = _held64(c, kind) if kind != "e4m3" else c["data"].view(torch.float8_e4m3fn).double()
            scale = c["scale"].double() if kind == "e4m3" else None
            at = 0
            for b, (n, m) in enumerate(zip(lens, new)):
                rows = x[at:at + m].double()
                at += m
                if not n:
                    continue
                pos = torch.arange(n - m, n, device="cuda")
                if freq is not None:
                    rows = _turn64(rows, pos, freq, 1.0, case["off"], case["inter"], False)
                values, sc = _stored64(rows.float(), kind)
                place = table[b].cuda().long()[pos // page]
                held[place, :, pos % page] = values
                if scale is not None:
                    scale[place, :, pos % page] = sc
            if kind == "e2m1":
                back = torch.zeros((case["B"], case["ctx"], case["H"], held.shape[-1]), dtype=torch.float64, device="cuda")
                for b, n in enumerate(lens):
                    back[b, :n] = _sequence64(held, s["table"][b], n, page)
                got.append(back)
            else:
                got.append((held, scale) if kind == "e4m3" else held)
        return got
    B, S, HA, Hkv, Dk, Dv = (case[n] for n in ("B", "S", "HA", "Hkv", "Dk", "Dv"))
    out = torch.zeros((B, S, HA, Dv), dtype=torch.float64, device="cuda")
    lse = torch.full((B, S, HA), -math.inf, dtype=torch.float64, device="cuda")
    kh, vh = _held64(s["k_cache"], "e2m1"), _held64(s["v_cache"], "e2m1")
    for b, n in enumerate(lens):
        if not n:
            continue
        k, v = _sequence64(kh, s["table"][b], n, page), _sequence64(vh, s["table"][b], n, page)
        for i in range(S):
            see = n - S + i + 1
            if see <= 0:
                continue
            ki, vi = k[:see], v[:see]
            if s["idx"] is not None:
                pick = s["idx"][b, i]
                pick = pick[pick >= 0].long()
                if not pick.numel():
                    continue
                ki, vi = k[pick], v[pick]
            for h in range(Hkv):
                g = slice(h * (HA // Hkv), (h + 1) * (HA // Hkv))
                t = (s["q"][b, i, g].double() @ ki[:, h].T) / math.sqrt(Dk)
                lse[b, i, g] = torch.logsumexp(t, -1)
                out[b, i, g] = torch.softmax(t, -1) @ vi[:, h]
    return (out, lse) if case["lse"] else out

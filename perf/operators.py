"""The serving operators of an NVFP4 key/value cache, as they are measured.

A request's keys and values are held in 4 bits, in pages.  One step of a
serving program plans the pages of the step's tokens on the GPU, normalises
and rotates queries and keys per head, writes keys and values into the cache,
and attends over it:

  plan      block tables, slots and positions from request lengths
  rope      RMS norm of each query and key head and the position rotation
  rope_bwd  its gradient (a training step on the same projection)
  append    the same for a serving step's tokens, keys and values quantized
            into the cache, and the written tokens read back
  attn      attention of a step's queries over the cache

``run`` computes them in plain torch operations, or, where ``own`` is true,
with the package's calls.

The cache of one layer (P pages of S tokens, H key/value heads of D values):
  k_codes [P, H, S, D/2]       byte j of a token: values 2j (low nibble), 2j+1
  k_scales [P, H, S, D/16]     one E4M3 byte per 16 values of a token
  v_codes [P, H, S/8, D/2, 8]  the same bytes, 8 consecutive tokens side by side
  v_scales [P, H, S/8, D/16, 8]
  k_amax, v_amax [H]           calibrated largest magnitudes, one per head
and a value is E2M1 code x block scale x amax / (6 * 256).
"""
import math
import random

import torch

own = False

DEV = "cuda"
SG = 256.0  # the 4/6 rule's largest block scale
EPS = 1e-6
BASE = 10000.0
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the scheduler's step between two tokens of a small batch: latency
        dict(name="plan_decode_32", op="plan", batch=32, page=16, ctx=8192, new=1),
        # a large batch in which most requests bring a prompt
        dict(name="plan_prompts_1024", op="plan", batch=1024, page=16, ctx=2048, new=128),
        # single tokens of 8 requests: latency
        dict(name="rope_tokens_8", op="rope", tokens=8, hq=32, hk=8, d=128, rot=128, pairs="halves"),
        # the 8192 x 4096 activation as 32 heads of 128, a whole prompt
        dict(name="rope_prompt_8192", op="rope", tokens=8192, hq=32, hk=8, d=128, rot=128, pairs="halves"),
        # a training step's gradient at an odd length, small heads, neighbours rotated
        dict(name="rope_bwd_1023_d64", op="rope_bwd", tokens=1023, hq=12, hk=4, d=64, rot=64, pairs="neighbours"),
        # the training step of the 8192-token prompt, part of each head rotated
        dict(name="rope_bwd_8192", op="rope_bwd", tokens=8192, hq=32, hk=8, d=128, rot=64, pairs="halves"),
        # one decoded token of each of 64 requests, from the fused projection
        dict(name="append_decode_64", op="append", tokens=64, hq=32, hk=8, d=128, rot=128, pairs="halves",
             page=16, select="4over6"),
        # a prompt of 8192 tokens
        dict(name="append_prompt_8192", op="append", tokens=8192, hq=32, hk=8, d=128, rot=128, pairs="halves",
             page=64, select="4over6"),
        # one user, one token over 8191 tokens: latency
        dict(name="attn_token_1", op="attn", batch=1, ctx=8190, new=1, hq=32, hk=8, d=128, page=64, window=0,
             lens="equal"),
        # a decode step of 64 requests of many lengths
        dict(name="attn_decode_64", op="attn", batch=64, ctx=8192, new=1, hq=32, hk=8, d=128, page=16, window=0,
             lens="ragged"),
        # a few very long requests, each checking 4 drafted tokens, wide head groups
        dict(name="attn_draft4_long", op="attn", batch=3, ctx=131072, new=4, hq=64, hk=8, d=128, page=64, window=0,
             lens="ragged"),
        # chunks of prompts behind cached tokens
        dict(name="attn_chunk_2x2048", op="attn", batch=2, ctx=6000, new=2048, hq=32, hk=8, d=128, page=64, window=0,
             lens="ragged"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "append", "attn", "attn", "attn"])
    if op == "plan":
        new = _spread(rng, 1, 128)
        return dict(op=op, batch=_spread(rng, 1, 1024), page=rng.choice([8, 16, 32, 64]), ctx=_spread(rng, 1, 8192),
                    new=new)
    d = rng.choice([64, 128, 256])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 4, 7, 8])
    if op in ("rope", "rope_bwd"):
        return dict(op=op, tokens=_spread(rng, 1, 8192 * 40 * 128 // (64 * 72) // (d // 64)), hq=min(hq, 64), hk=hk, d=d,
                    rot=rng.choice([d, d // 2]), pairs=rng.choice(["halves", "neighbours"]))
    if op == "append":
        return dict(op=op, tokens=_spread(rng, 1, 8192 * 128 // (2 * d)), hq=min(hq, 32), hk=hk, d=d, rot=rng.choice([d, d // 2]),
                    pairs=rng.choice(["halves", "neighbours"]), page=rng.choice([8, 16, 32, 64]),
                    select=rng.choice(["6", "4over6"]))
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _spread(rng, 16, 1024)])
    batch = _spread(rng, 1, 64) if new <= 8 else rng.randint(1, 2)
    ctx = _spread(rng, 1, min(131072, 64 * 8192 * 128 // (batch * d) // 2))
    if new > 8:
        ctx = min(ctx, 4096 * 4096 // (hq * d))
    return dict(op=op, batch=batch, ctx=ctx, new=new, hq=hq, hk=hk, d=d, page=rng.choice([8, 16, 32, 64]),
                window=rng.choice([0, 0, 0, _spread(rng, 64, 4096)]), lens=rng.choice(["equal", "ragged"]))


def _lengths(c):
    """(cached, new) tokens of each request, from the case alone."""
    r = random.Random(c["batch"] * 1000003 + c["ctx"] * 7 + c["new"])
    ctx, new = [], []
    for b in range(c["batch"]):
        equal = c.get("lens") == "equal" or b == 0
        ctx.append(c["ctx"] if equal else r.randint(c["ctx"] // 8, c["ctx"]))
        # the planner's batches mix prompts and single tokens; a chunk is a chunk
        new.append(c["new"] if c["op"] == "attn" or c["new"] == 1 or r.random() < 0.7 else 1)
    return ctx, new


# ------------------------------------------------------------------ state
def _table(n, rot):
    """cos and sin of position x frequency, in 64 bits, held in 32."""
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * f
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _heads(g, t, h, d):
    """Projections: normal, with a few channels that carry outliers."""
    x = torch.randn(t, h, d, device=DEV, generator=g)
    x *= 1.0 + 4.0 * (torch.rand(1, h, d, device=DEV, generator=g) < 0.05)
    return x.bfloat16()


def _weight(g, d):
    return (1.0 + 0.2 * torch.randn(d, device=DEV, generator=g)).bfloat16()


def _empty_cache(c, pages):
    h, s, d = c["hk"], c["page"], c["d"]
    z = lambda *n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    return dict(k_codes=z(pages, h, s, d // 2), k_scales=z(pages, h, s, d // 16), v_codes=z(pages, h, s // 8, d // 2, 8),
                v_scales=z(pages, h, s // 8, d // 16, 8))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op in ("plan", "attn"):
        ctx, new = _lengths(case)
        page = case["page"]
        have = [-(-n // page) for n in ctx]
        need = [-(-(n + m) // page) for n, m in zip(ctx, new)]
        total = sum(need)
        pages = total + total // 16 + 8
        order = torch.randperm(pages, device=DEV, generator=g, dtype=torch.int32)
    if op == "plan":
        width = max(need) + 4
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
        n = torch.tensor(have, device=DEV)
        first = n.cumsum(0) - n
        col = torch.arange(width, device=DEV)
        used = col[None, :] < n[:, None]
        table[used] = order[(first[:, None] + col[None, :])[used]]
        free = sum(have)
        return dict(s, ctx_lens=torch.tensor(ctx, dtype=torch.int32, device=DEV),
                    new_lens=torch.tensor(new, dtype=torch.int32, device=DEV), block_table=table,
                    free_pages=torch.cat([order[free:], torch.zeros(free, dtype=torch.int32, device=DEV)]),
                    free_count=torch.tensor([pages - free], dtype=torch.int32, device=DEV), tokens=sum(new), pages=pages)
    if op == "attn":
        width = max(need) + 1
        n = torch.tensor(need, device=DEV)
        first = n.cumsum(0) - n
        col = torch.arange(width, device=DEV)
        used = col[None, :] < n[:, None]
        table = torch.zeros((case["batch"], width), dtype=torch.int32, device=DEV)
        table[used] = order[(first[:, None] + col[None, :])[used]]
        s.update(_empty_cache(case, pages), block_table=table)
        h, d = case["hk"], case["d"]
        s["k_amax"] = 16.0 + 8.0 * torch.rand(h, device=DEV, generator=g)
        s["v_amax"] = 5.0 + torch.rand(h, device=DEV, generator=g)
        chan = 1.0 + 3.0 * (torch.rand(1, h, 1, d, device=DEV, generator=g) < 0.05)
        step = max(1, (1 << 25) // (h * page * d))
        for p in range(0, pages, step):
            q = min(pages, p + step)
            shape = (q - p, h, page, d)
            x = (torch.randn(shape, device=DEV, generator=g) * chan).bfloat16()
            codes, scales = _nvfp4(x, s["k_amax"].view(1, h, 1, 1), "6")
            s["k_codes"][p:q], s["k_scales"][p:q] = codes, scales
            x = torch.randn(shape, device=DEV, generator=g).bfloat16()
            codes, scales = _nvfp4(x, s["v_amax"].view(1, h, 1, 1), "6")
            s["v_codes"][p:q] = codes.view(q - p, h, page // 8, 8, d // 2).transpose(3, 4)
            s["v_scales"][p:q] = scales.view(q - p, h, page // 8, 8, d // 16).transpose(3, 4)
        t = sum(new)
        s["q"] = (_heads(g, t, case["hq"], d).float() * 0.7).bfloat16()
        lens = [a + b for a, b in zip(ctx, new)]
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEV) if case["new"] > 1 else None
        s["max_len"], s["max_new"] = max(lens), max(new)
        return s
    t, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
    qkv = _heads(g, t, hq + 2 * hk, d)  # the fused projection: q, k and v are views of it
    s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:])
    s["q_weight"], s["k_weight"] = _weight(g, d), _weight(g, d)
    top = 32768
    s["cos"], s["sin"] = _table(top, case["rot"])
    if op == "append" and t <= 64:  # single tokens of many requests
        s["positions"] = torch.randint(0, top, (t,), device=DEV, generator=g, dtype=torch.int32)
    else:
        s["positions"] = torch.arange(t, device=DEV, dtype=torch.int32) + int(seed) % 1000
    if op == "rope_bwd":
        s["dq_out"], s["dk_out"] = _heads(g, t, hq, d), _heads(g, t, hk, d)
    if op == "append":
        pages = -(-t // case["page"]) + 8 if t > 64 else t + 8
        s.update(_empty_cache(case, pages))
        order = torch.randperm(pages, device=DEV, generator=g)
        i = torch.arange(t, device=DEV)
        if t <= 64:
            s["slots"] = order[i] * case["page"] + torch.randint(0, case["page"], (t,), device=DEV, generator=g)
        else:
            s["slots"] = order[i // case["page"]] * case["page"] + i % case["page"]
        s["k_amax"] = 8.0 + 12.0 * torch.rand(hk, device=DEV, generator=g)
        s["v_amax"] = 12.0 + 12.0 * torch.rand(hk, device=DEV, generator=g)
    return s


# ------------------------------------------------------------------ NVFP4 in plain operations
def _fma(a, b, c):
    """a * b + c rounded once to 32 bits (the product of two 32-bit values is exact in 64)."""
    return (a.double() * b.double() + c.double()).float()


def _e2m1(y):
    a = y.abs()
    i = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return i + 8 * torch.signbit(y).int()


def _values(codes):
    t = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    return t[codes]


def _nvfp4(x, amax, select):
    """Codes (two a byte) and E4M3 scale bytes of bf16 x[..., D] under the outer amax, in binary32 steps."""
    alpha = amax / (6.0 * SG)
    b = x.float().unflatten(-1, (-1, 16))
    top = b.abs().amax(-1)

    def encode(to):
        raw = (top * (1.0 / (to * alpha))).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale = raw.float() * alpha
        inv = torch.where(scale == 0, 0.0, 1.0 / scale)
        codes = _e2m1(b * inv[..., None])
        return raw.view(torch.uint8), codes, scale

    s6, c6, f6 = encode(6.0)
    if select == "4over6":
        s4, c4, f4 = encode(4.0)

        def error(codes, f):
            r = _fma(-_values(codes), f[..., None], b).unflatten(-1, (4, 4))
            p = r[..., 0] * r[..., 0]
            p = _fma(r[..., 1], r[..., 1], p)
            p = _fma(r[..., 2], r[..., 2], p)
            p = _fma(r[..., 3], r[..., 3], p)
            return (p[..., 0] + p[..., 1]) + (p[..., 2] + p[..., 3])

        four = error(c4, f4) < error(c6, f6)
        s6, c6 = torch.where(four, s4, s6), torch.where(four[..., None], c4, c6)
    c = c6.flatten(-2)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), s6


def _decode(codes, scales):
    """E2M1 x E4M3 in 32 bits, without the outer scale."""
    t = _values(torch.arange(256, device=codes.device)[:, None] // torch.tensor([1, 16], device=codes.device) % 16)
    v = t[codes.int()].flatten(-2)
    f = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * f[..., None]).flatten(-2)


# ------------------------------------------------------------------ plain forms
def _plan(s):
    page, table = s["case"]["page"], s["block_table"]
    ctx, new = s["ctx_lens"].long(), s["new_lens"].long()
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    more = torch.where(need <= table.shape[1], need - have, 0)
    last = more.cumsum(0)
    free = s["free_count"].long()
    ok = (need <= table.shape[1]) & ((more == 0) | (last <= free))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    col = torch.arange(table.shape[1], device=DEV)
    fresh = (col[None, :] >= have[:, None]) & (col[None, :] < need[:, None]) & ok[:, None]
    at = (free - 1 - (last - more)[:, None] - (col[None, :] - have[:, None])).clamp(0, len(s["free_pages"]) - 1)
    table.copy_(torch.where(fresh, s["free_pages"][at], table))
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = ctx[b] + t - cu[b]
    slots = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return dict(cu_new=cu.int(), seq_lens=torch.where(ok, ctx + new, ctx).int(), positions=pos.int(),
                slots=torch.where(ok[b], slots, -1), block_table=table,
                free_count=(free - torch.where(ok, more, 0).sum()).int())


def _pairs(x, rot, how):
    """The two members of each rotated pair, and the rest of the head."""
    if how == "halves":
        return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]


def _unpairs(a, b, rest, how):
    if how == "halves":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _angles(s):
    p = s["positions"].long()
    return s["cos"][p][:, None].double(), s["sin"][p][:, None].double()


def _rope_one(s, x, w):
    """In 64 bits: what the cache keeps of a key in 4 bits turns on values next to a border."""
    c = s["case"]
    x = x.double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
    cos, sin = _angles(s)
    a, b, rest = _pairs(x, c["rot"], c["pairs"])
    return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, c["pairs"]).bfloat16()


def _rope_bwd_one(s, dy, x, w):
    c = s["case"]
    cos, sin = (v.float() for v in _angles(s))
    a, b, rest = _pairs(dy.float(), c["rot"], c["pairs"])
    g = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, c["pairs"])
    x, w = x.float(), w.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (g * n).double().sum((0, 1)).float()  # a long sum
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx.bfloat16(), dw


def _append(s):
    c = s["case"]
    h, d, page = c["hk"], c["d"], c["page"]
    q_out, k = _rope_one(s, s["q"], s["q_weight"]), _rope_one(s, s["k"], s["k_weight"])
    slots = s["slots"]
    p, o = slots // page, slots % page
    got = []
    for x, name in ((k, "k"), (s["v"], "v")):
        amax = s[name + "_amax"].view(1, h, 1)
        codes, scales = _nvfp4(x, amax, c["select"])
        if name == "k":
            s["k_codes"][p, :, o], s["k_scales"][p, :, o] = codes, scales
            codes, scales = s["k_codes"][p, :, o], s["k_scales"][p, :, o]
        else:
            s["v_codes"][p, :, o // 8, :, o % 8], s["v_scales"][p, :, o // 8, :, o % 8] = codes, scales
            codes, scales = s["v_codes"][p, :, o // 8, :, o % 8], s["v_scales"][p, :, o // 8, :, o % 8]
        got.append((_decode(codes.contiguous(), scales.contiguous()) * (amax / (6.0 * SG))).bfloat16())
    return dict(q=q_out, k=got[0], v=got[1])


def _gathered(s):
    """Keys and values of each request, [B, H, L, D], without the outer scale."""
    c = s["case"]
    h, d, page = c["hk"], c["d"], c["page"]
    n = -(-s["max_len"] // page)
    t = s["block_table"][:, :n].long()
    b = len(t)
    k = _decode(s["k_codes"][t], s["k_scales"][t]).permute(0, 2, 1, 3, 4).reshape(b, h, n * page, d)
    codes = s["v_codes"][t].permute(0, 2, 1, 3, 5, 4).reshape(b, h, n * page, d // 2)
    scales = s["v_scales"][t].permute(0, 2, 1, 3, 5, 4).reshape(b, h, n * page, d // 16)
    return k, _decode(codes, scales)


def _attn(s):
    c = s["case"]
    b, h, hq, d, m = c["batch"], c["hk"], c["hq"], c["d"], s["max_new"]
    group = hq // h
    k, v = _gathered(s)
    cu = s["cu_q"].long() if s["cu_q"] is not None else torch.arange(b + 1, device=DEV)
    lens = s["seq_lens"].long()
    i = torch.arange(m, device=DEV)
    row = (cu[:-1, None] + i).clamp(max=len(s["q"]) - 1)
    real = i[None] < (cu[1:] - cu[:-1])[:, None]
    q = s["q"][row].float().view(b, m, h, group, d).permute(0, 2, 3, 1, 4).reshape(b, h, group * m, d)
    scale = (s["k_amax"] / (6.0 * SG) / math.sqrt(d)).view(1, h, 1, 1)
    t = torch.matmul(q, k.transpose(-1, -2).contiguous()) * scale
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    t = t.view(b, h, group, m, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h, group * m, -1), torch.where((j[None] < lens[:, None])[:, None, :, None], v, 0.0))
    o = o.view(b, h, group, m, d) / torch.where(total == 0, 1.0, total) * (s["v_amax"] / (6.0 * SG)).view(1, h, 1, 1, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)[real].bfloat16()


# ------------------------------------------------------------------ the pass
def _own(s):
    import nvfp4_block_scaled_02_amd as nv

    c = s["case"]
    op = c["op"]
    if op == "plan":
        p = nv.kv_plan(s["ctx_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_count"],
                       page_size=c["page"], num_pages=s["pages"], tokens=s["tokens"])
        return dict(cu_new=p.cu_new, seq_lens=p.seq_lens, positions=p.positions, slots=p.slots,
                    block_table=s["block_table"], free_count=p.free_count)
    if op == "rope":
        q, k = nv.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos"], s["sin"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=EPS, pairs=c["pairs"])
        return dict(q=q, k=k)
    if op == "rope_bwd":
        dq, dk, dqw, dkw = nv.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["positions"], s["cos"],
                                               s["sin"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                               pairs=c["pairs"])
        return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
    if "cache" not in s:  # the handle that a program keeps for a layer
        s["cache"] = nv.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["k_amax"], s["v_amax"],
                                global_max=SG)
    if op == "append":
        q = nv.kv_append(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"], cos=s["cos"],
                         sin=s["sin"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, pairs=c["pairs"],
                         select=c["select"])
        k, v = nv.kv_read(s["cache"], s["slots"])
        return dict(q=q, k=k, v=v)
    return nv.kv_attention(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["cu_q"], max_seq_len=s["max_len"],
                           window=c["window"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "plan":
        return _plan(state)
    if op == "rope":
        return dict(q=_rope_one(state, state["q"], state["q_weight"]), k=_rope_one(state, state["k"], state["k_weight"]))
    if op == "rope_bwd":
        dq, dqw = _rope_bwd_one(state, state["dq_out"], state["q"], state["q_weight"])
        dk, dkw = _rope_bwd_one(state, state["dk_out"], state["k"], state["k_weight"])
        return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
    return _append(state) if op == "append" else _attn(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        page, b, t = case["page"], case["batch"], sum(new)
        more = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(ctx, new))
        old = sum(n % page != 0 for n in ctx)  # the started pages of the requests
        return dict(bytes=b * 8 + 4 + old * 4 + more * 8 + (b + 1) * 4 + b * 4 + t * 12 + 4, flops=0)
    if op == "attn":
        ctx, new = _lengths(case)
        hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
        window = case["window"] or 1 << 40
        cells = sum(min(n + i + 1, window) for n, m in zip(ctx, new) for i in range(m))
        keys = sum(n + m - max(0, n - window + 1) for n, m in zip(ctx, new))
        t = sum(new)
        return dict(bytes=keys * hk * (d + d // 8) + t * hq * d * 4 + sum(-(-(n + m) // page) for n, m in zip(ctx, new)) * 4 + len(ctx) * 8,
                    flops=4 * cells * hq * d)
    t, hq, hk, d, rot = case["tokens"], case["hq"], case["hk"], case["d"], case["rot"]
    angles = t * (rot * 4 + 4)
    if op == "rope":
        return dict(bytes=t * (hq + hk) * d * 4 + angles + 4 * d, flops=t * (hq + hk) * d * 8)
    if op == "rope_bwd":
        return dict(bytes=t * (hq + hk) * d * 6 + angles + 12 * d, flops=t * (hq + hk) * d * 14)
    return dict(bytes=t * (hq * d * 4 + hk * d * 4 + 2 * hk * (d // 2 + d // 16) + 2 * hk * d * 2) + angles + t * 8 + 4 * d,
                flops=t * (hq + hk) * d * 8 + t * hk * d * 30)


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers alone
    s = prepare(case, seed)
    e4m3 = torch.tensor([(m / 512 if e == 0 else (8 + m) / 8 * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=DEV)
    grid = torch.tensor(GRID, dtype=torch.float64, device=DEV)

    def nearest(x, values):
        """Index of the nearest of ascending values, a tie to the even index."""
        hi = torch.searchsorted(values, x).clamp(1, len(values) - 1)
        lo = hi - 1
        a, b = x - values[lo], values[hi] - x
        return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)

    def norm_rotate(x, w):
        x = x.to(torch.float64)
        t, h, d = x.shape
        r = case["rot"]
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w.to(torch.float64)
        place = torch.arange(r // 2, device=DEV)
        one, two = (place, place + r // 2) if case["pairs"] == "halves" else (2 * place, 2 * place + 1)
        at = s["positions"].long()
        z = s["cos"].double()[at] + 1j * s["sin"].double()[at]
        turned = torch.complex(y[..., one], y[..., two]) * z[:, None]
        y[..., one], y[..., two] = turned.real, turned.imag
        return y

    if op == "rope":
        return dict(q=norm_rotate(s["q"], s["q_weight"]), k=norm_rotate(s["k"], s["k_weight"]))
    if op == "rope_bwd":
        got = {}
        for n in "qk":
            with torch.enable_grad():
                x = s[n].double().detach().requires_grad_()
                w = s[n + "_weight"].double().detach().requires_grad_()
                y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
                r = case["rot"]
                at = s["positions"].long()
                cos, sin = s["cos"].double()[at][:, None], s["sin"].double()[at][:, None]
                rows = y[..., :r].unflatten(-1, (2, r // 2) if case["pairs"] == "halves" else (r // 2, 2))
                axis = -2 if case["pairs"] == "halves" else -1
                a, b = rows.select(axis, 0), rows.select(axis, 1)
                y = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], axis).flatten(-2), y[..., r:]], -1)
                got["d" + n], got["d" + n + "_weight"] = torch.autograd.grad(y, (x, w), s["d" + n + "_out"].double())
        return got
    if op == "append":
        def stored(x, amax):
            alpha = amax.double().view(1, -1, 1, 1) / (6 * SG)
            b = x.double().unflatten(-1, (-1, 16))
            top = b.abs().amax(-1, keepdim=True)
            best = None
            for to in (6, 4) if case["select"] == "4over6" else (6,):
                f = e4m3[nearest(top / (to * alpha), e4m3)] * alpha
                y = torch.where(f == 0, 0, b / torch.where(f == 0, 1, f))
                v = grid[nearest(y.abs().clamp(max=6), grid)] * y.sign() * f
                err = (v - b).square().sum(-1, keepdim=True)
                best = (v, err) if best is None else (torch.where(err < best[1], v, best[0]), torch.minimum(err, best[1]))
            return best[0].flatten(-2)

        k = norm_rotate(s["k"], s["k_weight"]).bfloat16()  # a key travels in bf16
        return dict(q=norm_rotate(s["q"], s["q_weight"]), k=stored(k, s["k_amax"]), v=stored(s["v"], s["v_amax"]))
    # attention, request by request
    h, hq, d, page = case["hk"], case["hq"], case["d"], case["page"]
    ctx, new = _lengths(case)
    out, t0 = [], 0
    signed = torch.cat([grid, -grid])
    for b, (n, m) in enumerate(zip(ctx, new)):
        length = n + m
        j = torch.arange(length, device=DEV)
        pg, o = s["block_table"][b].long()[j // page], j % page
        parts = []
        for head in range(h):
            kc, ks = s["k_codes"][pg, head, o].long(), s["k_scales"][pg, head, o].long()
            vc, vs = s["v_codes"][pg, head, o // 8, :, o % 8].long(), s["v_scales"][pg, head, o // 8, :, o % 8].long()
            k = signed[torch.stack([kc & 15, kc >> 4], -1).flatten(-2)] * e4m3[ks].repeat_interleave(16, -1) * (s["k_amax"][head].double() / (6 * SG))
            v = signed[torch.stack([vc & 15, vc >> 4], -1).flatten(-2)] * e4m3[vs].repeat_interleave(16, -1) * (s["v_amax"][head].double() / (6 * SG))
            q = s["q"][t0:t0 + m, head * (hq // h):(head + 1) * (hq // h)].double()
            a = torch.matmul(q.reshape(-1, d), k.T.contiguous()).view(m, hq // h, length) / math.sqrt(d)
            at = n + torch.arange(m, device=DEV)[:, None, None]
            hidden = j > at
            if case["window"]:
                hidden = hidden | (j <= at - case["window"])
            w = torch.softmax(a.masked_fill(hidden, -math.inf), -1)
            parts.append(torch.matmul(w.view(-1, length), v).view(m, hq // h, d))
        out.append(torch.cat(parts, 1))
        t0 += m
    return torch.cat(out)

"""The operators on an INT8 paged KV cache: what is measured, in plain form and
through the library.

Three operators, which belong together as one layer's cache path:

  append     rotate the new keys (and queries) by their positions, quantize keys
             and values to int8 with one scale for each page and head, and write
             them into the pages of their sequences;
  gather     read a range of positions of each sequence back as bf16;
  attention  attention of the new tokens over the cache: single tokens, a few
             tokens (a draft being checked) and long chunks, causal, with an
             optional tanh cap, distance bias, sliding window and prefix.

A cache is k_cache, v_cache int8 [pages, kv heads, page size, head dim] with
k_scale, v_scale fp32 [pages, kv heads]. Sequence b owns the pages
page_table[b, 0], page_table[b, 1], ...; its kv_len[b] tokens include the new
ones, which are rows seq_start[b] .. seq_start[b + 1] of the packed inputs.

`own` selects the library's calls; otherwise `run` is elementary torch in fp32.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def _case(name, op, hq, hkv, d, page, batch, q, ctx, **more):
    c = {"name": name, "op": op, "hq": hq, "hkv": hkv, "d": d, "page": page, "batch": batch, "q": q, "ctx": ctx,
         "ragged": False, "lens": 1, "pad": 0, "rot": d, "interleaved": False, "softcap": 0.0, "window": 0,
         "alibi": False, "prefix": 0}
    c.update(more)
    return c


def listed():
    return [
        # One decode step of 32 sequences of a 7B-shaped layer (32 heads of 128): 32 new tokens into the cache,
        # and the pages that they touched read back.
        _case("append_step_32", "append", 32, 32, 128, 64, 32, 1, 2048, ragged=True, lens=3),
        # A prefill batch of five prompts of odd lengths, grouped heads, keys rotated on half of the head.
        _case("append_prompts_ragged", "append", 32, 8, 128, 16, 5, 1531, 700, ragged=True, lens=5, rot=64, pad=7),
        # One whole prompt of 8192 tokens into an empty cache.
        _case("append_prompt_8192", "append", 32, 8, 128, 64, 1, 8192, 0),
        # A few short sequences read back: a prefix handed to another program, 64-wide heads.
        _case("gather_short", "gather", 16, 4, 64, 16, 4, 0, 333, ragged=True, lens=7),
        # A long context read back whole.
        _case("gather_32768", "gather", 32, 8, 128, 64, 1, 0, 32768),
        # The smallest step, where latency counts: one user, one token, a short context.
        _case("decode_1x512", "attention", 32, 32, 128, 64, 1, 1, 512),
        # The serving step of the 7B-shaped layer: 32 sequences, 4096 wide, contexts of 4096.
        _case("decode_32x4096", "attention", 32, 32, 128, 64, 32, 1, 4096),
        # Many users with contexts from a few tokens to 32768, grouped heads.
        _case("decode_64_ragged_32768", "attention", 32, 8, 128, 64, 64, 1, 32768, ragged=True, lens=11),
        # A draft of up to 4 tokens checked at once, capped scores, a sliding window, 64-wide heads, small pages.
        _case("verify_16x4_window", "attention", 16, 4, 64, 16, 16, 4, 5000, ragged=True, lens=13, softcap=30.0,
              window=2048),
        # The prefill of one prompt of the 7B-shaped layer.
        _case("prefill_2048", "attention", 32, 32, 128, 64, 1, 2048, 0),
        # Chunks of prompts behind cached contexts, odd lengths, a distance bias, a shared prefix seen by all.
        _case("prefill_chunks_ragged", "attention", 24, 8, 96, 32, 6, 777, 3001, ragged=True, lens=17, alibi=True,
              prefix=257, pad=5),
        # The longest prompt in one call.
        _case("prefill_8192", "attention", 32, 8, 128, 64, 1, 8192, 0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "decode", "decode", "prefill", "prefill"])
    d = rng.choice([64, 96, 128])
    hkv, group = rng.choice([(32, 1), (8, 4), (4, 4), (8, 3), (2, 8), (1, 16), (5, 2)])
    page = rng.choice([16, 32, 64, 128])
    c = _case("", "attention", hkv * group, hkv, d, page, 1, 1, 0, ragged=rng.random() < 0.7, lens=rng.randrange(1 << 20),
              rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.3, pad=rng.choice([0, 0, 3]))
    del c["name"]
    if op == "gather":
        c.update(op="gather", batch=_spread(rng, 1, 16), q=0)
        c["ctx"] = _spread(rng, 100, 32768 // c["batch"])
    elif op == "append":
        c.update(op="append", batch=_spread(rng, 1, 64))
        c["q"] = rng.choice([1, _spread(rng, 1, 8192 // c["batch"])])
        c["ctx"] = _spread(rng, 1, 2048)
    elif op == "decode":
        c.update(batch=_spread(rng, 1, 64), q=rng.choice([1, 1, 2, 4]))
        c["ctx"] = _spread(rng, 16, min(32768, (1 << 22) // (c["batch"] * hkv)))
    else:
        c.update(batch=_spread(rng, 1, 8))
        c["q"] = _spread(rng, 64, 4096 // c["batch"])
        c["ctx"] = rng.choice([0, _spread(rng, 1, 4096)])
    if c["op"] == "attention":
        c.update(softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, _spread(rng, 32, 4096)]),
                 alibi=rng.random() < 0.25, prefix=rng.choice([0, 0, _spread(rng, 1, 1000)]))
    return c


def _lens(case):
    """(new tokens, cached context) of each sequence."""
    r = random.Random(case["lens"])
    q, ctx = case["q"], case["ctx"]
    if not case["ragged"]:
        return [q] * case["batch"], [ctx] * case["batch"]
    qs = [q] + [r.randint(1, q) if q > 0 else 0 for _ in range(case["batch"] - 1)]
    cs = [ctx] + [_spread(r, 1, ctx) if ctx > 0 else 0 for _ in range(case["batch"] - 1)]
    return qs, cs


# ------------------------------------------------------------------ inputs
def _codes(shape, g):
    """int8 codes of about normal values, made in pieces of 2^26 values."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    for piece in flat.split(1 << 26):
        piece.copy_((torch.randn(piece.numel(), device="cuda", generator=g) * 40.0).round_().clamp_(-127, 127))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qs, cs = _lens(case)
    kv = [a + b for a, b in zip(qs, cs)]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    total, width = sum(qs), max(1, max(-(-n // page) for n in kv))
    need = sum(-(-n // page) for n in kv)
    pages = need + 3
    order = torch.randperm(pages, device="cuda", generator=g).tolist()
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(kv):
        m = -(-n // page)
        table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    starts = torch.tensor([0] + qs).cumsum(0).to(torch.int32)

    def i32(v):
        return torch.as_tensor(v, dtype=torch.int32).cuda()

    s = {
        "case": case,
        "page_table": table.cuda(), "seq_start": starts.cuda(), "kv_len": i32(kv),
        "k_cache": _codes((pages, hkv, page, d), g), "v_cache": _codes((pages, hkv, page, d), g),
        "k_scale": torch.rand((pages, hkv), device="cuda", generator=g) * 0.02 + 0.015,
        "v_scale": torch.rand((pages, hkv), device="cuda", generator=g) * 0.02 + 0.015,
        "max_q": max(qs), "max_kv": max(kv), "width": width,
    }
    rows = total + case["pad"]
    if case["op"] == "append":
        # the rows of one fused projection, seen as queries, keys and values
        fused = torch.randn((rows, hq + 2 * hkv, d), device="cuda", generator=g)
        fused = (fused * torch.exp(0.5 * torch.randn((rows, 1, 1), device="cuda", generator=g))).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        s["q_out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda")
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # what is read back: each sequence from the page that its first new token lies in
        first = [(n - m) // page * page for n, m in zip(kv, qs)]
    elif case["op"] == "gather":
        first = [0] * case["batch"]
    else:
        s["q"] = torch.randn((rows, hq, d), device="cuda", generator=g).to(torch.bfloat16)
        s["out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda")
        s["slopes"] = None
        if case["alibi"]:
            s["slopes"] = torch.exp2(-8.0 * (torch.arange(hq, device="cuda") + 1) / hq)
        s["prefix"] = i32([case["prefix"]] * case["batch"]) if case["prefix"] else None
        return s
    read = [n - f for n, f in zip(kv, first)]
    s["first"] = i32(first)
    s["read_start"] = torch.tensor([0] + read).cumsum(0).to(torch.int32).cuda()
    s["k_back"] = torch.zeros((sum(read), hkv, d), dtype=torch.bfloat16, device="cuda")
    s["v_back"] = torch.zeros((sum(read), hkv, d), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def _handles(s):
    """The cache and batch descriptions that a program keeps between steps."""
    if "handles" not in s:
        from int8_gemm_token_b200 import w8a8 as W
        s["handles"] = (W, W.PagedKVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]),
                        W.KVBatch(s["page_table"], s["seq_start"], s["kv_len"], s["max_q"], s["max_kv"]))
    return s["handles"]


def run(s):
    op = s["case"]["op"]
    if own:
        W, cache, batch = _handles(s)
        if op == "attention":
            c = s["case"]
            W.w8a8_kv_attention(s["q"], cache, batch, softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                                prefix_len=s["prefix"], out=s["out"])
            return {"out": s["out"]}
        got = {}
        if op == "append":
            W.w8a8_kv_append(s["k"], s["v"], cache, batch, cos=s["cos"], sin=s["sin"], q=s["q"], q_out=s["q_out"],
                             interleaved=s["case"]["interleaved"])
            got = {"q": s["q_out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        W.w8a8_kv_gather(cache, s["page_table"], s["first"], s["read_start"], k_out=s["k_back"], v_out=s["v_back"])
        return {**got, "k": s["k_back"], "v": s["v_back"]}
    if op == "attention":
        return {"out": _attention(s)}
    got = {}
    if op == "append":
        got = {"q": _append(s), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return {**got, "k": _read(s, "k"), "v": _read(s, "v")}


def _tokens(starts, rows):
    """(sequence, index in it, whether it is a token at all) of each packed row."""
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(starts[1:].long(), t, right=True)
    real = b < starts.numel() - 1
    b = b.clamp(max=starts.numel() - 2)
    return b, t - starts[b], real


def _rotate(x, pos, cos, sin, rot, interleaved):
    """x fp32 [tokens, heads, d] with its first `rot` values turned by the position's angles."""
    c, s = cos[pos][:, None], sin[pos][:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def _append(s):
    case = s["case"]
    page = case["page"]
    b, i, real = _tokens(s["seq_start"], s["k"].shape[0])
    new = s["seq_start"][1:] - s["seq_start"][:-1]
    pos = torch.where(real, s["kv_len"][b] - new[b] + i, 0).long()
    slot = torch.where(real, s["page_table"][b, pos // page], s["k_cache"].shape[0]).long()  # a page of no one for the rest
    args = (s["cos"], s["sin"], case["rot"], case["interleaved"])
    for name, x in (("k", _rotate(s["k"].float(), pos, *args)), ("v", s["v"].float())):
        codes, scale = s[name + "_cache"], s[name + "_scale"]
        pages, hkv, _, d = codes.shape
        amax = torch.zeros((pages + 1, hkv), device="cuda")
        amax.scatter_reduce_(0, slot[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        touched = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
        touched[slot] = True
        # a page keeps its scale if a token before the new ones lies in it and its scale is the larger
        first = s["kv_len"] - new
        old = torch.zeros(pages + 1, device="cuda")
        held = s["page_table"].gather(1, (first // page).clamp(max=s["width"] - 1).long()[:, None])[:, 0].long()
        held = torch.where((first % page > 0) & (new > 0), held, pages)
        old[held] = 1.0
        was = scale * old[:pages, None]
        now = torch.where(touched[:pages, None], torch.maximum(was, amax[:pages] / 127.0), scale)
        shrink = torch.where((now > was) & (was > 0), was / now, 1.0)
        codes.copy_((codes.float() * shrink[..., None, None]).round().clamp(-127, 127))
        inverse = torch.where(now > 0, 1.0 / now, 0.0)
        q = (x * torch.cat([inverse, inverse[:1]])[slot][..., None]).round().clamp(-127, 127).to(torch.int8)
        at = ((slot.clamp(max=pages - 1)[:, None] * hkv + torch.arange(hkv, device="cuda")) * page + (pos % page)[:, None])
        kept = codes.view(-1, d)
        wide = torch.cat([kept, kept[:1]])  # one row more, for rows that are no tokens
        wide[torch.where(real[:, None], at, kept.shape[0]).reshape(-1)] = q.reshape(-1, d)
        kept.copy_(wide[:-1])
        scale.copy_(now)
    turned = _rotate(s["q"].float(), pos, *args).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(real[:, None, None], turned, s["q_out"]))
    return s["q_out"]


def _read(s, name):
    codes, scale = s[name + "_cache"], s[name + "_scale"]
    page = s["case"]["page"]
    b, i, _ = _tokens(s["read_start"], s["k_back"].shape[0])
    pos = (s["first"][b] + i).long()
    slot = s["page_table"][b, pos // page].long()
    return (codes[slot, :, pos % page].float() * scale[slot][..., None]).to(torch.bfloat16)


def _attention(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group, rows, top = hq // hkv, s["q"].shape[0], s["max_q"]
    new = s["seq_start"][1:] - s["seq_start"][:-1]
    # keys and values of each sequence side by side, as the values they stand for
    table = s["page_table"].clamp(min=0).long()
    dense = []
    for name in ("k", "v"):
        x = s[name + "_cache"][table].float() * s[name + "_scale"][table][..., None, None]  # [b, page, head, token, d]
        dense.append(x.transpose(1, 2).reshape(table.shape[0], hkv, -1, d))
    keys, values = dense
    span = keys.shape[2]
    row = (s["seq_start"][:-1, None] + torch.arange(top, device="cuda")).clamp(max=rows - 1)
    q = s["q"][row].float()  # [b, i, head, d]
    q = q.view(-1, top, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(-1, hkv, group * top, d)
    x = (q @ keys.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    if case["softcap"]:
        x = x.mul_(1.0 / case["softcap"]).tanh_().mul_(case["softcap"])
    x = x.view(-1, hkv, group, top, span)
    i = (s["kv_len"] - new)[:, None, None] + torch.arange(top, device="cuda")[:, None]  # positions of the queries
    j = torch.arange(span, device="cuda")
    if s["slopes"] is not None:
        x += s["slopes"].view(hkv, group, 1, 1) * (j - i)[:, None, None].float()
    seen = (j <= i) & (j < s["kv_len"][:, None, None])
    if case["window"]:
        seen &= i - j < case["window"]
    if s["prefix"] is not None:
        seen |= (j < s["prefix"][:, None, None]) & (j < s["kv_len"][:, None, None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    most = x.amax(-1, keepdim=True)
    x.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    weight = x.sum(-1, keepdim=True)
    y = x.view(-1, hkv, group * top, span) @ values
    y = (y.view(-1, hkv, group, top, d) / torch.where(weight > 0, weight, 1.0)).to(torch.bfloat16)
    b, i, real = _tokens(s["seq_start"], rows)
    y = y.permute(0, 3, 1, 2, 4).reshape(-1, top, hq, d)[b, i.clamp(max=top - 1)]
    s["out"].copy_(torch.where(real[:, None, None], y, s["out"]))
    return s["out"]


# ------------------------------------------------------------------ floors
def _pairs(case):
    """(query, key) pairs that the masks leave, and keys that some query sees, over all sequences."""
    pairs = keys = 0
    for m, c in zip(*_lens(case)):
        n = m + c
        prefix = min(case["prefix"], n)
        lowest = n
        for p in range(c, n):
            low = max(0, p + 1 - case["window"]) if case["window"] else 0
            lowest = min(lowest, low)
            pairs += (p + 1 - low) + max(0, prefix - (p + 1)) + max(0, min(prefix, low))
        keys += (n - lowest if m else 0) + min(prefix, lowest if m else 0)
    return pairs, keys


def work(case):
    qs, cs = _lens(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    tokens = sum(qs)
    if case["op"] == "attention":
        pairs, keys = _pairs(case)
        return {"bytes": 2 * keys * hkv * d + 2 * 4 * hkv * keys / page + 2 * 2 * tokens * hq * d, "flops": 4.0 * pairs * hq * d}
    n = b = 0
    if case["op"] == "append":
        n = tokens * d * (2 * hkv + hq)
        b = tokens * d * (2 * hkv * 3 + hq * 4) + 4 * tokens * case["rot"]
        read = sum(m + c - c // page * page for m, c in zip(qs, cs))
    else:
        read = sum(m + c for m, c in zip(qs, cs))
    return {"bytes": b + 2 * read * hkv * d * 3 + 2 * 4 * hkv * read / page, "flops": 6.0 * n + 2.0 * read * hkv * d}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    kv, starts = s["kv_len"].tolist(), s["seq_start"].tolist()
    table = s["page_table"].tolist()
    wide = {}  # name -> (codes, scales) in 64 bits, page by page as they are needed

    def of_page(name, p):
        if (name, p) not in wide:
            wide[name, p] = (s[name + "_cache"][p].double(), s[name + "_scale"][p].double())
        return wide[name, p]

    def whole(name, b, n):
        m = -(-n // page)
        if case["op"] == "append":
            return torch.cat([of_page(name, table[b][k])[0] * of_page(name, table[b][k])[1][:, None, None]
                              for k in range(m)], 1)[:, :n]
        at = torch.tensor(table[b][:m], device="cuda")
        x = s[name + "_cache"][at].double() * s[name + "_scale"][at].double()[:, :, None, None]
        return torch.cat(list(x), 1)[:, :n]  # [head, token, d]

    if case["op"] == "attention":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        group = case["hq"] // case["hkv"]
        for b, n in enumerate(kv):
            lo, hi = starts[b], starts[b + 1]
            if hi == lo:
                continue
            keys, values = whole("k", b, n), whole("v", b, n)
            at_q = torch.arange(n - (hi - lo), n, device="cuda")[:, None]
            at_k = torch.arange(n, device="cuda")[None]
            hidden = at_k > at_q
            if case["window"]:
                hidden |= at_q - at_k >= case["window"]
            if case["prefix"]:
                hidden &= at_k >= case["prefix"]
            for h in range(case["hq"]):
                z = s["q"][lo:hi, h].double() @ keys[h // group].T / math.sqrt(case["d"])
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                if case["alibi"]:
                    z = z - s["slopes"][h].double() * (at_q - at_k)
                z = z.masked_fill(hidden, -math.inf)
                out[lo:hi, h] = torch.softmax(z, -1) @ values[h // group]
        return {"out": out}

    got = {}
    if case["op"] == "append":
        rot = case["rot"]
        half = rot // 2
        turned = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double()}
        first = [kv[b] - (starts[b + 1] - starts[b]) for b in range(len(kv))]
        pos = torch.cat([torch.arange(f, n) for f, n in zip(first, kv)] + [torch.zeros(case["pad"], dtype=torch.int64)]).cuda()
        cos, sin = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]
        for name in ("q", "k"):
            x = turned[name].clone()
            pair = x[..., :rot].unflatten(-1, (half, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_complex(pair.contiguous()) * torch.complex(cos.expand(pair.shape[:-1]), sin.expand(pair.shape[:-1]))
            z = torch.view_as_real(z)
            x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            turned[name] = x
        for b, n in enumerate(kv):
            for k in range(first[b] // page, -(-n // page) if n > first[b] else 0):
                lo, hi = max(first[b], k * page), min(n, (k + 1) * page)
                for name in ("k", "v"):
                    codes, was = of_page(name, table[b][k])
                    if lo == k * page:
                        was = torch.zeros_like(was)
                    x = turned[name][starts[b] + lo - first[b]:starts[b] + hi - first[b]].transpose(0, 1)
                    now = torch.maximum(was, x.abs().amax((1, 2)) / 127.0)
                    codes = torch.round(codes * (was / now)[:, None, None])
                    codes[:, lo - k * page:hi - k * page] = torch.round(x / now[:, None, None])
                    wide[name, table[b][k]] = (codes, now)
        total = starts[-1]
        got["q"] = turned["q"]
        got["q"][total:] = 0.0
        for name in ("k", "v"):
            got[name + "_scale"] = s[name + "_scale"].double()
            for (kind, p), (_, now) in wide.items():
                if kind == name:
                    got[name + "_scale"][p] = now
    starts_back, from_pos = s["read_start"].tolist(), s["first"].tolist()
    for name in ("k", "v"):
        rows = []
        for b, f in enumerate(from_pos):
            n = f + starts_back[b + 1] - starts_back[b]
            if n > f:
                rows.append(whole(name, b, n)[:, f:].transpose(0, 1))
        got[name] = torch.cat(rows)
    return got

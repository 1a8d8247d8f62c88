"""Workloads of the full-attention half of a hybrid decoder and of the end of a
speculative step: the paged cache of keys and values (quantised as it is written
and read back), the attention of a chunk of new tokens over it (prompts, drafts
to verify, single tokens), and the verification of drafted tokens against the
target's probabilities.

Each operator has a plain form in elementary torch operations (fp32; quotients
next to a rounding's border and running sums of probabilities in fp64) and, with
``own`` true, the calls of this package that compute the same.  ``exact`` is the
operators' definition in fp64, written apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
VOCAB = 151936  # the width of the candidate selector's rows

# Heads of a full-attention layer: 32 on 8 of 128, 16 on 2 of 256 (beside a
# delta mixer of 16 query/key heads), and a small model's 8 on 8 of 64.
WIDE = dict(hq=32, hkv=8, d=128)
DEEP = dict(hq=16, hkv=2, d=256)
SMALL = dict(hq=8, hkv=8, d=64)


def listed():
    return [
        # One stream's decode step: latency.
        dict(name="attend_decode_1", op="attend", b=1, t=1, ctx=4099, mix=0, kv="bf16", page=64,
             window=0, **DEEP),
        # A serving batch's decode step, contexts of very different lengths.
        dict(name="attend_decode_32", op="attend", b=32, t=1, ctx=8192, mix=1, kv="int8", page=64,
             window=0, **WIDE),
        # A large batch: the cache's bytes decide.
        dict(name="attend_decode_128", op="attend", b=128, t=1, ctx=16384, mix=2, kv="bf16",
             page=64, window=0, **WIDE),
        # The block's verification batch: 8 sequences of 4 drafted tokens.
        dict(name="attend_verify_8x4", op="attend", b=8, t=4, ctx=8192, mix=3, kv="e4m3", page=32,
             window=0, **DEEP),
        # The block's prefill size, one prompt with nothing before it.
        dict(name="attend_prompt_2048", op="attend", b=1, t=2048, ctx=2048, mix=0, kv="bf16",
             page=64, window=0, **WIDE),
        # A late chunk of a long prompt over a quantised cache.
        dict(name="attend_chunk_4096", op="attend", b=1, t=4096, ctx=16384, mix=0, kv="int8",
             page=64, window=0, **WIDE),
        # Continuous batching: chunks of prompts and single tokens in one call.
        dict(name="attend_ragged_13", op="attend", b=13, t=0, n=6007, ctx=9000, mix=4, kv="bf16",
             page=16, window=0, **DEEP),
        # A serving batch's new tokens written (and read back): latency.
        dict(name="cache_decode_32", op="cache", b=32, t=1, ctx=8192, mix=1, kv="int8", page=64,
             **WIDE),
        # A long prompt's keys and values.
        dict(name="cache_prompt_8192", op="cache", b=1, t=8192, ctx=8192, mix=0, kv="e4m3",
             page=64, **WIDE),
        # Prompts of very different lengths behind contexts that end inside pages.
        dict(name="cache_ragged_13", op="cache", b=13, t=0, n=6007, ctx=9000, mix=4, kv="int8",
             page=16, **DEEP),
        # Drafts of 4 tokens for 8 sequences; of 7 tokens for a large batch.
        dict(name="draft_8x4", op="draft", b=8, t=4, vocab=VOCAB, one_hot=False),
        dict(name="draft_128x7", op="draft", b=128, t=7, vocab=VOCAB, one_hot=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "cache", "cache", "draft"])
    if op == "draft":
        t = rng.randint(1, 8)
        vocab = rng.choice([VOCAB, _log(rng, 1000, 200000)])
        return dict(op="draft", b=_log(rng, 1, 128 * 7 * VOCAB // (t * max(vocab, VOCAB))), t=t,
                    vocab=vocab, one_hot=rng.random() < 0.25)
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    hq = hkv * rng.choice([1, 2, 3, 4, 8] if hkv < 8 else [1, 2, 4])
    kind = dict(kv=rng.choice(["bf16", "int8", "e4m3"]), page=rng.choice([16, 32, 64, 128, 256]),
                hq=hq, hkv=hkv, d=d, mix=rng.randint(1, 1 << 20))
    if op == "cache":
        n = _log(rng, 1, 8192 * 8 * 128 // (hkv * d) if hkv * d > 1024 else 8192)
        b = rng.choice([1, _log(rng, 1, 64)])
        return dict(op="cache", b=b, t=0, n=max(n, b), ctx=_log(rng, 1, 9000), **kind)
    kind["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    if rng.random() < 0.5:  # decode and verification
        t = rng.choice([1, 1, 2, 3, 4, 5, 8])
        ctx = _log(rng, t, 16384)
        b = _log(rng, 1, max(1, min(256, 128 * 16384 * 8 * 128 // (ctx * max(hkv * d, 1024)))))
        return dict(op="attend", b=b, t=t, ctx=ctx, **kind)
    n = _log(rng, 2, 4096 if hq * d <= 4096 else 2048)
    b = rng.choice([1, 1, _log(rng, 1, 13)])
    return dict(op="attend", b=b, t=0, n=max(n, b), ctx=_log(rng, n, 12288), **kind)


def lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence: ``t`` new ones
    each, or ``n`` in all; ``ctx`` is the longest context's length."""
    b, t, ctx = case["b"], case["t"], case["ctx"]
    g = torch.Generator().manual_seed(case["mix"])
    if t:
        new = [t] * b
    else:
        n = case["n"]
        if b > 3:  # half of the sequences decode: a single token each
            new = [1] * b
            cuts = torch.rand((b + 1) // 2, generator=g) ** 2 + 1e-3
            share = (cuts / cuts.sum() * (n - b)).long().tolist()
            for i, s in enumerate(share):
                new[2 * i if 2 * i < b else b - 1] += s
            new[0] += n - sum(new)
        else:
            new = [n // b] * b
            new[0] += n - sum(new)
    if b == 1:
        return new, [max(ctx, new[0])]
    before = (torch.rand(b, generator=g) * max(1, ctx - max(new))).long().tolist()
    before[b // 2] = max(0, ctx - new[b // 2])
    return new, [x + y for x, y in zip(before, new)]


def seen(case):
    """Pairs of a query and a key that it sees, and keys that any query sees."""
    pairs = keys = 0
    w = case.get("window", 0)
    for n, length in zip(*lengths(case)):
        first = length - n
        if not w:
            pairs += n * first + n * (n + 1) // 2
            keys += length
        else:
            short = max(0, min(n, w - 1 - first))  # queries with fewer than w keys before them
            pairs += short * first + short * (short + 1) // 2 + (n - short) * w
            keys += length - max(0, first - w + 1)
    return pairs, keys


def work(case):
    if case["op"] == "draft":
        b, t, v = case["b"], case["t"], case["vocab"]
        rows = 1 if case["one_hot"] else 2
        # the drafted tokens' probabilities, and one row (of both) to sample from
        return {"bytes": b * (4 * v * rows + 4 * t * (rows + 2) + 4 * (t + 1) + 8),
                "flops": b * (3 * v + 2 * t)}
    size = 2 if case["kv"] == "bf16" else 1
    row = case["hkv"] * case["d"]
    per_key = 2 * (row * size + (0 if size == 2 else 4 * case["hkv"]))
    if case["op"] == "cache":
        n = sum(lengths(case)[0])
        return {"bytes": n * (2 * 2 * row * 2 + 2 * per_key), "flops": 2 * 4 * n * row}
    pairs, keys = seen(case)
    n = sum(lengths(case)[0])
    return {"bytes": keys * per_key + n * 2 * 2 * case["hq"] * case["d"],
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ------------------------------------------------------------------ inputs

LEAST = 2.0 ** -126  # the smallest scale


def _scales(x, kv):
    """The scale of each row of x: for int8 the largest value's share of 127, for
    e4m3 the power of two that brings the largest value into (224, 448]."""
    top = x.double().abs().amax(-1)
    if kv == "int8":
        return (top / 127).float().clamp_min(LEAST)
    m, e = torch.frexp(top / 448)  # top / 448 = m 2^e with 1/2 <= m < 1
    e = torch.where(m == 0.5, e - 1, e)
    power = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e, exactly
    power = power.float().clamp_min(LEAST)
    return torch.where(top > 0, power, torch.full_like(power, LEAST))


def _codes(x, scale, kv):
    y = x.double() / scale.double()[..., None]
    return y.round().to(torch.int8) if kv == "int8" else y.float().to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV) * std

    if case["op"] == "draft":
        return _prepare_draft(case, g, normal)
    kv, page, hq, hkv, d = (case[x] for x in ("kv", "page", "hq", "hkv", "d"))
    new, length = lengths(case)
    b, n = case["b"], sum(new)
    per = [-(-x // page) for x in length]
    pages = sum(per) + 7  # some belong to nobody
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((b, max(per)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += p
    s = dict(case=case, table=table, new=new, length=length,
             lens=torch.tensor(length, dtype=torch.int32, device=DEV), cu=None)
    if not case["t"]:
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(b + 1)], dtype=torch.int32, device=DEV)
    shape = (pages, hkv, page, d)
    if case["op"] == "cache":
        # k and v are slices of one projected row
        row = normal(n, 2 * hkv * d)
        row *= torch.exp(normal(2 * hkv * d, std=0.5))  # channels of different sizes
        s["k"], s["v"] = (x.unflatten(1, (hkv, d)) for x in row.bfloat16().split(hkv * d, 1))
        store = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[kv]
        parts = [torch.zeros(shape, dtype=store, device=DEV) for _ in range(2)]
        scales = [torch.zeros(shape[:3], device=DEV) if kv != "bf16" else None for _ in range(2)]
    else:
        parts, scales = [], []
        for std in (1.0, 0.7):
            x = normal(*shape, std=std)
            x += normal(hkv, 1, d, std=0.3)  # a mean of each channel's own
            x = x.bfloat16()
            scale = None if kv == "bf16" else _scales(x, kv)
            parts.append(x if kv == "bf16" else _codes(x, scale, kv))
            scales.append(scale)
        row = normal(n, (hq + 2 * hkv) * d, std=2.0).bfloat16()
        s["q"] = row[:, :hq * d].unflatten(1, (hq, d))
    s["cache"] = (parts[0], parts[1], scales[0], scales[1])
    if own:
        import sparse_moe_decode_gb300 as moe
        s["attn"] = moe.PagedAttention(hq, hkv, d, page_size=page, kv_type=kv,
                                       window=case.get("window", 0), device=DEV)
        s["cache"] = moe.KVCache(*s["cache"])
    return s


def _prepare_draft(case, g, normal):
    b, t, v = case["b"], case["t"], case["vocab"]
    logits = normal(b, t + 1, v, std=3.0)
    target = torch.softmax(logits, -1)
    s = dict(case=case, target=target, draft=None,
             uniform=torch.rand((b, t + 1), generator=g, device=DEV))
    # the drafter's logits are the target's with an error
    near = torch.softmax(logits[:, :t] + normal(b, t, v, std=0.7), -1)
    if not case["one_hot"]:
        s["draft"] = near
    at = torch.rand((b, t, 1), generator=g, device=DEV, dtype=torch.float64)
    cum = near.double().cumsum(-1)
    tokens = torch.searchsorted(cum, at * cum[..., -1:], right=True)[..., 0].clamp_max(v - 1)
    if case["one_hot"]:  # a drafter without probabilities: often its likeliest token
        likely = torch.rand((b, t), generator=g, device=DEV) < 0.7
        tokens = torch.where(likely, near.argmax(-1), tokens)
    s["tokens"] = tokens.int()
    if own:
        import sparse_moe_decode_gb300 as moe
        s["verifier"] = moe.DraftVerifier(device=DEV)
    return s


# --------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"attend": _plain_attend, "cache": _plain_cache, "draft": _plain_draft}[op](s)


def _run_own(s, op):
    if op == "draft":
        tokens, accepted = s["verifier"].verify(s["target"], s["tokens"], s["uniform"],
                                                draft=s["draft"])
        return {"tokens": tokens, "accepted": accepted}
    if op == "attend":
        return {"out": s["attn"].attend(s["cache"], s["q"], s["table"], s["lens"], s["cu"])}
    s["attn"].write(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cu"])
    k, v = s["attn"].read(s["cache"], s["table"], s["lens"], s["cu"], rows=s["k"].shape[0])
    out = {"k": k, "v": v}
    if s["cache"].k_scale is not None:
        out.update(k_scale=s["cache"].k_scale, v_scale=s["cache"].v_scale)
    return out


def _places(s):
    """Page and offset of each new token's position."""
    page = s["case"]["page"]
    new = torch.tensor(s["new"], device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=DEV), new,
                                  output_size=sum(s["new"]))
    start = new.cumsum(0) - new
    at = s["lens"].long()[seq] - new[seq] + torch.arange(seq.shape[0], device=DEV) - start[seq]
    return s["table"][seq, at // page].long(), at % page


def _plain_cache(s):
    kv = s["case"]["kv"]
    page, at = _places(s)
    out = {}
    for name, store, scales in (("k", s["cache"][0], s["cache"][2]),
                                ("v", s["cache"][1], s["cache"][3])):
        x = s[name]
        if kv == "bf16":
            store[page, :, at] = x
            out[name] = store[page, :, at]
            continue
        scale = _scales(x, kv)
        # (indexing does not take every 8-bit type)
        store.view(torch.uint8)[page, :, at] = _codes(x, scale, kv).view(torch.uint8)
        scales[page, :, at] = scale
        back = store.view(torch.uint8)[page, :, at].view(store.dtype)
        out[name] = (back.float() * scales[page, :, at][..., None]).bfloat16()
        out[name + "_scale"] = scales
    return out


def _rows(s, pages, length):
    """Keys and values [.., Hkv, length, d] in fp32 of the given pages [.., p]."""
    out = []
    for store, scale in zip(s["cache"][:2], s["cache"][2:]):
        x = store.view(torch.uint8 if store.element_size() == 1 else torch.int16)[pages]
        x = x.view(store.dtype).float()
        if scale is not None:
            x = x * scale[pages][..., None]
        x = x.transpose(-4, -3).flatten(-3, -2)  # [.., Hkv, p * page, d]
        out.append(x[..., :length, :])
    return out


def _softmax_values(q, k, v, first, window, scale):
    """q [.., Hkv, g, n, d] at positions first + i, k and v [.., Hkv, L, d]."""
    n, length = q.shape[-2], k.shape[-2]
    score = (q.flatten(-3, -2) @ k.transpose(-1, -2)).unflatten(-2, q.shape[-3:-1]) * scale
    at = first + torch.arange(n, device=DEV)[:, None]
    key = torch.arange(length, device=DEV)
    hidden = key > at
    if window:
        hidden = hidden | (key <= at - window)
    hidden = hidden if hidden.dim() == 2 else hidden[:, None, None]
    score = score.masked_fill_(hidden, -math.inf)
    score = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    return (score.flatten(-3, -2) @ v).unflatten(-2, q.shape[-3:-1]) / total


def _plain_attend(s):
    c = s["case"]
    hkv, g, d, b = c["hkv"], c["hq"] // c["hkv"], c["d"], c["b"]
    scale = d ** -0.5
    q = s["q"].float().unflatten(1, (hkv, g)).permute(1, 2, 0, 3)  # [Hkv, g, N, d]
    out = torch.empty_like(q)
    if c["t"] and c["t"] <= 8:  # all sequences at once, padded to the longest
        t, step = c["t"], 16
        table = s["table"].clamp_min(0).long()
        for i in range(0, b, step):
            part = q[:, :, i * t:(i + step) * t].unflatten(2, (-1, t)).permute(2, 0, 1, 3, 4)
            longest = max(s["length"][i:i + step])
            k, v = _rows(s, table[i:i + step, :-(-longest // c["page"])], longest)
            first = (s["lens"][i:i + step].long() - t)[:, None, None]
            o = _softmax_values(part, k, torch.nan_to_num(v), first, c["window"], scale)
            out[:, :, i * t:(i + step) * t] = o.permute(1, 2, 0, 3, 4).flatten(2, 3)
    else:
        at = 0
        for i, (n, length) in enumerate(zip(s["new"], s["length"])):
            pages = s["table"][i, :-(-length // c["page"])].long()
            k, v = _rows(s, pages, length)
            for j in range(0, n, 1024):
                m = min(1024, n - j)
                end = length - n + j + m  # the keys behind the piece's last token
                out[:, :, at + j:at + j + m] = _softmax_values(
                    q[:, :, at + j:at + j + m], k[:, :end], v[:, :end], length - n + j,
                    c["window"], scale)
            at += n
    return {"out": out.permute(2, 0, 1, 3).flatten(1, 2).bfloat16()}


def _plain_draft(s):
    target, tokens, draft = s["target"], s["tokens"].long(), s["draft"]
    b, t = tokens.shape
    p = target[:, :t].gather(2, tokens[..., None])[..., 0].double()
    q = torch.ones_like(p) if draft is None else draft.gather(2, tokens[..., None])[..., 0].double()
    taken = s["uniform"][:, :t].double() * q < p
    accepted = taken.long().cumprod(1).sum(1)
    seq = torch.arange(b, device=DEV)
    weight = target[seq, accepted].double()
    at = accepted.clamp_max(t - 1)
    if draft is None:
        less = torch.zeros_like(weight)
        less.scatter_(1, tokens[seq, at][:, None], 1.0)
    else:
        less = draft[seq, at].double()
    rest = torch.where((accepted < t)[:, None], (weight - less).clamp_min(0.0), weight)
    # nothing is left where the target never exceeds the draft: the target itself
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, weight)
    cum = rest.cumsum(1)
    aim = s["uniform"][:, t].double()[:, None] * cum[:, -1:]
    sample = (cum <= aim).sum(1).clamp_max(target.shape[2] - 1)
    place = torch.arange(t + 1, device=DEV)
    drafted = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], 1)
    result = torch.where(place < accepted[:, None], drafted, torch.full_like(drafted, -1))
    result = torch.where(place == accepted[:, None], sample[:, None], result)
    return {"tokens": result.int(), "accepted": accepted.int()}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in fp64, one sequence (and one head) after another."""
    s = prepare(case, seed)
    return {"attend": _exact_attend, "cache": _exact_cache, "draft": _exact_draft}[case["op"]](s)


def _value(code, scale):
    return code.to(torch.float64) if scale is None else code.to(torch.float64) * scale.double()[..., None]


def _exact_attend(s):
    c = s["case"]
    page, d, w = c["page"], c["d"], c["window"]
    group = c["hq"] // c["hkv"]
    k_all, v_all, ks, vs = tuple(s["cache"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    start = 0
    for i, (n, length) in enumerate(zip(s["new"], s["length"])):
        key = torch.arange(length, device=DEV)
        pg, off = s["table"][i].long()[torch.div(key, page, rounding_mode="floor")], key % page
        for h in range(c["hkv"]):
            def take(store, scale):
                raw = store.view(torch.int8 if store.element_size() == 1 else torch.int16)[pg, h, off]
                return _value(raw.view(store.dtype), None if scale is None else scale[pg, h, off])
            kd, vd = take(k_all, ks), take(v_all, vs)
            heads = slice(h * group, (h + 1) * group)
            for j in range(0, n, 2048):
                rows = torch.arange(j, min(n, j + 2048), device=DEV)
                qd = s["q"][start + rows][:, heads].to(torch.float64)
                a = torch.einsum("ngd,kd->ngk", qd, kd) / math.sqrt(d)
                pos = length - n + rows
                ok = key[None] <= pos[:, None]
                if w > 0:
                    ok &= key[None] > pos[:, None] - w
                a = torch.where(ok[:, None], a, -math.inf)
                a = torch.exp(a - a.max(-1, keepdim=True).values)
                o = torch.einsum("ngk,kd->ngd", a, vd)
                out[start + rows, heads] = o / a.sum(-1)[..., None]
        start += n
    return {"out": out}


def _power_above(x):
    """The least power of two >= x (a logarithm may be off by a rounding)."""
    near = torch.round(torch.log2(x)).long().clamp(-1000, 1000)
    powers = torch.tensor([2.0 ** i for i in range(-1001, 1002)], dtype=torch.float64, device=DEV)
    low, mid, high = (powers[near + 1001 + i] for i in (-1, 0, 1))
    return torch.where(low >= x, low, torch.where(mid >= x, mid, high))


def _exact_cache(s):
    c = s["case"]
    page, kv = c["page"], c["kv"]
    out = {}
    for name, store, scale in (("k", s["cache"][0], s["cache"][2]),
                               ("v", s["cache"][1], s["cache"][3])):
        x = s[name].to(torch.float64)
        if kv == "bf16":
            out[name] = x
            continue
        top = x.abs().max(-1).values
        if kv == "int8":
            unit = torch.where(top > 0, top / 127, LEAST).float().to(torch.float64).clamp(min=LEAST)
            code = torch.round(x / unit[..., None])
        else:
            # the least power of two that is not below top / 448
            unit = _power_above(torch.clamp(top, min=1e-300) / 448.0)
            unit = torch.clamp(unit, min=LEAST)
            y = x / unit[..., None]
            # steps of 1/8 of the value's power of two, none below 2^-9
            size = torch.clamp(y.abs(), min=2.0 ** -6)
            above = _power_above(size)
            ulp = torch.where(above > size, above / 16, above / 8)
            code = torch.round(y / ulp) * ulp
        out[name] = code * unit[..., None]
        full = scale.to(torch.float64)
        start = 0
        for i, (n, length) in enumerate(zip(s["new"], s["length"])):
            pos = torch.arange(length - n, length, device=DEV)
            pg = s["table"][i].long()[torch.div(pos, page, rounding_mode="floor")]
            full[pg, :, pos % page] = unit[start:start + n]
            start += n
        out[name + "_scale"] = full
    return out


def _exact_draft(s):
    b, t = s["tokens"].shape
    tokens = torch.full((b, t + 1), -1, dtype=torch.int32, device=DEV)
    accepted = torch.zeros(b, dtype=torch.int32, device=DEV)
    drafted, u = s["tokens"].tolist(), s["uniform"].double().tolist()
    for i in range(b):
        a = 0
        while a < t:
            d = drafted[i][a]
            p = s["target"][i, a, d].item()
            q = 1.0 if s["draft"] is None else s["draft"][i, a, d].item()
            if not u[i][a] * q < p:
                break
            tokens[i, a] = d
            a += 1
        w = s["target"][i, a].to(torch.float64)
        if a < t:
            if s["draft"] is None:
                r = w.clone()
                r[drafted[i][a]] = max(0.0, r[drafted[i][a]].item() - 1.0)
            else:
                r = torch.relu(w - s["draft"][i, a].to(torch.float64))
            if r.sum().item() > 0.0:
                w = r
        cum = torch.cumsum(w, 0)
        aim = torch.tensor([u[i][t]], dtype=torch.float64, device=DEV) * cum[-1]
        tokens[i, a] = min(int(torch.searchsorted(cum, aim, right=True).item()), w.numel() - 1)
        accepted[i] = a
    return {"tokens": tokens, "accepted": accepted}

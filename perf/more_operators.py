"""The operators that serve long and shared contexts from the 4-bit KV cache, as cases that
can be measured.

Four operators around the paged NVFP4 cache:

  prefix   causal attention of a batch whose groups of sequences share long prefixes
           (one system prompt, one document): each prefix attended once for its group
  keys     the mean key of every page that an append has filled, in 8-bit integers
  select   the pages each query attends: the first, its last ones, and those whose mean
           key scores highest (8-bit integer products, the best head of a group counts)
  pages    causal attention over the selected pages alone

`own = False` computes them in elementary torch operations; `own = True` calls the
package's kernels.  A case is a dict of plain values; `prepare` makes what a server has
in hand before the call, `run` is one call.
"""
import math
import random

import numpy as np
import torch

own = False

F32 = torch.float32
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # four requests on one short system prompt: latency
        dict(name="prefix: four requests", op="prefix", batch=4, groups=1, q_len=1, prefix=2048, own=200, ragged=True,
             q_heads=32, kv_heads=8, head_dim=128, page=64),
        # an ordinary decoding batch on one long system prompt
        dict(name="prefix: system prompt", op="prefix", batch=64, groups=1, q_len=1, prefix=8192, own=1500, ragged=True,
             q_heads=64, kv_heads=8, head_dim=128, page=64),
        # checking drafts of four for three groups of requests, prefixes that end inside a
        # page, small heads, an odd group of five
        dict(name="prefix: drafts in three groups", op="prefix", batch=23, groups=3, q_len=4, prefix=4001, own=700,
             ragged=True, q_heads=40, kv_heads=8, head_dim=64, page=16),
        # many samples drawn from one long document
        dict(name="prefix: long document", op="prefix", batch=32, groups=1, q_len=1, prefix=65536, own=512, ragged=False,
             q_heads=64, kv_heads=8, head_dim=128, page=64),
        # one decoding step: a few of the sequences have just filled a page
        dict(name="keys: decode step", op="keys", tokens=64, kv_heads=8, head_dim=128, page=64, whole=False),
        # a long prompt of odd length has entered the cache
        dict(name="keys: prompt", op="keys", tokens=131000, kv_heads=8, head_dim=128, page=64, whole=True),
        # one request far into its context: latency
        dict(name="select: one sequence", op="select", batch=1, q_len=1, ctx=131072, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=64, top=32, first=1, last=2),
        # an ordinary decoding batch of ragged contexts
        dict(name="select: batch", op="select", batch=64, q_len=1, ctx=32768, ragged=True, q_heads=64, kv_heads=8,
             head_dim=128, page=64, top=64, first=1, last=4),
        # a chunk of a long prompt, small heads, an odd group of six, short pages
        dict(name="select: chunk", op="select", batch=1, q_len=2000, ctx=40000, ragged=False, q_heads=24, kv_heads=4,
             head_dim=64, page=32, top=48, first=1, last=2),
        # one request, 32 pages of its context: latency
        dict(name="pages: one sequence", op="pages", batch=1, q_len=1, ctx=131072, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=64, top=32, first=1, last=2),
        # the batch that selected 64 pages each
        dict(name="pages: batch", op="pages", batch=64, q_len=1, ctx=32768, ragged=True, q_heads=64, kv_heads=8,
             head_dim=128, page=64, top=64, first=1, last=4),
        # a chunk of a long prompt against what each of its queries selected, short pages
        dict(name="pages: chunk", op="pages", batch=1, q_len=1000, ctx=40000, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=32, top=48, first=1, last=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prefix", "prefix", "keys", "select", "pages", "pages"))
    d = rng.choice((64, 128))
    kv = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "keys":
        whole = rng.random() < 0.6
        tokens = _log(rng, 2 * page, min(131000, 131000 * 8 * 128 // (kv * d))) if whole else _log(rng, 1, 256)
        return dict(op=op, tokens=tokens, kv_heads=kv, head_dim=d, page=page, whole=whole)
    heads = kv * rng.choice((1, 3, 4, 5, 7, 8))
    while True:
        if op == "prefix":
            batch = _log(rng, 2, 64)
            q_len = 1 if rng.random() < 0.6 else rng.randint(2, 9)
            c = dict(op=op, batch=batch, groups=rng.randint(1, min(batch, 4)), q_len=q_len, prefix=_log(rng, 100, 65536),
                     own=max(q_len, _log(rng, 1, 2048)), ragged=rng.random() < 0.7, q_heads=heads, kv_heads=kv,
                     head_dim=d, page=page)
            w = work(c)
            if w["bytes"] <= 1e8 and w["flops"] <= 6e10:
                return c
            continue
        q_len = 1 if rng.random() < 0.6 else _log(rng, 2, 2000 if op == "select" else 1000)
        first, last = rng.randint(0, 2), rng.randint(1, 4)
        c = dict(op=op, batch=_log(rng, 1, 64) if q_len == 1 else rng.randint(1, 4), q_len=q_len,
                 ctx=max(q_len, _log(rng, 64, 131072)), ragged=rng.random() < 0.6, q_heads=heads, kv_heads=kv,
                 head_dim=d, page=page, top=first + last + _log(rng, 2, 64), first=first, last=last)
        queries = c["batch"] * q_len
        if op == "select":
            few = work(c)["flops"] == 0                             # no more pages than are kept: now and then
            if (queries * heads * (c["ctx"] // page) <= 1 << 26 and c["batch"] * c["ctx"] // page * kv * d <= 1 << 26
                    and (not few or rng.random() < 0.1)):
                return c
        elif (c["batch"] * c["ctx"] * kv * d <= 1 << 28 and queries * kv * d * c["top"] * page <= 12 << 30
              and work(c)["flops"] <= 2.5e10):
            return c


def _shared(case):
    """The sequences of a prefix case, by the case alone (what a scheduler hands over): the
    groups' first sequences, each group's prefix, each sequence's own tokens and queries."""
    b, g = case["batch"], case["groups"]
    r = random.Random(b * 1000003 + case["prefix"] * 31 + case["own"])
    starts = [0] + sorted(r.sample(range(1, b), g - 1)) + [b]
    ragged = case["ragged"]
    prefix = [case["prefix"]] + [r.randint(max(1, case["prefix"] // 4), case["prefix"]) if ragged else case["prefix"]
                                 for _ in range(g - 1)]
    mine = [r.randint(max(1, case["own"] // 8), case["own"]) if ragged else case["own"] for _ in range(b)]
    nq = [min(r.randint(1, case["q_len"]) if ragged else case["q_len"], n) for n in mine]
    return starts, prefix, mine, nq


def _lens(case):
    """The cached length and the number of new queries of each sequence, likewise."""
    b, ctx, q = case["batch"], case["ctx"], case["q_len"]
    if not case["ragged"]:
        return [ctx] * b, [q] * b
    r = random.Random(b * 1000003 + ctx * 31 + q)
    lens = [ctx] + [r.randint(max(1, ctx // 8), ctx) for _ in range(b - 1)]
    nq = [min(q, n) if i == 0 else min(r.randint(max(1, q // 4), q), n) for i, n in enumerate(lens)]
    return lens, nq


def work(case):
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    row = d // 2 + d // 16
    if case["op"] == "keys":
        full = case["tokens"] // page if case["whole"] else -(-case["tokens"] // page)
        return {"bytes": case["tokens"] * 8 + full * hk * (page * row + d + 4), "flops": full * hk * page * d * 2}
    hq = case["q_heads"]
    if case["op"] == "prefix":
        starts, prefix, mine, nq = _shared(case)
        tokens = sum(prefix) + sum(mine)
        pairs = 0
        for g, p in enumerate(prefix):
            for b in range(starts[g], starts[g + 1]):
                pairs += nq[b] * (p + mine[b]) - nq[b] * (nq[b] - 1) // 2
        return {"bytes": tokens * hk * 2 * row + sum(nq) * hq * (4 * d + 4) + -(-tokens // page) * 4,
                "flops": 4 * d * hq * pairs}
    lens, nq = _lens(case)
    queries = sum(nq)
    pages = sum(-(-n // page) for n in lens)
    if case["op"] == "select":
        scored = 0
        for n, m in zip(lens, nq):
            at = np.arange(n - m, n, dtype=np.int64) // page
            cand = np.clip(at - case["last"] + 1 - case["first"], 0, None)
            scored += int(cand[at + 1 > case["top"]].sum())
        return {"bytes": min(pages, scored) * (hk * (d + 4) + 4) + queries * (2 * hq * d + 4 * hk * case["top"]),
                "flops": 2 * d * hq * scored}
    pairs = touched = 0
    for n, m in zip(lens, nq):
        at = np.arange(n - m, n, dtype=np.int64)
        listed_pages = np.minimum(at // page + 1, case["top"])
        pairs += int(((listed_pages - 1) * page + at % page + 1).sum())
        touched += min(-(-n // page), int(listed_pages.sum()))
    return {"bytes": touched * page * hk * 2 * row + queries * (hq * (4 * d + 4) + 4 * hk * case["top"]),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------- 4-bit values
def _encode(y, g):
    """NVFP4 of float32 rows [..., heads, d] with one scale g per head: E2M1 codes (two
    a byte, the even element low) and an E4M3 scale per 16 elements."""
    b = y.unflatten(-1, (-1, 16))
    g = g[:, None]
    sc = ((b.abs().amax(-1) * (1.0 / 6.0)) / g).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (sc.to(F32) * g)[..., None]
    q = torch.where(step > 0, b / step, torch.zeros_like(b))
    a = q.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
         + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
         + (a > 5.0).to(torch.uint8))
    c = torch.where((step > 0) & torch.signbit(q), c + 8, c).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), sc


def _decode(codes, scales):
    """float32 E2M1 * E4M3 values (exact) of packed codes [..., d/2] and scales [..., d/16]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=F32, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).to(F32)[..., None]).flatten(-2)


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 29)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _fill_cache(s, gen, pages):
    """K with a mean of its own per head and element and a few outlier channels, V plain."""
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    outlier = 1.0 + 2.0 * (torch.rand(d, generator=gen, device=DEV) < 0.03)
    mean = 0.5 * _randn(gen, hk, d)
    for kv, g in (("k", 12.0), ("v", 5.5)):
        s[kv + "_global"] = g * (1.0 + 0.2 * torch.rand(hk, generator=gen, device=DEV)) / 2688.0
        codes = torch.empty((pages, hk, page, d // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((pages, hk, page, d // 16), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // (hk * page * d))
        for p in range(0, pages, step):
            y = _randn(gen, min(step, pages - p), page, hk, d)
            y = y * outlier + mean if kv == "k" else y
            c, sc = _encode(y.bfloat16().to(F32), s[kv + "_global"])
            codes[p:p + step] = c.transpose(1, 2)
            scales[p:p + step] = sc.view(torch.uint8).transpose(1, 2)
        s[kv + "_codes"], s[kv + "_scales"] = codes, scales


def _sequences(s, gen, lens, nq):
    """Block table, lengths and query starts of sequences with pages of their own; the
    number of pages."""
    page = s["case"]["page"]
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=DEV)
    first = 0
    for b, n in enumerate(need):
        table[b, :n] = order[first:first + n]
        first += n
    s["block_table"], s["seq_lens"] = table, _i32(lens)
    s["q_starts"] = _i32([0] + [int(v) for v in np.cumsum(nq)])
    return sum(need)


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": case}
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "keys":
        t = case["tokens"]
        pages = -(-t // page) + 7 if case["whole"] else t + 7
        order = torch.randperm(pages, generator=gen, device=DEV)
        at = torch.arange(t, device=DEV)
        if case["whole"]:                                       # one sequence's pages, row after row
            s["slots"] = order[at // page] * page + at % page
        else:                                                   # one token of t sequences; one in `page` fills its page
            row = torch.randint(0, page - 1, (t,), generator=gen, device=DEV)
            row[::page] = page - 1
            s["slots"] = order[:t] * page + row
        _fill_cache(s, gen, pages)
        s["key_codes"] = torch.zeros((pages, hk, d), dtype=torch.int8, device=DEV)
        s["key_scales"] = torch.zeros((pages, hk), dtype=F32, device=DEV)
    elif case["op"] == "prefix":
        starts, prefix, mine, nq = _shared(case)
        lens, table, used = [], [], 0
        for g, p in enumerate(prefix):
            common = list(range(used, used + -(-p // page)))    # the first sequence's, its last one cut off
            used += len(common)
            for b in range(starts[g], starts[g + 1]):
                lens.append(p + mine[b])
                tail = -(-lens[b] // page) - p // page
                keep = len(common) if b == starts[g] else p // page
                fresh = tail - (keep - p // page)
                table.append(common[:keep] + list(range(used, used + fresh)))
                used += fresh
        order = torch.randperm(used, generator=gen, device=DEV).to(torch.int32)
        wide = max(len(t) for t in table)
        s["block_table"] = order[torch.tensor([t + [0] * (wide - len(t)) for t in table], device=DEV)]
        s["seq_lens"] = _i32(lens)
        s["q_starts"] = _i32([0] + [int(v) for v in np.cumsum(nq)])
        s["group_starts"] = _i32(starts)
        s["prefix_lens"] = _i32([prefix[g] for g in range(len(prefix)) for _ in range(starts[g], starts[g + 1])])
        s["max_q"], s["max_prefix"], s["max_own"] = max(nq), max(prefix), max(mine)
        s["q"] = (_randn(gen, sum(nq), case["q_heads"], d) * 1.2).bfloat16()
        _fill_cache(s, gen, used)
    else:
        lens, nq = _lens(case)
        pages = _sequences(s, gen, lens, nq)
        s["q"] = (_randn(gen, sum(nq), case["q_heads"], d) * 1.2).bfloat16()
        s["max_len"] = max(lens)
        if case["op"] == "select":
            mean = _randn(gen, hk, d)
            key = mean + 0.4 * _randn(gen, pages, hk, d)        # pages' mean keys around their head's
            amax = key.abs().amax(-1)
            s["key_codes"] = (key * (127.0 / amax)[..., None]).round().to(torch.int8)
            s["key_scales"] = amax / 127.0
        else:
            _fill_cache(s, gen, pages)
            lists = []
            for n, m in zip(lens, nq):                          # the first and last ones, and some between
                at = torch.arange(n - m, n, device=DEV) // page
                wide = max(case["top"], int(at[-1]) + 1)
                j = torch.arange(wide, device=DEV)
                score = torch.rand((m, hk, wide), generator=gen, device=DEV)
                at = at[:, None, None]
                score = torch.where((j < case["first"]) | (j > at - case["last"]), 2.0, score)
                score = torch.where(j > at, -1.0, score)
                best, idx = score.topk(case["top"], dim=-1)
                idx = torch.where(best < 0, wide, idx).sort(-1).values
                lists.append(torch.where(idx == wide, -1, idx).to(torch.int32))
            s["pages"] = torch.cat(lists)
    if own:
        s["call"] = _call(s)
    return s


def _call(s):
    """The prepared call that a server keeps: its outputs and workspace, allocated once."""
    import nvfp4_quantization_amd as mxq
    case = s["case"]
    op = case["op"]
    if op == "select":
        keys = mxq.PageKeys(s["key_codes"], s["key_scales"], case["page"])
        return mxq.SelectPagesNVFP4(s["q"], keys, s["block_table"], s["seq_lens"], s["q_starts"], top=case["top"],
                                    first=case["first"], last=case["last"], max_seq_len=s["max_len"])
    cache = mxq.NVFP4KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["k_global"], s["v_global"])
    if op == "keys":
        return mxq.PageKeysNVFP4(cache, s["slots"], mxq.PageKeys(s["key_codes"], s["key_scales"], case["page"]))
    if op == "prefix":
        return mxq.AttentionPrefixNVFP4(s["q"], cache, s["block_table"], s["seq_lens"], s["q_starts"],
                                        s["group_starts"], s["prefix_lens"], max_q_len=s["max_q"],
                                        max_prefix_len=s["max_prefix"], max_own_len=s["max_own"], lse=True)
    return mxq.AttentionPagesNVFP4(s["q"], cache, s["block_table"], s["seq_lens"], s["q_starts"], s["pages"], lse=True)


# ------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"prefix": _prefix, "keys": _keys, "select": _select, "pages": _pages}[op](s)
    r = s["call"]()
    if op == "keys":
        return {"codes": s["key_codes"], "scales": s["key_scales"]}
    if op == "select":
        return {"pages": r}
    return {"out": r.out, "lse": r.lse}


def _rows(s, kv, at, off):
    """float32 K or V rows of cached tokens: at, off (page and row) -> [..., kv_heads, d]."""
    codes, sc = s[kv + "_codes"][at, :, off], s[kv + "_scales"][at, :, off]
    return _decode(codes, sc) * s[kv + "_global"][:, None]


def _prefix(s):
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hk
    starts, prefix, mine, nq = _shared(case)
    first, own_lens = s["q_starts"].long(), (s["seq_lens"] - s["prefix_lens"]).long()
    table = s["block_table"].long()
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], dtype=F32, device=DEV)
    for g, p in enumerate(prefix):
        b0, b1 = starts[g], starts[g + 1]
        nb, most, wide = b1 - b0, max(nq[b0:b1]), max(mine[b0:b1])
        t = torch.arange(p, device=DEV)
        pk, pv = (_rows(s, kv, table[b0, t // page], t % page).transpose(0, 1).contiguous() for kv in "kv")
        # the group's queries, padded: [kv, batch * q * group, d]
        i = torch.arange(most, device=DEV)
        run = (first[b0 + 1:b1 + 1] - first[b0:b1])[:, None]
        token, live = (first[b0:b1, None] + i).clamp(max=s["q"].shape[0] - 1), i < run
        q = s["q"].to(F32)[token].unflatten(2, (hk, group)).permute(2, 0, 1, 3, 4).reshape(hk, nb * most * group, d)
        x0 = torch.matmul(q, pk.transpose(1, 2).contiguous()) * (1.0 / math.sqrt(d))
        # each sequence's own tokens: [batch, kv, own, d]
        t = p + torch.arange(wide, device=DEV)
        slot = (t // page).clamp(max=table.shape[1] - 1)
        ok, ov = (_rows(s, kv, table[b0:b1][:, slot], (t % page)[None]).transpose(1, 2).contiguous() for kv in "kv")
        qb = q.unflatten(1, (nb, most * group)).transpose(0, 1).contiguous()
        x1 = torch.matmul(qb, ok.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(d))
        lens = own_lens[b0:b1, None]
        pos = lens - run + i
        see = (torch.arange(wide, device=DEV) <= pos[..., None]) & (torch.arange(wide, device=DEV) < lens[..., None])
        x1 = x1.unflatten(2, (most, group)).masked_fill_(~see[:, None, :, None], -math.inf)
        x1 = x1.transpose(0, 1).reshape(hk, nb * most * group, wide)
        top = torch.maximum(x0.amax(-1, keepdim=True), x1.amax(-1, keepdim=True))
        p0, p1 = (x0 - top).exp_(), (x1 - top).exp_()
        total = p0.sum(-1, keepdim=True) + p1.sum(-1, keepdim=True)
        o = torch.matmul(p0, pv)
        o += torch.matmul(p1.unflatten(1, (nb, most * group)).transpose(0, 1).contiguous(), ov).transpose(0, 1).flatten(1, 2)
        o = (o / total).reshape(hk, nb, most, group, d).permute(1, 2, 0, 3, 4).flatten(2, 3)
        l = (top + total.log()).reshape(hk, nb, most, group).permute(1, 2, 0, 3).flatten(2, 3)
        out[token[live]] = o[live].bfloat16()
        lse[token[live]] = l[live]
    return {"out": out, "lse": lse}


def _keys(s):
    """Sums over a page are sums of whole multiples of 2^-10 times the head's scale: in 64
    bits they are exact, and the codes do not hang on their order."""
    page = s["case"]["page"]
    slots = s["slots"]
    p = slots[slots % page == page - 1] // page
    step = max(1, (1 << 27) // (s["k_codes"].shape[1] * page * s["case"]["head_dim"]))
    for i in range(0, len(p), step):
        at = p[i:i + step]
        total = (_decode(s["k_codes"][at], s["k_scales"][at]).double() * 1024.0).sum(2)        # [pages, kv, d]
        amax = total.abs().amax(-1)
        codes = torch.where(amax[..., None] > 0, total * 127.0 / amax[..., None], 0.0)
        s["key_codes"][at] = codes.round().to(torch.int8)
        s["key_scales"][at] = (amax * s["k_global"].double() * (1.0 / (127.0 * 1024.0 * page))).to(F32)
    return {"codes": s["key_codes"], "scales": s["key_scales"]}


def _select(s):
    """Whole-number products in 32 bits are exact here (128 * 127 * 127 is below 2^24)."""
    case = s["case"]
    hk, page, top = case["kv_heads"], case["page"], case["top"]
    starts, most = s["q_starts"].long(), max(_lens(case)[1])
    run = (starts[1:] - starts[:-1])[:, None]
    i = torch.arange(most, device=DEV)
    token, live = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1), i < run
    q = s["q"].to(F32)
    step = q.abs().amax(-1) * (1.0 / 127.0)
    codes = torch.where(step[..., None] > 0, q / step[..., None], 0.0).round().clamp(-127.0, 127.0)
    rows = codes[token].unflatten(2, (hk, -1)).permute(0, 2, 1, 3, 4)                          # [batch, kv, q, group, d]
    step = step[token].unflatten(2, (hk, -1)).permute(0, 2, 1, 3)
    table = s["block_table"].long()
    key = s["key_codes"][table].to(F32).permute(0, 2, 3, 1).contiguous()                       # [batch, kv, d, pages]
    dot = torch.matmul(rows.flatten(2, 3).contiguous(), key).unflatten(2, (most, -1))
    score = (dot * step[..., None]).amax(3) * s["key_scales"][table].transpose(1, 2)[:, :, None]
    at = ((s["seq_lens"].long()[:, None] - run + i) // page)[:, None, :, None]
    j = torch.arange(table.shape[1], device=DEV)
    score = torch.where((j < case["first"]) | (j > at - case["last"]), math.inf, score)
    score = torch.where(j > at, -math.inf, score)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]         # ties: the lowest first
    order = torch.where(order > at, len(j), order).sort(-1).values
    order = torch.where(order == len(j), -1, order)
    order = torch.nn.functional.pad(order, (0, top - order.shape[-1]), value=-1)
    return {"pages": order.permute(0, 2, 1, 3)[live].to(torch.int32)}


def _pages(s):
    case = s["case"]
    hk, d, page, top = case["kv_heads"], case["head_dim"], case["page"], case["top"]
    group = case["q_heads"] // hk
    i = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(s["q_starts"][1:].long(), i, right=True)
    pos = (s["seq_lens"][seq] - s["q_starts"][seq + 1]).long() + i
    whole = len(i) * top >= s["k_codes"].shape[0]               # most pages are listed: decode each once

    def decoded(kv, *at):
        codes, sc = s[kv + "_codes"], s[kv + "_scales"]
        y = _decode(codes[at], sc[at]) if at else _decode(codes, sc)
        return y * s[kv + "_global"].view((hk, 1, 1, 1) if at else (hk, 1, 1))

    head = torch.arange(hk, device=DEV)[:, None]
    k, v = (decoded(kv) if whole else None for kv in "kv")
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], dtype=F32, device=DEV)
    step = max(1, (1 << 28) // (hk * top * page * d))
    for i in range(0, len(pos), step):
        here = s["pages"][i:i + step].long()                                                   # [n, kv, top]
        n = len(here)
        at = s["block_table"].long()[seq[i:i + step, None, None], here.clamp(min=0)]
        kk, vv = (y[at, head] if whole else decoded(kv, at, head) for kv, y in (("k", k), ("v", v)))
        kk, vv = kk.flatten(2, 3), vv.flatten(2, 3)                                            # [n, kv, top * page, d]
        q = s["q"][i:i + step].to(F32).unflatten(1, (hk, group))
        x = torch.matmul(q, kk.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(d))
        t = (here[..., None] * page + torch.arange(page, device=DEV)).flatten(2)
        see = (t >= 0) & (t <= pos[i:i + step, None, None])
        x = x.masked_fill_(~see[:, :, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = (x - m).exp_()
        total = p.sum(-1, keepdim=True)
        out[i:i + step] = (torch.matmul(p, vv) / total).flatten(1, 2).bfloat16()
        lse[i:i + step] = (m + total.log())[..., 0].reshape(n, -1)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"prefix": _exact_prefix, "keys": _exact_keys, "select": _exact_select, "pages": _exact_pages}[case["op"]](s)


def _exact_rows(s, kv, h):
    """All cached rows of head h in 64 bits: [pages * page, d]."""
    value = torch.tensor(list(E2M1) + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    c = s[kv + "_codes"][:, h].flatten(0, 1).int()
    rows = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.float64, device=DEV)
    rows[:, 0::2], rows[:, 1::2] = value[c & 15], value[c >> 4]
    sc = s[kv + "_scales"][:, h].flatten(0, 1).view(torch.float8_e4m3fn).double()
    return rows * sc.repeat_interleave(16, 1) * s[kv + "_global"][h].double()


def _exact_prefix(s):
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    starts, lens, prefix = s["q_starts"].tolist(), s["seq_lens"].tolist(), s["prefix_lens"].tolist()
    firsts = s["group_starts"].tolist()
    for h in range(hk):
        k, v = _exact_rows(s, "k", h), _exact_rows(s, "v", h)
        for b, n in enumerate(lens):
            leader = max(f for f in firsts[:-1] if f <= b)
            t = torch.arange(n, device=DEV)
            row = torch.where(t < prefix[b], s["block_table"][leader, (t // page).clamp(max=s["block_table"].shape[1] - 1)],
                              s["block_table"][b, t // page]).long() * page + t % page
            lo, hi = starts[b], starts[b + 1]
            hidden = t[None] > torch.arange(n - (hi - lo), n, device=DEV)[:, None]
            q = s["q"][lo:hi, h * group:(h + 1) * group].double()                              # [queries, group, d]
            x = (q.flatten(0, 1) @ k[row].T.contiguous() / math.sqrt(d)).unflatten(0, (hi - lo, group))
            x = torch.where(hidden[:, None], -math.inf, x)
            lse[lo:hi, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
            out[lo:hi, h * group:(h + 1) * group] = (torch.softmax(x, -1).flatten(0, 1) @ v[row]).unflatten(0, (hi - lo, group))
    return {"out": out, "lse": lse}


def _exact_keys(s):
    """Codes by whole-number arithmetic (the nearest of S * 127 / a, the even one of two)."""
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    codes, scales = s["key_codes"].clone(), s["key_scales"].double()
    slots = s["slots"].cpu().numpy()
    at = torch.from_numpy(np.unique(slots[slots % page == page - 1] // page)).to(DEV)
    twice = torch.tensor([int(2 * v) for v in E2M1] + [-int(2 * v) for v in E2M1], device=DEV)
    for h in range(hk):
        c = s["k_codes"][at, h].int()
        whole = torch.empty((len(at), page, d), dtype=torch.int64, device=DEV)
        whole[..., 0::2], whole[..., 1::2] = twice[c & 15], twice[c >> 4]
        sc = (s["k_scales"][at, h].view(torch.float8_e4m3fn).double() * 512).long()
        total = (whole * sc.repeat_interleave(16, -1)).sum(1)
        amax = total.abs().max(1, keepdim=True).values
        one = amax.clamp(min=1)
        down = torch.div(254 * total + one, 2 * one, rounding_mode="floor")                    # floor(x + 1/2)
        tie = (254 * total + one) % (2 * one) == 0
        down = torch.where(tie & (down % 2 != 0), down - 1, down)
        codes[at, h] = down.to(torch.int8)
        scales[at, h] = amax[:, 0].double() * float(s["k_global"][h]) / 130048.0 / page
    return {"codes": codes, "scales": scales}


def _exact_select(s):
    """The stated steps in numpy: whole-number products, each score rounded as the operator
    rounds it (two products in 32 bits)."""
    case = s["case"]
    hk, page, top, first, last = case["kv_heads"], case["page"], case["top"], case["first"], case["last"]
    group = case["q_heads"] // hk
    q = s["q"].float().cpu().numpy()
    key, scale = s["key_codes"].cpu().numpy().astype(np.float64), s["key_scales"].cpu().numpy()
    table, lens, starts = (s[n].cpu().numpy() for n in ("block_table", "seq_lens", "q_starts"))
    out = np.full((len(q), hk, top), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(hk):
            rows = table[b, :-(-int(n) // page)]
            kk, ks = key[rows, h], scale[rows, h]
            for i in range(starts[b], starts[b + 1]):
                at = (int(n) - int(starts[b + 1]) + i) // page
                if at + 1 <= top:
                    out[i, h, :at + 1] = np.arange(at + 1)
                    continue
                rows = q[i, h * group:h * group + group]
                st = np.abs(rows).max(1, keepdims=True) * np.float32(1.0 / 127.0)
                c = np.clip(np.rint(np.divide(rows, st, out=np.zeros_like(rows), where=st > 0)), -127, 127)
                dot = c.astype(np.float64) @ kk[:at + 1].T
                best = (dot.astype(np.float32) * st).max(0) * ks[:at + 1]
                inner = np.arange(first, at - last + 1)
                kept = inner[np.lexsort((inner, -best[inner]))[:top - first - last]]
                out[i, h] = np.sort(np.concatenate([np.arange(first), kept, np.arange(at - last + 1, at + 1)]))
    return {"pages": torch.from_numpy(out).to(DEV)}


def _exact_pages(s):
    case = s["case"]
    hk, d, page, top = case["kv_heads"], case["head_dim"], case["page"], case["top"]
    group = case["q_heads"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    starts, lens = s["q_starts"].tolist(), s["seq_lens"].tolist()
    step = max(1, (1 << 26) // (top * page * d))
    for h in range(hk):
        k, v = _exact_rows(s, "k", h), _exact_rows(s, "v", h)
        for b, n in enumerate(lens):
            for lo in range(starts[b], starts[b + 1], step):
                hi = min(lo + step, starts[b + 1])
                here = s["pages"][lo:hi, h].long()
                t = (here[..., None] * page + torch.arange(page, device=DEV)).flatten(1)       # [queries, tokens]
                row = (s["block_table"][b][here.clamp(min=0)].long()[..., None] * page + torch.arange(page, device=DEV)).flatten(1)
                pos = torch.arange(n - starts[b + 1] + lo, n - starts[b + 1] + hi, device=DEV)[:, None]
                x = (s["q"][lo:hi, h * group:(h + 1) * group].double()[:, :, None] * k[row][:, None]).sum(-1) / math.sqrt(d)
                x = torch.where(((t < 0) | (t > pos))[:, None], -math.inf, x)
                lse[lo:hi, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
                w = torch.softmax(x, -1)
                out[lo:hi, h * group:(h + 1) * group] = torch.matmul(w, v[row])
    return {"out": out, "lse": lse}

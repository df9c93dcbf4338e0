"""The serving operators around a 4-bit KV cache, as cases that can be measured.

Three operators, one attention layer's worth of them in the order a server calls them:

  norm     residual addition + root-mean-square norm -> FP8 E4M3 with 1x128 scales
           (the quantized input of the QKV or the gate / up projection)
  append   rotary positions on Q and K, then K and V into a paged NVFP4 cache
  attend   causal attention of ragged queries over that cache (paged, grouped heads,
           optional sliding window with first tokens that stay visible)

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
        # one token of a decoding request, hidden size of the large MoE workload: latency
        dict(name="norm: one token", op="norm", rows=1, n=7168, residual=True, bf16=False),
        # a prefill chunk of the large MoE workload; the router wants the BF16 norm too
        dict(name="norm: prefill chunk", op="norm", rows=16384, n=7168, residual=True, bf16=True),
        # one decoding step of a full batch: 64 sequences far apart in their contexts, a
        # few of them padding, half of the 128-element head rotated in adjacent pairs
        dict(name="append: decode step", op="append", tokens=64, q_heads=64, kv_heads=8, head_dim=128, rot=64,
             interleaved=True, page=64, pages=2048, far=1000000, scaling="none", padded=3),
        # a long prompt of odd length entering the cache, whole head rotated in halves,
        # frequencies stretched for a long context
        dict(name="append: prompt", op="append", tokens=8191, q_heads=32, kv_heads=8, head_dim=128, rot=128,
             interleaved=False, page=64, pages=136, far=131072, scaling="ramp", padded=0),
        # one request, a short context: latency
        dict(name="attend: one sequence", op="attend", batch=1, q_len=1, ctx=1000, ragged=False, q_heads=32,
             kv_heads=8, head_dim=128, page=64, window=0, sinks=0),
        # an ordinary decoding batch of ragged contexts
        dict(name="attend: batch", op="attend", batch=64, q_len=1, ctx=8192, ragged=True, q_heads=64, kv_heads=8,
             head_dim=128, page=64, window=0, sinks=0),
        # two very long contexts: the split over the cache matters
        dict(name="attend: long context", op="attend", batch=2, q_len=1, ctx=262144, ragged=False, q_heads=64,
             kv_heads=8, head_dim=128, page=64, window=0, sinks=0),
        # streaming decode: the last 4096 tokens and the first 4
        dict(name="attend: window and sinks", op="attend", batch=32, q_len=1, ctx=16384, ragged=True, q_heads=64,
             kv_heads=8, head_dim=128, page=128, window=4096, sinks=4),
        # checking a draft of a few tokens, small heads, an odd group of five
        dict(name="attend: draft of five", op="attend", batch=16, q_len=5, ctx=4001, ragged=True, q_heads=40,
             kv_heads=8, head_dim=64, page=16, window=0, sinks=0),
        # prompts attended as a whole
        dict(name="attend: prompt", op="attend", batch=2, q_len=4096, ctx=4096, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=64, window=0, sinks=0),
        # one chunk of a long prompt against what is cached already
        dict(name="attend: chunk", op="attend", batch=1, q_len=512, ctx=65536, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=64, window=0, sinks=0),
        # ragged chunks with a window, small heads, short pages
        dict(name="attend: ragged chunks", op="attend", batch=5, q_len=777, ctx=9001, ragged=True, q_heads=24,
             kv_heads=4, head_dim=64, page=16, window=1024, sinks=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "append", "attend", "attend"))
    if op == "norm":
        n = 128 * _log(rng, 4, 64)
        return dict(op=op, rows=_log(rng, 1, min(16384, 16384 * 7168 // n)), n=n, residual=rng.random() < 0.75,
                    bf16=rng.random() < 0.4)
    d = rng.choice((64, 128))
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 3, 4, 5, 7, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        tokens = _log(rng, 1, min(8191, 8191 * 48 // (heads + 2 * kv)))
        return dict(op=op, tokens=tokens, q_heads=heads, kv_heads=kv, head_dim=d, rot=rng.choice((d // 4, d // 2, d)),
                    interleaved=rng.random() < 0.5, page=page, pages=-(-tokens // page) + rng.randint(1, 64),
                    far=_log(rng, 16, 1000000), scaling=rng.choice(("none", "linear", "ramp")),
                    padded=rng.randint(0, tokens // 8))
    while True:
        q_len = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        c = dict(op=op, batch=_log(rng, 1, 64), q_len=q_len, ctx=max(q_len, _log(rng, 16, 200000)),
                 ragged=rng.random() < 0.6, q_heads=heads, kv_heads=kv, head_dim=d, page=page, window=0, sinks=0)
        if rng.random() < 0.35:
            c["window"] = _log(rng, 16, 8192)
            c["sinks"] = rng.choice((0, 1, 4, 17, 64))
        cells = c["batch"] * c["ctx"]
        w = work(c)
        if cells * kv * d <= 1 << 28 and cells * heads * q_len <= 1 << 30 and w["bytes"] <= 4e8 and w["flops"] <= 2.5e11:
            return c


def _lens(case):
    """The cached length and the number of new queries of each sequence: by the case
    alone (what a scheduler hands over), ragged ones spread over an eighth to the whole."""
    b, ctx, q = case["batch"], case["ctx"], case["q_len"]
    if not case["ragged"]:
        return [ctx] * b, [q] * b
    r = random.Random(b * 1000003 + ctx * 31 + q)
    lens = [ctx] + [r.randint(max(1, ctx // 8), ctx) for _ in range(b - 1)]
    nq = [min(q, n) if i == 0 else min(r.randint(max(1, q // 4), q), n) for i, n in enumerate(lens)]
    return lens, nq


def _visible(length, nq, window, sinks):
    """(query, key) pairs of one sequence, and the cached tokens that any query sees."""
    pos = np.arange(length - nq, length, dtype=np.int64)
    if not window:
        return int((pos + 1).sum()), length
    near = np.minimum(pos + 1, window)
    far = np.clip(np.minimum(sinks, pos + 1 - window), 0, None)
    first = max(0, length - nq - window + 1)
    return int((near + far).sum()), length - first + min(sinks, first)


def work(case):
    if case["op"] == "norm":
        m, n = case["rows"], case["n"]
        per = n * (2 + (4 if case["residual"] else 0) + 1 + (2 if case["bf16"] else 0)) + n // 128 * 4
        return {"bytes": m * per + 2 * n, "flops": 8 * m * n}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    row = d // 2 + d // 16
    if case["op"] == "append":
        t = case["tokens"] - case["padded"]
        return {"bytes": case["tokens"] * (4 * hq * d + 12) + t * hk * 2 * (2 * d + row + 2 * d),
                "flops": case["tokens"] * 3 * case["rot"] * (hq + hk) + t * hk * 2 * d * 4}
    pairs = tokens = queries = 0
    for length, nq in zip(*_lens(case)):
        p, t = _visible(length, nq, case["window"], case["sinks"])
        pairs, tokens, queries = pairs + p, tokens + t, queries + nq
    return {"bytes": tokens * hk * 2 * row + queries * hq * (4 * d + 4) + -(-tokens // case["page"]) * 4,
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
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32)


def _inv_freq(rot, scaling):
    """Angle per position of each rotated pair, in 64 bits: base^(-2i/rot); "linear"
    divides by 4; "ramp" divides the slow pairs by 16, leaves the fast ones and ramps in
    between (by how often a pair turns over 8192 positions).  And the factor on cos and sin."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return (f / 4.0).to(DEV), 1.0
    if scaling == "ramp":
        keep = ((f * 8192 / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        return (f * keep + f / 16.0 * (1.0 - keep)).to(DEV), 0.1 * math.log(16.0) + 1.0
    return f.to(DEV), 1.0


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        m, n = case["rows"], case["n"]
        spread = 1.0 + 9.0 * (torch.rand(n, generator=gen, device=DEV) < 0.01)      # a few outlier channels
        s["x"] = (_randn(gen, m, n) * 0.5).bfloat16()
        s["residual"] = (_randn(gen, m, n) * spread).bfloat16() if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * _randn(gen, n)).bfloat16()
    elif case["op"] == "append":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        qkv = _randn(gen, t, (hq + 2 * hk) * d).bfloat16()                          # one projection's output
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        far = case["far"]
        start = torch.randint(0, max(1, far - t), (1,), generator=gen, device=DEV)
        s["positions"] = ((torch.arange(t, device=DEV) + start) if t > 1024 else
                          torch.randint(0, far, (t,), generator=gen, device=DEV)).to(torch.int32)
        pages, page = case["pages"], case["page"]
        order = torch.randperm(pages, generator=gen, device=DEV)
        at = torch.arange(t, device=DEV)
        if t <= 1024 and pages >= t:                                                # one token of t sequences
            slots = order[:t] * page + torch.randint(0, page, (t,), generator=gen, device=DEV)
        else:                                                                       # one sequence's pages
            slots = order[at // page] * page + at % page
        if case["padded"]:
            slots[torch.randperm(t, generator=gen, device=DEV)[:case["padded"]]] = -1
        s["slots"] = slots.to(torch.int64)
        s["inv_freq"], s["factor"] = _inv_freq(case["rot"], case["scaling"])
        s["k_global"] = (4.5 + torch.rand(hk, generator=gen, device=DEV)) / 2688.0
        s["v_global"] = (4.0 + torch.rand(hk, generator=gen, device=DEV)) / 2688.0
        for kv in "kv":
            s[kv + "_codes"] = torch.randint(0, 256, (pages, hk, page, d // 2), generator=gen, device=DEV, dtype=torch.uint8)
            s[kv + "_scales"] = torch.randint(0x30, 0x7F, (pages, hk, page, d // 16), generator=gen, device=DEV, dtype=torch.uint8)
    else:
        hq, hk, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
        lens, nq = _lens(case)
        need = [-(-n // page) for n in lens]
        s["q"] = (_randn(gen, sum(nq), hq, d) * 1.2).bfloat16()
        order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=DEV)
        first = 0
        for b, n in enumerate(need):
            table[b, :n] = order[first:first + n]
            first += n
        s["block_table"] = table
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q_starts"] = torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32, device=DEV)
        s["max_q"], s["max_len"] = max(nq), max(lens)
        outlier = 1.0 + 2.0 * (torch.rand(d, generator=gen, device=DEV) < 0.03)
        for kv, g in (("k", 12.0), ("v", 5.5)):
            s[kv + "_global"] = g * (1.0 + 0.2 * torch.rand(hk, generator=gen, device=DEV)) / 2688.0
            codes = torch.empty((sum(need), hk, page, d // 2), dtype=torch.uint8, device=DEV)
            scales = torch.empty((sum(need), hk, page, d // 16), dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 26) // (hk * page * d))
            for p in range(0, sum(need), step):
                y = _randn(gen, min(step, sum(need) - p), page, hk, d) * (outlier if kv == "k" else 1.0)
                c, sc = _encode(y.bfloat16().to(F32), s[kv + "_global"])
                codes[p:p + step] = c.transpose(1, 2)
                scales[p:p + step] = sc.view(torch.uint8).transpose(1, 2)
            s[kv + "_codes"], s[kv + "_scales"] = codes, scales
    if own:
        s["call"] = _call(s)
    return s


def _call(s):
    """The prepared call that a server keeps: its outputs and workspace, allocated once."""
    import nvfp4_quantization_amd as mxq
    case = s["case"]
    if case["op"] == "norm":
        return mxq.AddRMSNormFP8(s["x"], s["weight"], residual=s["residual"], eps=1e-6, out_bf16=case["bf16"])
    cache = mxq.NVFP4KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["k_global"], s["v_global"])
    if case["op"] == "append":
        rope = mxq.RopePlan(s["inv_freq"], interleaved=case["interleaved"], factor=s["factor"])
        return mxq.RopeAppendNVFP4(s["q"], s["k"], s["v"], s["positions"], s["slots"], rope, cache, values=True)
    return mxq.AttentionNVFP4(s["q"], cache, s["block_table"], s["seq_lens"], s["q_starts"], max_q_len=s["max_q"],
                              max_seq_len=s["max_len"], window=case["window"], sinks=case["sinks"], lse=True)


# ------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _norm, "append": _append, "attend": _attend}[op](s)
    r = s["call"]()
    if op == "norm":
        out = {"q": r.q.view(torch.float8_e4m3fn), "scales": r.scales}
        if r.residual is not None:
            out["residual"] = r.residual
        if r.y is not None:
            out["y"] = r.y
        return out
    if op == "append":
        return _cache_outputs(s, r.q, r.k_values, r.v_values)
    return {"out": r.out, "lse": r.lse}


def _cache_outputs(s, q, k_values, v_values):
    """Q, the values that the new rows stand for, and the whole cache: its codes are whole
    numbers that have to be equal, its scales E4M3 values."""
    return {"q": q, "k_values": k_values, "v_values": v_values, "k_codes": s["k_codes"], "v_codes": s["v_codes"],
            "k_scales": s["k_scales"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"].view(torch.float8_e4m3fn)}


def _norm(s):
    z = s["x"]
    if s["residual"] is not None:
        z = (z.to(F32) + s["residual"].to(F32)).bfloat16()
    f = z.to(F32)
    # the mean in 64 bits, so that codes next to a rounding border do not hang on its order
    r = (1.0 / torch.sqrt(f.double().square().mean(-1, keepdim=True) + 1e-6)).to(F32)
    y = (f * r) * s["weight"].to(F32)
    b = y.unflatten(-1, (-1, 128))
    sc = b.abs().amax(-1).clamp(min=1e-10) * (1.0 / 448.0)
    out = {"q": (b / sc[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).flatten(-2), "scales": sc}
    if s["residual"] is not None:
        out["residual"] = z
    if s["case"]["bf16"]:
        out["y"] = y.bfloat16()
    return out


def _rotate(x, c, sn, rot, interleaved):
    """Rotary positions on the first `rot` elements of each head, rounded to BF16."""
    x = x.to(F32)
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * c - b * sn, b * c + a * sn
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, rest), -1).bfloat16()


def _append(s):
    case = s["case"]
    rot, inter, page = case["rot"], case["interleaved"], case["page"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]          # 64 bits: far positions
    c = (torch.cos(angle) * s["factor"]).to(F32)[:, None]
    sn = (torch.sin(angle) * s["factor"]).to(F32)[:, None]
    q = _rotate(s["q"], c, sn, rot, inter)
    k = _rotate(s["k"], c, sn, rot, inter)
    kept = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][kept]
    at, off = slot // page, slot % page
    got = {}
    for kv, y in (("k", k), ("v", s["v"])):
        g = s[kv + "_global"]
        codes, sc = _encode(y.to(F32), g)
        s[kv + "_codes"][at, :, off] = codes[kept]
        s[kv + "_scales"][at, :, off] = sc.view(torch.uint8)[kept]
        got[kv] = (_decode(codes, sc) * g[:, None]).bfloat16()
    return _cache_outputs(s, q, got["k"], got["v"])


def _attend(s):
    case = s["case"]
    hk, d, page, w = case["kv_heads"], case["head_dim"], case["page"], case["window"]
    lens, starts = s["seq_lens"].long(), s["q_starts"].long()
    nq = starts[1:] - starts[:-1]
    length, most = s["max_len"], s["max_q"]
    t = torch.arange(length, device=DEV)
    at, off = s["block_table"].long()[:, t // page], t % page

    def rows(kv):                                                     # [batch, kv_heads, length, d]
        codes, sc = s[kv + "_codes"][at, :, off], s[kv + "_scales"][at, :, off]
        return (_decode(codes, sc) * s[kv + "_global"][:, None]).transpose(1, 2).contiguous()

    i = torch.arange(most, device=DEV)
    token = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    live = i < nq[:, None]
    q = s["q"].to(F32)[token].unflatten(2, (hk, -1)).permute(0, 2, 1, 3, 4)      # [batch, kv, q, group, d]
    group = q.shape[3]
    q = q.reshape(q.shape[0], hk, most * group, d).contiguous()
    x = torch.matmul(q, rows("k").transpose(2, 3).contiguous()) * (1.0 / math.sqrt(d))
    pos = (lens - nq)[:, None] + i
    see = (t <= pos[..., None]) & (t < lens[:, None, None]) & live[..., None]
    if w:
        see = see & ((t > pos[..., None] - w) | (t < case["sinks"]))
    x = x.unflatten(2, (most, group)).masked_fill_(~see[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), rows("v")).unflatten(2, (most, group))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[live]                  # [queries, heads, d]
    return {"out": o.bfloat16(), "lse": lse.permute(0, 2, 1, 3).flatten(2, 3)[live]}


# ------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_norm(s):
    m, n = s["x"].shape
    out = {"q": torch.empty((m, n), dtype=torch.float8_e4m3fn, device=DEV),
           "scales": torch.empty((m, n // 128), dtype=torch.float64, device=DEV)}
    z = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).bfloat16()
    if s["residual"] is not None:
        out["residual"] = z
    z = z.double()
    y = z * torch.rsqrt((z * z).sum(1, keepdim=True) / n + 1e-6) * s["weight"].double()
    for g in range(n // 128):
        part = y[:, 128 * g:128 * g + 128]
        sc = torch.clamp(part.abs().max(1).values, min=1e-10) / 448
        out["scales"][:, g] = sc
        out["q"][:, 128 * g:128 * g + 128] = (part / sc[:, None]).to(torch.float8_e4m3fn)
    if s["case"]["bf16"]:
        out["y"] = y
    return out


def _exact_append(s):
    """Q in 64 bits; what the cache then holds is whole codes, which have no value in
    between: their places are left empty, and so are the values they stand for."""
    case = s["case"]
    q = s["q"].double()
    half = case["rot"] // 2
    z = torch.polar(torch.full((len(q), half), float(s["factor"]), dtype=torch.float64, device=DEV),
                    torch.outer(s["positions"].double(), s["inv_freq"]))
    first = slice(0, case["rot"], 2) if case["interleaved"] else slice(0, half)
    second = slice(1, case["rot"], 2) if case["interleaved"] else slice(half, case["rot"])
    turned = torch.complex(q[..., first], q[..., second]) * z[:, None]
    q[..., first], q[..., second] = turned.real, turned.imag
    return {"q": q, "k_values": None, "v_values": None, "k_codes": None, "v_codes": None, "k_scales": None,
            "v_scales": None}


def _exact_attend(s):
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hk
    value = torch.tensor(list(E2M1) + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    starts, lens = s["q_starts"].tolist(), s["seq_lens"].tolist()
    for b, n in enumerate(lens):
        pages = s["block_table"][b, :-(-n // page)].long()
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(n - (hi - lo), n, device=DEV)[:, None]
        key = torch.arange(n, device=DEV)[None]
        hidden = key > pos
        if case["window"]:
            hidden = hidden | ((pos - key >= case["window"]) & (key >= case["sinks"]))
        for h in range(hk):
            side = {}
            for kv in "kv":
                c = s[kv + "_codes"][pages, h].reshape(-1, d // 2)[:n].int()
                rows = torch.empty((n, d), dtype=torch.float64, device=DEV)
                rows[:, 0::2], rows[:, 1::2] = value[c & 15], value[c >> 4]
                sc = s[kv + "_scales"][pages, h].reshape(-1, d // 16)[:n].view(torch.float8_e4m3fn).double()
                side[kv] = rows * sc.repeat_interleave(16, 1) * s[kv + "_global"][h].double()
            for j in range(h * group, h * group + group):
                x = s["q"][lo:hi, j].double() @ side["k"].T.contiguous() / math.sqrt(d)
                x[hidden] = -math.inf
                lse[lo:hi, j] = torch.logsumexp(x, 1)
                out[lo:hi, j] = torch.softmax(x, 1) @ side["v"]
    return {"out": out, "lse": lse}

"""Plain forms of the calls around long and shared contexts, for the tests: numpy on the
host, written from the operators' definitions (whole-number and FP32 steps where the result
is stated bit for bit, 64 bits elsewhere)."""
import numpy as np
import torch

import nvfp4_quantization_amd as mxq
from tests import serve_util as su

TWICE = (2 * su.E2M1).astype(np.int64)


class Sequences:
    """Ragged sequences over a cache of random pages, on the host, and their device arrays.
    lens, nq: cached tokens and queries of each; `before` and `behind`: rows of q that belong to
    no sequence; order: "heads" [page][head][row] or "rows" [page][row][head]."""

    def __init__(self, lens, nq, hq, hk, d, page, seed=0, spare=3, before=0, behind=0, order="heads"):
        rng = np.random.default_rng(seed)
        self.lens, self.nq, self.hq, self.hk, self.d, self.page, self.order = list(lens), list(nq), hq, hk, d, page, order
        self.starts = before + np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.total = int(self.starts[-1]) + behind
        need = [-(-max(n, 0) // page) for n in lens]
        self.pages = sum(need) + spare
        ids = rng.permutation(self.pages).astype(np.int32)
        self.table = rng.integers(0, max(self.pages, 1), (len(lens), max(need + [1]) + 2)).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        (self.kc, self.ks, self.kg), (self.vc, self.vs, self.vg) = su.random_cache(rng, self.pages, hk, page, d)
        self.q = su.to_bf16((rng.standard_normal((self.total, hq, d)) * 1.3).astype(np.float32))
        self.rng = rng

    def device_cache(self, dev):
        def put(x):
            t = torch.from_numpy(x).to(dev)
            return t.transpose(1, 2).contiguous().transpose(1, 2) if self.order == "rows" else t
        return mxq.NVFP4KVCache(put(self.kc), put(self.ks), put(self.vc), put(self.vs), torch.from_numpy(self.kg).to(dev),
                                torch.from_numpy(self.vg).to(dev))

    def device_q(self, dev):
        return torch.from_numpy(self.q).bfloat16().to(dev)

    def device_sequences(self, dev):
        return (torch.from_numpy(self.table).to(dev), torch.tensor(self.lens, dtype=torch.int32, device=dev),
                torch.from_numpy(self.starts).to(dev))

    def length(self, b):
        return min(max(self.lens[b], 0), self.table.shape[1] * self.page)

    def queries(self):
        """(row of q, sequence, position) of every query."""
        for b in range(len(self.lens)):
            for i in range(self.nq[b]):
                yield int(self.starts[b]) + i, b, max(self.length(b) - self.nq[b] + i, -1)


# ------------------------------------------------------------------ mean keys
def page_keys_reference(kc, ks, kg, slots, codes, scales):
    """codes and scales (copies) with the mean keys of the pages whose last row is in slots."""
    pages, hk, page = kc.shape[:3]
    codes, scales = codes.copy(), scales.copy()
    for s in slots:
        if s < 0 or s >= pages * page or s % page != page - 1:
            continue
        p = int(s) // page
        for h in range(hk):
            if np.any((ks[p, h] & 0x7F) == 0x7F):
                codes[p, h], scales[p, h] = 0, np.nan
                continue
            v = np.empty((page, 2 * kc.shape[3]), np.int64)
            v[:, 0::2], v[:, 1::2] = TWICE[kc[p, h] & 15], TWICE[kc[p, h] >> 4]
            total = (v * np.repeat((su.E4M3[ks[p, h]] * 512).astype(np.int64), 16, axis=-1)).sum(0)
            a = int(np.abs(total).max())
            for d, t in enumerate(total):                        # Python's whole numbers: exact
                two, rest = divmod(2 * 127 * int(t), 2 * a) if a else (0, 0)
                codes[p, h, d] = two + (rest > a or (rest == a and two % 2 == 1))
            with np.errstate(over="ignore"):
                scales[p, h] = np.float32((np.float64(a) * np.float64(kg[h])) * (1.0 / (130048.0 * page)))
    return codes, scales


# ------------------------------------------------------------------ selection
def scores_reference(q, codes, scales):
    """FP32 scores of pages (codes [n][d], scales [n]) for the query rows q [group][d]."""
    with np.errstate(all="ignore"):
        top = np.abs(q).max(-1)
        step = np.where(np.isfinite(top), top, np.float32(0)) * np.float32(1.0 / 127.0)
        c = np.zeros(q.shape, np.int64)
        for h in range(len(q)):
            if step[h] > 0:
                c[h] = np.clip(np.rint(q[h] / step[h]), -127, 127).astype(np.int64)
        dot = c @ codes.astype(np.int64).T
        best = (dot.astype(np.float32) * step[:, None]).max(0)
        return best * scales


def select_reference(c, codes, scales, top, first, last, out):
    """out (a copy) with the selected pages of every query."""
    out = out.copy()
    group = c.hq // c.hk
    for row, b, pos in c.queries():
        current = pos // c.page if pos >= 0 else -1
        for h in range(c.hk):
            if current < top:
                out[row, h] = np.where(np.arange(top) <= current, np.arange(top), -1)
                continue
            at = c.table[b, :current + 1].astype(np.int64)
            ok = (at >= 0) & (at < c.pages)
            at = np.where(ok, at, 0)
            s = scores_reference(c.q[row, h * group:(h + 1) * group], codes[at, h], scales[at, h])
            real = ok & ~np.isnan(s)
            inner = np.arange(first, current + 1 - last)
            # by score from the largest, those without one last; equal ones by place
            kept = inner[np.lexsort((inner, -np.where(real, s, 0.0)[inner], ~real[inner]))]
            kept = kept[:top - first - last]
            out[row, h] = np.sort(np.concatenate([np.arange(first), kept, np.arange(current + 1 - last, current + 1)]))
    return out


# ------------------------------------------------------------------ attention over token lists
def attend_tokens(q, k, v, scale):
    """64-bit attention of one row over rows k, v: out, lse, mean |v|, sum |v|, the largest
    score's size (attention_bounds' arguments)."""
    d = q.shape[0]
    if len(k) == 0:
        return np.zeros(d), -np.inf, np.zeros(d), np.zeros(d), 0.0
    with np.errstate(invalid="ignore"):
        x = (k @ q) * scale
        m = x.max()
        p = np.exp(x - m)
        return (p @ v / p.sum(), m + np.log(p.sum()), p @ np.abs(v) / p.sum(), np.abs(v).sum(0),
                (np.abs(k) @ np.abs(q)).max() * scale)


def attention_over(c, tokens_of, scale):
    """out, lse and their bounds of every row and head; tokens_of(row, b, pos, kv head) gives the
    physical rows (page, row) that it sees.  Rows of no sequence come back NaN.

    attention_bounds counts everything but the rounding of a cut row's parts.  A part's output is
    rounded to FP16, divided by V's tensor scale and times 16: half a step is 2^-11 of it, or 2^-25
    / 16 of the tensor scale below FP16's normal range.  The join weighs parts by shares that add
    up to one, so the row is off by at most 2^-11 of the weighted mean of |part|, which is at most
    mean |v| and what the part itself is off by (its error times 2^-11: the factor 1.05), and by 2^-29
    of the tensor scale; then by as much of the rounding to BF16."""
    d, group = c.d, c.hq // c.hk
    out, lse = np.full((c.total, c.hq, d), np.nan), np.full((c.total, c.hq), np.nan)
    mean_v, sum_v, big = np.zeros((c.total, c.hq, d)), np.zeros((c.total, c.hq, d)), np.zeros((c.total, c.hq))
    k = su.decode_rows(c.kc, c.ks) * c.kg.astype(np.float64)[None, :, None, None]
    v = su.decode_rows(c.vc, c.vs) * c.vg.astype(np.float64)[None, :, None, None]
    for row, b, pos in c.queries():
        for h in range(c.hk):
            at, off = tokens_of(row, b, pos, h)
            kk, vv = k[at, h, off], v[at, h, off]
            for j in range(h * group, (h + 1) * group):
                out[row, j], lse[row, j], mean_v[row, j], sum_v[row, j], big[row, j] = attend_tokens(
                    c.q[row, j].astype(np.float64), kk, vv, scale)
    o, l = su.attention_bounds(out, lse, mean_v, sum_v, big, d)
    vg = np.repeat(np.abs(c.vg.astype(np.float64)), group)[None, :, None]
    return out, lse, o + (1 + 2.0 ** -8) * (1.05 * 2.0 ** -11 * mean_v + 2.0 ** -29 * vg), l


def listed_tokens(c, pages):
    """tokens_of for lists pages [total][hk][top]."""
    def tokens_of(row, b, pos, h):
        at, off = [], []
        for j in pages[row, h]:
            if j < 0 or pos < 0 or j > pos // c.page:
                continue
            n = min(c.page, pos + 1 - int(j) * c.page)
            at.append(np.full(n, c.table[b, j]))
            off.append(np.arange(n))
        if not at:
            return np.zeros(0, np.int64), np.zeros(0, np.int64)
        return np.concatenate(at), np.concatenate(off)
    return tokens_of


def random_lists(c, top, seed=0, first=1, last=2):
    """A list per row and head: the first and last pages and some between, -1 at the end; rows of
    no sequence hold lists too."""
    rng = np.random.default_rng(seed)
    out = rng.integers(0, 5, (c.total, c.hk, top)).astype(np.int32)
    for row, b, pos in c.queries():
        n = pos // c.page + 1 if pos >= 0 else 0
        for h in range(c.hk):
            if n <= top:
                pick = np.arange(n)
            else:
                inner = rng.permutation(np.arange(first, n - last))[:top - first - last]
                pick = np.sort(np.concatenate([np.arange(first), inner, np.arange(n - last, n)]))
            out[row, h] = -1
            out[row, h, :len(pick)] = pick
    return out


def check_attention(got_out, got_lse, want, what=""):
    """Device results (float arrays) against attention_over's within its bounds."""
    out, lse, out_by, lse_by = want
    live = ~np.isnan(lse)
    assert live.any() or lse.size == 0
    assert np.isfinite(got_out[live]).all(), what
    worst = np.abs(got_out[live] - out[live]) / out_by[live]
    assert worst.size == 0 or worst.max() <= 1.0, f"{what}: out off by {worst.max():.3f} of its bound"
    if got_lse is not None:
        empty = live & np.isneginf(lse)
        assert np.isneginf(got_lse[empty]).all(), what
        some = live & ~np.isneginf(lse)
        worst = np.abs(got_lse[some] - lse[some]) / lse_by[some]
        assert worst.size == 0 or worst.max() <= 1.0, f"{what}: lse off by {worst.max():.3f} of its bound"

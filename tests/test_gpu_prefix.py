"""Attention with shared prefixes on the GPU against the plain form of tests/context_util.py,
within bounds counted from its roundings (context_util.attention_over)."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import context_util as cu
from tests import serve_util as su
from tests.gpu_util import announce, assert_same, device, host

pytestmark = pytest.mark.gpu


def prefix_tokens(c, starts, prefix):
    """tokens_of for groups: the first prefix[b] tokens through the group's first sequence."""
    def leader(b):
        return max(s for s in starts[:-1] if s <= b)

    def tokens_of(row, b, pos, h):
        t = np.arange(pos + 1)
        shared = t < min(max(prefix[b], 0), c.table.shape[1] * c.page)
        at = np.where(shared, c.table[leader(b), t // c.page], c.table[b, t // c.page])
        return at.astype(np.int64), t % c.page
    return tokens_of


class Case(cu.Sequences):
    """Sequences of groups; what a sequence's own row of the table says of shared pages (whole
    ones) is not a page at all."""

    def __init__(self, starts, prefix, lens, nq, *args, **kw):
        super().__init__(lens, nq, *args, **kw)
        self.group_starts, self.prefix = list(starts), list(prefix)
        for b in range(len(lens)):
            if b not in self.group_starts[:-1]:
                self.table[b, :max(self.prefix[b], 0) // self.page] = -9
        for g in range(len(starts) - 1):                                 # the first one's row holds every prefix
            need = -(-max(self.prefix[starts[g]:starts[g + 1]] + [0]) // self.page)
            have = -(-max(lens[starts[g]], 0) // self.page)
            if need > self.table.shape[1]:
                self.table = np.concatenate([self.table, self.rng.integers(0, self.pages, (len(lens), need)).astype(np.int32)], 1)
            self.table[starts[g], have:need] = self.rng.integers(0, self.pages, max(need - have, 0))

    def prepared(self, dev, **kw):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
        kw.setdefault("max_q_len", max(self.nq))
        return mxq.AttentionPrefixNVFP4(self.device_q(dev), self.device_cache(dev), *self.device_sequences(dev),
                                        i32(self.group_starts), i32(self.prefix), **kw)

    def want(self, scale=None):
        return cu.attention_over(self, prefix_tokens(self, self.group_starts, self.prefix), scale or 1 / math.sqrt(self.d))


def run(c, dev, want=None, **kw):
    out = torch.full((c.total, c.hq, c.d), 7.0, dtype=torch.bfloat16, device=dev)
    call = c.prepared(dev, lse=True, out=out, **kw)
    call.out.lse.fill_(7.0)
    call.workspace.fill_(0xFF)                                           # whatever it holds: NaN here
    r = call()
    torch.cuda.synchronize()
    got, lse = su.f32_of_bf16(r.out), host(r.lse)
    want = want or c.want(kw.get("scale"))
    cu.check_attention(got, lse, want)
    none = np.isnan(want[1])
    assert (got[none] == 7.0).all() and (lse[none] == 7.0).all()
    r = call()
    torch.cuda.synchronize()
    assert np.array_equal(su.f32_of_bf16(r.out), got)                    # and it repeats
    return got, lse


@pytest.mark.parametrize("starts,prefix,lens,nq,hq,hk,d,page", [
    ([0, 3], [500, 500, 500], [510, 700, 501], [1, 1, 1], 8, 2, 128, 64),
    ([0, 2, 5], [100, 100, 333, 333, 333], [101, 164, 350, 900, 334], [1, 1, 1, 1, 1], 4, 4, 64, 16),
    ([0, 4], [256, 256, 256, 256], [300, 260, 257, 400], [3, 4, 1, 2], 10, 2, 64, 32),      # drafts of a group of five
    ([0, 40], [1000] * 40, [1001 + 7 * i for i in range(40)], [1] * 40, 16, 1, 128, 64),    # 640 rows of a group
    ([0, 1, 2, 30], [90, 0] + [200] * 28, [95, 120] + [230] * 28, [2, 1] + [1] * 28, 12, 3, 128, 16),
    ([0, 3], [128, 128, 128], [300, 192, 333], [100, 64, 3], 4, 2, 64, 64),                 # chunks: many rows of a sequence
    ([0, 2], [500, 500], [640, 541], [40, 41], 24, 2, 128, 32),
    ([0, 2], [65, 65], [66, 70], [1, 5], 24, 1, 64, 128),                                   # 24 rows a head
    ([0, 1], [777], [1500], [1], 8, 1, 128, 64),                                            # nobody to share with
    ([0, 200], [64] * 200, [65 + i % 9 for i in range(200)], [1] * 200, 2, 2, 64, 16),
])
def test_prefix(starts, prefix, lens, nq, hq, hk, d, page):
    dev = device()
    announce(f"prefix starts={starts} prefix={prefix[:4]} lens={lens[:4]} nq={nq[:4]} hq={hq} hk={hk} d={d} page={page}")
    c = Case(starts, prefix, lens, nq, hq, hk, d, page, seed=sum(lens), before=1, behind=2, order="rows" if d == 64 else "heads")
    want = c.want()
    run(c, dev, want)                                                    # planned for what the table can hold
    run(c, dev, want, max_prefix_len=max(prefix), max_own_len=max(n - p for n, p in zip(lens, prefix)))
    run(c, dev, want, max_prefix_len=1, max_own_len=1)                   # no pieces


@pytest.mark.parametrize("d,page,nq", [(64, 16, 1), (128, 64, 1), (128, 128, 9), (64, 32, 50)])
def test_prefixes_of_any_length(d, page, nq):
    """Of different lengths in one group: none, all of a sequence, longer than it, longer than the
    table, negative; sequences of no tokens, of no queries, with more queries than tokens."""
    dev = device()
    announce(f"any length d={d} page={page} nq={nq}")
    lens = [400, 400, 400, 64, 0, 30, 400, 333, 5]
    prefix = [300, 0, 400, 200, 100, 30, 1 << 30, -7, 3]
    runs = [nq, nq, nq, nq, nq, nq, 0, nq, nq + 3]
    need = -(-400 // page) + 2
    c = Case([0, 9], [min(p, 500) for p in prefix], lens, runs, 8, 4, d, page, seed=d + page)
    c.prefix = prefix
    c.table[0] = c.rng.integers(0, c.pages, c.table.shape[1])            # the first one's row: pages throughout
    assert c.table.shape[1] >= need
    run(c, dev)
    run(c, dev, max_prefix_len=64, max_own_len=64)


def test_many_groups():
    """More groups than a wave looks at in one step, some of them empty or without queries."""
    dev = device()
    batch = 150
    rng = np.random.default_rng(1)
    starts = [0] + sorted(int(v) for v in rng.integers(0, batch, 139)) + [batch]
    assert len(starts) - 1 == 140 and len(set(starts)) < len(starts)
    nq = [int(v) for v in rng.integers(0, 3, batch)]
    prefix = [0] * batch
    for g in range(140):
        for b in range(starts[g], starts[g + 1]):
            prefix[b] = 20 + 9 * (g % 7)
    lens = [p + int(rng.integers(3, 40)) for p in prefix]
    c = Case(starts, prefix, lens, nq, 4, 2, 64, 16, seed=3, behind=1)
    run(c, dev)


def test_same_as_whole_sequences():
    """Shared pages in every sequence's own row too, as a server has them: mxq_attention_nvfp4
    sees the same tokens."""
    dev = device()
    c = Case([0, 5], [320] * 5, [400, 321, 350, 500, 330], [1, 2, 1, 4, 1], 16, 2, 128, 32, seed=9)
    c.table[1:, :10] = c.table[0, :10]
    want = c.want()
    run(c, dev, want)
    r = mxq.mxq_attention_nvfp4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev), 4, lse=True)
    torch.cuda.synchronize()
    cu.check_attention(su.f32_of_bf16(r.out), host(r.lse), want)


@pytest.mark.parametrize("d,page,nq,batch", [(64, 16, 1, 3), (128, 64, 1, 3), (128, 32, 2, 30), (64, 64, 1, 40), (128, 128, 40, 3)])
def test_what_is_not_seen_stays_out(d, page, nq, batch):
    """A NaN scale in a shared token reaches the rows that see it and no other; in the tail of a
    cut-off page, past every sequence and in other pages it changes no bit; a page that may
    not be read makes the rows that see it NaN."""
    dev = device()
    announce(f"unseen d={d} page={page} nq={nq} batch={batch}")
    shared = 5 * page + 9                                                # ends inside a page

    def fresh():
        lens = [shared + nq + 11 * b for b in range(batch)]
        prefix = [shared - (b % 3) * 20 for b in range(batch)]           # not all share all of it
        return Case([0, batch], prefix, lens, [nq] * batch, 8, 2, d, page, seed=page + d)

    def results(c):
        r = c.prepared(dev, lse=True)()
        torch.cuda.synchronize()
        return su.f32_of_bf16(r.out), host(r.lse)

    clean, clean_lse = results(fresh())
    assert np.isfinite(clean).all()
    for t in (0, page + 3, shared - 41, shared - 21, shared - 1, shared, shared + page):
        for which in ("ks", "vs"):
            c = fresh()
            getattr(c, which)[c.table[0, t // page], 1, t % page, 2] = 0xFF
            got, lse = results(c)
            hit = np.zeros((c.total, c.hq), bool)
            seen = prefix_tokens(c, c.group_starts, c.prefix)
            for row, b, pos in c.queries():                              # (a page may be another sequence's)
                at, off = seen(row, b, pos, 1)
                hit[row, 4:] = ((at == c.table[0, t // page]) & (off == t % page)).any()
            assert_same("rows that do not see it", got[~hit], clean[~hit])
            assert_same("their log-sums", lse[~hit], clean_lse[~hit])
            if which == "ks":
                assert np.isnan(got[hit]).all() and np.isnan(lse[hit]).all()
            else:
                assert np.isnan(got[hit][:, 32:48]).all()
                assert_same("log-sums", lse[hit], clean_lse[hit])
    c = fresh()
    used = np.zeros((c.pages, page), bool)
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        mine = t >= c.prefix[b]
        used[c.table[b, t[mine] // page], t[mine] % page] = True
        used[c.table[0, t[~mine] // page], t[~mine] % page] = True
    for x in (c.ks, c.vs):
        x.transpose(0, 2, 1, 3)[~used] = 0x7F
    got, lse = results(c)
    assert_same("out", got, clean)
    assert_same("lse", lse, clean_lse)
    for bad in (c.pages, -1, 2147483647, -2147483648):
        c = fresh()
        c.table[0, 2] = bad
        got, lse = results(c)
        assert np.isnan(got).all() and np.isnan(lse).all()
        c = fresh()
        b = batch - 1
        c.table[b, shared // page] = bad
        got, lse = results(c)
        lo = int(c.starts[b])
        hit = np.zeros(c.total, bool)
        hit[lo:] = True
        assert np.isnan(got[hit]).all()
        assert_same("other sequences", got[~hit], clean[~hit])


def test_longer_runs_than_planned():
    """Queries past max_q_len are left as they were."""
    dev = device()
    for nq, most in ((5, 2), (60, 20)):
        c = Case([0, 2], [100, 100], [200, 180], [nq, 1], 4, 2, 64, 16, seed=nq)
        want = [x.copy() for x in c.want()]
        late = slice(int(c.starts[0]) + most, int(c.starts[1]))
        want[0][late], want[1][late] = np.nan, np.nan
        run(c, dev, want, max_q_len=most)


def test_scale_stream_and_strides():
    dev = device()
    c = Case([0, 3], [200, 200, 200], [230, 260, 201], [1, 1, 1], 6, 2, 64, 16, seed=8, behind=1)
    wide_q = torch.zeros((c.total, 10, c.d), dtype=torch.bfloat16, device=dev)
    wide_q[:, 2:8] = c.device_q(dev)
    wide_out = torch.full((c.total, 9, c.d), 3.0, dtype=torch.bfloat16, device=dev)
    table, lens, starts = c.device_sequences(dev)
    wide_table = torch.full((3, table.shape[1] + 5), 123456, dtype=torch.int32, device=dev)
    wide_table[:, :table.shape[1]] = table
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    stream = torch.cuda.Stream()
    r = mxq.mxq_attention_prefix_nvfp4(wide_q[:, 2:8], c.device_cache(dev), wide_table[:, :table.shape[1]], lens, starts,
                                       i32(c.group_starts), i32(c.prefix), 1, scale=0.2, lse=True, out=wide_out[:, 1:7],
                                       stream=stream)
    stream.synchronize()
    cu.check_attention(su.f32_of_bf16(wide_out[:, 1:7]), host(r.lse), c.want(0.2))
    assert (wide_out[:, 0] == 3).all() and (wide_out[:, 7:] == 3).all() and (wide_out[-1] == 3).all()


def test_workspace_and_empty_calls():
    dev = device()
    c = Case([0, 2], [100, 100], [130, 120], [1, 1], 4, 2, 64, 16)
    call = c.prepared(dev)
    with pytest.raises(mxq.MxqError, match="WORKSPACE_TOO_SMALL"):
        c.prepared(dev, workspace=torch.empty(call.workspace.numel() - 256, dtype=torch.uint8, device=dev))()
    c = Case([0, 1], [50], [100], [0], 4, 2, 64, 16)
    assert c.prepared(dev)().out.shape == (0, 4, 64)
    # a cache without pages: nothing to see
    c = Case([0, 2], [16, 16], [30, 40], [1, 2], 4, 2, 64, 16)
    empty = mxq.NVFP4KVCache(*[t[:0] for t in c.device_cache(dev).tensors()[:4]], *c.device_cache(dev).tensors()[4:])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    r = mxq.mxq_attention_prefix_nvfp4(c.device_q(dev), empty, *c.device_sequences(dev), i32([0, 2]), i32([16, 16]), 2, lse=True)
    torch.cuda.synchronize()
    assert (r.out == 0).all() and torch.isneginf(r.lse).all()


def test_graph():
    """A decoding step of a group, captured once: lengths, queries and the cache change between
    the replays, with other work between them."""
    dev = device()
    lens = [230, 260, 201, 333]
    c = Case([0, 4], [200] * 4, [n + 8 for n in lens], [1] * 4, 16, 2, 128, 64, seed=4)
    q, cache = c.device_q(dev), c.device_cache(dev)
    table, seq_lens, starts = c.device_sequences(dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    call = mxq.AttentionPrefixNVFP4(q, cache, table, seq_lens, starts, i32([0, 4]), i32([200] * 4), 1, lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        c.lens = [n + 2 * i for n in lens]
        c.q = su.to_bf16((c.rng.standard_normal(c.q.shape) * 1.3).astype(np.float32))
        seq_lens.copy_(i32(c.lens))
        q.copy_(c.device_q(dev))
        graph.replay()
        torch.cuda.synchronize()
        cu.check_attention(su.f32_of_bf16(call.out.out), host(call.out.lse), c.want())
        call.out.out.fill_(9.0)
        call.workspace.fill_(0xFF)


@pytest.mark.parametrize("graph", [False, True])
def test_decoding_behind_a_shared_prompt(graph):
    """Steps of a server: each sequence of two groups appends a token to pages of its own, then all
    attend over prompt and tokens; captured once and replayed too."""
    dev = device()
    hk, hq, d, page, batch = 2, 8, 64, 16, 5
    starts, prefix = [0, 3, 5], [100, 100, 100, 64, 64]
    own = [3, 17, 1, 30, 2]
    c = Case(starts, prefix, [p + n + 12 for p, n in zip(prefix, own)], [1] * batch, hq, hk, d, page, seed=2)
    cache = c.device_cache(dev)
    table, seq_lens, q_starts = c.device_sequences(dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    gen = torch.Generator(device=dev).manual_seed(5)
    qkv = torch.empty((batch, hq + 2 * hk, d), dtype=torch.bfloat16, device=dev)
    positions, slots = i32([0] * batch), torch.zeros(batch, dtype=torch.int64, device=dev)
    append = mxq.RopeAppendNVFP4(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], positions, slots, mxq.rope_plan(d), cache)
    attend = mxq.AttentionPrefixNVFP4(append.out.q, cache, table, seq_lens, q_starts, i32(starts), i32(prefix), 1, lse=True)
    recorded = None
    for i in range(6):
        now = torch.tensor([p + n + i for p, n in zip(prefix, own)], device=dev)
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=dev))
        positions.copy_(now)
        slots.copy_(table[torch.arange(batch, device=dev), now // page].long() * page + now % page)
        seq_lens.copy_(now + 1)
        if graph and recorded is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                recorded = torch.cuda.CUDAGraph()
                with torch.cuda.graph(recorded, stream=side):
                    append(), attend()
            torch.cuda.current_stream().wait_stream(side)
        recorded.replay() if graph else (append(), attend())
        torch.cuda.synchronize()
        c.kc, c.ks, c.vc, c.vs = (host(t) for t in cache.tensors()[:4])
        c.lens, c.q = [int(v) + 1 for v in now], su.f32_of_bf16(append.out.q)
        cu.check_attention(su.f32_of_bf16(attend.out.out), host(attend.out.lse), c.want())

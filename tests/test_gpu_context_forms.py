"""Every form that the calls for long and shared contexts take by shape, against the plain forms of
tests/context_util.py: the widths, tiles and page layouts of the kernels, scores by way of the
workspace, and joins of more parts than a wave holds at once."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import context_util as cu
from tests import serve_util as su
from tests.gpu_util import announce, assert_same, device, host
from tests.test_gpu_pages import random_keys, run_pages, run_select
from tests.test_gpu_prefix import Case, run

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection
def select_by_workspace(c, codes, scales, top, first, last, dev, **kw):
    """A selection whose scores are made by work-groups of their own."""
    keys = mxq.PageKeys(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), c.page)
    fill = np.full((c.total, c.hk, top), -77, np.int32)
    call = mxq.SelectPagesNVFP4(c.device_q(dev), keys, *c.device_sequences(dev), top=top, first=first, last=last,
                                out=torch.from_numpy(fill).to(dev), **kw)
    assert call.workspace is not None
    call.workspace.fill_(0xFF)                                           # whatever it holds: above every score
    got = call()
    torch.cuda.synchronize()
    assert_same(f"pages of {c.lens} {c.nq}", host(got), cu.select_reference(c, codes, scales, top, first, last, fill))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,hk", [(1, 4), (2, 2), (3, 3), (4, 8), (5, 1), (8, 2), (12, 2), (16, 1), (24, 2), (40, 1)])
def test_scores_by_way_of_the_workspace(group, hk, d):
    """Few queries of long sequences: planned for more than they hold, for just what they hold, and for
    1024 pages of some 1300; one short sequence among them; NaN scales and unreadable pages."""
    dev = device()
    announce(f"scores by workspace group={group} hk={hk} d={d}")
    page = 16
    c = cu.Sequences([page * 1300 + 5, 300, page * 1100], [2, 1, 1], group * hk, hk, d, page, seed=group + d, before=1, behind=1)
    assert c.total * hk <= 64
    codes, scales = random_keys(c, 1)
    select_by_workspace(c, codes, scales, 40, 1, 2, dev, max_seq_len=1 << 20)
    select_by_workspace(c, codes, scales, 40, 1, 2, dev)
    select_by_workspace(c, codes, scales, 40, 1, 2, dev, max_seq_len=1024 * page)
    select_by_workspace(c, codes, scales, 300, 2, 3, dev)                # more than the shortlist takes
    c.table[:, ::7] = c.pages
    c.table[2, 100] = -1
    scales[::5] = np.nan
    c.q[1] = -np.abs(c.q[1])
    c.q[2, 0, 3] = np.inf
    select_by_workspace(c, codes, scales, 64, 1, 2, dev)
    codes[:, :, 1:] = 0                                                  # ties: a score of few values
    select_by_workspace(c, np.sign(codes), np.ones_like(scales), 40, 1, 2, dev)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 7, 13, 20])
def test_select_widths(group, d):
    """The forms for few queries, for some hundreds, and for long runs of them."""
    dev = device()
    announce(f"select widths group={group} d={d}")
    page = 16
    for lens, nq, hk, top in (([1500], [3], 2, 10),                      # 16 waves a query
                              ([1700, 40, 900], [100, 30, 40], 2, 12),   # four
                              ([1200, 1300], [300, 270], 4, 9)):         # several queries a work-group
        c = cu.Sequences(lens, nq, group * hk, hk, d, page, seed=group + len(lens), before=2, behind=1)
        codes, scales = random_keys(c, 1)
        run_select(c, codes, scales, top, 1, 2, dev)


@pytest.mark.parametrize("lens,nq,hq,hk,d", [
    ([20000], [2], 8, 2, 128),                                           # by way of the workspace
    ([900, 333], [2, 1], 6, 2, 64),
    ([1500, 700], [300, 260], 8, 4, 128),
])
def test_select_strides(lens, nq, hq, hk, d):
    """q inside a wider buffer whose other heads are NaN, a table with a row stride."""
    dev = device()
    announce(f"select strides lens={lens} nq={nq} hq={hq} hk={hk} d={d}")
    c = cu.Sequences(lens, nq, hq, hk, d, 16, seed=hq, behind=1)
    codes, scales = random_keys(c, 1)
    keys = mxq.PageKeys(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), c.page)
    wide_q = torch.full((c.total, hq + 5, d), float("nan"), dtype=torch.bfloat16, device=dev)
    wide_q[:, 3:3 + hq] = c.device_q(dev)
    table, seq_lens, starts = c.device_sequences(dev)
    wide_table = torch.full((len(lens), table.shape[1] + 5), 123456, dtype=torch.int32, device=dev)
    wide_table[:, :table.shape[1]] = table
    fill = np.full((c.total, hk, 20), -77, np.int32)
    out = torch.from_numpy(fill).to(dev)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    mxq.mxq_select_pages_nvfp4(wide_q[:, 3:3 + hq], keys, wide_table[:, :table.shape[1]], seq_lens, starts, top=20, out=out,
                               stream=stream)
    stream.synchronize()
    assert_same("pages", host(out), cu.select_reference(c, codes, scales, 20, 1, 2, fill))


# ------------------------------------------------------------------ attention over listed pages
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("group,nq,hk", [(5, 3, 2), (24, 3, 2), (33, 2, 1), (2, 257, 8), (17, 257, 8)])
def test_listed_pages_forms(group, nq, hk, page, d):
    """16 or 32 rows, one tile of them or two, a work-group a unit or a wave a unit, short pages or long."""
    dev = device()
    announce(f"pages forms group={group} nq={nq} hk={hk} page={page} d={d}")
    c = cu.Sequences([page * 5 + 7 + nq], [nq], group * hk, hk, d, page, seed=page + group, before=1, behind=1)
    run_pages(c, cu.random_lists(c, 4, seed=d), dev)


def parts_of(call, c):
    """How many parts a row's workspace holds (FP32 elements, maximum and sum)."""
    return call.workspace.numel() // (c.total * c.hq * (c.d * 4 + 8))


@pytest.mark.parametrize("d,top,least", [(128, 100, 25), (128, 150, 37), (128, 200, 50), (128, 700, 175), (64, 160, 40),
                                         (64, 300, 73), (64, 340, 85), (64, 700, 175)])
def test_many_parts_of_a_list(d, top, least):
    """One query and cached head: the join takes 36 parts at a time (heads of 64: 72).  The row's largest
    scores in the first part, in the last, in neither; a list that leaves the last parts empty, one that
    leaves all but one."""
    dev = device()
    announce(f"parts of a list d={d} top={top}")
    page = 64
    for loud in (None, 0, top - 1):
        c = cu.Sequences([page * top - 3], [1], 4, 1, d, page, seed=top)
        if loud is not None:                                             # K of a page eight times as large
            c.ks[c.table[0, loud]] = np.minimum(c.ks[c.table[0, loud]] + 0x18, 0x7E)
        lists = np.arange(top, dtype=np.int32).reshape(1, 1, top)
        _, _, call = run_pages(c, lists, dev)
        assert parts_of(call, c) >= least
        for entries in (1, 5, top - 9):
            short = lists.copy()
            short[..., entries:] = -1
            run_pages(c, short, dev)


# ------------------------------------------------------------------ shared prefixes
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("batch,nq,group,groups", [
    (4, 1, 3, 1),                                                        # 16 rows of both kinds
    (4, 1, 7, 1), (3, 3, 7, 3),                                          # 32
    (14, 1, 3, 1),                                                       # 128 rows of a group, 16 of a sequence
    (3, 8, 4, 1), (7, 1, 20, 2),                                         # 32 of a sequence
    (3, 9, 4, 1), (2, 150, 1, 2),                                        # 128 of both
])
def test_prefix_forms(batch, nq, group, groups, page, d):
    dev = device()
    announce(f"prefix forms batch={batch} nq={nq} group={group} groups={groups} page={page} d={d}")
    starts = [batch * g // groups for g in range(groups + 1)]
    prefix = [3 * page + 5 + (b % 2) * 20 for b in range(batch)]
    c = Case(starts, prefix, [p + nq + 9 * b for b, p in enumerate(prefix)], [nq] * batch, 2 * group, 2, d, page, seed=page + d)
    run(c, dev)


@pytest.mark.parametrize("d,prefix,own,least", [(128, 20000, 50, 78), (64, 40000, 50, 150), (128, 40, 12000, 46), (64, 9000, 20000, 100)])
def test_many_parts_of_a_prefix(d, prefix, own, least):
    """A row's parts of both kinds in several passes of the join; the largest scores in the prefix's first
    page, its last, or the sequence's own last one."""
    dev = device()
    announce(f"parts of a prefix d={d} prefix={prefix} own={own}")
    page = 64
    for loud in (None, 0, prefix // page - 1, (prefix + own - 1) // page):
        c = Case([0, 2], [prefix] * 2, [prefix + own, prefix + 1], [1, 1], 4, 1, d, page, seed=own)
        if loud is not None:
            c.ks[c.table[0, loud]] = np.minimum(c.ks[c.table[0, loud]] + 0x18, 0x7E)
        run(c, dev, max_prefix_len=prefix, max_own_len=own)
        assert parts_of(c.prepared(dev, max_prefix_len=prefix, max_own_len=own), c) >= least


def test_more_parts_than_tokens():
    """Planned for far longer prefixes and sequences than there are: 256 parts, nearly all empty."""
    dev = device()
    announce("more parts than tokens")
    for d, page in ((64, 16), (128, 64)):
        c = Case([0, 2], [100, 130], [140, 131], [1, 1], 4, 1, d, page, seed=d, behind=1)
        run(c, dev, max_prefix_len=1 << 24, max_own_len=1 << 24)
        assert parts_of(c.prepared(dev, max_prefix_len=1 << 24, max_own_len=1 << 24), c) == 256


@pytest.mark.parametrize("what", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("d,page,batch,nq,group", [(64, 16, 4, 1, 3), (128, 64, 3, 3, 7), (128, 16, 14, 1, 3), (64, 64, 2, 150, 1)])
def test_rows_beside_one_that_is_no_number(batch, nq, group, page, d, what):
    """NaN, infinities or the largest numbers in one query and head: every other row's bits stay."""
    dev = device()
    announce(f"one row of {what} batch={batch} nq={nq} group={group} page={page} d={d}")
    c = Case([0, batch], [4 * page + 3] * batch, [5 * page + nq + 9 * b for b in range(batch)], [nq] * batch, 2 * group, 2, d, page,
             seed=page + d)
    c.table[1:, :4] = c.table[0, :4]                                     # (for the lists: a row of its own for each)
    lists = torch.from_numpy(cu.random_lists(c, 4, seed=d)).to(dev)

    def results():
        shared = c.prepared(dev, lse=True)()
        listed = mxq.mxq_attention_pages_nvfp4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev), lists, lse=True)
        torch.cuda.synchronize()
        return [su.f32_of_bf16(shared.out), host(shared.lse), su.f32_of_bf16(listed.out), host(listed.lse)]

    clean = results()
    assert all(np.isfinite(x).all() for x in clean)
    row, head = c.total // 2, c.hq - 1
    c.q[row, head, ::3] = su.to_bf16(np.full(c.d, what, np.float32))[::3]
    got = results()
    for x, y in zip(got, clean):
        if what != 3e38:
            assert np.isnan(x[row, head]).all()
        x, y = x.copy(), y.copy()
        x[row, head] = y[row, head] = 0
        assert_same("the other rows", x, y)


# ------------------------------------------------------------------ mean keys on two streams
def test_mean_keys_and_selection_on_two_streams():
    """Two servers' steps at once: each updates mean keys and selects by them, on a stream of its own."""
    dev = device()
    announce("mean keys on two streams")

    def server(seed, hq, hk, d, page):
        c = cu.Sequences([page * 60 + 3, page * 33], [1, 1], hq, hk, d, page, seed=seed)
        cache, keys = c.device_cache(dev), mxq.PageKeys(
            torch.zeros((c.pages, hk, d), dtype=torch.int8, device=dev), torch.zeros((c.pages, hk), device=dev), page)
        update = mxq.PageKeysNVFP4(cache, torch.arange(c.pages * page, device=dev), keys)
        select = mxq.SelectPagesNVFP4(c.device_q(dev), keys, *c.device_sequences(dev), top=12)
        return update, select, keys

    servers = [server(1, 8, 2, 128, 16), server(2, 6, 3, 64, 32)]
    want = []
    for update, select, keys in servers:
        update(), select()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (keys.codes, keys.scales, select.out)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for _, select, keys in servers:
            for t in (keys.codes, keys.scales, select.out):
                t.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            for s, (update, select, _) in zip(streams, servers):
                update(s), select(s)
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for (_, select, keys), expected in zip(servers, want):
            for got, w in zip((keys.codes, keys.scales, select.out), expected):
                assert torch.equal(got, w)

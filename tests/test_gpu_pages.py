"""Mean keys, page selection and attention over listed pages on the GPU against plain forms
(tests/context_util.py): keys and selections bit for bit, attention within bounds counted from
its roundings (context_util.attention_over)."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import context_util as cu
from tests import serve_util as su
from tests.gpu_util import announce, assert_same, device, host

pytestmark = pytest.mark.gpu


def f32(t):
    return su.f32_of_bf16(t)


# ------------------------------------------------------------------ mean keys
def keys_case(pages, hk, page, d, seed, order="heads"):
    return cu.Sequences([page], [1], hk, hk, d, page, seed=seed, spare=pages - 1, order=order)


def run_keys(c, slots, dev):
    cache = c.device_cache(dev)
    rng = np.random.default_rng(9)
    codes = rng.integers(-128, 128, (c.pages, c.hk, c.d)).astype(np.int8)
    scales = rng.random((c.pages, c.hk)).astype(np.float32)
    keys = mxq.PageKeys(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), c.page)
    mxq.mxq_page_keys_nvfp4(cache, torch.from_numpy(slots).to(dev), keys)
    torch.cuda.synchronize()
    want_codes, want_scales = cu.page_keys_reference(c.kc, c.ks, c.kg, slots, codes, scales)
    assert_same("codes", host(keys.codes), want_codes)
    got = host(keys.scales)
    assert np.array_equal(np.isnan(got), np.isnan(want_scales))
    assert_same("scales", np.nan_to_num(got), np.nan_to_num(want_scales))


@pytest.mark.parametrize("pages,hk,page,d,order", [
    (9, 1, 16, 64, "heads"), (9, 3, 16, 128, "rows"), (7, 2, 32, 128, "heads"), (7, 8, 64, 128, "heads"),
    (5, 5, 64, 64, "rows"), (4, 2, 128, 64, "heads"), (3, 2, 512, 128, "heads"), (3, 1, 256, 64, "rows"),
])
def test_page_keys(pages, hk, page, d, order):
    dev = device()
    announce(f"keys pages={pages} hk={hk} page={page} d={d} {order}")
    c = keys_case(pages, hk, page, d, pages * 7 + d, order)
    # last rows of some pages, other rows, padding and rows past the cache
    slots = np.array([page - 1, 2 * page - 2, 3 * page - 1, -1, pages * page, pages * page + page - 1, -page - 1, page],
                     np.int64)
    run_keys(c, slots, dev)
    run_keys(c, np.arange(pages * page, dtype=np.int64), dev)            # a whole prompt
    run_keys(c, np.array([page - 1], np.int64), dev)
    run_keys(c, np.array([5, 6], np.int64), dev)                         # nothing full


@pytest.mark.parametrize("hk,page,d", [(8, 16, 128), (16, 64, 64), (8, 128, 128)])
def test_page_keys_many_slots(hk, page, d):
    """Enough slots that a wave looks at several, in order and shuffled."""
    dev = device()
    pages = 1100 // (page // 16) + 1
    announce(f"many slots hk={hk} page={page} d={d}")
    c = keys_case(pages, hk, page, d, 3)
    slots = np.arange(pages * page, dtype=np.int64)
    assert slots.size * hk > 8192
    run_keys(c, slots[:-page // 2], dev)
    np.random.default_rng(4).shuffle(slots)
    run_keys(c, slots[:-3], dev)


@pytest.mark.parametrize("d", [64, 128])
def test_page_keys_extremes(d):
    """The largest sums (512 rows of 6 * 448), zeros, one element alone, halves that go to the
    even number, NaN scales in one head only, a tensor scale that overflows the scale."""
    dev = device()
    c = keys_case(6, 2, 512, d, 8)
    c.kc[0], c.ks[0] = 0x77, 0x7E                                        # all 6 * 448
    c.kc[1], c.ks[1] = 0xFF, 0x7E                                        # all -6 * 448
    c.kc[2] = 0                                                          # zeros (and -0 below)
    c.kc[2, :, :, 0] = 0x80
    c.kc[3], c.ks[3] = 0, 0x01                                           # one element of the smallest step
    c.kc[3, :, 7, 5] = 0x10
    c.kc[4] = 0                                                          # 127 : 64 quotients k / 2
    c.ks[4] = 0x38
    c.kc[4, :, 0, 0] = 0x77
    c.kc[4, :, 1:22, 0] = 0x07
    c.ks[5, 1, 300, d // 16 - 1] = 0xFF
    run_keys(c, np.arange(6, dtype=np.int64) * 512 + 511, dev)
    c.kg[:] = [3e38, 1e-38]
    run_keys(c, np.arange(6, dtype=np.int64) * 512 + 511, dev)


# ------------------------------------------------------------------ selection
def random_keys(c, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    codes = rng.integers(-127, 128, (c.pages, c.hk, c.d)).astype(np.int8)
    return codes, (rng.random((c.pages, c.hk)) * spread + 0.01).astype(np.float32)


def run_select(c, codes, scales, top, first, last, dev, max_seq_len=None):
    keys = mxq.PageKeys(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), c.page)
    fill = np.full((c.total, c.hk, top), -77, np.int32)
    out = torch.from_numpy(fill).to(dev)
    mxq.mxq_select_pages_nvfp4(c.device_q(dev), keys, *c.device_sequences(dev), top=top, first=first, last=last,
                               max_seq_len=max_seq_len, out=out)
    torch.cuda.synchronize()
    want = cu.select_reference(c, codes, scales, top, first, last, fill)
    assert_same(f"pages of {c.lens} {c.nq}", host(out), want)


@pytest.mark.parametrize("lens,nq,hq,hk,d,page,top,first,last", [
    ([1000], [1], 8, 2, 128, 16, 8, 1, 2),
    ([1, 16, 17, 0, 500], [1, 1, 1, 1, 1], 4, 4, 64, 16, 5, 1, 1),
    ([900, 40, 333], [5, 3, 0], 6, 2, 64, 32, 7, 2, 3),
    ([2048, 64 * 9 + 1], [33, 2], 24, 1, 128, 64, 6, 0, 1),              # 24 rows a head
    ([3000], [4], 40, 1, 64, 16, 64, 1, 4),                              # 40 rows a head
    ([700, 700], [3, 9], 15, 3, 128, 16, 4, 1, 3),                       # nothing but the first and last
    ([5000, 300], [2, 2], 16, 2, 128, 16, 33, 0, 2),
    ([260], [1], 2, 1, 128, 128, 1, 0, 1),
    ([10, 2], [14, 5], 4, 2, 64, 16, 3, 1, 1),                           # more queries than tokens
    ([20000], [3], 8, 1, 64, 16, 100, 3, 5),
    ([9000, 9000], [70, 70], 4, 4, 64, 16, 40, 1, 2),
])
def test_select(lens, nq, hq, hk, d, page, top, first, last):
    dev = device()
    announce(f"select lens={lens} nq={nq} hq={hq} hk={hk} d={d} page={page} top={top} first={first} last={last}")
    c = cu.Sequences(lens, nq, hq, hk, d, page, seed=sum(lens), before=2, behind=3)
    codes, scales = random_keys(c, 1)
    run_select(c, codes, scales, top, first, last, dev)
    if max(lens) > 300 * page:                                           # scores that do not fit what is held
        run_select(c, codes, scales, top, first, last, dev, max_seq_len=page)


def test_select_ties():
    """Equal scores go to the lower page: keys of few values, all the same, zeros of both signs."""
    dev = device()
    c = cu.Sequences([3001, 800], [3, 2], 8, 2, 64, 16, seed=2)
    rng = np.random.default_rng(3)
    codes = np.repeat(rng.integers(-127, 128, (1, c.hk, c.d)), c.pages, 0).astype(np.int8)
    ones = np.ones((c.pages, c.hk), np.float32)
    run_select(c, codes, ones, 20, 1, 2, dev)
    run_select(c, codes, rng.integers(0, 3, ones.shape).astype(np.float32), 20, 1, 2, dev)
    run_select(c, codes * (rng.integers(0, 2, (c.pages, 1, 1)) * 2 - 1).astype(np.int8), ones, 50, 1, 2, dev)
    run_select(c, codes * 0, ones, 20, 0, 1, dev)
    c.q[:] = 0
    c.q[::2] = -0.0
    run_select(c, codes, ones, 20, 1, 2, dev)


def test_select_values_at_the_edges():
    """NaN and infinite scales, pages that may not be read, rows of q with infinities, NaN,
    subnormals and the largest numbers."""
    dev = device()
    c = cu.Sequences([2000, 1500], [8, 8], 6, 2, 128, 16, seed=5)
    codes, scales = random_keys(c, 6)
    rng = np.random.default_rng(7)
    scales[rng.random(scales.shape) < 0.3] = np.nan
    scales[rng.random(scales.shape) < 0.05] = np.inf
    c.table[0, rng.random(c.table.shape[1]) < 0.1] = c.pages
    c.table[1, rng.random(c.table.shape[1]) < 0.1] = -5
    c.table[1, 3] = 2147483647
    c.q[0, 0, 3] = np.inf
    c.q[1, 1, 100] = np.nan
    c.q[2] = np.nan
    c.q[3, :3] = su.to_bf16(np.full((3, 128), 3e38, np.float32))
    c.q[4] = c.q[4] * np.float32(2.0 ** -130)
    c.q[4] = su.to_bf16(c.q[4])
    c.q[5, 2] = 0
    c.q[5, 2, 77] = np.float32(2.0 ** -133)
    run_select(c, codes, scales, 30, 1, 2, dev)
    scales[:] = np.nan
    run_select(c, codes, scales, 30, 1, 2, dev)


# ------------------------------------------------------------------ attention over listed pages
def run_pages(c, lists, dev, lse=True, want=None, scale=None):
    out = torch.full((c.total, c.hq, c.d), 7.0, dtype=torch.bfloat16, device=dev)
    call = mxq.AttentionPagesNVFP4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev),
                                   torch.from_numpy(lists).to(dev), lse=lse, out=out, scale=scale)
    if lse:
        call.out.lse.fill_(7.0)
    if call.workspace is not None:
        call.workspace.fill_(0xFF)                                       # whatever it holds: NaN here
    r = call()
    torch.cuda.synchronize()
    got, got_lse = f32(r.out), host(r.lse)
    if want is None:
        want = cu.attention_over(c, cu.listed_tokens(c, lists), scale or 1 / math.sqrt(c.d))
    cu.check_attention(got, got_lse, want)
    none = np.isnan(want[1])
    assert (got[none] == 7.0).all() and (got_lse is None or (got_lse[none] == 7.0).all())
    r = call()
    torch.cuda.synchronize()
    assert np.array_equal(f32(r.out), got)                               # and it repeats
    return got, got_lse, call


@pytest.mark.parametrize("lens,nq,hq,hk,d,page,top", [
    ([1000], [1], 8, 2, 128, 16, 8),
    ([1, 16, 17, 0, 500], [1, 1, 1, 1, 1], 4, 4, 64, 16, 5),
    ([900, 40, 333], [5, 3, 0], 6, 2, 64, 32, 7),
    ([2048, 577], [17, 2], 24, 1, 128, 64, 6),                           # 24 rows a head
    ([3000], [3], 40, 1, 64, 16, 40),                                    # 40 rows a head
    ([1500], [2], 70, 1, 128, 64, 9),
    ([700, 90], [3, 9], 15, 3, 128, 16, 4),
    ([3000, 300], [2, 2], 16, 2, 128, 128, 5),
    ([5000], [2], 4, 1, 64, 1024, 3),                                    # pages of many tiles
    ([10, 2], [14, 5], 4, 2, 64, 16, 3),                                 # more queries than tokens
    ([400, 500], [150, 150], 8, 8, 64, 16, 5),                           # a wave a unit
    ([600], [300], 8, 8, 128, 64, 4),
    ([333], [270], 160, 8, 64, 32, 3),                                   # 20 rows a head, a wave a unit
])
def test_attention_pages(lens, nq, hq, hk, d, page, top):
    dev = device()
    announce(f"pages lens={lens} nq={nq} hq={hq} hk={hk} d={d} page={page} top={top}")
    c = cu.Sequences(lens, nq, hq, hk, d, page, seed=sum(lens) + d, before=1, behind=2, order="rows" if d == 64 else "heads")
    run_pages(c, cu.random_lists(c, top, seed=4), dev)


@pytest.mark.parametrize("page,d,nq", [(16, 64, 1), (16, 128, 160), (32, 128, 2), (64, 128, 3), (64, 64, 300), (128, 64, 1)])
def test_lists_of_any_shape(page, d, nq):
    """Entries that add nothing in any place (negative, past the query's page, the largest
    numbers), pages twice, any order, none at all."""
    dev = device()
    announce(f"lists page={page} d={d} nq={nq}")
    c = cu.Sequences([page * 11 + 5 + nq], [nq], 16, 8, d, page, seed=page)
    rng = np.random.default_rng(page + d)
    lists = rng.integers(-3, 16, (c.total, c.hk, 9)).astype(np.int32)
    lists[rng.random(lists.shape) < 0.1] = 2147483647
    lists[rng.random(lists.shape) < 0.1] = -2147483648
    lists[0, 0] = -1                                                     # nothing
    lists[0, 1] = 3                                                      # one page nine times
    lists[0, 2] = [-1] * 8 + [0]
    run_pages(c, lists, dev)


def test_split_lists_and_their_workspace():
    """One query's list over several work-groups: parts meet in the workspace, some of them
    empty; too small a workspace is refused."""
    dev = device()
    c = cu.Sequences([9000], [1], 8, 2, 128, 64, seed=1)
    lists = cu.random_lists(c, 120, seed=2)
    got, _, call = run_pages(c, lists, dev)
    assert call.workspace is not None
    short = lists.copy()
    short[0, 0, 3:] = -1
    short[0, 1] = -1
    got, lse, _ = run_pages(c, short, dev)
    assert (got[0, 4:] == 0).all() and np.isneginf(lse[0, 4:]).all()
    with pytest.raises(mxq.MxqError, match="WORKSPACE_TOO_SMALL"):
        mxq.mxq_attention_pages_nvfp4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev),
                                      torch.from_numpy(lists).to(dev),
                                      workspace=torch.empty(call.workspace.numel() - 256, dtype=torch.uint8, device=dev))


@pytest.mark.parametrize("page,d,nq,top", [(16, 64, 1, 40), (16, 128, 3, 12), (32, 64, 150, 5), (64, 128, 1, 30), (64, 64, 2, 5),
                                           (128, 128, 130, 3)])
def test_what_is_not_seen_stays_out(page, d, nq, top):
    """NaN scales in tokens past a query, in pages that it does not list and past the
    sequence change no bit; NaN in a token that it sees makes K's rows and V's blocks NaN; a page
    that may not be read makes the rows that list it NaN and no other."""
    dev = device()
    announce(f"unseen page={page} d={d} nq={nq} top={top}")

    def fresh():
        c = cu.Sequences([page * 45 + 7], [nq], 16, 8 if nq > 100 else 4, d, page, seed=page + d)
        return c, cu.random_lists(c, top, seed=1)

    c, lists = fresh()
    clean, clean_lse, _ = run_pages(c, lists, dev)
    n, group = c.lens[0], c.hq // c.hk
    seen = np.zeros((c.total, c.hk, n), bool)
    for row, b, pos in c.queries():
        for h in range(c.hk):
            for j in lists[row, h]:
                if j >= 0:
                    seen[row, h, j * page:min((j + 1) * page, pos + 1)] = True
    last = n - 1
    unlisted = np.nonzero(~seen.any((0, 1)))[0]
    targets = [last, n - nq, 3] + ([int(unlisted[len(unlisted) // 2])] if unlisted.size else [])
    for t in sorted(set(targets)):
        for which in ("ks", "vs"):
            c, lists = fresh()
            h = 1
            getattr(c, which)[c.table[0, t // page], h, t % page, 1] = 0x7F
            got = []
            call = mxq.AttentionPagesNVFP4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev),
                                           torch.from_numpy(lists).to(dev), lse=True)
            r = call()
            torch.cuda.synchronize()
            got, lse = f32(r.out), host(r.lse)
            hit = np.zeros((c.total, c.hq), bool)
            hit[:, h * group:(h + 1) * group] = seen[:, h, t][:, None]
            assert_same("rows that do not see it", got[~hit], clean[~hit])
            assert_same("their log-sums", lse[~hit], clean_lse[~hit])
            if which == "ks":
                assert np.isnan(got[hit]).all() and np.isnan(lse[hit]).all()
            else:
                assert np.isnan(got[hit][:, 16:32]).all()
                assert_same("log-sums", lse[hit], clean_lse[hit])
    # rows past the sequence in its last page, and every page that is not the sequence's
    c, lists = fresh()
    at = c.table[0, last // page]
    for which in ("ks", "vs"):
        getattr(c, which)[at, :, last % page + 1:] = 0xFF
        rest = np.setdiff1d(np.arange(c.pages), c.table[0, :last // page + 1])
        getattr(c, which)[rest] = 0x7F
    call = mxq.AttentionPagesNVFP4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev),
                                   torch.from_numpy(lists).to(dev), lse=True)
    r = call()
    torch.cuda.synchronize()
    assert_same("out", f32(r.out), clean)
    assert_same("lse", host(r.lse), clean_lse)
    # unreadable pages
    for bad in (c.pages, -1, 2147483647, -2147483648):
        c, lists = fresh()
        j = int(lists[0, 0, 1])
        c.table[0, j] = bad
        call = mxq.AttentionPagesNVFP4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev),
                                       torch.from_numpy(lists).to(dev), lse=True)
        r = call()
        torch.cuda.synchronize()
        hit = np.repeat(seen[:, :, j * page:(j + 1) * page].any(-1), group, axis=1)
        assert np.isnan(f32(r.out)[hit]).all()
        assert_same("other rows", f32(r.out)[~hit], clean[~hit])


def test_listing_every_page_is_attention_over_the_sequence():
    """Lists of all pages in order: the same tokens as mxq_attention_nvfp4, within both bounds."""
    dev = device()
    c = cu.Sequences([1111, 130], [3, 1], 8, 2, 128, 32, seed=3)
    lists = np.tile(np.arange(40, dtype=np.int32), (c.total, c.hk, 1))
    want = cu.attention_over(c, cu.listed_tokens(c, lists), 1 / math.sqrt(c.d))
    run_pages(c, lists, dev, want=want)
    r = mxq.mxq_attention_nvfp4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev), 3, lse=True)
    torch.cuda.synchronize()
    cu.check_attention(f32(r.out), host(r.lse), want)


def test_strides_and_another_stream():
    """q and out inside wider buffers, a table with a row stride; on a stream of its own."""
    dev = device()
    c = cu.Sequences([500, 310], [2, 1], 6, 2, 64, 16, seed=8, behind=1)
    lists = cu.random_lists(c, 9)
    want = cu.attention_over(c, cu.listed_tokens(c, lists), 0.2)
    wide_q = torch.zeros((c.total, 10, c.d), dtype=torch.bfloat16, device=dev)
    wide_q[:, 2:8] = c.device_q(dev)
    wide_out = torch.full((c.total, 9, c.d), 3.0, dtype=torch.bfloat16, device=dev)
    table, lens, starts = c.device_sequences(dev)
    wide_table = torch.full((2, table.shape[1] + 5), 123456, dtype=torch.int32, device=dev)
    wide_table[:, :table.shape[1]] = table
    stream = torch.cuda.Stream()
    r = mxq.mxq_attention_pages_nvfp4(wide_q[:, 2:8], c.device_cache(dev), wide_table[:, :table.shape[1]], lens, starts,
                                      torch.from_numpy(lists).to(dev), scale=0.2, lse=True, out=wide_out[:, 1:7],
                                      stream=stream)
    stream.synchronize()
    cu.check_attention(f32(wide_out[:, 1:7]), host(r.lse), want)
    assert (wide_out[:, 0] == 3).all() and (wide_out[:, 7:] == 3).all() and (wide_out[-1] == 3).all()


def test_empty_calls():
    dev = device()
    c = cu.Sequences([100], [0], 4, 2, 64, 16)
    lists = torch.zeros((0, 2, 4), dtype=torch.int32, device=dev)
    r = mxq.mxq_attention_pages_nvfp4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev), lists)
    assert r.out.shape == (0, 4, 64)
    # a cache without pages: nothing to see
    c = cu.Sequences([0, 50], [1, 2], 4, 2, 64, 16, spare=0)
    empty = mxq.NVFP4KVCache(*[t[:0] for t in c.device_cache(dev).tensors()[:4]], *c.device_cache(dev).tensors()[4:])
    keys = mxq.PageKeys.allocate(empty)
    pages = mxq.mxq_select_pages_nvfp4(c.device_q(dev), keys, *c.device_sequences(dev), top=4)
    assert (pages == -1).all()
    r = mxq.mxq_attention_pages_nvfp4(c.device_q(dev), empty, *c.device_sequences(dev),
                                      torch.zeros((3, 2, 4), dtype=torch.int32, device=dev), lse=True)
    torch.cuda.synchronize()
    assert (r.out == 0).all() and torch.isneginf(r.lse).all()
    mxq.mxq_page_keys_nvfp4(empty, torch.tensor([15, -1], device=dev), keys)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the calls together
@pytest.mark.parametrize("graph", [False, True])
def test_decoding_with_selected_pages(graph):
    """Steps of a server: append, mean keys, selection, attention over what was selected; each
    against the plain forms of what the cache holds then.  Captured once and replayed too, with
    other work between the replays."""
    dev = device()
    page, hk, hq, d, batch, top = 16, 2, 8, 64, 3, 5
    lens = [157, 30, 301]
    c = cu.Sequences([n + 40 for n in lens], [1] * batch, hq, hk, d, page, seed=12)
    cache = c.device_cache(dev)
    keys = mxq.PageKeys.allocate(cache)
    table, _, starts = c.device_sequences(dev)
    # the prompts' keys
    prompt = torch.cat([table[b].long().repeat_interleave(page)[:n] * page + torch.arange(n, device=dev) % page
                        for b, n in enumerate(lens)])
    mxq.mxq_page_keys_nvfp4(cache, prompt, keys)
    gen = torch.Generator(device=dev).manual_seed(3)
    qkv = torch.empty((batch, (hq + 2 * hk), d), dtype=torch.bfloat16, device=dev)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    positions = torch.empty(batch, dtype=torch.int32, device=dev)
    slots = torch.empty(batch, dtype=torch.int64, device=dev)
    rope = mxq.rope_plan(d)
    append = mxq.RopeAppendNVFP4(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], positions, slots, rope, cache)
    update = mxq.PageKeysNVFP4(cache, slots, keys)
    select = mxq.SelectPagesNVFP4(append.out.q, keys, table, seq_lens, starts, top=top, max_seq_len=400)
    attend = mxq.AttentionPagesNVFP4(append.out.q, cache, table, seq_lens, starts, select.out, lse=True)

    def step():
        append(), update(), select(), attend()

    def inputs(i):
        now = torch.tensor([n + i for n in lens], device=dev)
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=dev))
        positions.copy_(now)
        slots.copy_(table[torch.arange(batch, device=dev), now // page].long() * page + now % page)
        seq_lens.copy_(now + 1)

    recorded = None
    for i in range(20):                                                  # every sequence fills a page
        inputs(i)
        if graph and recorded is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                recorded = torch.cuda.CUDAGraph()
                with torch.cuda.graph(recorded, stream=side):
                    step()
            torch.cuda.current_stream().wait_stream(side)
        recorded.replay() if graph else step()
        torch.cuda.synchronize()
        if i % 5 != 4:
            continue
        c.kc, c.ks, c.vc, c.vs = (host(t) for t in cache.tensors()[:4])
        c.lens, c.q = [n + i + 1 for n in lens], f32(append.out.q)
        full = np.concatenate([c.table[b, :n // page].astype(np.int64) * page + page - 1 for b, n in enumerate(c.lens)])
        codes, scales = cu.page_keys_reference(c.kc, c.ks, c.kg, full, np.zeros(keys.codes.shape, np.int8),
                                               np.zeros(keys.scales.shape, np.float32))
        used = full // page
        assert_same("mean keys", host(keys.codes)[used], codes[used])
        assert_same("their scales", host(keys.scales)[used], scales[used])
        pages = cu.select_reference(c, codes, scales, top, 1, 2, host(select.out))
        assert_same("pages", host(select.out), pages)
        want = cu.attention_over(c, cu.listed_tokens(c, pages), 1 / math.sqrt(d))
        cu.check_attention(f32(attend.out.out), host(attend.out.lse), want)


# runs of queries long enough that a work-group takes several, whose scores share the keys
@pytest.mark.parametrize("lens,nq,hq,hk,d,page,top,first,last", [
    ([3000, 700], [500, 44], 4, 4, 64, 16, 20, 1, 2),                    # one row a head: 64 queries
    ([1500, 900], [300, 260], 8, 4, 128, 16, 12, 0, 1),                  # two
    ([2500], [530], 24, 6, 64, 16, 70, 2, 4),                            # four; just 64 to choose
    ([2600, 40, 1999], [300, 40, 211], 18, 3, 128, 16, 80, 1, 3),        # six of eight; more than 64
    ([1999, 1200], [251, 300], 22, 2, 64, 16, 9, 1, 2),                  # eleven of sixteen
    ([5200], [1100], 16, 1, 128, 16, 40, 1, 2),
    ([9000, 40], [300, 1], 4, 4, 64, 16, 30, 1, 2),                      # scores of 512 candidates a query
])
def test_select_long_runs(lens, nq, hq, hk, d, page, top, first, last):
    dev = device()
    announce(f"select runs lens={lens} nq={nq} hq={hq} hk={hk} d={d} page={page} top={top} first={first} last={last}")
    c = cu.Sequences(lens, nq, hq, hk, d, page, seed=sum(lens), before=5, behind=3)
    codes, scales = random_keys(c, 1)
    run_select(c, codes, scales, top, first, last, dev)
    run_select(c, codes, scales, top, first, last, dev, max_seq_len=page)
    codes[:, :, 1:] = 0                                                  # ties: a score of few values
    run_select(c, np.sign(codes), np.ones_like(scales), top, first, last, dev)
    c.table[:, ::7] = c.pages
    scales[::5] = np.nan
    run_select(c, codes, scales, top, first, last, dev)


@pytest.mark.parametrize("lens,nq,hq,hk,d,page,top", [
    ([20000], [1], 8, 1, 64, 16, 500),                                   # more than the shortlist takes: 16 waves
    ([9000, 8000], [150, 150], 8, 2, 64, 16, 300),                       # four waves a query
    ([8000], [600], 4, 1, 64, 16, 230),                                  # a wave a query
    ([9000], [2], 40, 1, 128, 16, 256),
])
def test_select_many_pages(lens, nq, hq, hk, d, page, top):
    dev = device()
    announce(f"many pages lens={lens} nq={nq} hq={hq} hk={hk} d={d} top={top}")
    c = cu.Sequences(lens, nq, hq, hk, d, page, seed=top)
    codes, scales = random_keys(c, 1)
    run_select(c, codes, scales, top, 1, 2, dev)
    scales = np.round(scales * 3)                                        # ties, zeros
    run_select(c, np.sign(codes), scales, top, 1, 2, dev)

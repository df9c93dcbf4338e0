"""The calls around long and shared contexts on the host: argument errors before anything is
enqueued (fake device addresses, so without a GPU only) and the binding's own checks on CPU
tensors."""
import ctypes
import os

import pytest
import torch

import nvfp4_quantization_amd as mxq
from nvfp4_quantization_amd import pages as pg
from nvfp4_quantization_amd import serve

OK, INVALID, MISALIGNED, WS_SMALL, UNSUPPORTED, HIP = range(6)
A = 1 << 20          # a fake, 256-byte aligned device address: never dereferenced on these paths
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake device addresses: run where no GPU is visible")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mxq.LIB_PATH):
        pytest.skip("libmxq.so not built")
    return mxq.lib()


def kv(**over):
    f = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, k_global=A, v_global=A, num_pages=10, page_size=16, kv_heads=2,
             head_dim=128, code_stride_page=2 * 16 * 64, code_stride_head=16 * 64, code_stride_token=64,
             scale_stride_page=2 * 16 * 8, scale_stride_head=16 * 8, scale_stride_token=8)
    f.update(over)
    return serve._KV(**f)


def keys(**over):
    f = dict(codes=A, scales=A, num_pages=10, page_size=16, kv_heads=2, head_dim=128)
    f.update(over)
    return pg._Keys(**f)


def page_keys(L, c=None, slots=A, tokens=4, k=None):
    return L.mxq_page_keys_nvfp4(ctypes.byref(c or kv()), slots, tokens, ctypes.byref(k or keys()), None)


def select(L, q=A, ld_q=1024, hq=8, total=4, k=None, table=A, ld_table=5, pages=5, lens=A, starts=A, batch=2, max_len=80,
           top=4, first=1, last=2, out=A, ws=None, ws_bytes=0):
    return L.mxq_select_pages_nvfp4(q, ld_q, hq, total, ctypes.byref(k or keys()), table, ld_table, pages, lens, starts, batch,
                                    max_len, top, first, last, out, ws, ws_bytes, None)


def attend(L, q=A, ld_q=1024, hq=8, total=400, out=A, ld_out=1024, lse=A, c=None, table=A, ld_table=5, table_pages=5, lens=A,
           starts=A, batch=2, pages=A, top=4, scale=0.1, ws=None, ws_bytes=0):
    return L.mxq_attention_pages_nvfp4(q, ld_q, hq, total, out, ld_out, lse, ctypes.byref(c or kv()), table, ld_table,
                                       table_pages, lens, starts, batch, pages, top, scale, ws, ws_bytes, None)


@no_gpu
def test_page_keys_errors(L):
    assert page_keys(L, tokens=0) == OK and page_keys(L, tokens=0, slots=None) == OK
    assert page_keys(L, tokens=-1) == INVALID
    assert page_keys(L, slots=None) == INVALID
    assert page_keys(L, slots=A + 4) == MISALIGNED
    for over in (dict(num_pages=9), dict(page_size=32), dict(kv_heads=3), dict(head_dim=64), dict(num_pages=-1),
                 dict(codes=None), dict(scales=None), dict(kv_heads=0), dict(page_size=0)):
        assert page_keys(L, k=keys(**over)) == INVALID, over
    assert page_keys(L, k=keys(codes=A + 8)) == MISALIGNED
    assert page_keys(L, k=keys(scales=A + 2)) == MISALIGNED
    big = dict(page_size=1024, code_stride_head=1024 * 64, code_stride_page=2 * 1024 * 64, scale_stride_head=1024 * 8,
               scale_stride_page=2 * 1024 * 8)
    assert page_keys(L, c=kv(**big), k=keys(page_size=1024)) == UNSUPPORTED      # past what sums hold
    assert page_keys(L, c=kv(head_dim=96), k=keys(head_dim=96)) == UNSUPPORTED
    assert page_keys(L, tokens=1 << 31) == UNSUPPORTED
    assert page_keys(L, tokens=(1 << 31) - 200) == UNSUPPORTED                   # more waves than a launch holds
    assert L.mxq_page_keys_nvfp4(None, A, 4, ctypes.byref(keys()), None) == INVALID
    assert L.mxq_page_keys_nvfp4(ctypes.byref(kv()), A, 4, None, None) == INVALID


@no_gpu
def test_select_errors(L):
    assert select(L, total=0) == OK and select(L, total=0, q=None, out=None) == OK
    for over in (dict(total=-1), dict(hq=0), dict(hq=7), dict(batch=0), dict(max_len=-1), dict(pages=-1), dict(ld_table=4),
                 dict(first=-1), dict(last=0), dict(top=0), dict(top=2), dict(first=3), dict(ld_q=1016), dict(q=None),
                 dict(out=None), dict(lens=None), dict(starts=None), dict(table=None), dict(k=keys(codes=None))):
        assert select(L, **over) == INVALID, over
    assert select(L, first=(1 << 31) - 1, last=(1 << 31) - 1, top=(1 << 31) - 1) == INVALID   # their sum is formed wider
    for over in (dict(ld_q=1028), dict(q=A + 8), dict(out=A + 2), dict(lens=A + 1), dict(starts=A + 2), dict(table=A + 2)):
        assert select(L, **over) == MISALIGNED, over
    for over in (dict(top=65537), dict(batch=65536), dict(total=1 << 28), dict(total=1 << 23), dict(k=keys(page_size=1024)),
                 dict(k=keys(head_dim=32)), dict(ld_q=1 << 40), dict(ld_table=1 << 40),
                 dict(pages=1 << 31, ld_table=1 << 31), dict(max_len=1 << 31)):
        assert select(L, **over) == UNSUPPORTED, over
    # one query of a long sequence: its scores go through the workspace
    need = mxq.mxq_select_pages_nvfp4_workspace_size(8, 2, 16, 1, 1, 100000)
    assert need > 0 and need % 256 == 0
    long = dict(total=1, batch=1, max_len=100000)
    assert select(L, **long) == INVALID
    assert select(L, **long, ws=A, ws_bytes=need - 1) == WS_SMALL
    assert select(L, **long, ws=A + 128, ws_bytes=need) == MISALIGNED
    size = mxq.mxq_select_pages_nvfp4_workspace_size
    assert size(8, 2, 16, 64, 64, 1000) == 0
    for args in ((0, 1, 16, 1, 1, 99999), (8, 3, 16, 1, 1, 99999), (8, 2, 24, 1, 1, 99999), (8, 2, 1024, 1, 1, 1 << 30),
                 (8, 2, 16, 0, 1, 99999), (8, 2, 16, 1, 0, 99999), (8, 2, 16, 1, 1, -1), (8, 2, 16, 1, 1, 1 << 31)):
        assert size(*args) == 0


@no_gpu
def test_attention_pages_errors(L):
    assert attend(L, total=0) == OK
    for over in (dict(total=-1), dict(hq=0), dict(hq=7), dict(batch=0), dict(table_pages=-1), dict(ld_table=4), dict(top=0),
                 dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ld_q=1016), dict(ld_out=1016),
                 dict(q=None), dict(out=None), dict(pages=None), dict(lens=None), dict(starts=None), dict(table=None),
                 dict(c=kv(k_codes=None))):
        assert attend(L, **over) == INVALID, over
    for over in (dict(ld_q=1028), dict(ld_out=1028), dict(q=A + 8), dict(out=A + 8), dict(lse=A + 2), dict(pages=A + 2),
                 dict(lens=A + 1), dict(starts=A + 2), dict(table=A + 2)):
        assert attend(L, **over) == MISALIGNED, over
    big = dict(page_size=1 << 20, code_stride_head=64 << 20, code_stride_page=128 << 20, scale_stride_head=8 << 20,
               scale_stride_page=16 << 20)
    for over in (dict(top=65537), dict(batch=65536), dict(total=1 << 28), dict(c=kv(head_dim=96)),
                 dict(c=kv(**big), top=1025), dict(ld_q=1 << 40), dict(ld_out=1 << 40)):
        assert attend(L, **over) == UNSUPPORTED, over
    # one query, a long list: several parts
    need = mxq.mxq_attention_pages_nvfp4_workspace_size(8, 2, 128, 16, 1, 1024)
    assert need > 0 and need % 256 == 0
    assert attend(L, total=1, top=1024) == INVALID
    assert attend(L, total=1, top=1024, ws=A, ws_bytes=need - 1) == WS_SMALL
    assert attend(L, total=1, top=1024, ws=A + 128, ws_bytes=need) == MISALIGNED


def test_attention_pages_workspace_size(L):
    size = mxq.mxq_attention_pages_nvfp4_workspace_size
    assert size(8, 2, 128, 64, 4000, 32) == 0
    for args in ((0, 1, 128, 64, 1, 9), (8, 3, 128, 64, 1, 9), (8, 2, 96, 64, 1, 9), (8, 2, 128, 48, 1, 9), (8, 2, 128, 64, 0, 9),
                 (8, 2, 128, 64, 1, 0), (8, 2, 128, 64, 1, 1 << 17)):
        assert size(*args) == 0


def cpu_case():
    cache = mxq.NVFP4KVCache.allocate(6, 16, 2, 64, 1.0, 1.0, device="cpu")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    seqs = (torch.zeros(2, 5, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.tensor([0, 1, 3], dtype=torch.int32))
    return cache, mxq.PageKeys.allocate(cache), q, seqs


def test_binding_checks():
    cache, keys_, q, seqs = cpu_case()
    slots = torch.zeros(3, dtype=torch.int64)
    assert keys_.codes.shape == (6, 2, 64) and keys_.scales.shape == (6, 2) and keys_.page_size == 16
    with pytest.raises(ValueError, match="expected a GPU"):
        mxq.mxq_page_keys_nvfp4(cache, slots, keys_)
    with pytest.raises(ValueError, match="expected a GPU"):
        mxq.mxq_select_pages_nvfp4(q, keys_, *seqs, top=4)
    lists = torch.zeros(3, 2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="expected a GPU"):
        mxq.mxq_attention_pages_nvfp4(q, cache, *seqs, lists)
    for bad, error in ((slots.int(), TypeError), (torch.zeros(2, 3, dtype=torch.int64), ValueError),
                       (torch.zeros(6, dtype=torch.int64)[::2], ValueError), ([1, 2], TypeError)):
        with pytest.raises(error):
            mxq.PageKeysNVFP4(cache, bad, keys_)
    for args in ((keys_.codes.int(), keys_.scales, 16), (keys_.codes, keys_.scales.double(), 16),
                 (keys_.codes, keys_.scales[:5], 16), (keys_.codes[:, :, ::2], keys_.scales, 16),
                 (keys_.codes, keys_.scales, 0), (keys_.codes, keys_.scales, 1 << 32)):
        with pytest.raises((TypeError, ValueError)):
            mxq.PageKeys(*args)
    for over in (dict(top=0), dict(top=(1 << 32) + 4), dict(top=4, first=-1), dict(top=4, last=0), dict(top=4, last=(1 << 32) + 1),
                 dict(top=4, first=(1 << 32)), dict(top=4, out=torch.zeros(3, 2, 5, dtype=torch.int32)),
                 dict(top=4, out=torch.zeros(3, 2, 4, dtype=torch.int64)), dict(top=4, out=torch.zeros(3, 2, 8, dtype=torch.int32)[:, :, ::2])):
        with pytest.raises((TypeError, ValueError)):
            mxq.SelectPagesNVFP4(q, keys_, *seqs, **over)
    with pytest.raises(ValueError, match="q must be"):
        mxq.SelectPagesNVFP4(q[..., :32], keys_, *seqs, top=4)
    for bad in (lists.long(), lists[:2], lists[:, :1], torch.zeros(3, 2, 8, dtype=torch.int32)[:, :, ::2]):
        with pytest.raises((TypeError, ValueError)):
            mxq.AttentionPagesNVFP4(q, cache, *seqs, bad)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        mxq.AttentionPagesNVFP4(q, cache, *seqs, lists, workspace=torch.zeros(512, dtype=torch.uint8)[::2])
    with pytest.raises(ValueError, match="as many rows as q"):
        mxq.AttentionPagesNVFP4(q, cache, *seqs, lists, out=torch.zeros(2, 4, 64, dtype=torch.bfloat16))
    for table, lens, starts in ((seqs[0].long(), *seqs[1:]), (seqs[0], seqs[1][:1], seqs[2]), (seqs[0], seqs[1], seqs[2][:2]),
                                (seqs[0].T.contiguous().T, *seqs[1:])):
        with pytest.raises((TypeError, ValueError)):
            mxq.SelectPagesNVFP4(q, keys_, table, lens, starts, top=4)
        with pytest.raises((TypeError, ValueError)):
            mxq.AttentionPagesNVFP4(q, cache, table, lens, starts, lists)


# ------------------------------------------------------------------ shared prefixes
def prefix(L, q=A, ld_q=1024, hq=8, total=4, out=A, ld_out=1024, lse=A, c=None, table=A, ld_table=5, table_pages=5, lens=A,
           starts=A, batch=3, groups_at=A, prefix_at=A, groups=2, max_q=2, max_prefix=40, max_own=40, scale=0.1, ws=A,
           ws_bytes=1 << 40):
    return L.mxq_attention_prefix_nvfp4(q, ld_q, hq, total, out, ld_out, lse, ctypes.byref(c or kv()), table, ld_table,
                                        table_pages, lens, starts, batch, groups_at, prefix_at, groups, max_q, max_prefix,
                                        max_own, scale, ws, ws_bytes, None)


@no_gpu
def test_attention_prefix_errors(L):
    assert prefix(L, total=0) == OK and prefix(L, max_q=0) == OK
    for over in (dict(total=-1), dict(hq=0), dict(hq=7), dict(batch=0), dict(groups=0), dict(groups=-1), dict(max_q=-1),
                 dict(max_prefix=-1), dict(max_own=-1), dict(table_pages=-1), dict(ld_table=4), dict(scale=0.0),
                 dict(scale=float("nan")), dict(scale=float("inf")), dict(ld_q=1016), dict(ld_out=1016), dict(q=None),
                 dict(out=None), dict(lens=None), dict(starts=None), dict(table=None), dict(groups_at=None),
                 dict(prefix_at=None), dict(ws=None), dict(c=kv(k_codes=None))):
        assert prefix(L, **over) == INVALID, over
    for over in (dict(ld_q=1028), dict(ld_out=1028), dict(q=A + 8), dict(out=A + 8), dict(lse=A + 2), dict(groups_at=A + 2),
                 dict(prefix_at=A + 1), dict(lens=A + 1), dict(starts=A + 2), dict(table=A + 2), dict(ws=A + 128)):
        assert prefix(L, **over) == MISALIGNED, over
    for over in (dict(batch=65536), dict(groups=4097), dict(total=1 << 28), dict(c=kv(head_dim=96)), dict(ld_q=1 << 40),
                 dict(ld_out=1 << 40), dict(max_q=1 << 31), dict(total=1 << 27, max_q=1 << 27, batch=65535)):
        assert prefix(L, **over) == UNSUPPORTED, over
    need = mxq.mxq_attention_prefix_nvfp4_workspace_size(8, 2, 128, 3, 2, 4, 2, 40, 40)
    assert need > 0 and need % 256 == 0
    assert prefix(L, ws_bytes=need - 1) == WS_SMALL


def test_attention_prefix_workspace_size(L):
    size = mxq.mxq_attention_prefix_nvfp4_workspace_size
    base = (8, 2, 128, 3, 2, 4, 2, 40, 40)
    assert size(*base) >= 2 * 4 * 8 * (128 * 2 + 8)                      # a part of each kind at least
    for i, v in ((0, 0), (1, 3), (2, 96), (3, 0), (3, 65536), (4, 0), (4, 4097), (5, 0), (5, 1 << 30), (6, 0), (7, -1), (8, -1)):
        assert size(*base[:i], v, *base[i + 1:]) == 0
    # no estimate, however large, plans more parts than a row's join takes
    for tokens in (1, 1 << 20, 1 << 40, (1 << 63) - 1):
        assert size(8, 2, 64, 1, 1, 1, 1, tokens, tokens) <= 512 * 8 * (64 * 2 + 8) + 255


def test_prefix_binding_checks():
    cache, _, q, seqs = cpu_case()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    good = (i32(0, 2), i32(4, 4), 2)
    with pytest.raises(ValueError, match="expected a GPU"):
        mxq.mxq_attention_prefix_nvfp4(q, cache, *seqs, *good)
    for bad in ((i32(0), i32(4, 4), 2), (i32(0, 2), i32(4), 2), (i32(0, 2).long(), i32(4, 4), 2), (i32(0, 2), i32(4, 4).float(), 2),
                (i32(0, 9, 2)[::2], i32(4, 4), 2), (i32(0, 2), i32(4, 4, 4)[::2], 2), ([0, 2], i32(4, 4), 2)):
        with pytest.raises((TypeError, ValueError)):
            mxq.AttentionPrefixNVFP4(q, cache, *seqs, *bad)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        mxq.AttentionPrefixNVFP4(q, cache, *seqs, *good, workspace=torch.zeros(512, dtype=torch.uint8)[::2])


@no_gpu
def test_prefix_rows_that_no_launch_joins(L):
    """A wave joins a query row and head, four a work-group: 2^26 of them are more threads than a
    launch holds, and the call is refused before anything is enqueued."""
    size = mxq.mxq_attention_prefix_nvfp4_workspace_size
    shape = dict(hq=64, ld_q=64 * 128, ld_out=64 * 128, c=kv(kv_heads=8, code_stride_page=8 * 16 * 64, scale_stride_page=8 * 16 * 8),
                 batch=1, groups=1, max_q=1)
    assert size(64, 8, 128, 1, 1, 1 << 20, 1, 40, 40) == 0
    assert size(64, 8, 128, 1, 1, (1 << 20) - 1, 1, 40, 40) > 0
    assert prefix(L, total=1 << 20, **shape) == UNSUPPORTED
    # one query head each, so every count can be had: 2^26 - 4 rows are 2^32 - 256 threads
    assert size(1, 1, 64, 1, 1, (1 << 26) - 4, 1, 40, 40) > 0
    for rows in range((1 << 26) - 3, (1 << 26) + 1):
        assert size(1, 1, 64, 1, 1, rows, 1, 40, 40) == 0

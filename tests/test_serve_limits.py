"""Limits of the serving calls on the host: shapes that a launch or a plan could not
hold, and tensors that the binding must not hand to a kernel.  The C calls get fake device
addresses, so they run where no GPU is visible."""
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests.test_serve_boundary import HIP, INVALID, MISALIGNED, UNSUPPORTED, WS_SMALL, A, L, attend, kv, no_gpu  # noqa: F401


def attend_wide(L, heads, batch, group=1):
    """One query for `batch` sequences of `heads` cached heads of 64."""
    c = kv(heads=heads, d=64, pages=1, c=(heads * 512, 512, 32), s=(heads * 64, 64, 4))
    return attend(L, ld_q=heads * group * 64, ld_out=heads * group * 64, hq=heads * group, tq=1, cache=c, b=batch, mq=1)


@no_gpu
@pytest.mark.parametrize("heads,batch", [(257, 65535), (1024, 16384), (32768, 65535), (65538, 65535), (131072, 32768),
                                         (131072, 32769)])
@pytest.mark.parametrize("group", [1, 20])
def test_units_past_a_launch_are_refused(L, heads, batch, group):
    """batch * kv_heads from 2^24 on, 2^31, 2^32 and a little past them (where 32 bits would
    wrap to no work-groups, or to a few): refused, and the size query asks for nothing."""
    assert heads * batch >= 1 << 24
    assert attend_wide(L, heads, batch, group) == UNSUPPORTED
    assert mxq.mxq_attention_nvfp4_workspace_size(heads * group, heads, 64, batch, 1, 1, 64) == 0


@no_gpu
def test_units_up_to_the_limit_reach_the_launch(L):
    assert attend_wide(L, 256, 65535) == HIP          # (which fails: there is no GPU)


# ------------------------------------------------------------------ the binding
def cpu_calls():
    """One prepared call of each kind on tensors in host memory."""
    cache = mxq.NVFP4KVCache.allocate(2, 16, 1, 64, 1.0, 1.0, device="cpu")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    ints = torch.arange(3, dtype=torch.int32)
    return [mxq.AddRMSNormFP8(x, torch.ones(256, dtype=torch.bfloat16)),
            mxq.RopeAppendNVFP4(q, q, q, ints[:2], ints[:2].long(), mxq.rope_plan(64, device="cpu"), cache),
            mxq.AttentionNVFP4(q, cache, ints[:2, None], ints[:2], ints, 1)]


@pytest.mark.parametrize("stream", [None, 0, 1 << 20])
def test_tensors_in_host_memory_are_refused(stream):
    """Before a stream is looked up or anything is enqueued: a kernel would read host addresses."""
    for call in cpu_calls():
        with pytest.raises(ValueError, match="GPU"):
            call(stream)


def attention_args(tokens=1, heads=4, pages=1):
    cache = mxq.NVFP4KVCache.allocate(2, 16, 1, 64, 1.0, 1.0, device="cpu")
    return (torch.zeros(tokens, heads, 64, dtype=torch.bfloat16), cache, torch.zeros(1, pages, dtype=torch.int32),
            torch.ones(1, dtype=torch.int32), torch.tensor([0, tokens], dtype=torch.int32), tokens)


def test_workspaces_with_gaps_or_repeats_are_refused():
    """Their element count is not the bytes behind the first one: the kernels would write past
    the end of a repeated byte, and into what lies between strided ones."""
    need = mxq.mxq_attention_nvfp4_workspace_size(4, 1, 64, 1, 1, 1, 1 << 20)
    assert need > 0
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            mxq.AttentionNVFP4(*attention_args(), max_seq_len=1 << 20, workspace=bad)
    mxq.AttentionNVFP4(*attention_args(), max_seq_len=1 << 20, workspace=torch.zeros(need, dtype=torch.uint8))


@no_gpu
def test_tables_that_could_hold_more_than_a_sequence(L):
    """The default length to plan for is what the table can hold, or the most that the library
    takes: 32769 pages of 65536 tokens are past it."""
    cache = mxq.NVFP4KVCache.allocate(1, 1 << 16, 1, 64, 1.0, 1.0, device="cpu")
    q, _, table, *rest = attention_args(pages=32769)
    call = mxq.AttentionNVFP4(q, cache, table, *rest)
    assert call.workspace is not None
    assert call._fn(*call._args, None) in (HIP, MISALIGNED)       # past the checks of shapes


@no_gpu
@pytest.mark.parametrize("residual", [False, True])
def test_one_row_has_no_stride(residual):
    """torch reports any stride for a dimension of one: a column seen transposed is a row."""
    column = torch.zeros(256, 1, dtype=torch.bfloat16)
    assert column.t().stride() == (1, 1)
    call = mxq.AddRMSNormFP8(column.t(), torch.ones(256, dtype=torch.bfloat16), column.t() if residual else None)
    assert call._fn(*call._args, None) == HIP


@no_gpu
def test_long_work_is_cut(L):
    """Few units over long contexts are cut, and then the workspace is checked."""
    q = mxq.mxq_attention_nvfp4_workspace_size
    for shape in [(64, 8, 128, 2, 2, 1, 262144), (32, 8, 128, 1, 512, 512, 65536), (8, 8, 64, 4, 16, 4, 100000),
                  (4, 2, 128, 2, 6, 3, 1 << 20)]:
        assert q(*shape) > 0, shape
    need = q(4, 2, 128, 2, 6, 3, 1 << 20)
    assert attend(L, ml=1 << 20, wsb=need) == HIP                 # taken, and no GPU to launch on
    assert attend(L, ml=1 << 20, wsb=need - 1) == WS_SMALL
    assert attend(L, ml=1 << 20, ws=None) == INVALID
    assert attend(L, ml=1 << 20, ws=A + 128) == MISALIGNED

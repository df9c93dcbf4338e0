"""Rows whose work is cut into parts, where few of many tokens add to an element: its sum is a small
number beside the row's other ones, and has to reach the output with no other rounding to fewer
bits than the last.

K is zero, so that all tokens weigh the same; V is zero but for the smallest number (0.5 * 2^-9)
in a few tokens, S of them for an element: out = S 2^-10 vg / tokens, lse = ln(tokens).

How far it may be off: every weight is the same 2^x (off by at most 2^-22, numerator and
denominator alike but for its rounding to FP16, which takes 512 (1 +- 2^-22) to 512); sums of up
to 2^10 tiles' equal numbers in FP32 by at most 2^10 2^-24 with their last 10 adds; the division, the tensor
scale and the join by fewer than 2^-20.  All of it is below 2^-13 of the value; then BF16's half
step, 2^-8 of it.  (context_util.attention_over allows parts rounded to FP16 too, a rounding that the
calls do not make.)"""
import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import context_util as cu
from tests import serve_util as su
from tests.gpu_util import announce, device, host
from tests.test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


def few_tokens(c, table, tokens):
    """V's smallest number in a few of the first `tokens` tokens of a row of the table; how many
    of them for each element."""
    c.kc[:], c.ks[:], c.vc[:], c.vs[:] = 0, 0x38, 0, 0x01
    count = 1 + np.arange(c.d) % 5
    for e, n in enumerate(count):
        for t in (977 * np.arange(n) + 31 * e) % tokens:
            c.vc[table[t // c.page], :, t % c.page, e // 2] |= 0x10 if e % 2 else 0x01
    return count


def check(c, r, count, tokens):
    """tokens: that each row of q sees."""
    out, lse = su.f32_of_bf16(r.out).astype(np.float64), host(r.lse)
    head_vg = np.repeat(c.vg.astype(np.float64), c.hq // c.hk)
    want = count * 2.0 ** -10 * head_vg[None, :, None] / tokens[:, None, None]
    off = np.abs(out - want) / want
    assert off.max() <= 2.0 ** -8 + 2.0 ** -13, f"off by {off.max():.5f}, at most {2.0 ** -8:.5f} allowed"
    assert np.abs(lse - np.log(tokens)[:, None]).max() <= 2.0 ** -12


@pytest.mark.parametrize("prefix,own,batch,nq,hq,d,page", [
    (58000, 1, 1, 1, 8, 64, 64),                                         # a wave a tile: 16 rows
    (58000, 3, 3, 1, 8, 128, 32),                                        # 32
    (58000, 1, 20, 1, 8, 64, 64),                                        # 128 rows of the prefix
    (5, 58000, 1, 1, 8, 128, 64),                                        # the sequence's own tokens
    (5, 58000, 1, 8, 24, 64, 16),                                        # 128 rows of them
])
def test_prefix(prefix, own, batch, nq, hq, d, page):
    dev = device()
    announce(f"small parts prefix={prefix} own={own} batch={batch} nq={nq} hq={hq} d={d} page={page}")
    c = Case([0, batch], [prefix] * batch, [prefix + own] * batch, [nq] * batch, hq, 1, d, page, seed=d, spare=1)
    count = few_tokens(c, c.table[0], 50000)
    r = c.prepared(dev, lse=True, max_prefix_len=1, max_own_len=1)()     # one part of each kind
    torch.cuda.synchronize()
    tokens = np.array([pos + 1.0 for _, _, pos in c.queries()])
    check(c, r, count, tokens)


@pytest.mark.parametrize("d,page", [(64, 64), (128, 16)])
def test_listed_pages(d, page):
    dev = device()
    announce(f"small parts of lists d={d} page={page}")
    c = cu.Sequences([61700], [256], 8, 1, d, page, seed=d, spare=1)
    count = few_tokens(c, c.table[0], 29000)                             # (all in the first part of two)
    top = -(-c.lens[0] // page)
    lists = torch.arange(top, dtype=torch.int32, device=dev).expand(c.total, 1, top).contiguous()
    call = mxq.AttentionPagesNVFP4(c.device_q(dev), c.device_cache(dev), *c.device_sequences(dev), lists, lse=True)
    assert call.workspace is not None
    r = call()
    torch.cuda.synchronize()
    check(c, r, count, np.array([pos + 1.0 for _, _, pos in c.queries()]))

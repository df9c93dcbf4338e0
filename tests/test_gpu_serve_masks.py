"""What must not reach a query of the attention over the NVFP4 cache, in every form of it: pages
shorter and longer than a tile, both head sizes, one and two column tiles of few rows and the
form for many, windows with and without first tokens, units of their own and cut ones (the
token then lies in a part that is not the first, so that a NaN has to come through the join)."""
import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import serve_util as su
from tests.gpu_util import announce, assert_same, device, host
from tests.test_gpu_serve import Case

pytestmark = pytest.mark.gpu


def case(page, d, nq, window, sinks):
    first = 1200 if window < 2000 else 4000
    return Case([first, 333], [nq, 1], 8, 2, d, page, window=window, sinks=sinks, seed=page + nq, spare=0)


def results(c, dev, cut):
    """max_seq_len only sizes the split: of one tile, none; long enough, units in several parts
    (few rows: shares of the line of 512 work-groups, of eight tiles here; many: of four)."""
    few = c.nq[0] * 4 <= 32
    call = c.run(dev, poison=False, max_seq_len=64 if not cut else 1 << 22 if few else c.lens[0])
    assert (call.workspace is not None) == cut
    r = call()
    torch.cuda.synchronize()
    return su.f32_of_bf16(r.out), host(r.lse)


def seeing(c, tokens):
    """Which of the first sequence's queries see one of the tokens."""
    p = np.arange(c.lens[0] - c.nq[0], c.lens[0])[:, None]
    t = np.asarray(tokens)[None]
    return ((t <= p) & ((c.window == 0) | (t > p - c.window) | (t < c.sinks))).any(1)


# 4 .. 160 query rows a cached head.  A short window leaves too few tiles to cut for few rows
FORMS = [(page, d, nq, window, sinks, cut) for page in (16, 32, 64, 128) for d in (64, 128) for nq in (1, 3, 7, 40)
         for window, sinks, cut in ((0, 0, False), (0, 0, True), (200, 5, False), (200, 5, True))
         if not (cut and window and nq < 9)]
FORMS += [(page, d, nq, 2600, 5, True) for page in (16, 64) for d in (64, 128) for nq in (1, 7)]


@pytest.mark.parametrize("page,d,nq,window,sinks,cut", FORMS)
def test_nan_rows_and_blocks(page, d, nq, window, sinks, cut):
    """A NaN block scale in K makes the rows that see its token NaN (and their log-sums), in V
    that block of 16 elements; every other bit is as without it."""
    dev = device()
    announce(f"NaN page={page} d={d} nq={nq} window={window} sinks={sinks} cut={cut}")
    clean, clean_lse = results(case(page, d, nq, window, sinks), dev, cut)
    assert np.isfinite(clean).all() and np.isfinite(clean_lse).all()
    n = case(page, d, nq, window, sinks).lens[0]
    # in a later part, before every window, among the first tokens, the first query's own one
    # and (for several queries) the last's
    for at in sorted({n - 100, 600, 3, n - nq, n - 1}):
        for which in "kv":
            c = case(page, d, nq, window, sinks)
            seen = seeing(c, [at])
            block = 1 if d == 64 else 5
            (c.ks if which == "k" else c.vs)[c.table[0, at // page], 1, at % page, block] = 0x7F if at & 1 else 0xFF
            out, lse = results(c, dev, cut)
            what = f"{which} token {at}"
            assert_same(what + ": the other cached head", out[:, :4], clean[:, :4])
            assert_same(what + ": the other sequence", out[nq:], clean[nq:])
            assert_same(what + ": unseen", out[:nq][~seen], clean[:nq][~seen])
            assert_same(what + ": unseen, log-sums", lse[:nq][~seen], clean_lse[:nq][~seen])
            if which == "k":
                assert np.isnan(out[:nq][seen][:, 4:]).all(), what
                assert np.isnan(lse[:nq][seen][:, 4:]).all(), what
            else:
                assert np.isnan(out[:nq][seen][:, 4:, 16 * block:16 * block + 16]).all(), what
                assert_same(what + ": log-sums", lse, clean_lse)


@pytest.mark.parametrize("page,d,nq,window,sinks,cut", FORMS)
def test_bad_pages(page, d, nq, window, sinks, cut):
    """A page number outside the cache: rows that see one of its tokens are NaN, every other bit
    is as without it."""
    dev = device()
    announce(f"bad page, page={page} d={d} nq={nq} window={window} sinks={sinks} cut={cut}")
    clean, _ = results(case(page, d, nq, window, sinks), dev, cut)
    n = case(page, d, nq, window, sinks).lens[0]
    for at, number in ((n - 100, -1), (600, 1 << 30), (3, None), (n - 1, -(1 << 31))):
        c = case(page, d, nq, window, sinks)
        first = at // page * page
        seen = seeing(c, range(first, min(first + page, n)))
        c.table[0, at // page] = c.kc.shape[0] if number is None else number
        out, lse = results(c, dev, cut)
        what = f"page of token {at}"
        assert np.isnan(out[:nq][seen]).all() and np.isnan(lse[:nq][seen]).all(), what
        assert_same(what + ": unseen", out[:nq][~seen], clean[:nq][~seen])
        assert_same(what + ": the other sequence", out[nq:], clean[nq:])


def test_what_lies_between_rows_of_q_stays_out():
    """Q inside a wider buffer whose other columns are NaN and infinite: no bit of the output
    depends on them, and the buffer is as it was."""
    dev = device()
    for d, nq in ((64, 1), (128, 3), (128, 40), (64, 40)):
        announce(f"between rows of q d={d} nq={nq}")
        c = Case([170, 33], [nq, 1], 4, 2, d, 16, seed=3)
        call = c.run(dev)
        plain = call()
        rows, width = nq + 1, 4 * d
        wide = torch.full((rows, width + 64), float("nan"), dtype=torch.bfloat16, device=dev)
        wide[:, width:width + 32] = float("inf")
        wide[:, 16:16 + width] = c.q.to(dev).flatten(1)
        before = wide.clone()
        r = mxq.mxq_attention_nvfp4(wide[:, 16:16 + width].unflatten(1, (4, d)), call._cache,
                                    torch.from_numpy(c.table).to(dev), torch.tensor(c.lens, dtype=torch.int32, device=dev),
                                    torch.from_numpy(c.starts).to(dev), nq, 170, lse=True)
        torch.cuda.synchronize()
        assert torch.equal(r.out, plain.out) and torch.equal(r.lse, plain.lse)
        assert torch.equal(wide.view(torch.int16), before.view(torch.int16))

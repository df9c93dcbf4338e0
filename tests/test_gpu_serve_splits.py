"""Attention over the paged NVFP4 cache: the ways the work is spread over the chip, against
64 bits.  max_seq_len only sizes that split, so each case runs with a bound of one tile (a
work-group per sequence and cached head) and with one far past its lengths (work-groups that
share all tiles, cut units and their join)."""
import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests.gpu_util import announce, device
from tests.test_gpu_serve import Case

pytestmark = pytest.mark.gpu

RNG = np.random.default_rng(77)
SHORT = [int(n) for n in RNG.integers(0, 140, 300)]

CASES = {
    "rows first, pages of 64": dict(lens=[300, 64, 1], nq=[1, 1, 1], hq=8, hk=2, d=128, page=64, rows_first=True),
    "rows first, pages of 128, drafts": dict(lens=[300, 129], nq=[5, 2], hq=8, hk=2, d=128, page=128, rows_first=True),
    "rows first, d64": dict(lens=[300, 64, 700], nq=[1, 4, 3], hq=8, hk=2, d=64, page=64, rows_first=True),
    "rows first, prompt": dict(lens=[200, 90], nq=[90, 90], hq=4, hk=2, d=64, page=64, rows_first=True),
    "pages of 64, group 24": dict(lens=[700, 64, 65], nq=[1, 1, 1], hq=24, hk=1, d=128, page=64),
    "pages of 128, d64, group 5 drafts": dict(lens=[513, 128, 4], nq=[5, 5, 4], hq=10, hk=2, d=64, page=128),
    "pages of 64, d64": dict(lens=[64, 63, 500], nq=[1, 1, 1], hq=8, hk=1, d=64, page=64),
    "pages of 32, group 17": dict(lens=[333, 32, 31], nq=[1, 1, 1], hq=17, hk=1, d=128, page=32),
    "one long among short": dict(lens=SHORT[:100] + [9000] + SHORT[100:160], nq=[1] * 161, hq=2, hk=1, d=128, page=64),
    "two long, drafts": dict(lens=[5000, 20, 7000, 1], nq=[3, 2, 3, 3], hq=8, hk=1, d=64, page=16),
    "without queries between": dict(lens=SHORT, nq=[int(n % 3 != 1) for n in range(300)], hq=4, hk=2, d=64, page=16),
    "first and last empty": dict(lens=[0, 0, 500, 0, 700, 0], nq=[1, 0, 1, 1, 1, 0], hq=8, hk=2, d=128, page=64),
    "windows": dict(lens=[n * 9 for n in SHORT[:40]], nq=[1] * 40, hq=4, hk=2, d=128, page=16, window=200, sinks=4),
    "sinks alone": dict(lens=[300, 80], nq=[1, 5], hq=4, hk=2, d=64, page=16, sinks=70),
    "window past everything": dict(lens=[300, 80], nq=[2, 40], hq=4, hk=2, d=64, page=16, window=(1 << 31) - 1,
                                   sinks=(1 << 31) - 1),
    "sinks in the window's tile": dict(lens=[170, 140], nq=[1, 30], hq=4, hk=2, d=128, page=64, window=50, sinks=100),
    "chunks in three parts": dict(lens=[520], nq=[256], hq=32, hk=16, d=64, page=64),
    "chunks in many parts": dict(lens=[4000], nq=[9], hq=8, hk=2, d=128, page=16),
}


@pytest.mark.parametrize("name", list(CASES))
def test_both_splits(name):
    dev = device()
    c = Case(seed=len(name), **CASES[name])
    for bound in (64, 1 << 22):
        announce(f"splits {name} {bound}")
        r = c.run(dev, max_seq_len=bound)()
        torch.cuda.synchronize()
        c.check(r)


def test_more_units_than_the_line_takes():
    dev = device()
    announce("1100 sequences")
    c = Case([n % 97 for n in range(1100)], [1] * 1100, 2, 1, 64, 16, seed=3)
    r = c.run(dev, max_seq_len=1 << 22)()
    torch.cuda.synchronize()
    c.check(r)


def test_two_streams_at_once():
    """Two prepared calls, each with its own workspace, in flight together and in turns."""
    dev = device()
    cases = [Case([3000, 100], [1, 1], 8, 2, 128, 64, seed=1), Case([2500, 900, 10], [2, 1, 3], 8, 2, 64, 16, seed=2),
             Case([1500], [30], 8, 2, 128, 64, seed=3)]
    calls = [c.run(dev) for c in cases]
    want = []
    for call in calls:
        r = call()
        torch.cuda.synchronize()
        want.append((r.out.clone(), r.lse.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for call in calls:
            call.out.out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for call, s in zip(calls, streams):
                call(s)
        torch.cuda.synchronize()
        for call, (o, l) in zip(calls, want):
            assert torch.equal(call.out.out, o) and torch.equal(call.out.lse, l)


def test_cache_without_pages():
    """No page can be read, so every sequence is empty: zeros, and a lse of -inf."""
    dev = device()
    for nq in (1, 40):
        announce(f"no pages, {nq} queries")
        cache = mxq.NVFP4KVCache.allocate(0, 64, 2, 128, 1.0, 1.0, device=dev)
        q = torch.ones(nq, 8, 128, dtype=torch.bfloat16, device=dev)
        r = mxq.mxq_attention_nvfp4(q, cache, torch.zeros(1, 9, dtype=torch.int32, device=dev),
                                    torch.tensor([500], dtype=torch.int32, device=dev),
                                    torch.tensor([0, nq], dtype=torch.int32, device=dev), nq, 5000, lse=True)
        torch.cuda.synchronize()
        assert not r.out.any() and bool(torch.isneginf(r.lse).all())


def test_graph_of_cut_units():
    """A captured call whose work-groups cut units, replayed while the lengths grow, with eager
    calls of another workspace between."""
    dev = device()
    c = Case([3000, 40, 2000], [1, 1, 1], 8, 2, 128, 64, seed=5)
    call, other = c.run(dev, poison=False, max_seq_len=4000), c.run(dev, poison=False, max_seq_len=4000)
    lens, other_lens = call._tensors[4], other._tensors[4]
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        for t in (lens, other_lens):
            t.copy_(torch.tensor([2900 + 20 * i, 40 - i, 1000 + 300 * i], dtype=torch.int32))
        r = other()
        torch.cuda.synchronize()
        call.out.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out.out, r.out) and torch.equal(call.out.lse, r.lse), f"replay {i}"


def test_one_prompt_in_a_wide_batch():
    """One run of 8192 queries among single ones: most of the row tiles that the widths allow
    for hold nothing (batch * row tiles * heads = 2^17 of them)."""
    dev = device()
    announce("wide batch")
    rng = np.random.default_rng(6)
    cache = mxq.NVFP4KVCache.allocate(8, 64, 8, 64, 1.0, 1.0, device=dev)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape, dtype=np.uint8)))
    cache.k_scales.fill_(0x38)
    cache.v_scales.fill_(0x38)
    batch, run = 64, 8192
    q = torch.from_numpy(rng.standard_normal((run + batch - 1, 32, 64), dtype=np.float32)).bfloat16().to(dev)
    table = torch.arange(batch, dtype=torch.int32, device=dev)[:, None] % 8
    lens = torch.full((batch,), 64, dtype=torch.int32, device=dev)
    starts = torch.tensor([0] + [run + i for i in range(batch)], dtype=torch.int32, device=dev)
    r = mxq.mxq_attention_nvfp4(q, cache, table, lens, starts, run, 64, lse=True)
    alone = mxq.mxq_attention_nvfp4(q[run - 64:run], cache, table[:1], lens[:1],
                                    torch.tensor([0, 64], dtype=torch.int32, device=dev), 64, 64, lse=True)
    torch.cuda.synchronize()
    assert not r.out[:run - 64].any() and bool(torch.isneginf(r.lse[:run - 64]).all())
    assert torch.equal(r.out[run - 64:run], alone.out) and torch.equal(r.lse[run - 64:run], alone.lse)
    singles = mxq.mxq_attention_nvfp4(q[run:], cache, table[1:], lens[1:],
                                      torch.arange(batch, dtype=torch.int32, device=dev), 40, 64)
    torch.cuda.synchronize()
    assert torch.equal(r.out[run:], singles.out)


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("kg", [2.0 ** -126, 2.0 ** -60, 2.0 ** 100])
def test_extreme_tensor_scales(nq, kg):
    """Queries of zeros and of tiny and huge elements under K scales at the ends of their range:
    masked scores stay masked, whatever the factor on them comes to."""
    dev = device()
    announce(f"extreme scales {nq} {kg}")
    c = Case([100, 70], [nq, nq], 4, 2, 64, 16, seed=9)
    c.kg[:] = kg
    amp = torch.tensor([0.0, 2.0 ** -110, 1.0, 2.0 ** -60])[:, None]
    c.q = (c.q.float() * amp * (2.0 ** -100 if kg > 1 else 1.0)).bfloat16()
    r = c.run(dev)()
    torch.cuda.synchronize()
    c.check(r)


@pytest.mark.parametrize("nq", [1, 40])
def test_smallest_v_scale(nq):
    """V's tensor scale at the smallest normal number, many tokens: the output keeps its bits."""
    dev = device()
    announce(f"smallest v scale {nq}")
    c = Case([190], [nq], 4, 2, 128, 16, seed=11)
    plain = c.run(dev)()
    ratio = (c.vg.astype(np.float64) / 2.0 ** -126)
    c.vg[:] = 2.0 ** -126
    r = c.run(dev)()
    torch.cuda.synchronize()
    scale = torch.from_numpy(np.repeat(ratio, 2))[None, :, None].to(dev)
    want, got = plain.out.double(), r.out.double() * scale
    # two roundings to BF16 (2^-8 each) and FP32 ones far below; an output under 2^-126 is
    # subnormal, off by at most half of BF16's smallest step: 2^-134, brought up by `scale`
    assert bool(((got - want).abs() <= 2.0 ** -6.9 * want.abs() + 2.0 ** -134 * scale).all())

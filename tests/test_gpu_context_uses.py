"""The calls for long and shared contexts in ways their own tests leave out: caches and mean keys
past 32-bit offsets, calls of different graphs that share a workspace, and calls on two streams
at once.  All compare with the same call made alone, bit for bit."""
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import context_util as cu
from tests.gpu_util import announce, device
from tests.test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


def i32(dev, *v):
    return torch.tensor(v, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("nq", [1, 40])
def test_past_4_gib(nq):
    """The same pages at the far end of a cache whose mean keys alone are past 4 GiB (K and V are
    the same storage here: 34 GiB of codes, 4 of scales)."""
    dev = device()
    if torch.cuda.get_device_properties(0).total_memory < 96 << 30:
        pytest.skip("needs 48 GiB")
    announce(f"past 4 GiB nq={nq}")
    hk, page, d = 2, 16, 128
    c = cu.Sequences([700, 650], [nq, nq], 4, hk, d, page, seed=nq, spare=0)
    c.table = c.table % c.pages
    far_pages = (1 << 32) // (hk * d) + 4096
    codes = torch.empty((far_pages, hk, page, d // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((far_pages, hk, page, d // 16), dtype=torch.uint8, device=dev)
    key_codes = torch.empty((far_pages, hk, d), dtype=torch.int8, device=dev)
    key_scales = torch.empty((far_pages, hk), dtype=torch.float32, device=dev)
    g = torch.from_numpy(c.kg).to(dev)
    near_kv = [torch.from_numpy(x).to(dev) for x in (c.kc, c.ks)]
    codes[-c.pages:], scales[-c.pages:] = near_kv
    assert (far_pages - c.pages) * hk * d > 1 << 32

    def results(kc, ks, keys, first_page):
        cache = mxq.NVFP4KVCache(kc, ks, kc, ks, g, g)
        q, (table, lens, starts) = c.device_q(dev), c.device_sequences(dev)
        table += first_page
        slots = torch.arange(c.pages, device=dev) * page + page - 1 + first_page * page
        mxq.mxq_page_keys_nvfp4(cache, slots, keys)
        select = mxq.mxq_select_pages_nvfp4(q, keys, table, lens, starts, top=9)
        over_pages = mxq.mxq_attention_pages_nvfp4(q, cache, table, lens, starts, select, lse=True)
        shared = mxq.mxq_attention_prefix_nvfp4(q, cache, table, lens, starts, i32(dev, 0, 2), i32(dev, 600, 600), nq, lse=True)
        torch.cuda.synchronize()
        return [keys.codes[first_page:first_page + c.pages], keys.scales[first_page:first_page + c.pages], select,
                over_pages.out, over_pages.lse, shared.out, shared.lse]

    near_keys = mxq.PageKeys(torch.zeros((c.pages, hk, d), dtype=torch.int8, device=dev),
                             torch.zeros((c.pages, hk), dtype=torch.float32, device=dev), page)
    near = results(*near_kv, near_keys, 0)
    far = results(codes, scales, mxq.PageKeys(key_codes, key_scales, page), far_pages - c.pages)
    assert all(torch.isfinite(x).all() for x in near if x.is_floating_point())
    for what, a, b in zip(("codes", "scales", "pages", "out", "lse", "shared out", "shared lse"), near, far):
        assert torch.equal(a, b), what


def calls(dev, workspaces):
    """Prepared calls of different sizes that all cut their rows, over sequences of their own."""
    a = Case([0, 4], [900] * 4, [1000, 930, 1200, 905], [1] * 4, 16, 2, 128, 64, seed=1)
    b = cu.Sequences([3000], [1], 8, 2, 128, 16, seed=2)
    e = Case([0, 40], [1000] * 40, [1003 + 7 * i for i in range(40)], [1] * 40, 16, 1, 64, 16, seed=3)
    lists = torch.from_numpy(cu.random_lists(b, 100)).to(dev)
    keys = mxq.PageKeys(torch.randint(-127, 128, (b.pages, 2, 128), dtype=torch.int8, device=dev,
                                      generator=torch.Generator(device=dev).manual_seed(5)),
                        torch.ones((b.pages, 2), device=dev), 16)
    kw = lambda i: {} if workspaces is None else dict(workspace=workspaces[i])
    return [a.prepared(dev, lse=True, **kw(0)),
            mxq.AttentionPagesNVFP4(b.device_q(dev), b.device_cache(dev), *b.device_sequences(dev), lists, lse=True, **kw(1)),
            e.prepared(dev, lse=True, **kw(2)),
            mxq.SelectPagesNVFP4(b.device_q(dev), keys, *b.device_sequences(dev), top=30, max_seq_len=1 << 18, **kw(3))]


def outputs(call):
    return [call.out] if isinstance(call.out, torch.Tensor) else [call.out.out, call.out.lse]


def alone(dev):
    """Each call's outputs, made alone, and its workspace's size."""
    made = calls(dev, None)
    assert all(x.workspace is not None for x in made)
    for x in made:
        x()
        torch.cuda.synchronize()
    return [[t.clone() for t in outputs(x)] for x in made], [x.workspace.numel() for x in made]


def test_graphs_that_share_a_workspace():
    """A graph per call, one workspace: replayed in any order, with other work between."""
    dev = device()
    announce("graphs that share a workspace")
    want, sizes = alone(dev)
    workspace = torch.full((max(sizes),), 0xFF, dtype=torch.uint8, device=dev)
    made, graphs = calls(dev, [workspace] * 4), []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in made:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                x()
            graphs.append(graph)
    torch.cuda.current_stream().wait_stream(side)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (2, 2, 0, 3), (1, 3, 0, 2)):
        for x in made:
            for t in outputs(x):
                t.fill_(-7)
        for i in order:
            graphs[i].replay()
        made[order[0]]()                                                 # and one made eagerly behind them
        torch.cuda.synchronize()
        for i in set(order):
            for a, b in zip(outputs(made[i]), want[i]):
                assert torch.equal(a, b), (order, i)
        workspace.fill_(0xFF)


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams, many behind one another."""
    dev = device()
    announce("two streams at once")
    want, _ = alone(dev)
    made = calls(dev, None)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for i, x in enumerate(made):
            x(streams[i % 2])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for i, x in enumerate(made):
        for a, b in zip(outputs(x), want[i]):
            assert torch.equal(a, b), i

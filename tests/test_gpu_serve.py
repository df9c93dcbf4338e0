"""The serving operators on the GPU against plain 64-bit forms (tests/serve_util.py):
the norm and the append byte for byte, the attention within bounds counted from its
roundings (serve_util.attention_bounds)."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import serve_util as su
from tests.gpu_util import announce, assert_same, device, host

pytestmark = pytest.mark.gpu


def bf16(rng, *shape, amp=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * amp).astype(np.float32)).bfloat16()


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("m,n,res,options,y,transposed", [
    (1, 128, False, 0, False, False),
    (3, 384, True, 0, True, False),
    (5, 7168, True, 0, True, True),
    (2, 8192, False, 1, True, False),
    (3, 8320, True, 1, False, True),            # just past one chunk a thread
    (2, 16384, True, 0, True, False),
    (2, 32768, True, 0, False, False),          # the widest row
    (700, 640, True, 0, True, False),
    (1300, 4096, True, 0, True, False),
])
def test_norm(m, n, res, options, y, transposed):
    dev = device()
    announce(f"norm {m}x{n} res={res} options={options} y={y} transposed={transposed}")
    rng = np.random.default_rng(m * 7 + n)
    x, w = bf16(rng, m, n), bf16(rng, n) + 1
    r = bf16(rng, m, n, amp=3.0) if res else None
    got = mxq.mxq_add_rmsnorm_quant_fp8(x.to(dev), w.to(dev), r.to(dev) if res else None, 1e-5, options, y, transposed)
    torch.cuda.synchronize()
    rows = np.unique(np.linspace(0, m - 1, min(m, 40)).astype(int))
    z, yy, codes, scales = su.norm_reference(su.f32_of_bf16(x)[rows], su.f32_of_bf16(r)[rows] if res else None,
                                             su.f32_of_bf16(w), 1e-5, options)
    assert_same("q", host(got.q)[rows], codes)
    assert_same("scales", (host(got.scales).T if transposed else host(got.scales))[rows], scales)
    if res:
        assert_same("residual", su.f32_of_bf16(got.residual)[rows], z)
    if y:
        assert_same("y", su.f32_of_bf16(got.y)[rows], su.to_bf16(yy))


def test_norm_strides_and_in_place():
    """Rows inside wider buffers, the residual updated in place, and the same through the
    sum buffer x itself; rows and columns around them stay as they were."""
    dev = device()
    rng = np.random.default_rng(5)
    m, n, wide = 37, 512, 800
    xb, rb = bf16(rng, m, wide).to(dev), bf16(rng, m, wide).to(dev)
    w = bf16(rng, n).to(dev)
    x, r = xb[:, 8:8 + n], rb[:, 16:16 + n]
    before = rb.clone()
    z, _, codes, scales = su.norm_reference(su.f32_of_bf16(x), su.f32_of_bf16(r), su.f32_of_bf16(w), 1e-6, 0)
    got = mxq.mxq_add_rmsnorm_quant_fp8(x, w, r, residual_out=r)
    torch.cuda.synchronize()
    assert_same("q", host(got.q), codes)
    assert_same("scales", host(got.scales), scales)
    assert_same("residual", su.f32_of_bf16(rb[:, 16:16 + n]), z)
    assert torch.equal(rb[:, :16], before[:, :16]) and torch.equal(rb[:, 16 + n:], before[:, 16 + n:])
    rb.copy_(before)
    got = mxq.mxq_add_rmsnorm_quant_fp8(x, w, r, residual_out=x)
    torch.cuda.synchronize()
    assert_same("q (into x)", host(got.q), codes)
    assert_same("residual (into x)", su.f32_of_bf16(x), z)


def test_norm_special_values():
    """Zero rows, tiny and huge values, NaN and infinities: the stated steps give what they
    give (eps alone under a zero row; NaN codes 0x7F; a row with an infinity has r = 0)."""
    dev = device()
    n = 256
    x = torch.zeros(8, n)
    x[1] = 1e-30
    x[2] = torch.linspace(-3e38, 3e38, n)
    x[3] = torch.linspace(-1, 1, n)
    x[3, 5] = float("nan")
    x[4] = 1.0
    x[4, 200] = float("inf")
    x[5, 7] = -1.5
    x[6] = torch.linspace(1e-20, 1e-18, n)
    x[7] = -0.0
    x = x.bfloat16()
    w = torch.linspace(-2, 2, n).bfloat16()
    for eps in (1e-6, 0.0):
        got = mxq.mxq_add_rmsnorm_quant_fp8(x.to(dev), w.to(dev), None, eps, out_bf16=True)
        torch.cuda.synchronize()
        _, y, codes, scales = su.norm_reference(su.f32_of_bf16(x), None, su.f32_of_bf16(w), eps, 0)
        assert_same("q", host(got.q), codes)
        assert_same("scales", host(got.scales), scales)
        a, b = su.f32_of_bf16(got.y), su.to_bf16(y)
        assert np.array_equal(np.isnan(a), np.isnan(b))
        assert_same("y", np.where(np.isnan(a), 0, a), np.where(np.isnan(b), 0, b))


# ------------------------------------------------------------------ rotary append
def paged(rng, pages, hk, page, d, dev, rows_first=False):
    """A cache of known bytes; rows_first: [pages][page][heads] order, seen transposed."""
    t = []
    for width in (d // 2, d // 16) * 2:
        shape = (pages, page, hk, width) if rows_first else (pages, hk, page, width)
        b = torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).to(dev)
        t.append(b.transpose(1, 2) if rows_first else b)
    kg = torch.from_numpy((0.5 + rng.random(hk)).astype(np.float32) * 5 / 2688)
    vg = torch.from_numpy((0.5 + rng.random(hk)).astype(np.float32) * 5 / 2688)
    return mxq.NVFP4KVCache(t[0], t[1], t[2], t[3], kg.to(dev), vg.to(dev))


@pytest.mark.parametrize("t,hq,hk,d,rot,inter,page,rows_first,far", [
    (1, 8, 1, 128, 128, False, 16, False, 10),
    (7, 4, 2, 64, 64, True, 16, False, 5000),
    (33, 5, 5, 64, 16, False, 32, True, 1000000),
    (50, 12, 4, 128, 64, True, 64, False, 2147483647),
    (19, 0, 3, 128, 96, False, 16, True, 131072),     # K and V alone; 96 of 128 rotated
    (130, 3, 1, 64, 0, False, 128, False, 77),        # nothing rotated
    (2100, 2, 1, 64, 32, True, 64, False, 400000),
])
def test_append(t, hq, hk, d, rot, inter, page, rows_first, far):
    dev = device()
    announce(f"append t={t} hq={hq} hk={hk} d={d} rot={rot} inter={inter} page={page} far={far}")
    rng = np.random.default_rng(t * 31 + d + rot)
    pages = -(-t // page) + 3
    cache = paged(rng, pages, hk, page, d, dev, rows_first)
    before = [host(x).copy() for x in cache.tensors()[:4]]
    qkv = bf16(rng, t, (hq + 2 * hk) * d + 16, amp=1.5)
    pos = rng.integers(0, far, t, dtype=np.int64).astype(np.int32)
    pos[0] = far - 1
    slots = rng.permutation(pages * page)[:t].astype(np.int64)
    slots[rng.random(t) < 0.15] = -1
    if t > 3:
        slots[2] = pages * page + 5                   # past the cache: padding too
    plan = mxq.rope_plan(rot, interleaved=inter, scaling="ramp" if rot else "none", scale=4.0 if rot else 1.0,
                         trained_length=4096, device=dev)
    dq = qkv.to(dev)
    q = dq[:, :hq * d].unflatten(1, (hq, d)) if hq else None
    k = dq[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    v = dq[:, (hq + hk) * d:(hq + 2 * hk) * d].unflatten(1, (hk, d))
    got = mxq.mxq_rope_append_nvfp4(q, k, v, torch.from_numpy(pos).to(dev), torch.from_numpy(slots).to(dev), plan, cache,
                                    values=True)
    torch.cuda.synchronize()
    f = host(plan.inv_freq)
    kk = su.rope_reference(su.f32_of_bf16(k), pos, f, plan.factor, inter)
    vv = su.f32_of_bf16(v)
    if hq:
        assert_same("q", su.f32_of_bf16(got.q), su.rope_reference(su.f32_of_bf16(q), pos, f, plan.factor, inter))
    keep = (slots >= 0) & (slots < pages * page)
    for name, y, g, ci, si, values in (("k", kk, cache.k_global, 0, 1, got.k_values),
                                       ("v", vv, cache.v_global, 2, 3, got.v_values)):
        gh = host(g)
        codes, scales = su.encode_rows(y, gh)
        before[ci][slots[keep] // page, :, slots[keep] % page] = codes[keep]
        before[si][slots[keep] // page, :, slots[keep] % page] = scales[keep]
        assert_same(name + " codes", host(cache.tensors()[ci]), before[ci])
        assert_same(name + " scales", host(cache.tensors()[si]), before[si])
        want = su.to_bf16(su.decode_rows(codes, scales).astype(np.float32) * gh[None, :, None])
        assert_same(name + " values", su.f32_of_bf16(values), want)


def test_append_special_values():
    """NaN and infinite K / V blocks, zero blocks, values far above and below what the
    tensor scale was calibrated for."""
    dev = device()
    rng = np.random.default_rng(3)
    t, hk, d, page = 6, 2, 64, 16
    k, v = bf16(rng, t, hk, d), bf16(rng, t, hk, d)
    k[0, 0, 3] = float("nan")
    v[1, 1, 40] = float("inf")
    v[2] = 0
    k[3, 1] *= 1e6
    k[4, 0] *= 1e-6
    v[5, 0, :16] = -0.0
    cache = paged(rng, 2, hk, page, d, dev)
    pos = np.zeros(t, np.int32)
    plan = mxq.rope_plan(32, device=dev)
    got = mxq.mxq_rope_append_nvfp4(None, k.to(dev), v.to(dev), torch.from_numpy(pos).to(dev),
                                    torch.arange(t, device=dev), plan, cache, values=True)
    torch.cuda.synchronize()
    for name, y, g, c, s, val in (("k", k, cache.k_global, cache.k_codes, cache.k_scales, got.k_values),
                                  ("v", v, cache.v_global, cache.v_codes, cache.v_scales, got.v_values)):
        yy = su.f32_of_bf16(y)
        if name == "k":
            yy = su.rope_reference(yy, pos, host(plan.inv_freq), 1.0, False)
        codes, scales = su.encode_rows(yy, host(g))
        assert_same(name + " codes", host(c)[0, :, :t].transpose(1, 0, 2), codes)
        assert_same(name + " scales", host(s)[0, :, :t].transpose(1, 0, 2), scales)
        with np.errstate(invalid="ignore"):
            want = su.to_bf16(su.decode_rows(codes, scales).astype(np.float32) * host(g)[None, :, None])
        a = su.f32_of_bf16(val)
        assert np.array_equal(np.isnan(a), np.isnan(want))
        assert_same(name + " values", np.where(np.isnan(a), 0, a), np.where(np.isnan(want), 0, want))


def test_append_q_in_place():
    dev = device()
    rng = np.random.default_rng(9)
    for inter in (False, True):
        q, k = bf16(rng, 40, 6, 128).to(dev), bf16(rng, 40, 1, 128).to(dev)
        cache = paged(rng, 3, 1, 16, 128, dev)
        pos = torch.arange(40, dtype=torch.int32, device=dev) * 999
        slots = torch.arange(40, device=dev)
        plan = mxq.rope_plan(128, interleaved=inter, device=dev)
        want = mxq.mxq_rope_append_nvfp4(q, k, k, pos, slots, plan, cache).q.clone()
        got = mxq.mxq_rope_append_nvfp4(q, k, k, pos, slots, plan, cache, q_out=q).q
        torch.cuda.synchronize()
        assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


# ------------------------------------------------------------------ attention
class Case:
    def __init__(self, lens, nq, hq, hk, d, page, window=0, sinks=0, seed=0, q_amp=1.0, rows_first=False, spare=2,
                 behind=0):
        rng = np.random.default_rng(seed * 1009 + d + page + hq)
        self.lens, self.nq, self.window, self.sinks, self.d, self.page = lens, nq, window, sinks, d, page
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        (self.kc, self.ks, self.kg), (self.vc, self.vs, self.vg) = su.random_cache(rng, pages, hk, page, d)
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.q = bf16(rng, int(self.starts[-1]) + behind, hq, d, amp=q_amp)
        self.rows_first = rows_first

    def run(self, dev, lse=True, max_seq_len=None, poison=True, out=None, **kw):
        t = [torch.from_numpy(x.copy()) for x in (self.kc, self.ks, self.vc, self.vs)]
        if poison:                                    # rows past a sequence's end hold NaN scales
            used = np.zeros((self.kc.shape[0], self.page), bool)
            for b, n in enumerate(self.lens):
                for i in range(n):
                    used[self.table[b, i // self.page], i % self.page] = True
            for x in (t[1], t[3]):
                x.transpose(1, 2)[torch.from_numpy(~used)] = 0x7F
        if self.rows_first:
            t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in t]
        cache = mxq.NVFP4KVCache(*[x.to(dev) if not self.rows_first else x.transpose(1, 2).to(dev).transpose(1, 2)
                                   for x in t], torch.from_numpy(self.kg).to(dev), torch.from_numpy(self.vg).to(dev))
        call = mxq.AttentionNVFP4(self.q.to(dev), cache, torch.from_numpy(self.table).to(dev),
                                  torch.tensor(self.lens, dtype=torch.int32, device=dev),
                                  torch.from_numpy(self.starts).to(dev), max(max(self.nq), 1),
                                  max(self.lens) if max_seq_len is None else max_seq_len, window=self.window,
                                  sinks=self.sinks, lse=lse, out=out, **kw)
        if call.workspace is not None:
            call.workspace.fill_(0xFF)                # any contents
        return call

    def check(self, r, rows=None):
        want, lse, bo, bl = su.attention_reference(
            su.f32_of_bf16(self.q), self.kc, self.ks, self.vc, self.vs, self.kg, self.vg, self.table, self.lens,
            self.starts, 1.0 / math.sqrt(self.d), self.window, self.sinks)
        n = int(self.starts[-1])
        bo, bl = bo[:n], bl[:n]
        got = su.f32_of_bf16(r.out)[:n].astype(np.float64)
        off = np.abs(got - want[:n])
        bad = np.argwhere(~(off <= bo))
        assert not len(bad), f"out: {len(bad)} of {off.size}, first {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"
        if r.lse is not None:
            g = host(r.lse)[:n].astype(np.float64)
            empty = np.isinf(lse[:n])
            assert np.array_equal(np.isneginf(g), empty)
            diff = np.abs(np.where(empty, 0, g) - np.where(empty, 0, lse[:n]))
            assert bool((diff <= bl).all()), f"lse off by {diff.max()}"


CASES = {
    "one token": dict(lens=[1], nq=[1], hq=1, hk=1, d=64, page=16),
    "two tokens, group 8": dict(lens=[2], nq=[1], hq=8, hk=1, d=128, page=16),
    "decode ragged": dict(lens=[1, 15, 16, 17, 63, 64, 65, 200, 333], nq=[1] * 9, hq=8, hk=2, d=128, page=16),
    "decode ragged d64": dict(lens=[1, 31, 32, 33, 127, 129, 300], nq=[1] * 7, hq=6, hk=2, d=64, page=32),
    "empty sequences": dict(lens=[0, 40, 0, 7], nq=[1, 1, 0, 1], hq=4, hk=2, d=128, page=16),
    "more queries than tokens": dict(lens=[3, 0, 70], nq=[5, 4, 2], hq=4, hk=2, d=64, page=16),
    "group 16": dict(lens=[150, 90], nq=[1, 1], hq=32, hk=2, d=128, page=64),
    "group 24": dict(lens=[150, 90], nq=[1, 2], hq=24, hk=1, d=128, page=64),
    "group 5 draft": dict(lens=[100, 61, 7], nq=[4, 3, 7], hq=10, hk=2, d=64, page=16),
    "one head each": dict(lens=[77, 130], nq=[1, 3], hq=3, hk=3, d=128, page=16),
    "pages of 128": dict(lens=[127, 128, 129, 513], nq=[1, 1, 1, 1], hq=8, hk=2, d=128, page=128),
    "rows first": dict(lens=[90, 33], nq=[1, 9], hq=8, hk=2, d=128, page=16, rows_first=True),
    "window": dict(lens=[200, 64, 65, 3], nq=[1, 1, 1, 1], hq=8, hk=2, d=128, page=16, window=64),
    "window 1": dict(lens=[100, 5], nq=[1, 2], hq=4, hk=1, d=64, page=16, window=1),
    "window and sinks": dict(lens=[300, 40, 129], nq=[1, 1, 3], hq=8, hk=2, d=128, page=32, window=33, sinks=5),
    "sinks past the window": dict(lens=[300, 90], nq=[1, 20], hq=4, hk=2, d=64, page=16, window=10, sinks=70),
    "window chunks": dict(lens=[700, 150, 257], nq=[200, 150, 1], hq=6, hk=2, d=64, page=16, window=100, sinks=3),
    "prompt": dict(lens=[190, 65], nq=[190, 65], hq=4, hk=2, d=128, page=64),
    "prompt d64": dict(lens=[257, 130, 1], nq=[257, 130, 1], hq=4, hk=1, d=64, page=16),
    "chunk": dict(lens=[520, 300], nq=[70, 33], hq=8, hk=2, d=128, page=64),
    "chunk group 3": dict(lens=[410, 128], nq=[43, 128], hq=6, hk=2, d=128, page=16),
    "sharp scores": dict(lens=[300, 90], nq=[1, 17], hq=8, hk=2, d=128, page=16, q_amp=12.0),
    "flat scores": dict(lens=[600], nq=[2], hq=8, hk=2, d=128, page=16, q_amp=1e-3),
    "huge queries": dict(lens=[130], nq=[9], hq=4, hk=2, d=64, page=16, q_amp=1e4),
    "long decode": dict(lens=[5000, 2999], nq=[1, 1], hq=8, hk=2, d=128, page=64),
    "long chunk": dict(lens=[3000], nq=[20], hq=8, hk=2, d=64, page=64),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attention(name):
    dev = device()
    announce(f"attention {name}")
    c = Case(seed=len(name), **CASES[name])
    r = c.run(dev)()
    torch.cuda.synchronize()
    c.check(r)


def test_attention_underestimated_length():
    """max_seq_len only sizes the split: a sequence that outgrew it is still right."""
    dev = device()
    for nq in ([1, 1], [40, 3]):
        c = Case([3000, 100], nq, 8, 2, 128, 16, seed=4)
        for bound in (0, 1, 500):
            announce(f"underestimated {nq} {bound}")
            r = c.run(dev, max_seq_len=bound)()
            torch.cuda.synchronize()
            c.check(r)


def test_attention_overestimated_length():
    dev = device()
    c = Case([300, 100, 1], [1, 2, 1], 8, 2, 128, 16, seed=4)
    r = c.run(dev, max_seq_len=1 << 20)()
    torch.cuda.synchronize()
    c.check(r)


def test_attention_rows_behind_stay():
    """Rows of q that belong to no sequence, and queries past max_q_len, keep what out and
    lse held."""
    dev = device()
    for nq in ([1, 2], [30, 70]):
        c = Case([100, 90], nq, 8, 2, 64, 16, seed=2, behind=5)
        call = c.run(dev)
        call.out.out.fill_(7.0)
        call.out.lse.fill_(-3.0)
        r = call()
        torch.cuda.synchronize()
        c.check(r)
        assert (r.out[-5:] == 7.0).all() and (r.lse[-5:] == -3.0).all()
    c = Case([100], [50], 8, 2, 64, 16, seed=2)
    call = c.run(dev)
    short = mxq.AttentionNVFP4(c.q.to(dev), call._cache, torch.from_numpy(c.table).to(dev),
                               torch.tensor(c.lens, dtype=torch.int32, device=dev), torch.from_numpy(c.starts).to(dev),
                               20, 100, lse=True)
    short.out.out.fill_(7.0)
    r, full = short(), call()
    torch.cuda.synchronize()
    assert torch.equal(r.out[:20], full.out[:20]) and (r.out[20:] == 7.0).all()


def test_attention_masked_nan_stays_out():
    """A query's output does not depend on tokens it does not see: NaN K and V rows after
    it, and before its window, change no bit; a visible NaN K row makes the row NaN, a
    visible NaN V block at least that block."""
    dev = device()
    for window, nq, d in ((0, 40, 128), (0, 40, 64), (16, 40, 64), (0, 3, 128)):
        announce(f"masked NaN window={window} nq={nq} d={d}")
        c = Case([120], [nq], 4, 2, d, 16, window=window, seed=6)
        clean = c.run(dev)()
        torch.cuda.synchronize()
        c.check(clean)
        at = 120 - nq + 1                             # the second query's own position
        page, row = c.table[0, at // 16], at % 16
        for which in ("k", "v"):
            d2 = Case([120], [nq], 4, 2, d, 16, window=window, seed=6)
            (d2.ks if which == "k" else d2.vs)[page, 1, row, 2] = 0x7F
            r = d2.run(dev)()
            torch.cuda.synchronize()
            a, b = su.f32_of_bf16(r.out), su.f32_of_bf16(clean.out)
            assert_same("heads of the other cached head", a[:, :2], b[:, :2])
            assert_same("the query before", a[0], b[0])
            seen = slice(1, nq if not window else min(nq, 1 + window))
            assert np.isnan(a[seen, 2:, 32:48]).all()
            if which == "k":
                assert np.isnan(a[seen, 2:]).all()
            if window and nq > 1 + window:
                assert_same("queries past the window", a[1 + window:], b[1 + window:])


def test_attention_bad_pages():
    """A page number outside the cache is never followed: queries that see one of its
    tokens come out NaN, the others as without it; so do lengths past the table."""
    dev = device()
    for nq in (1, 50):
        for bad in (-1, 1 << 30, 10):
            announce(f"bad page {bad} nq={nq}")
            c = Case([120, 60], [nq, 1], 4, 2, 128, 16, seed=8, spare=0)
            clean = c.run(dev, poison=False)()
            pages = c.kc.shape[0]
            c.table[0, 5] = bad if bad != 10 else pages           # tokens 80 .. 95
            r = c.run(dev, poison=False)()
            torch.cuda.synchronize()
            a, b = su.f32_of_bf16(r.out), su.f32_of_bf16(clean.out)
            hit = np.arange(120 - nq, 120) >= 80
            assert np.isnan(a[:nq][hit]).all()
            assert_same("before the page", a[:nq][~hit], b[:nq][~hit])
            assert_same("the other sequence", a[nq:], b[nq:])
    c = Case([120], [2], 4, 2, 128, 16, seed=8)
    full = c.run(dev, poison=False)()
    c.lens = [128]
    whole = c.run(dev, poison=False)()
    c.lens = [1 << 30]                                            # read as the table's 8 pages: 128 tokens
    r = c.run(dev, poison=False, max_seq_len=128)()
    torch.cuda.synchronize()
    assert_same("length past the table", su.f32_of_bf16(r.out), su.f32_of_bf16(whole.out))
    assert not torch.equal(full.out, whole.out)


def test_attention_cache_past_4gib():
    """Offsets past 32 bits: the same pages at the far end of a cache of 6 GiB."""
    dev = device()
    if torch.cuda.get_device_properties(0).total_memory < 32 << 30:
        pytest.skip("needs 16 GiB")
    for nq in (1, 40):
        announce(f"past 4 GiB nq={nq}")
        c = Case([150], [nq], 4, 2, 128, 16, seed=1, spare=0)
        near = c.run(dev, poison=False)()
        pages = c.kc.shape[0]
        far_pages = (6 << 30) // (2 * 16 * 64)
        big = [torch.zeros((far_pages, 2, 16, w), dtype=torch.uint8, device=dev) for w in (64, 8, 64, 8)]
        for b, x in zip(big, (c.kc, c.ks, c.vc, c.vs)):
            b[-pages:] = torch.from_numpy(x).to(dev)
        cache = mxq.NVFP4KVCache(*big, torch.from_numpy(c.kg).to(dev), torch.from_numpy(c.vg).to(dev))
        r = mxq.mxq_attention_nvfp4(c.q.to(dev), cache, torch.from_numpy(c.table + (far_pages - pages)).to(dev),
                                    torch.tensor([150], dtype=torch.int32, device=dev),
                                    torch.from_numpy(c.starts).to(dev), nq, 150)
        torch.cuda.synchronize()
        assert torch.equal(r.out, near.out)
        slots = torch.tensor([(far_pages - 1) * 16 + 3], device=dev)
        k = bf16(np.random.default_rng(0), 1, 2, 128).to(dev)
        mxq.mxq_rope_append_nvfp4(None, k, k, torch.zeros(1, dtype=torch.int32, device=dev), slots,
                                  mxq.rope_plan(0, device=dev), cache)
        torch.cuda.synchronize()
        codes, scales = su.encode_rows(su.f32_of_bf16(k), c.vg)
        assert_same("far codes", host(big[2][-1, :, 3]), codes[0])
        assert_same("far scales", host(big[3][-1, :, 3]), scales[0])
        del big, cache


def test_attention_repeats_bit_for_bit():
    dev = device()
    for name in ("decode ragged", "long decode", "chunk", "long chunk"):
        c = Case(seed=1, **CASES[name])
        call = c.run(dev)
        first = call()
        o, l = first.out.clone(), first.lse.clone()
        for _ in range(3):
            r = call()
        torch.cuda.synchronize()
        assert torch.equal(r.out, o) and torch.equal(r.lse, l)


def test_attention_padded_q_rows():
    """Q inside a wider QKV buffer, out with a stride of its own."""
    dev = device()
    c = Case([70, 33], [3, 33], 4, 2, 128, 16, seed=3)
    plain = c.run(dev)()
    wide = torch.zeros(36, 4 * 128 + 256, dtype=torch.bfloat16, device=dev)
    wide[:, :512] = c.q.to(dev).flatten(1)
    keep = c.q
    call = c.run(dev)
    out = torch.full((36, 600), 5.0, dtype=torch.bfloat16, device=dev)
    strided = mxq.AttentionNVFP4(wide[:, :512].unflatten(1, (4, 128)), call._cache, torch.from_numpy(c.table).to(dev),
                                 torch.tensor(c.lens, dtype=torch.int32, device=dev),
                                 torch.from_numpy(c.starts).to(dev), 33, 70, out=out[:, :512].unflatten(1, (4, 128)))
    r = strided()
    torch.cuda.synchronize()
    assert torch.equal(r.out, plain.out) and (out[:, 512:] == 5.0).all() and keep is c.q


# ------------------------------------------------------------------ streams, graphs, a run together
def test_side_stream_and_graph():
    """The three calls in a row on another stream, and captured into a graph that is
    replayed with new inputs and eager work in between."""
    dev = device()
    rng = np.random.default_rng(12)
    hq, hk, d, page, n, b = 8, 2, 128, 16, 1024, 3
    cache = mxq.NVFP4KVCache.allocate(16, page, hk, d, 5.0, 5.0, device=dev)
    cache.k_codes.copy_(torch.from_numpy(rng.integers(0, 256, cache.k_codes.shape, dtype=np.uint8)))
    cache.v_codes.copy_(torch.from_numpy(rng.integers(0, 256, cache.v_codes.shape, dtype=np.uint8)))
    cache.k_scales.fill_(0x30)
    cache.v_scales.fill_(0x34)
    x, res, w = bf16(rng, b, n).to(dev), bf16(rng, b, n).to(dev), bf16(rng, n).to(dev)
    qkv = bf16(rng, b, (hq + 2 * hk) * d).to(dev)
    table = torch.arange(15, dtype=torch.int32, device=dev).view(3, 5)
    lens = torch.tensor([70, 33, 1], dtype=torch.int32, device=dev)
    starts = torch.arange(4, dtype=torch.int32, device=dev)
    plan = mxq.rope_plan(d, device=dev)
    norm = mxq.AddRMSNormFP8(x, w, res, out_bf16=True)
    pos, slots = lens - 1, torch.empty(3, dtype=torch.int64, device=dev)

    def place():
        slots.copy_(table.long().gather(1, (pos.long() // page)[:, None])[:, 0] * page + pos.long() % page)

    place()
    app = mxq.RopeAppendNVFP4(qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                              qkv[:, (hq + hk) * d:].unflatten(1, (hk, d)), pos, slots, plan, cache)
    att = mxq.AttentionNVFP4(app.out.q, cache, table, lens, starts, 1, 80, lse=True)

    def step(stream=None):
        norm(stream), app(stream), att(stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (norm.out.q, norm.out.scales, norm.out.y, app.out.q, cache.k_codes, cache.v_scales,
                                    att.out.out, att.out.lse)]

    step()
    want = results()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        att.out.out.zero_()
        step(s)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(bf16(rng, b, n))
        qkv.copy_(bf16(rng, b, (hq + 2 * hk) * d))
        lens.add_(1)
        pos.copy_(lens - 1)
        place()
        step()                                        # eager
        want = results()
        att.out.out.zero_()
        norm.out.q.zero_()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(results(), want)), f"replay {i}"


def test_serving_steps_together():
    """A prompt, a chunk and three decoding steps through norm, append and attention: the
    attention of every step against 64 bits on what the cache holds by then."""
    dev = device()
    rng = np.random.default_rng(21)
    hq, hk, d, page, n = 6, 2, 64, 16, 256
    cache = mxq.NVFP4KVCache.allocate(14, page, hk, d, 4.5, 4.5, device=dev)
    table = torch.from_numpy(rng.permutation(14).astype(np.int32).reshape(2, 7)).to(dev)
    w = bf16(rng, n).to(dev)
    weight = bf16(rng, n, (hq + 2 * hk) * d, amp=n ** -0.5).to(dev)
    plan = mxq.rope_plan(32, interleaved=True, device=dev)
    lens = [0, 0]
    for nq in ([40, 9], [13, 20], [1, 1], [1, 1], [1, 0]):
        lens = [a + b for a, b in zip(lens, nq)]
        t = sum(nq)
        x = mxq.mxq_add_rmsnorm_quant_fp8(bf16(rng, t, n).to(dev), w, bf16(rng, t, n).to(dev), out_bf16=True)
        qkv = (x.y.float() @ weight.float()).bfloat16()
        pos = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, nq)]).astype(np.int32)
        seq = np.repeat(np.arange(2), nq)
        tab = host(table)
        slots = torch.from_numpy(tab[seq, pos // page].astype(np.int64) * page + pos % page).to(dev)
        app = mxq.mxq_rope_append_nvfp4(qkv[:, :hq * d].unflatten(1, (hq, d)),
                                        qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                                        qkv[:, (hq + hk) * d:].unflatten(1, (hk, d)), torch.from_numpy(pos).to(dev),
                                        slots, plan, cache)
        starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        r = mxq.mxq_attention_nvfp4(app.q, cache, table, torch.tensor(lens, dtype=torch.int32, device=dev),
                                    torch.from_numpy(starts).to(dev), max(nq), max(lens), lse=True)
        torch.cuda.synchronize()
        c = [host(z) for z in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.k_global, cache.v_global)]
        want, lse, bo, bl = su.attention_reference(su.f32_of_bf16(app.q), *c, tab, lens, starts, 1 / math.sqrt(d))
        assert (np.abs(su.f32_of_bf16(r.out) - want) <= bo).all()
        assert (np.abs(host(r.lse) - lse) <= bl).all()


def test_empty_calls():
    dev = device()
    w = torch.ones(256, dtype=torch.bfloat16, device=dev)
    r = mxq.mxq_add_rmsnorm_quant_fp8(torch.empty(0, 256, dtype=torch.bfloat16, device=dev), w)
    assert r.q.shape == (0, 256)
    cache = mxq.NVFP4KVCache.allocate(2, 16, 1, 64, 1.0, 1.0, device=dev)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=dev)
    mxq.mxq_rope_append_nvfp4(e, e, e, torch.empty(0, dtype=torch.int32, device=dev),
                              torch.empty(0, dtype=torch.int64, device=dev), mxq.rope_plan(64, device=dev), cache)
    a = mxq.mxq_attention_nvfp4(e, cache, torch.zeros(1, 1, dtype=torch.int32, device=dev),
                                torch.zeros(1, dtype=torch.int32, device=dev),
                                torch.zeros(2, dtype=torch.int32, device=dev), 1)
    torch.cuda.synchronize()
    assert a.out.shape == (0, 1, 64)


def test_library_refusals_raise():
    dev = device()
    x = torch.zeros(2, 192, dtype=torch.bfloat16, device=dev)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_add_rmsnorm_quant_fp8(x, torch.ones(192, dtype=torch.bfloat16, device=dev))
    cache = mxq.NVFP4KVCache.allocate(2, 48, 1, 64, 1.0, 1.0, device=dev)        # 48 rows a page
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=dev)
    one = torch.zeros(1, dtype=torch.int32, device=dev)
    with pytest.raises(mxq.MxqError):
        mxq.mxq_attention_nvfp4(q, cache, one[None], one, torch.tensor([0, 1], dtype=torch.int32, device=dev), 1)

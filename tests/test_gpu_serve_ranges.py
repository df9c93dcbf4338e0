"""The serving calls at the ends of what their arguments may hold: tensor scales, scores and
angles far from the ordinary, and tokens that a query does not see."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from tests import serve_util as su
from tests.gpu_util import announce, assert_same, device, host
from tests.test_gpu_serve import Case, bf16

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the append's tensor scales
@pytest.mark.parametrize("g", [2.0 ** -126, 1.7 * 2.0 ** -126, 1.3 * 2.0 ** -120, 1.1 * 2.0 ** -100, 1.9 * 2.0 ** -75,
                               1.2 * 2.0 ** 75, 1.5 * 2.0 ** 125, 1.3 * 2.0 ** 126, 1.999 * 2.0 ** 127])
def test_append_tensor_scales(g):
    """Blocks over the whole range of block scales (and below and above it) under every normal
    tensor scale: the stated divisions, also where a step or an inverse is not normal."""
    dev = device()
    announce(f"append tensor scale {g}")
    rng = np.random.default_rng(int(math.log2(g)) + 500)
    t, hk, d = 64, 2, 128
    # a block's largest value is 6 * scale * g: scales 2^-11 .. 2^10 as far as BF16 goes
    amp = 6.0 * g * 2.0 ** rng.uniform(-11, 10, (t, hk, d // 16, 1))
    y = np.clip(rng.uniform(-1, 1, (t, hk, d // 16, 16)) * amp, -3e38, 3e38).reshape(t, hk, d)
    k = torch.from_numpy(y.astype(np.float32)).bfloat16()
    v = (k.flip(0).float() * 0.5).bfloat16()
    scale = torch.full((hk,), g, dtype=torch.float64).float()
    cache = mxq.NVFP4KVCache.allocate(t // 16, 16, hk, d, 1.0, 1.0, device=dev)
    cache.k_global.copy_(scale)
    cache.v_global.copy_(scale)
    got = mxq.mxq_rope_append_nvfp4(None, k.to(dev), v.to(dev), torch.zeros(t, dtype=torch.int32, device=dev),
                                    torch.arange(t, device=dev), mxq.rope_plan(0, device=dev), cache, values=True)
    torch.cuda.synchronize()
    for name, x, codes, scales, values in (("k", k, cache.k_codes, cache.k_scales, got.k_values),
                                           ("v", v, cache.v_codes, cache.v_scales, got.v_values)):
        want_codes, want_scales = su.encode_rows(su.f32_of_bf16(x), scale.numpy())
        assert_same(name + " scales", host(scales.transpose(1, 2).reshape(t, hk, d // 16)), want_scales)
        assert_same(name + " codes", host(codes.transpose(1, 2).reshape(t, hk, d // 2)), want_codes)
        with np.errstate(over="ignore"):
            want = su.to_bf16(su.decode_rows(want_codes, want_scales).astype(np.float32) * scale.numpy()[None, :, None])
        assert_same(name + " values", su.f32_of_bf16(values), want)


# ------------------------------------------------------------------ angles
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_angles_past_the_reduction(interleaved):
    """Angles below 2^45 are turned by, whatever position and frequency make them up; from
    there on, and for frequencies that are no numbers, the pair is NaN."""
    dev = device()
    announce(f"angles interleaved={interleaved}")
    rng = np.random.default_rng(4)
    freq = np.array([1.0, 2.0 ** 13 + 0.3, 2.0 ** 14, 2.0 ** 20, 1e30, 1e300, np.inf, np.nan])
    pos = np.array([0, 1, 1000, -5, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 30], np.int64).astype(np.int32)
    q = bf16(rng, 8, 2, 64)
    k = bf16(rng, 8, 1, 64)
    cache = mxq.NVFP4KVCache.allocate(1, 16, 1, 64, 4.0, 4.0, device=dev)
    plan = mxq.RopePlan(torch.from_numpy(freq).to(dev), interleaved=interleaved)
    got = mxq.mxq_rope_append_nvfp4(q.to(dev), k.to(dev), k.to(dev), torch.from_numpy(pos).to(dev),
                                    torch.arange(8, device=dev), plan, cache)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        theta = pos.astype(np.float64)[:, None] * freq
        bad = ~(np.abs(theta) < 2.0 ** 45)
        want = su.rope_reference(su.f32_of_bf16(q), pos, freq, 1.0, interleaved)
    pair = np.repeat(bad, 2, 1) if interleaved else np.concatenate([bad, bad], 1)
    pair = np.broadcast_to(pair[:, None], (8, 2, 16))
    a = su.f32_of_bf16(got.q)
    assert np.array_equal(np.isnan(a[..., :16]), pair)
    assert_same("angles in range", np.where(pair, 0, a[..., :16]), np.where(pair, 0, want[..., :16]))
    assert_same("unrotated", a[..., 16:], want[..., 16:])


# ------------------------------------------------------------------ what a query does not see
@pytest.mark.parametrize("nq,hq", [(3, 8), (7, 8), (60, 8), (100, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_unseen_tokens_change_no_bit(nq, hq, d):
    """The last query's own token gets the largest key along that query (its score raises the
    running maximum wherever it is seen) and other values: no bit of an earlier query changes."""
    dev = device()
    announce(f"unseen nq={nq} hq={hq} d={d}")
    changed = 0
    for seed in range(4):
        results = []
        for other in (False, True):
            c = Case([1400 + seed], [nq], hq, 2, d, 16, seed=seed, q_amp=0.3)
            if other:
                at = c.lens[0] - 1
                page, row = c.table[0, at // 16], at % 16
                for kv in range(2):
                    code = 7 + 8 * (c.q[-1, kv * (hq // 2)].float().numpy() < 0).astype(np.uint8)
                    c.kc[page, kv, row] = code[0::2] | (code[1::2] << 4)
                c.ks[page, :, row] = 0x7E
                c.vs[page, :, row] = 0x70
            r = c.run(dev)()
            torch.cuda.synchronize()
            results.append((r.out.clone(), r.lse.clone()))
        (a, la), (b, lb) = results
        assert not torch.equal(a[-1], b[-1])
        changed += int((a[:-1] != b[:-1]).sum()) + int((la[:-1] != lb[:-1]).sum())
    assert changed == 0
# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("nq,hq", [(1, 8), (5, 8), (3, 32), (60, 8)])
@pytest.mark.parametrize("amp", [1e6, 1e8, 1e12, 1e31])
@pytest.mark.parametrize("bound", [64, 1 << 22])
def test_scores_past_a_weight_range(nq, hq, amp, bound):
    """Scores so large that one step of FP32 at them is more than the weights' own range: where
    the best token leads by more than the scores' rounding, the output is that token's value
    and the log-sum its score."""
    dev = device()
    announce(f"scores nq={nq} hq={hq} amp={amp} bound={bound}")
    d, hk = 128, 2
    c = Case([700, 1, 130], [nq, 1, nq], hq, hk, d, 16, seed=nq, q_amp=amp)
    r = c.run(dev, max_seq_len=bound)()
    torch.cuda.synchronize()
    out, lse = su.f32_of_bf16(r.out).astype(np.float64), host(r.lse).astype(np.float64)
    q = su.f32_of_bf16(c.q).astype(np.float64)
    checked = 0
    for b, n in enumerate(c.lens):
        at, off = c.table[b][np.arange(n) // 16], np.arange(n) % 16
        for h in range(hq):
            kv = h // (hq // hk)
            k = su.decode_rows(c.kc[at, kv, off], c.ks[at, kv, off]) * float(c.kg[kv])
            v = su.decode_rows(c.vc[at, kv, off], c.vs[at, kv, off]) * float(c.vg[kv])
            for i in range(c.starts[b], c.starts[b + 1]):
                seen = n - int(c.starts[b + 1]) + int(i) + 1
                x = k[:seen] @ q[i, h] / math.sqrt(d)
                # the scores' rounding (serve_util.attention_bounds): d + 8 of 2^-24 of sum |q k|
                off_by = (d + 8) * 2.0 ** -24 * (np.abs(k[:seen]) @ np.abs(q[i, h])).max() / math.sqrt(d) + 2.0 ** -20
                best = int(x.argmax())
                lead = x[best] - np.delete(x, best).max() if seen > 1 else np.inf
                assert np.isfinite(out[i, h]).all() and abs(lse[i, h] - x[best]) <= off_by + math.log(seen) + 2.0 ** -22 * abs(x[best])
                if lead <= 2 * off_by + 40.0:
                    continue
                checked += 1
                # the others' weights are below e^-40; its own is rounded to FP16 for the product and
                # not in the sum (half a step: 2^-11), the output to BF16 (2^-8), the rest is FP32
                e = np.abs(out[i, h] - v[best])
                assert (e <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * np.abs(v[best]) + 1e-12).all(), (e / np.abs(v[best])).max()
    assert checked > 0.5 * q.shape[0] * hq




# ------------------------------------------------------------------ Q's power of two
@pytest.mark.parametrize("nq", [1, 6, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ratio", [-20, -29, -33])
def test_small_elements_beside_a_large_one(ratio, d, nq):
    """One element of Q, whose keys are zero, 2^-ratio times the others, which make the scores:
    they are exact down to 2^-31 of it, and off by at most 2^-39 of it below."""
    dev = device()
    announce(f"ratio 2^{ratio} d={d} nq={nq}")
    c = Case([150, 70], [nq, 1], 4, 2, d, 16, seed=5, spare=0)
    c.kc[..., 0] &= 0xF0                                          # element 0 of every key
    q = np.clip(c.q.float().numpy(), -2, 2) * 2.0 ** ratio
    q[..., 0] = 1.5
    c.q = torch.from_numpy(q).bfloat16()
    scale = 2.0 ** -ratio / math.sqrt(d)
    call = c.run(dev)
    r = mxq.mxq_attention_nvfp4(c.q.to(dev), call._cache, torch.from_numpy(c.table).to(dev),
                                torch.tensor(c.lens, dtype=torch.int32, device=dev), torch.from_numpy(c.starts).to(dev),
                                nq, max(c.lens), scale=scale, lse=True)
    torch.cuda.synchronize()
    want, lse, _, _ = su.attention_reference(su.f32_of_bf16(c.q), c.kc, c.ks, c.vc, c.vs, c.kg, c.vg, c.table, c.lens,
                                             c.starts, scale)
    k = np.abs(su.decode_rows(c.kc, c.ks)) * c.kg.astype(np.float64)[None, :, None, None]
    v = np.abs(su.decode_rows(c.vc, c.vs)) * c.vg.astype(np.float64)[None, :, None, None]
    # serve_util.attention_bounds, with the largest sums of any token, and beside a score's FP32
    # roundings Q's: half of FP16's smallest step, 2^-25, where the largest element is at least
    # 2^14, for every element that is not exact (all below 2^-31: 8 bits from 2^-24 on)
    small = 2.0 * 2.0 ** ratio
    q_off = 0.0 if ratio >= -24 else 2.0 ** -39 * 1.5
    delta = ((d + 8) * 2.0 ** -24 * small + q_off) * k.sum(-1).max() * scale + 2.0 ** -22
    e = v.max() * (2 * delta + 2.0 ** -11) * 1.05 + 2.0 ** -34 * v.max() * 150
    off = np.abs(su.f32_of_bf16(r.out) - want)
    assert (off <= 2.0 ** -8 * (np.abs(want) + e) + e).all(), off.max()
    assert (np.abs(host(r.lse) - lse) <= delta + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all()
    # (scores of zero, as of elements that were lost, would not pass)
    seen = [n - k + 1 + i for n, k in zip(c.lens, c.nq) for i in range(k)]
    assert np.abs(lse - np.log(seen)[:, None]).max() > 2 * delta + 2.0 ** -18


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("q_power,kg_power,scale_power", [(-30, -100, 119), (-90, -50, 127), (120, -126, -6), (100, -3, -109),
                                                          (-60, 100, -50), (110, -110, -12), (0, -126, 114)])
def test_factors_that_cancel(q_power, kg_power, scale_power, nq):
    """Queries, K's tensor scale and the softmax scale at far ends of their ranges whose product
    is ordinary: no step between loses bits of it."""
    dev = device()
    announce(f"factors 2^{q_power} 2^{kg_power} 2^{scale_power} nq={nq}")
    c = Case([100, 70], [nq, nq], 4, 2, 64, 16, seed=13)
    c.kg[:] = np.array([1.0, 1.37]) * 2.0 ** kg_power
    c.q = (c.q.double() * 2.0 ** q_power).bfloat16()
    scale = float(np.float32(2.0 ** scale_power * 1.3))
    call = c.run(dev)
    r = mxq.mxq_attention_nvfp4(c.q.to(dev), call._cache, torch.from_numpy(c.table).to(dev),
                                torch.tensor(c.lens, dtype=torch.int32, device=dev), torch.from_numpy(c.starts).to(dev),
                                nq, 100, scale=scale, lse=True)
    torch.cuda.synchronize()
    want, lse, bo, bl = su.attention_reference(su.f32_of_bf16(c.q), c.kc, c.ks, c.vc, c.vs, c.kg, c.vg, c.table, c.lens,
                                               c.starts, scale)
    assert 0.1 < (lse.max() - lse.min()) < 1e4
    assert (np.abs(su.f32_of_bf16(r.out) - want) <= bo).all()
    assert (np.abs(host(r.lse) - lse) <= bl).all()

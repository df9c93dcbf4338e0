"""The serving calls on the host: argument errors before anything is enqueued (fake
device addresses, so without a GPU only), the binding's own checks on CPU tensors, the
workspace query and the rotary plans."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import nvfp4_quantization_amd as mxq
from nvfp4_quantization_amd import serve
from tests import serve_util as su

OK, INVALID, MISALIGNED, WS_SMALL, UNSUPPORTED, HIP = range(6)
A = 1 << 20          # a fake, 256-byte aligned device address: never dereferenced on these paths


def _gpu_visible() -> bool:
    return torch.cuda.device_count() > 0


no_gpu = pytest.mark.skipif(_gpu_visible(), reason="fake device addresses: run where no GPU is visible")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mxq.LIB_PATH):
        pytest.skip("libmxq.so not built")
    return mxq.lib()


def norm(L, x=A, ldx=256, res=A, ld_res=256, ro=A, ld_ro=256, w=A, eps=1e-6, m=4, n=256, options=0, y=None, ld_y=0,
         q=A, ldq=256, s=A, sr=2, sg=1):
    return L.mxq_add_rmsnorm_quant_fp8(x, ldx, res, ld_res, ro, ld_ro, w, eps, m, n, options, y, ld_y, q, ldq, s, sr, sg,
                                       None)


@no_gpu
def test_norm_argument_errors(L):
    assert norm(L, options=2) == INVALID
    assert norm(L, m=-1) == INVALID
    assert norm(L, ldx=128) == INVALID
    assert norm(L, res=None) == INVALID                           # residual_out without a residual
    assert norm(L, ro=None) == INVALID
    assert norm(L, ld_ro=248) == INVALID
    assert norm(L, y=A, ld_y=128) == INVALID
    assert norm(L, eps=-1.0) == INVALID
    assert norm(L, eps=float("nan")) == INVALID
    assert norm(L, eps=float("inf")) == INVALID
    assert norm(L, w=None) == INVALID
    assert norm(L, sr=-1) == INVALID
    assert norm(L, n=200, ldx=200, ld_res=200, ld_ro=200, ldq=208) == MISALIGNED
    assert norm(L, ldq=264) == MISALIGNED
    assert norm(L, ld_res=260) == MISALIGNED
    assert norm(L, y=A, ld_y=260) == MISALIGNED
    assert norm(L, w=A + 8) == MISALIGNED
    assert norm(L, s=A + 2) == MISALIGNED
    big = 32768 + 128
    assert norm(L, n=big, ldx=big, ld_res=big, ld_ro=big, ldq=big) == UNSUPPORTED
    assert norm(L, m=1 << 31) == UNSUPPORTED
    assert norm(L, m=1 << 23) == UNSUPPORTED                      # more work-groups than a launch takes
    assert norm(L, ld_res=1 << 40) == UNSUPPORTED
    assert norm(L, sg=1 << 40) == UNSUPPORTED
    assert norm(L, m=0, x=None, q=None, s=None, w=None) == OK


def kv(**kw):
    a = dict(kc=A, ks=A, vc=A, vs=A, kg=A, vg=A, pages=4, page=16, heads=2, d=128, c=(2048, 1024, 64), s=(256, 128, 8))
    a.update(kw)
    return serve._KV(a["kc"], a["ks"], a["vc"], a["vs"], a["kg"], a["vg"], a["pages"], a["page"], a["heads"], a["d"],
                     *a["c"], *a["s"])


BAD_CACHES = [
    (dict(kg=None), INVALID), (dict(vs=None), INVALID), (dict(heads=0), INVALID), (dict(pages=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=1 << 21), UNSUPPORTED), (dict(c=(2048, 1024, 72)), MISALIGNED), (dict(s=(256, 128, 12)), MISALIGNED),
    (dict(c=(2048, -1024, 64)), INVALID), (dict(c=(2048, 1024, 32)), INVALID), (dict(s=(256, 128, 0)), INVALID),
    (dict(kc=A + 8), MISALIGNED), (dict(vs=A + 4), MISALIGNED), (dict(vg=A + 2), MISALIGNED),
    (dict(c=(1 << 39, 1024, 64)), UNSUPPORTED), (dict(c=(1 << 29, 1 << 29, (1 << 24) + 16)), UNSUPPORTED), (dict(s=(1 << 60, 1 << 60, 8)), UNSUPPORTED),
]


def append(L, q=A, ld_q=512, hq=4, qo=A, ld_qo=512, k=A, ld_k=256, v=A, ld_v=256, t=3, pos=A, slots=A, rot=128, flags=0,
           factor=1.0, freq=A, rope=True, cache=None, kvals=None, vvals=None):
    r = serve._Rope(freq, rot, flags, factor)
    c = cache if cache is not None else kv()
    return L.mxq_rope_append_nvfp4(q, ld_q, hq, qo, ld_qo, k, ld_k, v, ld_v, t, pos, slots,
                                   ctypes.byref(r) if rope else None, ctypes.byref(c), kvals, vvals, None)


@no_gpu
def test_append_argument_errors(L):
    for kw, want in BAD_CACHES:
        assert append(L, cache=kv(**kw)) == want, kw
    assert append(L, rope=False) == INVALID
    assert append(L, flags=2) == INVALID
    assert append(L, rot=144) == INVALID
    assert append(L, rot=-16) == INVALID
    assert append(L, rot=24) == MISALIGNED
    assert append(L, freq=None) == INVALID
    assert append(L, factor=float("inf")) == INVALID
    assert append(L, t=-1) == INVALID
    assert append(L, hq=-1) == INVALID
    assert append(L, ld_q=256) == INVALID
    assert append(L, ld_k=128) == INVALID
    assert append(L, ld_v=260) == MISALIGNED
    assert append(L, q=None) == INVALID
    assert append(L, v=None) == INVALID
    assert append(L, slots=None) == INVALID
    assert append(L, slots=A + 4) == MISALIGNED
    assert append(L, k=A + 8) == MISALIGNED
    assert append(L, kvals=A + 2) == MISALIGNED
    assert append(L, t=1 << 31) == UNSUPPORTED
    assert append(L, t=1 << 30) == UNSUPPORTED                    # more threads than a launch takes
    assert append(L, ld_k=1 << 40) == UNSUPPORTED
    assert append(L, t=0, k=None, v=None, slots=None, pos=None) == OK


def attend(L, q=A, ld_q=512, hq=4, tq=6, out=A, ld_out=512, lse=None, cache=None, table=A, ld_t=4, pages=4, lens=A,
           starts=A, b=2, mq=3, ml=64, scale=0.1, window=0, sinks=0, ws=A, wsb=1 << 30):
    c = cache if cache is not None else kv()
    return L.mxq_attention_nvfp4(q, ld_q, hq, tq, out, ld_out, lse, ctypes.byref(c), table, ld_t, pages, lens, starts, b,
                                 mq, ml, scale, window, sinks, ws, wsb, None)


@no_gpu
def test_attention_argument_errors(L):
    for kw, want in BAD_CACHES:
        assert attend(L, cache=kv(**kw)) == want, kw
    assert attend(L, hq=5, ld_q=640, ld_out=640) == INVALID       # not a multiple of the cached heads
    assert attend(L, hq=0) == INVALID
    assert attend(L, b=0) == INVALID
    assert attend(L, mq=-1) == INVALID
    assert attend(L, ml=-1) == INVALID
    assert attend(L, ld_t=3) == INVALID
    assert attend(L, window=-1) == INVALID
    assert attend(L, sinks=-1) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(L, scale=bad) == INVALID
    assert attend(L, ld_q=256) == INVALID
    assert attend(L, ld_out=516) == MISALIGNED
    assert attend(L, out=A + 8) == MISALIGNED
    assert attend(L, lse=A + 1) == MISALIGNED
    assert attend(L, table=A + 2) == MISALIGNED
    assert attend(L, table=None) == INVALID
    assert attend(L, lens=None) == INVALID
    assert attend(L, b=65536) == UNSUPPORTED
    assert attend(L, tq=1 << 30) == UNSUPPORTED
    assert attend(L, ld_t=1 << 40) == UNSUPPORTED
    assert attend(L, tq=0, q=None) == OK
    assert attend(L, mq=0, q=None) == OK


@no_gpu
def test_attention_workspace(L):
    q = mxq.mxq_attention_nvfp4_workspace_size
    for shape in [(32, 8, 128, 1, 1, 1, 1 << 20), (64, 8, 128, 64, 64, 1, 8192), (32, 8, 128, 1, 512, 512, 65536),
                  (8, 8, 64, 3, 40, 17, 100), (4, 2, 128, 2, 6, 3, 1 << 20)]:
        need = q(*shape)
        assert need % 256 == 0 and need < 1 << 30
    need = q(4, 2, 128, 2, 6, 3, 1 << 20)
    if need:
        assert attend(L, ml=1 << 20, wsb=need - 1) == WS_SMALL
        assert attend(L, ml=1 << 20, ws=None) == INVALID
        assert attend(L, ml=1 << 20, ws=A + 128) == MISALIGNED
    for bad in [(0, 1, 128, 1, 1, 1, 1), (4, 0, 128, 1, 1, 1, 1), (4, 3, 128, 1, 1, 1, 1), (4, 2, 96, 1, 1, 1, 1),
                (4, 2, 128, 0, 1, 1, 1), (4, 2, 128, 1, 0, 1, 1), (4, 2, 128, 1, 1, 0, 1), (4, 2, 128, 1, -1, 1, 1)]:
        assert q(*bad) == 0


# ------------------------------------------------------------------ the binding's own checks
def cpu_cache(pages=3, heads=2, page=16, d=64):
    return mxq.NVFP4KVCache.allocate(pages, page, heads, d, 4.0, [3.0, 5.0], device="cpu")


def test_cache_checks():
    c = cpu_cache()
    assert c.head_dim == 64 and c.k_codes.shape == (3, 2, 16, 32) and c.k_scales.shape == (3, 2, 16, 4)
    assert np.array_equal(c.v_global.numpy(), np.array([3.0, 5.0], np.float32) * np.float32(1 / 2688))
    t = list(c.tensors())
    for i, bad in [(0, t[0].float()), (1, t[1][..., :3]), (2, t[2][:2]), (3, t[3].to(torch.int8)), (4, t[4][:1]),
                   (5, t[5].double()), (2, t[2].transpose(1, 2).contiguous().transpose(1, 2))]:
        u = list(t)
        u[i] = bad
        with pytest.raises((TypeError, ValueError)):
            mxq.NVFP4KVCache(*u)


def test_prepared_call_checks():
    """What the binding refuses by itself: nothing reaches the library."""
    c = cpu_cache()
    rope = mxq.rope_plan(32, device="cpu")
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    pos, slots = torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)
    mxq.RopeAppendNVFP4(q, k, k, pos, slots, rope, c)             # accepted (and not run)
    for args in [(q.float(), k, k, pos, slots), (q[:4], k, k, pos, slots), (q, k[:, :1], k, pos, slots),
                 (q, k, k[..., :32], pos, slots), (q, k, k, pos.long(), slots), (q, k, k, pos, slots.int()),
                 (q, k, k, pos[:4], slots), (q.transpose(1, 2).contiguous().transpose(1, 2), k, k, pos, slots)]:
        with pytest.raises((TypeError, ValueError)):
            mxq.RopeAppendNVFP4(*args, rope, c)
    with pytest.raises(ValueError):
        mxq.RopeAppendNVFP4(None, k, k, pos, slots, rope, c, q_out=q)
    table, lens, starts = (torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                           torch.zeros(3, dtype=torch.int32))
    mxq.AttentionNVFP4(q, c, table, lens, starts, 3)
    for args in [(q, c, table.long(), lens, starts), (q, c, table, lens[:1], starts), (q, c, table, lens, starts[:2]),
                 (q[0], c, table, lens, starts), (q, c, table, lens.float(), starts)]:
        with pytest.raises((TypeError, ValueError)):
            mxq.AttentionNVFP4(*args, 3)
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    mxq.AddRMSNormFP8(x, w)
    for args in [(x.float(), w), (x, w[:128]), (x, w, x[:2]), (x[0], w), (x.t().contiguous().t(), w)]:
        with pytest.raises((TypeError, ValueError)):
            mxq.AddRMSNormFP8(*args)
    with pytest.raises(ValueError):
        mxq.AddRMSNormFP8(x, w, residual_out=x)


def test_rope_plans():
    """The scalings of the frequencies, against their definitions."""
    d = 64
    f = 10000.0 ** (-np.arange(0, d, 2) / d)
    plain = mxq.rope_plan(d, device="cpu")
    assert plain.rot_dim == d and plain.factor == 1.0 and np.allclose(plain.inv_freq.numpy(), f, rtol=1e-14)
    assert np.allclose(mxq.rope_plan(d, scaling="linear", scale=8.0, device="cpu").inv_freq.numpy(), f / 8, rtol=1e-14)
    b = mxq.rope_plan(d, scaling="base", scale=8.0, device="cpu").inv_freq.numpy()
    assert b[0] == 1.0 and abs(b[-1] / (f[-1] / 8) - 1) < 1e-12
    r = mxq.rope_plan(d, scaling="ramp", scale=8.0, trained_length=4096, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    got = r.inv_freq.numpy()
    assert np.allclose(got[turns > 32], f[turns > 32]) and np.allclose(got[turns < 1], f[turns < 1] / 8)
    assert (np.diff(got) < 0).all() and abs(r.factor - (0.1 * math.log(8) + 1)) < 1e-15
    for bad in (dict(scaling="other"), dict(scaling="ramp", scale=2.0), dict(scale=0.5)):
        with pytest.raises(ValueError):
            mxq.rope_plan(d, device="cpu", **bad)
    with pytest.raises(ValueError):
        mxq.rope_plan(63, device="cpu")
    assert mxq.rope_plan(0, device="cpu").rot_dim == 0


def test_reference_attention_by_hand():
    """The tests' 64-bit attention on a case worked by hand: two tokens, equal keys, so
    the output is the mean of the values; one visible token gives its value."""
    kc = np.full((1, 1, 16, 32), 0x22, np.uint8)                  # every element 1.0
    ks = np.full((1, 1, 16, 4), 0x38, np.uint8)                   # scale 1.0
    vc = kc.copy()
    vc[0, 0, 1] = 0x44                                            # token 1: 2.0
    q = np.ones((2, 1, 64), np.float32)
    one = np.ones(1, np.float32)
    out, lse, _, _ = su.attention_reference(q, kc, ks, vc, ks, one, 2 * one, [[0]], [2], [0, 2], 0.125)
    assert np.allclose(out[0], 2.0) and np.allclose(out[1], 3.0)
    assert np.allclose(lse[:, 0], [8.0, 8.0 + math.log(2)])
